// Verification of drafted tokens against the target's probabilities.
//
// At token c of a sequence (its first to begin with) the children are tried in
// order.  With p and q the target's and the draft's probabilities after c, a
// child x is accepted with probability min(1, r(x) / q(x)), r = p; after each
// rejection r becomes max(0, r - q), divided by its sum.  Undivided, r is
// max(0, p - c0 q) for one number c0: r' = max(0, max(0, p - c0 q) - Z q) =
// max(0, p - (c0 + Z) q), Z the sum of the r before (1 for p itself), so
//     accept x if (c0 + u_x Z) q(x) < p(x), else c0 += Z, Z = sum_j max(0, p_j - c0 q_j)
// and a whole row is read only after a rejection and for the token that ends
// the path, which is drawn from the last r.  Without q a draft was certain:
// accepted with probability r(x), and r loses x when it is rejected.
//
// Sums are taken in integers, multiples of 2^-60: their order changes nothing,
// so the token drawn does not depend on how a row was split.
#include "drafts.cuh"

#include <cooperative_groups.h>

namespace gdn {

static __device__ int g_verify_error;     // debug: a store's index
static __device__ int g_verify_skipped;   // an offset or token of the caller's, out of range

struct VerifyArgs {
    DraftTokens d;
    const void* p;
    const void* q;            // null: certain drafts
    int64_t ld_p, ld_q;
    const int32_t* tokens;
    const float* u;           // null: greedy
    const float* u_next;
    int32_t* rows;
    int32_t* ids;
    int32_t* count;
    int32_t* node;
    int32_t* next;
    int vocab;
};

constexpr int VF_THREADS = 512;
constexpr int VF_WARPS = VF_THREADS / 32;
constexpr int VF_MOST = 16;               // CTAs of a cluster

__device__ __forceinline__ float vf_value(const float* p) { return *p; }
__device__ __forceinline__ float vf_value(const uint16_t* p) { return bf16_bits_to_float(*p); }

// A probability: what is negative or no number counts as 0, what is above 1 as 1.
__device__ __forceinline__ float vf_prob(float x) { return x > 0.0f ? fminf(x, 1.0f) : 0.0f; }

// x in [0, 1] as a multiple of 2^-60 (what is below is cut off).
__device__ __forceinline__ uint64_t vf_fixed(float x) {
    const uint32_t b = __float_as_uint(x), e = b >> 23;
    const uint64_t m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    return e >= 90 ? m << (e - 90) : e > 66 ? m >> (90 - e) : 0ull;
}

// x in [0, 1) as a multiple of 2^-64.
__device__ __forceinline__ uint64_t vf_fraction(float x) {
    if (x >= 1.0f) return ~0ull;
    if (!(x > 0.0f)) return 0ull;
    const uint32_t b = __float_as_uint(x), e = b >> 23;
    const uint64_t m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    return e >= 86 ? m << (e - 86) : e > 62 ? m >> (86 - e) : 0ull;
}

// A score as an integer of the same order, NaN the lowest.
__device__ __forceinline__ uint32_t vf_order(float x) {
    const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
    return x != x ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint64_t vf_warp_sum(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ uint64_t vf_warp_max(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t y = __shfl_xor_sync(0xffffffffu, x, o);
        x = y > x ? y : x;
    }
    return x;
}

struct VerifySmem {
    // what the first CTA of the cluster read, in all of them: the same to the bit, so that they take the same turns
    int first, n;
    int parent[GDN_MAX_NEW], token[GDN_MAX_NEW];
    float u[GDN_MAX_NEW], p[GDN_MAX_NEW], q[GDN_MAX_NEW];    // p and q of the token in its parent's row
    float u_next;
    uint64_t total[2][VF_MOST];           // the CTAs' sums (or largest scores), by the parity of the row's turn
    uint64_t warp_sum[VF_WARPS];
    int gone[GDN_MAX_NEW];
    int found;
};

// A cluster per sequence, each of whose warps has a run of the vocabulary.  The
// first CTA gathers all that the decisions need but the sums of rows and gives it
// to the others; from there each CTA takes the same decisions, and they meet
// (one barrier, their sums sent around before it) once per row that is read.
template <class T>
__global__ void __launch_bounds__(VF_THREADS) verify_kernel(const __grid_constant__ VerifyArgs a) {
    namespace cg = cooperative_groups;
    __shared__ VerifySmem sm;
    const cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int s = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T* P = static_cast<const T*>(a.p);
    const T* Q = static_cast<const T*>(a.q);
    const bool greedy = !a.u;
    pdl_wait();
    pdl_trigger();
    cluster.sync();                       // every CTA is there: their memory may be written
    if (rank == 0 && tid < GDN_MAX_NEW) {
        int first;
        const int n = draft_range(a.d, s, first, g_verify_skipped);
        int parent = -2, token = -1;
        float u = 0.0f, p = 0.0f, q = 0.0f;
        if (tid < n) {
            parent = draft_parent(draft_ancestors(a.d, first, tid));
            token = a.tokens[first + tid];
            if (tid > 0 && (token < 0 || token >= a.vocab)) {
                atomicCAS(&g_verify_skipped, 0, static_cast<int>(ERR_INDEX));
                token = -1;
            }
            if (!greedy) {
                u = a.u[first + tid];
                if (parent >= 0 && token >= 0) {
                    p = vf_prob(vf_value(P + (first + parent) * a.ld_p + token));
                    if (Q) q = vf_prob(vf_value(Q + (first + parent) * a.ld_q + token));
                }
            }
        }
        for (int c = 0; c < ctas; ++c) {
            VerifySmem* to = cluster.map_shared_rank(&sm, c);
            to->parent[tid] = parent;
            to->token[tid] = token;
            to->u[tid] = u;
            to->p[tid] = p;
            to->q[tid] = q;
            if (tid == 0) {
                to->first = first;
                to->n = n;
                to->u_next = n && !greedy ? a.u_next[s] : 0.0f;
            }
        }
    }
    cluster.sync();
    const int n = sm.n, first = sm.first;
    if (n == 0) {
        if (rank == 0 && tid == 0) {
            a.count[s] = 0;
            a.node[s] = a.next[s] = -1;
        }
        return;
    }
    const int run = (a.vocab + ctas * VF_THREADS - 1) / (ctas * VF_THREADS) * 32;      // a warp's part of a row
    const int j0 = min((rank * VF_WARPS + warp) * run, a.vocab), j1 = min(j0 + run, a.vocab);
    int cur = 0, depth = 0, n_gone = 0, turn = 0;
    uint64_t C = 0, Z = 1ull << 60;       // c0 in multiples of 2^-50; the sum of the residual
    bool summed = false;                  // Z is the sum of this row
    int best = -1;
    const T* p = P + static_cast<int64_t>(first) * a.ld_p;
    const T* q = Q ? Q + static_cast<int64_t>(first) * a.ld_q : nullptr;
    const auto weight = [&](int j) -> uint64_t {
        const uint64_t x = vf_fixed(vf_prob(vf_value(p + j)));
        if (!C) return x;
        const uint64_t y = vf_fixed(vf_prob(vf_value(q + j)));
        const uint64_t c = C == 1ull << 50 ? y : (__umul64hi(y, C) << 14) | (y * C >> 50);
        return x > c ? x - c : 0ull;
    };
    const auto is_gone = [&](int x) {
        for (int g = 0; g < n_gone; ++g)
            if (sm.gone[g] == x) return true;
        return false;
    };
    // the CTAs' numbers, each put together with a CTA's others, in every CTA
    const auto spread = [&](uint64_t x) {
        uint64_t* all = sm.total[turn & 1];
        ++turn;
        if (tid < ctas) *cluster.map_shared_rank(all + rank, tid) = x;
        cluster.sync();
        return all;
    };
    const auto sum_row = [&]() {
        uint64_t w = 0;
#pragma unroll 4
        for (int j = j0 + lane; j < j1; j += 32) w += weight(j);
        if (lane < n_gone && sm.gone[lane] >= j0 && sm.gone[lane] < j1) w -= weight(sm.gone[lane]);
        if (lane + 32 < n_gone && sm.gone[lane + 32] >= j0 && sm.gone[lane + 32] < j1) w -= weight(sm.gone[lane + 32]);
        w = vf_warp_sum(w);
        if (lane == 0) sm.warp_sum[warp] = w;
        __syncthreads();
        uint64_t x = 0;
#pragma unroll
        for (int i = 0; i < VF_WARPS; ++i) x += sm.warp_sum[i];
        const uint64_t* all = spread(x);
        Z = 0;
        for (int c = 0; c < ctas; ++c) Z += all[c];
        summed = true;
    };
    const auto find_best = [&]() {
        uint64_t top = 0;
#pragma unroll 4
        for (int j = j0 + lane; j < j1; j += 32) {
            const uint64_t v = static_cast<uint64_t>(vf_order(vf_value(p + j))) << 32 | (0xffffffffu - j);
            top = v > top ? v : top;
        }
        top = vf_warp_max(top);
        if (lane == 0) sm.warp_sum[warp] = top;
        __syncthreads();
        top = 0;
#pragma unroll
        for (int i = 0; i < VF_WARPS; ++i) top = sm.warp_sum[i] > top ? sm.warp_sum[i] : top;
        const uint64_t* all = spread(top);
        for (int c = 0; c < ctas; ++c) top = all[c] > top ? all[c] : top;
        best = static_cast<int>(0xffffffffu - static_cast<uint32_t>(top));
    };
    int path = 0, id = -1;                // thread d: the path's token d and the one after it
    if (greedy) find_best();
    for (int i = 1; i < n; ++i) {
        if (sm.parent[i] != cur) continue;
        const int x = sm.token[i];
        bool ok;
        if (greedy) {
            ok = x == best;
        } else {
            const double z = static_cast<double>(Z) * 0x1p-60, c0 = static_cast<double>(C) * 0x1p-50;
            const double px = sm.p[i], qx = sm.q[i], u = sm.u[i];
            ok = x >= 0 && (Q ? (c0 + u * z) * qx < px : !is_gone(x) && u * z < px);
        }
        if (ok) {
            if (tid == depth) {
                path = cur;
                id = x;
            }
            cur = i;
            ++depth;
            n_gone = 0;
            C = 0;
            Z = 1ull << 60;
            summed = false;
            p = P + static_cast<int64_t>(first + i) * a.ld_p;
            if (Q) q = Q + static_cast<int64_t>(first + i) * a.ld_q;
            if (greedy) find_best();
        } else if (!greedy) {
            if (Q) {
                C += Z >> 10;
            } else if (x >= 0 && !is_gone(x)) {
                __syncthreads();
                if (tid == 0) sm.gone[n_gone] = x;
                __syncthreads();
                ++n_gone;
            }
            sum_row();
        }
    }
    int winner = 0, next = best;
    if (!greedy) {
        if (!summed) sum_row();
        if (Z == 0) {                     // nothing is left of the residual: the target's own row
            C = 0;
            n_gone = 0;
            sum_row();
        }
        // the first place whose running sum passes u * Z, that is its whole part: the CTA, its warp's run, the place
        const uint64_t limit = __umul64hi(vf_fraction(sm.u_next), Z);
        const uint64_t* all = sm.total[(turn - 1) & 1];
        uint64_t before = 0;
        while (winner < ctas && before + all[winner] <= limit) before += all[winner++];
        next = -1;
        if (winner == ctas) {
            winner = 0;                   // the row has nothing
        } else if (rank == winner) {
            int w = 0;
            while (w < VF_WARPS - 1 && before + sm.warp_sum[w] <= limit) before += sm.warp_sum[w++];
            const int k0 = min((rank * VF_WARPS + w) * run, a.vocab), k1 = min(k0 + run, a.vocab);
            const int per = (run + VF_THREADS - 1) / VF_THREADS, m0 = min(k0 + tid * per, k1), m1 = min(m0 + per, k1);
            const auto at = [&](int j) -> uint64_t { return is_gone(j) ? 0 : weight(j); };
            uint64_t mine = 0;
            for (int j = m0; j < m1; ++j) mine += at(j);
            uint64_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            __syncthreads();              // warp_sum has been read
            if (lane == 31) sm.warp_sum[warp] = upto;
            __syncthreads();
            for (int i = 0; i < warp; ++i) before += sm.warp_sum[i];
            before += upto - mine;
            if (before <= limit && before + mine > limit)
                for (int j = m0; j < m1; ++j) {
                    before += at(j);
                    if (before > limit) {
                        sm.found = j;
                        break;
                    }
                }
            __syncthreads();
            next = sm.found;
        }
    }
    if (rank != winner) return;
    if (tid == depth) {
        path = cur;
        id = next;
    }
    if (tid < n && GDN_IN_RANGE(g_verify_error, first + tid < a.d.n_tokens)) {
        a.rows[first + tid] = tid <= depth ? first + path : -1;
        a.ids[first + tid] = tid <= depth ? id : -1;
    }
    if (tid == 0) {
        a.count[s] = depth + 1;
        a.node[s] = cur;
        a.next[s] = next;
    }
}

template <class T>
static cudaError_t verify_launch(const VerifyArgs& a, cudaStream_t st) {
    static PerDeviceOnce once;
    once.run([](int) { cudaFuncSetAttribute(verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
    const int ctas = a.d.n_seqs <= 8 ? 16 : 8;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.d.n_seqs * ctas);
    cfg.blockDim = dim3(VF_THREADS);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

cudaError_t launch_verify(const DraftTokens& d, bool bf16, const void* p, int64_t ld_p, const void* q, int64_t ld_q, int64_t vocab,
                          const int32_t* tokens, const float* u, const float* u_next, int32_t* rows, int32_t* ids, int32_t* count,
                          int32_t* node, int32_t* next, cudaStream_t st) {
    const VerifyArgs a{d, p, q, ld_p, ld_q, tokens, u, u_next, rows, ids, count, node, next, static_cast<int>(vocab)};
    return bf16 ? verify_launch<uint16_t>(a, st) : verify_launch<float>(a, st);
}

int* verify_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_verify_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

int* verify_skipped_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_verify_skipped) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdn
