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

// max(0, p - c0 q), c0 a multiple of 2^-50
__device__ __forceinline__ uint64_t vf_weight(float p, float q, uint64_t c0) {
    const uint64_t a = vf_fixed(vf_prob(p)), b = vf_fixed(vf_prob(q));
    const uint64_t c = (__umul64hi(b, c0) << 14) | (b * c0 >> 50);
    return a > c ? a - c : 0ull;
}

// The sum over the block's threads.
__device__ __forceinline__ uint64_t vf_block_sum(uint64_t x, uint64_t* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    uint64_t r = 0;
    for (int w = 0; w < VF_WARPS; ++w) r += red[w];
    return r;
}

// A score as an integer of the same order, NaN the lowest.
__device__ __forceinline__ uint32_t vf_order(float x) {
    const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
    return x != x ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <class T>
__global__ void __launch_bounds__(VF_THREADS) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ uint64_t red[VF_WARPS];
    __shared__ uint64_t part[VF_THREADS];
    __shared__ int gone[GDN_MAX_NEW];
    __shared__ int found;
    const int s = blockIdx.x, tid = threadIdx.x;
    int first;
    const int n = draft_range(a.d, s, first, g_verify_skipped);
    if (n == 0) {
        if (tid == 0) {
            a.count[s] = 0;
            a.node[s] = a.next[s] = -1;
        }
        return;
    }
    const T* P = static_cast<const T*>(a.p);
    const T* Q = static_cast<const T*>(a.q);
    const bool greedy = !a.u;
    const int per = (a.vocab + VF_THREADS - 1) / VF_THREADS;        // a thread's part of a row
    const int j0 = min(tid * per, a.vocab), j1 = min(j0 + per, a.vocab);
    int cur = 0, depth = 0, n_gone = 0;
    uint64_t C = 0, Z = 1ull << 60;
    double c0 = 0.0;
    int best = -1;
    const T* p = P + static_cast<int64_t>(first) * a.ld_p;
    const T* q = a.q ? Q + static_cast<int64_t>(first) * a.ld_q : nullptr;
    const auto weight = [&](int j) { return a.q ? vf_weight(vf_value(p + j), vf_value(q + j), C) : vf_fixed(vf_prob(vf_value(p + j))); };
    const auto is_gone = [&](int x) {
        for (int g = 0; g < n_gone; ++g)
            if (gone[g] == x) return true;
        return false;
    };
    // the sum of the part's weights, those of rejected certain drafts left out
    const auto part_sum = [&]() {
        uint64_t w = 0;
        for (int j = j0; j < j1; ++j) w += weight(j);
        if (!a.q)
            for (int g = 0; g < n_gone; ++g)
                if (gone[g] >= j0 && gone[g] < j1) w -= weight(gone[g]);
        return w;
    };
    const auto find_best = [&]() {
        uint64_t top = 0;
        for (int j = j0; j < j1; ++j) {
            const uint64_t v = static_cast<uint64_t>(vf_order(vf_value(p + j))) << 32 | (0xffffffffu - j);
            top = v > top ? v : top;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t v = __shfl_xor_sync(0xffffffffu, top, o);
            top = v > top ? v : top;
        }
        __syncthreads();
        if ((tid & 31) == 0) red[tid >> 5] = top;
        __syncthreads();
        top = 0;
        for (int w = 0; w < VF_WARPS; ++w) top = red[w] > top ? red[w] : top;
        return static_cast<int>(0xffffffffu - static_cast<uint32_t>(top));
    };
    if (greedy) best = find_best();
    for (int i = 1; i < n; ++i) {
        if (draft_parent(draft_ancestors(a.d, first, i)) != cur) continue;
        const int x = a.tokens[first + i];
        const bool known = x >= 0 && x < a.vocab;
        if (!known && tid == 0) atomicCAS(&g_verify_skipped, 0, static_cast<int>(ERR_INDEX));
        bool ok;
        if (greedy) {
            ok = x == best;
        } else if (!known) {
            ok = false;
        } else {
            const double u = a.u[first + i], z = static_cast<double>(Z) * 0x1p-60, px = vf_prob(vf_value(p + x));
            ok = a.q ? (c0 + u * z) * vf_prob(vf_value(q + x)) < px : u * z < (is_gone(x) ? 0.0 : px);
        }
        if (ok) {
            if (tid == 0 && GDN_IN_RANGE(g_verify_error, first + depth < a.d.n_tokens)) {
                a.rows[first + depth] = first + cur;
                a.ids[first + depth] = x;
            }
            cur = i;
            ++depth;
            n_gone = 0;
            C = 0;
            c0 = 0.0;
            Z = 1ull << 60;
            p = P + static_cast<int64_t>(first + i) * a.ld_p;
            if (a.q) q = Q + static_cast<int64_t>(first + i) * a.ld_q;
            if (greedy) best = find_best();
        } else if (!greedy) {
            if (a.q) {
                C += Z >> 10;
                c0 += static_cast<double>(Z) * 0x1p-60;
            } else if (known && !is_gone(x)) {
                __syncthreads();
                if (tid == 0) gone[n_gone] = x;
                __syncthreads();
                ++n_gone;
            }
            Z = vf_block_sum(part_sum(), red);
        }
    }
    int next = best;
    if (!greedy) {
        uint64_t w = part_sum();
        uint64_t total = vf_block_sum(w, red);
        if (total == 0) {                 // nothing is left of the residual: the target's own row
            C = 0;
            n_gone = 0;
            w = part_sum();
            total = vf_block_sum(w, red);
        }
        // the first place whose running sum passes u * total, that is its whole part
        const float u = a.u_next[s];
        uint64_t U = 0;
        if (u >= 1.0f) U = ~0ull;
        else if (u > 0.0f) {
            const uint32_t b = __float_as_uint(u), e = b >> 23;
            const uint64_t m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
            U = e >= 86 ? m << (e - 86) : e > 62 ? m >> (86 - e) : 0ull;
        }
        const uint64_t limit = __umul64hi(U, total);
        part[tid] = w;
        if (tid == 0) found = -1;
        __syncthreads();
        uint64_t before = 0;
        for (int t = 0; t < tid; ++t) before += part[t];
        if (before <= limit && before + w > limit) {
            for (int j = j0; j < j1; ++j) {
                before += !a.q && is_gone(j) ? 0ull : weight(j);
                if (before > limit) {
                    found = j;
                    break;
                }
            }
        }
        __syncthreads();
        next = found;
    }
    if (tid == 0) {
        a.rows[first + depth] = first + cur;
        a.ids[first + depth] = next;
        a.count[s] = depth + 1;
        a.node[s] = cur;
        a.next[s] = next;
    }
    for (int i = depth + 1 + tid; i < n; i += VF_THREADS) a.rows[first + i] = a.ids[first + i] = -1;
}

cudaError_t launch_verify(const DraftTokens& d, bool bf16, const void* p, int64_t ld_p, const void* q, int64_t ld_q, int64_t vocab,
                          const int32_t* tokens, const float* u, const float* u_next, int32_t* rows, int32_t* ids, int32_t* count,
                          int32_t* node, int32_t* next, cudaStream_t st) {
    const VerifyArgs a{d, p, q, ld_p, ld_q, tokens, u, u_next, rows, ids, count, node, next, static_cast<int>(vocab)};
    if (bf16)
        verify_kernel<uint16_t><<<d.n_seqs, VF_THREADS, 0, st>>>(a);
    else
        verify_kernel<float><<<d.n_seqs, VF_THREADS, 0, st>>>(a);
    return cudaGetLastError();
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
