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
// Sums are taken in integers, multiples of 2^-44: their order changes nothing,
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
__device__ __forceinline__ float vf_prob(float x) { return __saturatef(x); }

// x + e, x in [0, 1] and |e| <= 2^-23, as a multiple of 2^-44, in two parts: hi
// multiples of 2^-22 and lo.  Adding 3 (1.5 times 2^-21) rounds to the last place
// of numbers of that size, which then stands in the low bits.
struct Fixed {
    uint32_t hi;
    int32_t lo;
    __device__ __forceinline__ int64_t all() const { return (static_cast<int64_t>(hi) << 22) + lo; }
};
__device__ __forceinline__ Fixed vf_fixed(float x, float e) {
    const float t = __fadd_rn(x, 3.0f);
    const float r = __fadd_rn(__fsub_rn(x, __fsub_rn(t, 3.0f)), e);      // the difference is exact
    const float v = __fadd_rn(r, 0x1.8p-21f);
    return {__float_as_uint(t) - 0x40400000u, static_cast<int32_t>(__float_as_uint(v) - 0x35400000u)};
}

// max(0, p - c q), c = ch + cl: the product's and the difference's roundings go
// into a second number, so that together they are good to 2^-47.
__device__ __forceinline__ Fixed vf_residual(float p, float q, float ch, float cl) {
    const float m = __fmul_rn(ch, q), d = __fsub_rn(p, m);
    const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, d), m), __fmaf_rn(cl, q, __fmaf_rn(ch, q, -m)));
    const bool some = __fadd_rn(d, e) > 0.0f;
    const Fixed f = vf_fixed(d, e);
    return {some ? f.hi : 0u, some ? f.lo : 0};
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

__device__ __forceinline__ int64_t vf_warp_sum(int64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ uint64_t vf_warp_max(uint64_t x) {
    const uint32_t hi = static_cast<uint32_t>(x >> 32), a = __reduce_max_sync(0xffffffffu, hi);
    return static_cast<uint64_t>(a) << 32 | __reduce_max_sync(0xffffffffu, hi == a ? static_cast<uint32_t>(x) : 0u);
}

// What the decisions need but the sums of rows: read by the first CTA of the
// cluster and taken from it by the others, the same to the bit, so that all take
// the same turns.
struct VerifyNodes {
    uint64_t children[GDN_MAX_NEW];
    int token[GDN_MAX_NEW];
    float u[GDN_MAX_NEW], p[GDN_MAX_NEW], q[GDN_MAX_NEW];    // p and q of the token in its parent's row
    float u_next;
    int first, n, pad;
};

struct VerifySmem {
    VerifyNodes node;
    uint64_t total[2][VF_MOST];           // the CTAs' sums, by the parity of the row's turn
    uint64_t top[2][VF_MOST * VF_WARPS];  // the warps' largest keys, likewise
    uint64_t warp_sum[VF_WARPS];
    int gone[GDN_MAX_NEW];                // rejected certain drafts
    int found;
};

// A row in runs of whole 16-byte vectors, one per warp of the cluster; the
// elements before the first vector go with the first run, those after the last
// one with the last.
template <class T>
struct VerifyRow {
    static constexpr int VEC = 16 / sizeof(T);
    const T *p, *q;
    int head, vecs, per, runs, vocab;
    bool q_aligned;
    __device__ __forceinline__ VerifyRow(const T* p_, const T* q_, int vocab_, int runs_) : p(p_), q(q_), runs(runs_), vocab(vocab_) {
        head = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / static_cast<int>(sizeof(T)), vocab);
        vecs = (vocab - head) / VEC;
        per = (vecs + runs - 1) / runs;
        q_aligned = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    }
    __device__ __forceinline__ int vec(int r) const { return min(r * per, vecs); }
    __device__ __forceinline__ int begin(int r) const { return r == 0 ? 0 : head + vec(r) * VEC; }
    __device__ __forceinline__ int end(int r) const { return r == runs - 1 ? vocab : head + vec(r + 1) * VEC; }
    __device__ __forceinline__ int run_of(int j) const {
        if (j < head || vecs == 0) return j < head ? 0 : runs - 1;
        const int v = (j - head) / VEC;
        return v < vecs ? v / per : runs - 1;
    }
    // the elements of vector v
    static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[VEC]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (VEC == 4) {
                x[e] = __uint_as_float(u[e]);
            } else {
                x[2 * e] = __uint_as_float(u[e] << 16);
                x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ uint4 load_p(int v) const { return *reinterpret_cast<const uint4*>(p + head + v * VEC); }
    __device__ __forceinline__ uint4 load_q(int v) const {
        const T* at = q + head + v * VEC;
        if (q_aligned) return *reinterpret_cast<const uint4*>(at);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (VEC == 4) w[e] = __float_as_uint(at[e]);
            else w[e] = at[2 * e] | static_cast<uint32_t>(at[2 * e + 1]) << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// A lane's share of the weights of vectors v, v + 32, ... below v1: max(0, p - c q)
// (REST) or p.  Functions of their own, a copy each: unrolled into every place
// that reads a row they do not fit the instruction cache.
template <class T, bool REST>
__device__ __noinline__ int64_t vf_sum_vectors(const VerifyRow<T> row, int v, int v1, float ch, float cl) {
    using Row = VerifyRow<T>;
    constexpr int BATCH = 16 / Row::VEC;  // vectors that a thread has in flight
    int64_t w = 0;
#pragma unroll 1
    for (; v < v1; v += 32 * BATCH) {
        uint4 x[BATCH], y[BATCH];         // past the run: zeros
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            x[k] = v + 32 * k < v1 ? row.load_p(v + 32 * k) : make_uint4(0, 0, 0, 0);
            if (REST) y[k] = v + 32 * k < v1 ? row.load_q(v + 32 * k) : make_uint4(0, 0, 0, 0);
        }
        uint32_t hi = 0;
        int32_t lo = 0;                   // 16 times 2^22 at most
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            float xe[Row::VEC], ye[Row::VEC];
            Row::unpack(x[k], xe);
            if (REST) Row::unpack(y[k], ye);
#pragma unroll
            for (int e = 0; e < Row::VEC; ++e) {
                const Fixed f = REST ? vf_residual(vf_prob(xe[e]), vf_prob(ye[e]), ch, cl) : vf_fixed(vf_prob(xe[e]), 0.0f);
                hi += f.hi;
                lo += f.lo;
            }
        }
        w += (static_cast<int64_t>(hi) << 22) + lo;
    }
    return w;
}

// The key of a score: the larger the score, and of equal ones the lower the
// place, the larger the key.
__device__ __forceinline__ uint64_t vf_key(float x, int j) { return static_cast<uint64_t>(vf_order(x)) << 32 | (0xffffffffu - j); }

// The key of a lane's largest score above -inf among its vectors, 0 if there is
// none.  A vector is looked at element by element only where its largest one is
// a new record of the lane's, which its first few mostly are.
template <class T>
__device__ __noinline__ uint64_t vf_top_vectors(const VerifyRow<T> row, int v, int v1) {
    using Row = VerifyRow<T>;
    constexpr int BATCH = 4;
    float top = __uint_as_float(0xff800000u);
    int at = -1;
#pragma unroll 1
    for (; v < v1; v += 32 * BATCH) {
        uint4 x[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) x[k] = row.load_p(min(v + 32 * k, v1 - 1));   // the last one again changes nothing
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            float xe[Row::VEC];
            Row::unpack(x[k], xe);
            float m = xe[0];
#pragma unroll
            for (int e = 1; e < Row::VEC; ++e) m = fmaxf(m, xe[e]);
            if (m > top) {
                top = m;
#pragma unroll
                for (int e = Row::VEC - 1; e >= 0; --e)
                    if (xe[e] == m) at = row.head + min(v + 32 * k, v1 - 1) * Row::VEC + e;
            }
        }
    }
    return at < 0 ? 0 : vf_key(top, at);
}

// An integer below 2^53 times 2^-44 as two floats, off by at most 2^-49 of it: what
// 63 rejections of a row's sum below 8 come to is below 504 times 2^44.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair vf_pair(int64_t x) {
    // three parts that a float holds, 23, 15 and 15 bits
    const uint32_t low = static_cast<uint32_t>(x);
    const float a = static_cast<float>(static_cast<uint32_t>(x >> 30)) * 0x1p-14f;
    const float b = static_cast<float>(low >> 15 & 0x7fffu) * 0x1p-29f, c = static_cast<float>(low & 0x7fffu) * 0x1p-44f;
    const float m = __fadd_rn(b, c), e = __fsub_rn(c, __fsub_rn(m, b));      // b is 0 or more than c
    const float s = __fadd_rn(a, m);      // a is 0 or more than m
    return {s, __fadd_rn(__fsub_rn(m, __fsub_rn(s, a)), e)};
}

// (c0 + u z) q < p, in pairs of floats: sm_103a has next to no units for 64 bits,
// and every warp decides for itself.  With c0 = 0 and z = 1 it is exact.
__device__ __forceinline__ bool vf_accepted(Pair c0, float u, Pair z, float q, float p) {
    const float m = __fmul_rn(u, z.hi), me = __fmaf_rn(u, z.lo, __fmaf_rn(u, z.hi, -m));      // u z
    const float s = __fadd_rn(c0.hi, m), t = __fsub_rn(s, c0.hi);                             // c0 + u z
    const float se = __fadd_rn(__fadd_rn(__fsub_rn(c0.hi, __fsub_rn(s, t)), __fsub_rn(m, t)), __fadd_rn(c0.lo, me));
    const float x = __fmul_rn(s, q), xe = __fmaf_rn(se, q, __fmaf_rn(s, q, -x));              // times q
    const float d = __fsub_rn(p, x);      // exact where p and x are near each other
    return __fadd_rn(d, -xe) > 0.0f;
}

// A cluster per sequence, each of whose warps has a run of the vocabulary.  The
// CTAs meet once at the start and once per row that is read, their sums sent
// around before the barrier.  What bounds it is that rows follow one another: a row
// of 150001 fp32 p and q takes some 2.5 us (the loads' latency, 22 instructions an
// element, the sums and the barrier; 1.7 of them with a vocabulary of 1000), the
// gathering before the first some 4.  One chain of 5: 9.4 us; 32 greedy chains of up
// to 6 (128000 bf16): 14; 16 trees of 12 to 32: 30.  Certain drafts (no q): the same
// trees 20, 32 chains of 2 to 6 (128000 bf16) 9.5.  Decisions in fp64 had been 4 us
// more for the one chain.
template <class T>
__global__ void __launch_bounds__(VF_THREADS, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
    namespace cg = cooperative_groups;
    using Row = VerifyRow<T>;
    constexpr int VEC = Row::VEC;
    __shared__ __align__(16) VerifySmem sm;
    const cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int s = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T* P = static_cast<const T*>(a.p);
    const T* Q = static_cast<const T*>(a.q);
    const bool greedy = !a.u;
    if (tid == 0) sm.found = -1;
    pdl_wait();
    pdl_trigger();
    if (rank == 0) {
        if (tid < GDN_MAX_NEW) sm.node.children[tid] = 0;
        __syncthreads();
        int first;
        const int n = draft_range(a.d, s, first, g_verify_skipped);
        if (tid == 0) {
            sm.node.first = first;
            sm.node.n = n;
            sm.node.u_next = n && !greedy ? a.u_next[s] : 0.0f;
        }
        if (tid < n) {
            const int parent = draft_parent(draft_ancestors(a.d, first, tid));
            int token = a.tokens[first + tid];
            float u = greedy ? 0.0f : a.u[first + tid], p = 0.0f, q = 0.0f;
            if (tid > 0 && (token < 0 || token >= a.vocab)) {
                atomicCAS(&g_verify_skipped, 0, static_cast<int>(ERR_INDEX));
                token = -1;
            }
            if (!greedy && parent >= 0 && token >= 0) {
                p = vf_prob(vf_value(P + (first + parent) * a.ld_p + token));
                if (Q) q = vf_prob(vf_value(Q + (first + parent) * a.ld_q + token));
            }
            if (parent >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&sm.node.children[parent]), 1ull << tid);
            sm.node.token[tid] = token;
            sm.node.u[tid] = u;
            sm.node.p[tid] = p;
            sm.node.q[tid] = q;
        }
    }
    cluster.sync();                       // the first CTA has its nodes, and all are there
    if (rank) {
        const uint32_t* from = reinterpret_cast<const uint32_t*>(cluster.map_shared_rank(&sm.node, 0));
        for (int e = tid; e < static_cast<int>(sizeof(VerifyNodes) / 4); e += VF_THREADS) reinterpret_cast<uint32_t*>(&sm.node)[e] = from[e];
    }
    __syncthreads();
    const int n = sm.node.n, first = sm.node.first;
    if (n == 0) {
        if (rank == 0 && tid == 0) {
            a.count[s] = 0;
            a.node[s] = a.next[s] = -1;
        }
        cluster.sync();                   // the first CTA's memory is read until here
        return;
    }
    const int mine = rank * VF_WARPS + warp, runs = ctas * VF_WARPS;
    int cur = 0, depth = 0, n_gone = 0, turn = 0;
    int64_t C = 0, Z = 1ll << 44;         // c0 and the sum of the residual, in multiples of 2^-44
    Pair c0 = {0.0f, 0.0f};
    bool summed = false;                  // the CTAs' and warps' sums are those of this residual
    int best = -1;
    const auto row_of = [&](int i) {
        return Row(P + static_cast<int64_t>(first + i) * a.ld_p, Q ? Q + static_cast<int64_t>(first + i) * a.ld_q : nullptr, a.vocab, runs);
    };
    Row row = row_of(0);
    const auto weight = [&](int j) -> int64_t {
        const float x = vf_prob(vf_value(row.p + j));
        return (C ? vf_residual(x, vf_prob(vf_value(row.q + j)), c0.hi, c0.lo) : vf_fixed(x, 0.0f)).all();
    };
    const auto is_gone = [&](int x) {
        for (int g = 0; g < n_gone; ++g)
            if (sm.gone[g] == x) return true;
        return false;
    };
    // the CTAs' numbers in every CTA
    const auto spread = [&](uint64_t x) {
        uint64_t* all = sm.total[turn & 1];
        ++turn;
        if (tid < ctas) *cluster.map_shared_rank(all + rank, tid) = x;
        cluster.sync();
        return all;
    };
    // the row's sum (of what C says is left; rejected certain drafts are still in it)
    const auto sum_row = [&]() {
        int64_t w = 0;
        if (mine == 0 && lane < row.head) w += weight(lane);
        if (mine == runs - 1 && row.head + row.vecs * VEC + lane < a.vocab) w += weight(row.head + row.vecs * VEC + lane);
        const int v0 = row.vec(mine) + lane, v1 = row.vec(mine + 1);
        w += C ? vf_sum_vectors<T, true>(row, v0, v1, c0.hi, c0.lo) : vf_sum_vectors<T, false>(row, v0, v1, 0.0f, 0.0f);
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
    // the largest key, from warps to warps: putting a CTA's together first, as the sums do, takes 0.4 us more a row
    const auto top_of_all = [&](uint64_t top) {
        uint64_t* all = sm.top[turn & 1];
        ++turn;
        top = vf_warp_max(top);
        if (lane < ctas) *cluster.map_shared_rank(all + mine, lane) = top;
        cluster.sync();
        top = 0;
        for (int r = lane; r < runs; r += 32) top = all[r] > top ? all[r] : top;
        return vf_warp_max(top);
    };
    const auto find_best = [&]() {
        uint64_t top = vf_top_vectors<T>(row, row.vec(mine) + lane, row.vec(mine + 1));
        const auto take = [&](int j) {
            const float x = vf_value(row.p + j);
            const uint64_t k = x > __uint_as_float(0xff800000u) ? vf_key(x, j) : 0;
            top = k > top ? k : top;
        };
        const int tail = row.head + row.vecs * VEC + lane;
        if (mine == 0 && lane < row.head) take(lane);
        if (mine == runs - 1 && tail < a.vocab) take(tail);
        top = top_of_all(top);
        if (top == 0) {                   // nothing above -inf: its first place, or the row's where there is none
            for (int j = row.begin(mine) + lane; j < row.end(mine); j += 32) {
                const uint64_t k = vf_key(vf_value(row.p + j), j);
                top = k > top ? k : top;
            }
            top = top_of_all(top);
        }
        best = static_cast<int>(0xffffffffu - static_cast<uint32_t>(top));
    };
    int path = 0, id = -1;                // thread d: the path's token d and the one after it
    uint64_t left = sm.node.children[0];  // children still to be tried
    bool read = greedy, over = false;     // the row is to be read; the target's own row takes a residual's place
    int drop = -1;                        // a rejected certain draft, to be taken off the row's sum
    for (;;) {
        if (read) {
            if (greedy) find_best();
            else sum_row();
            read = false;
        }
        if (drop >= 0) {
            const int x = sm.node.token[drop];
            if (x >= 0 && !is_gone(x)) {
                Z -= vf_fixed(sm.node.p[drop], 0.0f).all();
                __syncthreads();
                if (tid == 0) sm.gone[n_gone] = x;
                __syncthreads();
                ++n_gone;
            }
            drop = -1;
        }
        if (!left) {
            if (greedy || (summed && (Z != 0 || over))) break;
            if (summed) {                 // nothing is left of the residual
                C = 0;
                n_gone = 0;
                over = true;
            }
            read = true;
            continue;
        }
        const int i = __ffsll(static_cast<long long>(left)) - 1, x = sm.node.token[i];
        bool ok;
        if (greedy) {
            ok = x == best;
        } else {
            // a certain draft's q is 1, and what it was taken off the row shows in z alone
            ok = x >= 0 && vf_accepted(c0, sm.node.u[i], vf_pair(Z), Q ? sm.node.q[i] : 1.0f, sm.node.p[i]) && !is_gone(x);
        }
        if (ok) {
            if (tid == depth) {
                path = cur;
                id = x;
            }
            cur = i;
            ++depth;
            left = sm.node.children[i];
            n_gone = 0;
            C = 0;
            c0 = {0.0f, 0.0f};
            Z = 1ll << 44;
            summed = false;
            row = row_of(i);
            read = greedy;
            continue;
        }
        left &= left - 1;
        if (Q) {
            C += Z;
            c0 = vf_pair(C);
            read = true;
        } else if (!greedy) {
            drop = i;
            read = !summed;
        }
    }
    int winner = 0, next = best;
    if (!greedy) {
        uint64_t* all = sm.total[(turn - 1) & 1];
        if (n_gone) {
            __syncthreads();
            if (tid == 0)
                for (int g = 0; g < n_gone; ++g) {
                    const int r = row.run_of(sm.gone[g]);
                    const int64_t w = weight(sm.gone[g]);
                    all[r / VF_WARPS] -= w;
                    if (r / VF_WARPS == rank) sm.warp_sum[r % VF_WARPS] -= w;
                }
            __syncthreads();
        }
        // the first place whose running sum passes u * Z, that is its whole part: the CTA, its warp's run, the place
        const uint64_t limit = __umul64hi(vf_fraction(sm.node.u_next), static_cast<uint64_t>(Z));
        uint64_t before = 0;
        while (winner < ctas && before + all[winner] <= limit) before += all[winner++];
        next = -1;
        if (winner == ctas) {
            winner = 0;                   // the row has nothing
        } else if (rank == winner) {
            int w = 0;
            while (w < VF_WARPS - 1 && before + sm.warp_sum[w] <= limit) before += sm.warp_sum[w++];
            const int k0 = row.begin(rank * VF_WARPS + w), k1 = row.end(rank * VF_WARPS + w);
            const int per = (k1 - k0 + VF_THREADS - 1) / VF_THREADS, m0 = min(k0 + tid * per, k1), m1 = min(m0 + per, k1);
            const auto at = [&](int j) -> uint64_t { return is_gone(j) ? 0 : weight(j); };
            uint64_t own = 0;
            for (int j = m0; j < m1; ++j) own += at(j);
            uint64_t upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            __syncthreads();              // warp_sum has been read
            if (lane == 31) sm.warp_sum[warp] = upto;
            __syncthreads();
            for (int i = 0; i < warp; ++i) before += sm.warp_sum[i];
            before += upto - own;
            if (before <= limit && before + own > limit)
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
    // as many CTAs as run at once, two to an SM: 32 greedy sequences of a vocabulary of 128000 took 24.4 us with 16 CTAs
    // each, 16.6 with 8, 16.9 with 4; 64 sampled ones of 100000 35.7, 17.1 and 11.4; one of 150001
    // 9.4, 10.2 and 12.7
    int ctas = VF_MOST;
    while (ctas > 1 && a.d.n_seqs * ctas > 2 * 152) ctas >>= 1;
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
