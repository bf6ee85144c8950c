// The GDN layer over drafted tokens: the short conv and the delta rule along a
// chain or a tree of up to 64 tokens of each sequence, which leave the held
// state alone, and the commit of the accepted path into it.
//
// The recurrence along the path to token i, S_i = a_i S_p (I - b_i k_i k_i^T) +
// b_i v_i k_i^T with p its parent, is S_i = a_i S_p + u_i k_i^T for u_i = b_i
// (v_i - a_i S_p k_i).  With g_i the sum of log a over i and its ancestors,
//     u_i = b_i (v_i - e^{g_i} S_0 k_i - sum_{j anc i} e^{g_i - g_j} (k_j . k_i) u_j)
//     o_i = S_i q_i = e^{g_i} S_0 q_i + sum_{j anc i, i} e^{g_i - g_j} (k_j . q_i) u_j
// so no state but S_0 is formed, S_0 is read once for all tokens of the
// sequence, and the state after any token n follows from the u:
//     S_n = e^{g_n} S_0 + sum_{j anc n, n} e^{g_n - g_j} u_j k_j^T.
#include "drafts.cuh"

namespace gdn {

static __device__ int g_draft_error;      // a value beyond fp16; debug: a store's index
static __device__ int g_draft_skipped;    // an offset or node of the caller's, out of range

constexpr float LOG_A_MIN = -1.0e4f;      // e^-10000 is 0 in fp32, and sums of it stay finite (a = 0: log a = -inf)

// N bytes from global to shared memory, without a register in between.
template <int N>
__device__ __forceinline__ void cp_async(void* to, const void* from) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 32 bytes of a state: one access where the states start on 32 bytes (WIDE), two
// where they start on 16; the pieces lie whole multiples of 32 behind the start.
template <bool WIDE>
__device__ __forceinline__ void load_state(const float* p, uint32_t (&w)[8]) {
    if constexpr (WIDE) {
        load32(p, w);
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>(p), y = *reinterpret_cast<const uint4*>(p + 4);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
    }
}
template <bool WIDE>
__device__ __forceinline__ void store_state(float* p, const uint32_t (&w)[8]) {
    if constexpr (WIDE) {
        store32(p, w);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(p + 4) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
static bool on_32_bytes(const float* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; }

// ------------------------------------------------------------ conv

struct ConvTreeArgs {
    DraftTokens d;
    const uint16_t* qkvz;
    int64_t ld_qkvz;
    const float* ba;
    int64_t ld_ba;
    const float* tail;     // [n_seqs][c_conv][3]
    const float* conv_w;   // [c_conv][4]
    const float* A_log;
    const float* dt_bias;
    uint16_t* out;         // fp16 [n_tokens][c_conv]
    float* log_a;
    float* b;
    int c_conv, n_heads, n_qk_norm, n_q, hv, col_blocks;
    bool wide;             // rows of qkvz start on 16 bytes
    float eps, q_scale;
};

constexpr int CT_THREADS = 128;
constexpr int CT_COLS = 256;               // channels of a block
constexpr int CT_SLOTS = CT_COLS / 8;      // threads of a token

// Block (CT_COLS channels, sequence): all raw inputs of the sequence's tokens to
// shared memory at once, each read once, and from there to the up to four tokens
// that have them as a tap.  A thread has 8 channels, their weights in registers, of
// every fourth token.  The last block of x computes the gates.  48 trees of 20 to
// 64 tokens, 8192 channels: 33 us, 2.2 TB/s (35 in blocks of 512 channels, 44 with
// 512 threads); with a warp walking a head's tokens from L1 it was 51.  What bounds it is this order of a block's work: all
// copies, a wait for all of them, then up to 16 tokens a thread, so that loads and arithmetic do not overlap within a
// block (DRAM 14 %, 0.39 instructions issued a cycle and scheduler); a third fewer instructions changed nothing.
template <int D>
__global__ void __launch_bounds__(CT_THREADS, 6) conv_tree_kernel(const __grid_constant__ ConvTreeArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];    // raw inputs [token][CT_COLS] bf16, the conv state [CT_COLS][3] fp32
    __shared__ uint64_t anc[GDN_MAX_NEW];
    __shared__ __align__(16) int at[GDN_MAX_NEW][4];     // the taps' tokens, oldest first; -1, -2, -3: the conv state
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.y, tid = threadIdx.x;
    int first;
    const int n = draft_range(a.d, s, first, g_draft_skipped);
    if (n == 0) return;
    if (static_cast<int>(blockIdx.x) == a.col_blocks) {
        for (int e = tid; e < n * a.hv; e += CT_THREADS) {
            const int64_t t = first + e / a.hv;
            const int h = e % a.hv;
            if (GDN_IN_RANGE(g_draft_error, t < a.d.n_tokens))
                gate_values(a.ba[t * a.ld_ba + h], a.ba[t * a.ld_ba + a.hv + h], a.A_log[h], a.dt_bias[h], a.log_a[t * a.hv + h],
                            a.b[t * a.hv + h]);
        }
        return;
    }
    const int col0 = blockIdx.x * CT_COLS, slot = tid % CT_SLOTS, c0 = col0 + 8 * slot;
    const bool in = c0 < a.c_conv;         // heads are whole multiples of 8 channels
    float* tail = reinterpret_cast<float*>(raw + a.d.max_new * CT_COLS * 2);
    if (in)
        for (int i = tid / CT_SLOTS; i < n; i += CT_THREADS / CT_SLOTS) {
            unsigned char* to = raw + (i * CT_SLOTS + slot) * 16;
            const uint16_t* src = a.qkvz + static_cast<int64_t>(first + i) * a.ld_qkvz + c0;
            if (a.wide) {
                cp_async<16>(to, src);
            } else {
                cp_async<8>(to, src);
                cp_async<8>(to + 8, src + 4);
            }
        }
    for (int e = tid; e < CT_COLS * 3; e += CT_THREADS)
        if (col0 * 3 + e < a.c_conv * 3) cp_async<4>(tail + e, a.tail + (static_cast<int64_t>(s) * a.c_conv + col0) * 3 + e);
    if (tid < n) anc[tid] = draft_ancestors(a.d, first, tid);
    F2 w[4][4];                            // taps of channels 2e and 2e + 1
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float4* src = reinterpret_cast<const float4*>(a.conv_w + static_cast<int64_t>(in ? c0 + 2 * e : 0) * 4);
        const float4 x = src[0], y = src[1];
        w[0][e] = f2(x.x, y.x);
        w[1][e] = f2(x.y, y.y);
        w[2][e] = f2(x.z, y.z);
        w[3][e] = f2(x.w, y.w);
    }
    __syncthreads();
    if (tid < n) {
        int x = tid;
        at[tid][3] = x;
#pragma unroll
        for (int m = 2; m >= 0; --m) {
            x = x < 0 ? x - 1 : draft_parent(anc[x]);
            at[tid][m] = x;
        }
    }
    cp_async_wait();
    __syncthreads();
    const int head = c0 / D;
    const bool norm = head < a.n_qk_norm;
    const float mul = head < a.n_q ? a.q_scale : 1.0f;
    const float* mine = tail + 24 * slot;
    bool over = false;
    // a warp's lanes share the token
    for (int i = tid / CT_SLOTS; i < n; i += CT_THREADS / CT_SLOTS) {
        const int4 taps = *reinterpret_cast<const int4*>(at[i]);
        const int row[4] = {taps.x, taps.y, taps.z, taps.w};
        F2 y[4];                           // as conv4_silu has it, two channels at a time
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            F2 v[4];
            if (m < 3 && row[m] < 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = f2(mine[6 * e + 3 + row[m]], mine[6 * e + 6 + row[m]]);
            } else {
                const uint4 x = *reinterpret_cast<const uint4*>(raw + (max(row[m], 0) * CT_SLOTS + slot) * 16);
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = f2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = m ? f2_fma(w[m][e], v[e], y[e]) : f2_mul(w[m][e], v[e]);
        }
        F2 sq = f2(0.0f, 0.0f);
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float l = -1.4426950408889634f;
            float t0, t1;
            f2_split(f2_mul(y[e], f2(l, l)), t0, t1);
            f2_split(f2_add(f2(ex2_ftz(t0), ex2_ftz(t1)), f2(1.0f, 1.0f)), t0, t1);
            y[e] = f2_mul(y[e], f2(rcp_ftz(t0), rcp_ftz(t1)));
            sq = f2_fma(y[e], y[e], sq);
        }
        float ss, s1;
        f2_split(sq, ss, s1);
        ss += s1;
#pragma unroll
        for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float f = norm ? rsqrtf(ss + a.eps) * mul : 1.0f;
        uint32_t out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y0, y1;
            f2_split(f2_mul(y[e], f2(f, f)), y0, y1);
            top = fmaxf_nan(top, fmaxf_nan(fabsf(y0), fabsf(y1)));
            out[e] = f16x2_bits(y0, y1);
        }
        over |= in && !((norm ? fmaxf_nan(top, ss <= 3.0e38f ? 0.0f : ss) : top) <= 65504.0f);
        if (in && GDN_IN_RANGE(g_draft_error, first + i < a.d.n_tokens && c0 + 8 <= a.c_conv))
            *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(first + i) * a.c_conv + c0) =
                make_uint4(out[0], out[1], out[2], out[3]);
    }
    if (over) atomicCAS(&g_draft_error, 0, static_cast<int>(ERR_RANGE));
}

template <int D>
static cudaError_t conv_tree_launch(const ConvTreeArgs& a, dim3 grid, cudaStream_t st) {
    constexpr int TAIL = CT_COLS * 12;
    static PerDeviceOnce once;
    once.run([](int) { cudaFuncSetAttribute(conv_tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, GDN_MAX_NEW * CT_COLS * 2 + TAIL); });
    return launch_dependent(conv_tree_kernel<D>, grid, dim3(CT_THREADS), static_cast<size_t>(a.d.max_new * CT_COLS * 2 + TAIL), st, a);
}

cudaError_t launch_conv_tree(const gdn_layer& L, const DraftTokens& d, const uint16_t* qkvz, int64_t ld_qkvz, const float* ba, int64_t ld_ba,
                             const float* tail, uint16_t* out, float* log_a, float* b, cudaStream_t st) {
    ConvTreeArgs a;
    a.d = d;
    a.qkvz = qkvz;
    a.ld_qkvz = ld_qkvz;
    a.ba = ba;
    a.ld_ba = ld_ba;
    a.tail = tail;
    a.conv_w = L.conv_w;
    a.A_log = L.A_log;
    a.dt_bias = L.dt_bias;
    a.out = out;
    a.log_a = log_a;
    a.b = b;
    a.n_heads = 2 * L.n_qk_heads + L.n_v_heads;
    a.c_conv = a.n_heads * L.dk;
    a.n_qk_norm = 2 * L.n_qk_heads;
    a.n_q = L.n_qk_heads;
    a.hv = L.n_v_heads;
    a.col_blocks = (a.c_conv + CT_COLS - 1) / CT_COLS;
    a.eps = L.eps_l2;
    a.q_scale = L.q_scale;
    a.wide = reinterpret_cast<uintptr_t>(qkvz) % 16 == 0 && ld_qkvz % 8 == 0;
    const dim3 grid(a.col_blocks + (L.gate_log_a ? 0 : 1), d.n_seqs);
    return L.dk == 128 ? conv_tree_launch<128>(a, grid, st) : conv_tree_launch<64>(a, grid, st);
}

// ------------------------------------------------------------ delta rule

struct DeltaTreeArgs {
    DraftTokens d;
    const uint16_t* qkv;   // fp16 [n_tokens][c_conv]
    const float* log_a;    // [n_tokens][hv]
    const float* b;
    const float* state;    // [n_seqs][hv][D][D]
    uint16_t* o;           // fp16 [n_tokens][hv][D]
    float* delta;          // [n_tokens][hv][D]
    int hv, ratio, c_qk, c_conv, c_v;
};

__device__ __forceinline__ float clamp_log_a(float la) { return la < LOG_A_MIN ? LOG_A_MIN : la; }

// Sums of log a along paths of up to 64 tokens, whose differences enter an
// exponential: two floats each, so a difference keeps fp32's relative accuracy
// where the sums themselves are large.
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 sum2(Sum2 a, Sum2 b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    const float h = s + e;
    return {h, e - (h - s)};
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Products of fp32 operands on the tensor cores: tf32 takes the upper 11 bits of
// each, so an operand is the nearest such number and a rest, whose upper 11 bits
// count (cutting x off instead of rounding it would give the rest x's sign, and
// what is cut off the rest one direction: 3.7e-7 of S_0 k, not 1e-7).  Of the four
// products the one of the two rests (2^-24 of the whole) is left out.
struct Tf32 {
    uint32_t hi, lo;
};
// By an addition and a mask, or by a conversion, which is the faster one only where little else is converted
// (delta_few_kernel: 32.4 us with it, 33.5 without; delta_tree_kernel 72.5 and 70.2).
__device__ __forceinline__ Tf32 tf32(float x) {
    const uint32_t hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    return {hi, __float_as_uint(x - __uint_as_float(hi))};
}
__device__ __forceinline__ Tf32 tf32_by_conversion(uint32_t x) {
    uint32_t hi;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(__uint_as_float(x)));
    return {hi, __float_as_uint(__uint_as_float(x) - __uint_as_float(hi))};
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// What counts as finite where products of two parts are taken: from 2^128 - 2^116 =
// 3.40274e38 on the first part rounds to infinity, and 0 times that is no number.
constexpr float TF32_MAX = 3.4e38f;
// c [16 rows][8 tokens i] += x [16 rows][8 tokens j] m [j][i].  x is laid out as the
// products are (lane g, t: rows g, g + 8, tokens 2t, 2t + 1), which makes the tokens
// 2t and 2t + 1 the operands' indices t and t + 4; m0, m1: m[2t][g], m[2t + 1][g].
__device__ __forceinline__ void mma_rows(float (&c)[4], const float (&x)[4], float m0, float m1) {
    const Tf32 a0 = tf32(x[0]), a1 = tf32(x[2]), a2 = tf32(x[1]), a3 = tf32(x[3]), b0 = tf32(m0), b1 = tf32(m1);
    mma_tf32(c, a0.lo, a1.lo, a2.lo, a3.lo, b0.hi, b1.hi);
    mma_tf32(c, a0.hi, a1.hi, a2.hi, a3.hi, b0.lo, b1.lo);
    mma_tf32(c, a0.hi, a1.hi, a2.hi, a3.hi, b0.hi, b1.hi);
}

constexpr int DT_U = 20;                    // floats between the tokens of a warp's 16 rows: lanes 2t * 20 + g differ in their banks

// The pieces that both kernels of the delta rule over drafts are made of.

// Rows g and g + 8 of S_0 as operands: columns 8t .. 8t+7 of each 32, a row's
// largest taken to [2^13, 2^14), then the fp16 number nearest and the one nearest
// to the rest.  What they lose is 2^-23 of an element or 2^-38 of the largest.
template <int KB>
struct StateOperand {
    uint32_t h0[KB][4], h1[KB][4], l0[KB][4], l1[KB][4];
    float back[2];
    // get(m, b, w): the eight columns of block b, of row g (m = 0) or g + 8
    template <class Get>
    __device__ __forceinline__ explicit StateOperand(const Get& get) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float top = 0.0f;               // of the numbers; a NaN stays one without it
            uint32_t w[8];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                get(m, b, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(__uint_as_float(w[e])));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t e8 = min(max(__float_as_uint(top) >> 23, 14u), 254u);
            const float scale = __uint_as_float((267u - e8) << 23);
            back[m] = __uint_as_float((e8 - 13u) << 23);
            const F2 scale2 = f2(scale, scale);
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                get(m, b, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const F2 x = f2_mul(f2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1])), scale2);
                    float x0, x1;
                    f2_split(x, x0, x1);
                    const __half2 hh = __floats2half2_rn(x0, x1);
                    const float2 f = __half22float2(hh);
                    f2_split(f2_sub(x, f2(f.x, f.y)), x0, x1);
                    (m ? h1 : h0)[b][e] = *reinterpret_cast<const uint32_t*>(&hh);
                    (m ? l1 : l0)[b][e] = f16x2_bits(x0, x1);
                }
            }
        }
    }
    // e^{g_i} S_0 times the rows of eight tokens, rows g and g + 8 by tokens 2t and 2t + 1
    __device__ __forceinline__ void times(const uint4* rows, int sw, float e0, float e1, float (&x)[4]) const {
        float c[4] = {}, d[4] = {};
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            const uint4 y = rows[(4 * b) ^ sw];
            mma_f16(c, h0[b][0], h1[b][0], h0[b][1], h1[b][1], y.x, y.y);
            mma_f16(d, l0[b][0], l1[b][0], l0[b][1], l1[b][1], y.x, y.y);
            mma_f16(c, h0[b][2], h1[b][2], h0[b][3], h1[b][3], y.z, y.w);
            mma_f16(d, l0[b][2], l1[b][2], l0[b][3], l1[b][3], y.z, y.w);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = (c[m] + d[m]) * back[m >> 1] * (m & 1 ? e1 : e0);
    }
};

// What all rows of a head share, in shared memory.
struct DeltaTokens {
    const uint4 *ks, *qs;    // fp16 rows in units of 16 bytes, unit x of row r at x ^ 4 (r & 1)
    float *kk, *qk;          // [j][i], pitch floats apart: -e^{g_i - g_j} k_j . k_i, 0 where j is no ancestor of i;
                             // e^{g_i - g_j} k_j . q_i, where j is one or i itself
    float* inv;              // per block of 8 tokens [j][i]: u_i = sum_j inv[j][i] r_j
    uint64_t* anc;           // ancestors
    uint64_t* uni;           // per block: its ancestors before it
    Sum2* g;
    int* up;
    float* eg;
    const float* b;
    int pitch;
};

// A warp: ancestors in, sums along the paths out.  By doubling: after a round that
// looked 2^m tokens back, a token holds the sum of the nearest 2^(m + 1) of its
// path.  mask and log a of the lane's tokens lane and lane + 32.
__device__ __forceinline__ void delta_sums(const DeltaTokens& d, int n, const uint64_t (&mask)[2], const float (&log_a)[2]) {
    const int lane = threadIdx.x & 31, np = (n + 7) & ~7;
    Sum2 sum[2];
    int up[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int i = lane + 32 * m;
        const uint64_t x = i < n ? mask[m] & ((1ull << i) - 1) : 0ull;
        sum[m] = {i < n ? clamp_log_a(log_a[m]) : 0.0f, 0.0f};
        up[m] = draft_parent(x);
        if (i < np) {
            d.anc[i] = x;
            d.g[i] = sum[m];
            d.up[i] = up[m];
        }
    }
    __syncwarp();
    for (int step = 1; step < n; step <<= 1) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
            if (up[m] >= 0) {
                sum[m] = sum2(sum[m], d.g[up[m]]);
                up[m] = d.up[up[m]];
            }
        __syncwarp();
#pragma unroll
        for (int m = 0; m < 2; ++m)
            if (lane + 32 * m < np) {
                d.g[lane + 32 * m] = sum[m];
                d.up[lane + 32 * m] = up[m];
            }
        __syncwarp();
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
        if (lane + 32 * m < np) d.eg[lane + 32 * m] = expf(sum[m].hi + sum[m].lo);
    if (lane < np / 8) {
        uint64_t all = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) all |= d.anc[8 * lane + c];
        d.uni[lane] = all & ((1ull << 8 * lane) - 1);
    }
}

// A warp: the products of tokens j = 16 jt .. with the block of tokens i = 8 bi ..
template <int D>
__device__ __forceinline__ void delta_products(const DeltaTokens& d, int np, int jt, int bi) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, sw = t ^ (4 * (g & 1));
    constexpr int UNITS = D / 8;
    float c[2][2][4] = {};                  // with keys, with queries; two chains each
    const int j0 = 16 * jt + g;
    const bool second = 16 * jt + 8 < np;
    const int i0 = 8 * bi + 2 * t;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
        const int unit = (4 * b) ^ sw;
        const uint4 x0 = d.ks[j0 * UNITS + unit], x1 = second ? d.ks[(j0 + 8) * UNITS + unit] : make_uint4(0, 0, 0, 0);
        const uint4 y = d.ks[(8 * bi + g) * UNITS + unit], z = d.qs[(8 * bi + g) * UNITS + unit];
        mma_f16(c[0][0], x0.x, x1.x, x0.y, x1.y, y.x, y.y);
        mma_f16(c[1][0], x0.x, x1.x, x0.y, x1.y, z.x, z.y);
        mma_f16(c[0][1], x0.z, x1.z, x0.w, x1.w, y.z, y.w);
        mma_f16(c[1][1], x0.z, x1.z, x0.w, x1.w, z.z, z.w);
    }
    const uint64_t anc[2] = {d.anc[i0], d.anc[i0 + 1]};
    const Sum2 gi[2] = {d.g[i0], d.g[i0 + 1]}, gj[2] = {d.g[j0], d.g[second ? j0 + 8 : j0]};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int j = j0 + 8 * (m >> 1), i = i0 + (m & 1);
        const bool on = anc[m & 1] >> j & 1;
        const float w = expf((gi[m & 1].hi - gj[m >> 1].hi) + (gi[m & 1].lo - gj[m >> 1].lo));
        if (m < 2 || second) {
            d.kk[j * d.pitch + i] = on ? -w * (c[0][0][m] + c[0][1][m]) : 0.0f;
            d.qk[j * d.pitch + i] = on || i == j ? w * (c[1][0][m] + c[1][1][m]) : 0.0f;
        }
    }
}

// Eight lanes of a warp: the inverse of block bi's system, a column each.
__device__ __forceinline__ void delta_inverse(const DeltaTokens& d, int bi) {
    const int lane = threadIdx.x & 31;
    if (lane >= 8) return;
    float m[8][8], out[8];
    uint32_t on[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        on[i] = static_cast<uint32_t>(d.anc[8 * bi + i] >> 8 * bi);
#pragma unroll
        for (int j = 0; j < i; ++j) m[i][j] = d.kk[(8 * bi + j) * d.pitch + 8 * bi + i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float sum = i == lane ? 1.0f : 0.0f;
#pragma unroll
        for (int j = 0; j < i; ++j) sum = on[i] >> j & 1 ? fmaf(m[i][j], out[j], sum) : sum;
        out[i] = sum * d.b[8 * bi + i];
        d.inv[64 * bi + 8 * lane + i] = out[i];
    }
}

// A block of 8 tokens of a warp's 16 rows.  r, xq: v - e^g S_0 k and e^g S_0 q, rows
// g and g + 8 by tokens 2t and 2t + 1; us: the warp's u of earlier tokens; bad: tokens
// whose u in row lane % 16 is not finite.  Leaves u and o in r's layout.
__device__ __forceinline__ void delta_block(const DeltaTokens& d, int bi, float (&r)[4], float (&xq)[4], float* us, uint64_t& bad,
                                            float (&u)[4], float (&o)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint64_t before = d.uni[bi];
    for (int jb = 0; jb < bi; ++jb) {
        if (!(before >> 8 * jb & 0xff)) continue;
        const int j = 8 * jb + 2 * t;
        const float x[4] = {us[j * DT_U + g], us[(j + 1) * DT_U + g], us[j * DT_U + g + 8], us[(j + 1) * DT_U + g + 8]};
        mma_rows(r, x, d.kk[j * d.pitch + 8 * bi + g], d.kk[(j + 1) * d.pitch + 8 * bi + g]);
        mma_rows(xq, x, d.qk[j * d.pitch + 8 * bi + g], d.qk[(j + 1) * d.pitch + 8 * bi + g]);
    }
    const int j = 8 * bi + 2 * t;
#pragma unroll
    for (int m = 0; m < 4; ++m) u[m] = 0.0f;
    mma_rows(u, r, d.inv[64 * bi + 16 * t + g], d.inv[64 * bi + 16 * t + 8 + g]);
    const float sum = ((fabsf(r[0]) + fabsf(r[1])) + (fabsf(r[2]) + fabsf(r[3]))) + ((fabsf(u[0]) + fabsf(u[1])) + (fabsf(u[2]) + fabsf(u[3])));
    if (!__any_sync(0xffffffffu, bad != 0 || !(sum <= TF32_MAX))) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            us[(j + (m & 1)) * DT_U + g + 8 * (m >> 1)] = u[m];
            o[m] = xq[m];
        }
        mma_rows(o, u, d.qk[j * d.pitch + 8 * bi + g], d.qk[(j + 1) * d.pitch + 8 * bi + g]);
        __syncwarp();
        return;
    }
    // token by token: lane r works on row r, with r and S_0 q by way of the block's place in us
    const int row = lane & 15;
    float v[8], w[8], ou[8];
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
        for (int m = 0; m < 4; ++m) us[(j + (m & 1)) * DT_U + g + 8 * (m >> 1)] = pass ? xq[m] : r[m];
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) (pass ? w : v)[c] = us[(8 * bi + c) * DT_U + row];
        __syncwarp();
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int i = 8 * bi + c;
        float x = v[c] * d.b[i];
        if (bad & d.anc[i]) x = __uint_as_float(0x7fffffffu);
        ou[c] = x;
        if (!(fabsf(x) <= TF32_MAX)) {
            bad |= 1ull << i;
            x = 0.0f;
        }
        const float* kr = d.kk + i * d.pitch + 8 * bi;
        const float* qr = d.qk + i * d.pitch + 8 * bi;
#pragma unroll
        for (int e = c; e < 8; ++e) {
            if (e > c) v[e] = fmaf(kr[e], x, v[e]);
            w[e] = fmaf(qr[e], x, w[e]);
        }
        if (bad & (d.anc[i] | 1ull << i)) w[c] = __uint_as_float(0x7fffffffu);
    }
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {  // o, u, and last the u that others may take
#pragma unroll
        for (int c = 0; c < 8; ++c) us[(8 * bi + c) * DT_U + row] = pass == 0 ? w[c] : pass == 2 && (bad >> (8 * bi + c) & 1) ? 0.0f : ou[c];
        __syncwarp();
        if (pass < 2) {
#pragma unroll
            for (int m = 0; m < 4; ++m) (pass ? u : o)[m] = us[(j + (m & 1)) * DT_U + g + 8 * (m >> 1)];
            __syncwarp();
        }
    }
}

// u and o of a block to global memory; true if an o is beyond fp16.
__device__ __forceinline__ bool delta_store(const DeltaTreeArgs& a, int first, int n, int bi, int64_t col, const float (&u)[4], const float (&o)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    bool over = false;
    const int64_t at = static_cast<int64_t>(first + 8 * bi + 2 * t) * a.c_v + col + g;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int i = 8 * bi + 2 * t + (m & 1);
        if (i < n && GDN_IN_RANGE(g_draft_error, first + i < a.d.n_tokens)) {
            const int64_t to = at + static_cast<int64_t>(m & 1 ? a.c_v : 0) + 8 * (m >> 1);
            a.delta[to] = u[m];
            a.o[to] = __half_as_ushort(__float2half_rn(o[m]));
            over |= !(fabsf(o[m]) <= 65504.0f);
        }
    }
    return over;
}

// Shared memory of delta_tree_kernel for np tokens (a multiple of 8) and a
// number of warps: byte offsets.
template <int D>
struct DeltaTreeSmem {
    int k, q, kk, qk, inv, u, anc, uni, g, up, eg, b, end;
    __host__ __device__ DeltaTreeSmem(int np, int warps) {
        k = 0;
        q = k + np * D * 2;
        kk = q + np * D * 2;
        qk = kk + np * (np + 4) * 4;        // a pitch of np + 4 for the banks of lanes 2t * pitch + g
        inv = qk + np * (np + 4) * 4;
        u = inv + np * 32;                  // per warp [token][16 rows]
        anc = u + warps * np * DT_U * 4;
        uni = anc + np * 8;
        g = uni + 64;
        up = g + np * 8;
        eg = up + np * 4;
        b = eg + np * 4;
        end = b + np * 4;
    }
};

// A warp holds 16 rows of S_0; the rows of u and o follow from them alone, so
// warps meet only for what all rows share, the decayed products of keys and
// queries.  S_0 is read once, straight into operands of the tensor cores (the k
// index is permuted alike in both operands: thread t of a quad holds columns 8t ..
// 8t+7 of each 32).  Keys and queries are fp16 as they come.
//
// Tokens go in blocks of 8.  With r_i = v_i - e^{g_i} S_0 k_i + what the ancestors
// before the block add, the block's u are its unit lower-triangular system's
// inverse times r; the inverse (8 x 8, the same for all rows, taken once per CTA),
// the earlier u and the block's own enter as products of fp32 operands on the
// tensor cores, whose layout never changes in between.  Numbers that are not
// finite would reach tokens that do not descend from theirs (0 times them), so a
// warp that meets one goes through the block token by token.
//
// The products are mma.sync: S_0 goes from registers that loaded it into operands,
// where tcgen05 would want both halves of it written to shared memory first, twice
// its bytes, for products of 16 to 128 columns.
//
// This kernel: a CTA for a head, or for part of its rows, of a sequence.  24 trees
// of 24 to 64 tokens over 32 heads of 128: 60 us; S_0 alone could be read in 15.
// A CTA's phases follow one another (S_0, the tokens' products, the blocks in turn:
// 16300 of 51000 cycles of 64 tokens are these), with two CTAs to an SM and 0.47
// instructions issued a cycle and scheduler.  At the 128 registers that two CTAs
// leave a thread, heads of 128 spill 16 bytes.
template <int D, bool WIDE>
__global__ void __launch_bounds__(256, 2) delta_tree_kernel(const __grid_constant__ DeltaTreeArgs a) {
    constexpr int KB = D / 32;              // blocks of 32 columns
    constexpr int UNITS = D / 8;            // 16-byte units of a row of keys
    extern __shared__ __align__(16) unsigned char raw[];
    pdl_wait();
    pdl_trigger();
    const int warps = blockDim.x >> 5, parts = D / (16 * warps);
    const int h = blockIdx.x / parts, part = blockIdx.x % parts, s = blockIdx.y, hk = h / a.ratio;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int r0 = (part * warps + warp) * 16;              // the warp's rows
    uint32_t w0[KB][8], w1[KB][8];                          // rows g and g + 8
    {
        const float* S = a.state + ((static_cast<int64_t>(s) * a.hv + h) * D + r0 + g) * D + 8 * t;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            load_state<WIDE>(S + 32 * b, w0[b]);
            load_state<WIDE>(S + 8 * D + 32 * b, w1[b]);
        }
    }
    int first;
    const int n = draft_range(a.d, s, first, g_draft_skipped);
    if (n == 0) return;
    const int np = (n + 7) & ~7, nb = np / 8;
    const DeltaTreeSmem<D> at(np, warps);
    uint4* ks = reinterpret_cast<uint4*>(raw + at.k);
    uint4* qs = reinterpret_cast<uint4*>(raw + at.q);
    float* bs = reinterpret_cast<float*>(raw + at.b);
    const DeltaTokens d = {ks, qs, reinterpret_cast<float*>(raw + at.kk), reinterpret_cast<float*>(raw + at.qk),
                           reinterpret_cast<float*>(raw + at.inv), reinterpret_cast<uint64_t*>(raw + at.anc),
                           reinterpret_cast<uint64_t*>(raw + at.uni), reinterpret_cast<Sum2*>(raw + at.g),
                           reinterpret_cast<int*>(raw + at.up), reinterpret_cast<float*>(raw + at.eg), bs, np + 4};
    float* us = reinterpret_cast<float*>(raw + at.u) + warp * np * DT_U;
    // v of a block, in the products' layout
    const uint16_t* vs = a.qkv + static_cast<int64_t>(first) * a.c_conv + 2 * a.c_qk + h * D + r0;
    const auto load_v = [&](int bi, uint16_t (&v)[4]) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = 8 * bi + 2 * t + (m & 1);
            v[m] = i < n ? vs[static_cast<int64_t>(i) * a.c_conv + g + 8 * (m >> 1)] : static_cast<uint16_t>(0);
        }
    };
    uint16_t vn[4];
    if (warp == 0) {
        uint64_t mask[2];
        float la[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int i = lane + 32 * m;
            const int64_t row = static_cast<int64_t>(first + i) * a.hv + h;
            mask[m] = i < n && a.d.tree ? a.d.tree[first + i] : ~0ull;
            la[m] = i < n ? a.log_a[row] : 0.0f;
            if (i < np) bs[i] = i < n ? a.b[row] : 0.0f;
        }
        delta_sums(d, n, mask, la);
        load_v(0, vn);
    } else {
        load_v(0, vn);
        for (int e = tid - 32; e < np * UNITS; e += blockDim.x - 32) {
            const int i = e / UNITS, x = e % UNITS, to = i * UNITS + (x ^ (4 * (i & 1)));
            if (i < n) {
                const uint16_t* row = a.qkv + static_cast<int64_t>(first + i) * a.c_conv + hk * D + 8 * x;
                cp_async<16>(qs + to, row);
                cp_async<16>(ks + to, row + a.c_qk);
            } else {
                qs[to] = ks[to] = make_uint4(0, 0, 0, 0);
            }
        }
    }
    const StateOperand<KB> S0([&](int m, int b, uint32_t (&w)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = m ? w1[b][e] : w0[b][e];
    });
    cp_async_wait();
    __syncthreads();
    const int sw = t ^ (4 * (g & 1));       // the unit of columns 8t .. 8t+7 in rows of g's parity
    // where a block has ancestors, in turn
    for (int bi = 0, turn = warp; bi < nb; ++bi) {
        const uint64_t before = d.uni[bi];
#pragma unroll 1
        for (int jt = 0; 2 * jt <= bi; ++jt) {
            if (2 * jt + 1 < bi && !(before >> 16 * jt & 0xffff)) continue;
            if (turn == 0) delta_products<D>(d, np, jt, bi);
            turn = turn == 0 ? warps - 1 : turn - 1;
        }
    }
    __syncthreads();
    for (int bi = warp; bi < nb; bi += warps) delta_inverse(d, bi);
    float xk[4], xq[4];
    const auto with_state = [&](int bi) {
        const float e0 = d.eg[8 * bi + 2 * t], e1 = d.eg[8 * bi + 2 * t + 1];
        S0.times(ks + (8 * bi + g) * UNITS, sw, e0, e1, xk);
        S0.times(qs + (8 * bi + g) * UNITS, sw, e0, e1, xq);
    };
    with_state(0);
    __syncthreads();
    uint64_t bad = 0;
    bool over = false;
    for (int bi = 0; bi < nb; ++bi) {
        float r[4], u[4], o[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) r[m] = __half2float(__ushort_as_half(vn[m]));
        if (bi + 1 < nb) load_v(bi + 1, vn);
#pragma unroll
        for (int m = 0; m < 4; ++m) r[m] -= xk[m];
        delta_block(d, bi, r, xq, us, bad, u, o);
        if (bi + 1 < nb) with_state(bi + 1);
        over |= delta_store(a, first, n, bi, h * D + r0, u, o);
    }
    if (over) atomicCAS(&g_draft_error, 0, static_cast<int>(ERR_RANGE));
}

// The same for sequences of up to 8 tokens, a block: S_0 is used once, so its
// numbers go from the load to the tensor cores without being kept, as two tf32
// numbers each against keys and queries in fp32 (22 bits of S_0 count, at every
// size).  Nothing but reading S_0 takes long, so the rest hides behind it: the
// loads come first, and a warp of its own takes the products of the tokens while
// the others have S_0 times keys and queries.  64 chains of up to 8 tokens over 32
// heads of 128 (146 MB): 31.4 us, 4.65 TB/s; reading S_0 and nothing else takes
// 22.8.  With S_0 kept in operands as above it was 52; fetched a head ahead into
// shared memory by CTAs that stay, 45 (its way through shared memory cost more
// than the waits it saved).
constexpr int DF_WARPS = 4;                 // 64 rows of a head to a CTA (31.4 us for 64 chains of up to 8 over 32 heads of 128; 32.5 with 128)
template <int D>
struct DeltaFewSmem {
    static constexpr int W = DF_WARPS, ROW = D + 4;           // floats of a row of keys: lanes g * ROW + 8t differ in their banks
    float k[8][ROW], q[8][ROW];
    uint4 k16[8 * D / 8], q16[8 * D / 8];                   // as delta_products takes them
    float kk[8 * 12], qk[8 * 12], inv[64], us[W][8 * DT_U];
    uint64_t anc[8], uni[8];
    Sum2 g[8];
    int up[8];
    float eg[8], b[8];
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(32 * (DF_WARPS + 1), 4) delta_few_kernel(const __grid_constant__ DeltaTreeArgs a) {
    using Smem = DeltaFewSmem<D>;
    constexpr int KB = D / 32, UNITS = D / 8, W = DF_WARPS, PARTS = D / 16 / W;
    __shared__ __align__(16) Smem sm;
    pdl_wait();
    pdl_trigger();
    const int h = blockIdx.x / PARTS, s = blockIdx.y, hk = h / a.ratio;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int r0 = (blockIdx.x % PARTS * W + warp) * 16;
    const DeltaTokens d = {sm.k16, sm.q16, sm.kk, sm.qk, sm.inv, sm.anc, sm.uni, sm.g, sm.up, sm.eg, sm.b, 12};
    int first;
    if (warp == W) {
        const int n = draft_range(a.d, s, first, g_draft_skipped);
        if (n == 0) return;
        uint64_t mask[2] = {~0ull, 0};
        float la[2] = {0.0f, 0.0f};
        const int64_t row = static_cast<int64_t>(first + lane) * a.hv + h;
        if (lane < n) {
            if (a.d.tree) mask[0] = a.d.tree[first + lane];
            la[0] = a.log_a[row];
        }
        if (lane < 8) sm.b[lane] = lane < n ? a.b[row] : 0.0f;
        delta_sums(d, n, mask, la);
        __syncthreads();
        delta_products<D>(d, 8, 0, 0);
        __syncwarp();
        delta_inverse(d, 0);
        __syncthreads();
        return;
    }
    uint32_t w[KB][2][8];                                   // rows g and g + 8
    {
        const float* S = a.state + ((static_cast<int64_t>(s) * a.hv + h) * D + r0 + g) * D + 8 * t;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            load_state<WIDE>(S + 32 * b, w[b][0]);
            load_state<WIDE>(S + 8 * D + 32 * b, w[b][1]);
        }
    }
    const int n = draft_range(a.d, s, first, g_draft_skipped);
    if (n == 0) return;
    const uint16_t* rows = a.qkv + static_cast<int64_t>(first) * a.c_conv;
    for (int e = tid; e < 8 * UNITS; e += 32 * W) {
        const int i = e / UNITS, c = e % UNITS, to = i * UNITS + (c ^ (4 * (i & 1)));
        const uint16_t* row = rows + static_cast<int64_t>(i) * a.c_conv + hk * D + 8 * c;
        const uint4 zero = make_uint4(0, 0, 0, 0), x = i < n ? *reinterpret_cast<const uint4*>(row) : zero;
        const uint4 y = i < n ? *reinterpret_cast<const uint4*>(row + a.c_qk) : zero;
        sm.q16[to] = x;
        sm.k16[to] = y;
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            *reinterpret_cast<float2*>(&sm.q[i][8 * c + 2 * m]) = __half22float2(*reinterpret_cast<const __half2*>(&xs[m]));
            *reinterpret_cast<float2*>(&sm.k[i][8 * c + 2 * m]) = __half22float2(*reinterpret_cast<const __half2*>(&ys[m]));
        }
    }
    float r[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int i = 2 * t + (m & 1);
        r[m] = i < n ? __half2float(__ushort_as_half(rows[static_cast<int64_t>(i) * a.c_conv + 2 * a.c_qk + h * D + r0 + g + 8 * (m >> 1)])) : 0.0f;
    }
    __syncthreads();
    float kh[4] = {}, kl[4] = {}, qh[4] = {}, ql[4] = {};
#pragma unroll
    for (int b = 0; b < KB; ++b) {
        float ke[8], qe[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            *reinterpret_cast<float4*>(&ke[4 * e]) = *reinterpret_cast<const float4*>(&sm.k[g][32 * b + 8 * t + 4 * e]);
            *reinterpret_cast<float4*>(&qe[4 * e]) = *reinterpret_cast<const float4*>(&sm.q[g][32 * b + 8 * t + 4 * e]);
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const Tf32 a0 = tf32_by_conversion(w[b][0][e]), a1 = tf32_by_conversion(w[b][1][e]), a2 = tf32_by_conversion(w[b][0][e + 1]),
                       a3 = tf32_by_conversion(w[b][1][e + 1]);
            const uint32_t k0 = __float_as_uint(ke[e]), k1 = __float_as_uint(ke[e + 1]), q0 = __float_as_uint(qe[e]), q1 = __float_as_uint(qe[e + 1]);
            mma_tf32(kh, a0.hi, a1.hi, a2.hi, a3.hi, k0, k1);
            mma_tf32(qh, a0.hi, a1.hi, a2.hi, a3.hi, q0, q1);
            mma_tf32(kl, a0.lo, a1.lo, a2.lo, a3.lo, k0, k1);
            mma_tf32(ql, a0.lo, a1.lo, a2.lo, a3.lo, q0, q1);
        }
    }
    __syncthreads();
    float xq[4], u[4], o[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float e = d.eg[2 * t + (m & 1)];
        r[m] -= (kh[m] + kl[m]) * e;
        xq[m] = (qh[m] + ql[m]) * e;
    }
    uint64_t bad = 0;
    delta_block(d, 0, r, xq, sm.us[warp], bad, u, o);
    if (delta_store(a, first, n, 0, h * D + r0, u, o)) atomicCAS(&g_draft_error, 0, static_cast<int>(ERR_RANGE));
}

template <int D, bool WIDE>
static cudaError_t delta_tree_launch(const DeltaTreeArgs& a, cudaStream_t st) {
    const int np = (a.d.max_new + 7) & ~7, heads = a.hv * a.d.n_seqs;
    static PerDeviceOnce once;
    once.run([](int) {
        cudaFuncSetAttribute(delta_tree_kernel<D, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, DeltaTreeSmem<D>(GDN_MAX_NEW, D / 16).end);
    });
    // up to 8 tokens the kernel for them is the faster one at any number of heads (of 128: 1 head 2.7 us and 3.8, 32 heads
    // 2.8 and 4.0, 160 4.7 and 5.5, 512 9.9 and 12.1, 2048 31 and 41; of 64: 2.5 and 3.3, 32 heads 2.5 and 3.4, 512 3.8 and 4.5)
    if (a.d.max_new <= 8)
        return launch_dependent(delta_few_kernel<D, WIDE>, dim3(a.hv * (D / 16 / DF_WARPS), a.d.n_seqs), dim3(32 * (DF_WARPS + 1)), 0, st, a);
    // a head of 128 in two CTAs while each finds an SM of its own (76 heads, 16 tokens: 5.2 us in two, 5.7 whole; 64 tokens:
    // 16.1 and 18.0; 80 heads: 5.9 and 5.7, 19.2 and 18.0), else a CTA a head; in four parts it was never faster, a head of
    // 64 not in two
    const int warps = D == 128 && 2 * heads <= 152 ? 4 : D / 16;
    return launch_dependent(delta_tree_kernel<D, WIDE>, dim3(a.hv * (D / 16 / warps), a.d.n_seqs), dim3(32 * warps),
                            static_cast<size_t>(DeltaTreeSmem<D>(np, warps).end), st, a);
}

cudaError_t launch_delta_tree(const gdn_layer& L, const DraftTokens& d, const uint16_t* qkv, const float* log_a, const float* b,
                              const float* state, uint16_t* o, float* delta, cudaStream_t st) {
    DeltaTreeArgs a;
    a.d = d;
    a.qkv = qkv;
    a.log_a = log_a;
    a.b = b;
    a.state = state;
    a.o = o;
    a.delta = delta;
    a.hv = L.n_v_heads;
    a.ratio = L.n_v_heads / L.n_qk_heads;
    a.c_qk = L.n_qk_heads * L.dk;
    a.c_v = L.n_v_heads * L.dv;
    a.c_conv = 2 * a.c_qk + a.c_v;
    if (on_32_bytes(state)) return L.dk == 128 ? delta_tree_launch<128, true>(a, st) : delta_tree_launch<64, true>(a, st);
    return L.dk == 128 ? delta_tree_launch<128, false>(a, st) : delta_tree_launch<64, false>(a, st);
}

// ------------------------------------------------------------ commit

struct CommitArgs {
    DraftTokens d;
    const uint16_t* qkv;
    const float* log_a;
    const float* delta;
    const int32_t* node;     // [n_seqs], -1: nothing accepted
    const float* state_in;
    float* state_out;
    const uint16_t* qkvz;
    int64_t ld_qkvz;
    const float* tail_in;    // null: no conv state
    float* tail_out;
    int hv, ratio, c_qk, c_conv;
};

constexpr int CM_THREADS = 256;
constexpr int CM_CHANNELS = 4;             // of the conv state, per thread

// The accepted token of sequence s, -1 where there is none; n: its tokens.
__device__ __forceinline__ int commit_node(const CommitArgs& a, int s, int n) {
    const int node = a.node[s];
    if (node >= -1 && node < n) return node;
    atomicCAS(&g_draft_skipped, 0, static_cast<int>(ERR_INDEX));
    return -1;
}

// Block (rows of a value head, sequence): a thread has 8 columns of CH rows, all
// of them loaded before it is known what is accepted (the loads are what bounds
// the kernel); then a rank-1 update per token of the path, from shared memory.  64
// sequences of 32 heads of 128 (281 MB): 53 us, 5.3 TB/s; a copy of the states
// takes 42.
// Blocks past the heads: the conv state, CM_CHANNELS channels a thread.
template <int D, int CH, bool WIDE>
__global__ void __launch_bounds__(CM_THREADS, 4) commit_kernel(const __grid_constant__ CommitArgs a) {
    constexpr int COLS = D / 8, STEP = CM_THREADS / COLS, PARTS = D / (STEP * CH);
    constexpr int ROWS = STEP * CH;
    extern __shared__ __align__(16) float cm[];        // per token of the path: k [D], then u of the block's rows
    __shared__ Sum2 la[GDN_MAX_NEW + 1];
    __shared__ float w[GDN_MAX_NEW + 1];
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int first;
    if (static_cast<int>(blockIdx.x) >= a.hv * PARTS) {
        const int n = draft_range(a.d, s, first, g_draft_skipped), node = commit_node(a, s, n);
        int at[3];                         // tokens, or -1, -2, -3: the old state from its newest entry on
        at[2] = node;
#pragma unroll
        for (int m = 1; m >= 0; --m) at[m] = at[m + 1] < 0 ? at[m + 1] - 1 : draft_parent(draft_ancestors(a.d, first, at[m + 1]));
        const int64_t base = static_cast<int64_t>(s) * a.c_conv;
        float x[CM_CHANNELS][3];
#pragma unroll
        for (int k = 0; k < CM_CHANNELS; ++k) {
            const int c = ((blockIdx.x - a.hv * PARTS) * CM_CHANNELS + k) * CM_THREADS + tid;
            if (c >= a.c_conv) break;
#pragma unroll
            for (int m = 0; m < 3; ++m)
                x[k][m] = at[m] < 0 ? a.tail_in[(base + c) * 3 + 3 + at[m]] : bf16_bits_to_float(a.qkvz[(first + at[m]) * a.ld_qkvz + c]);
        }
#pragma unroll
        for (int k = 0; k < CM_CHANNELS; ++k) {
            const int c = ((blockIdx.x - a.hv * PARTS) * CM_CHANNELS + k) * CM_THREADS + tid;
            if (c >= a.c_conv || !GDN_IN_RANGE(g_draft_error, s < a.d.n_seqs)) break;
#pragma unroll
            for (int m = 0; m < 3; ++m) a.tail_out[(base + c) * 3 + m] = x[k][m];
        }
        return;
    }
    const int h = blockIdx.x / PARTS, row0 = blockIdx.x % PARTS * (STEP * CH), hk = h / a.ratio;
    const int col = tid % COLS * 8, row = tid / COLS;
    const int64_t base = ((static_cast<int64_t>(s) * a.hv + h) * D + row0 + row) * D + col;
    uint32_t v[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) load_state<WIDE>(a.state_in + base + j * STEP * D, v[j]);
    const int n = draft_range(a.d, s, first, g_draft_skipped), node = commit_node(a, s, n);
    const uint64_t on = node < 0 ? 0ull : draft_ancestors(a.d, first, node) | 1ull << node;
    const int np = __popcll(on);
    // a warp for every eighth token of the path
    int at = 0;
    for (uint64_t m = on; m; m &= m - 1, ++at) {
        if (at % (CM_THREADS / 32) != warp) continue;
        const int64_t t = first + __ffsll(static_cast<long long>(m)) - 1;
        float* to = cm + at * (D + ROWS);
        for (int e = lane; e < COLS; e += 32) {
            const uint4 x = *reinterpret_cast<const uint4*>(a.qkv + t * a.c_conv + a.c_qk + hk * D + 8 * e);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) *reinterpret_cast<float2*>(to + 8 * e + 2 * c) = __half22float2(*reinterpret_cast<const __half2*>(&u[c]));
        }
        for (int e = lane; e < ROWS; e += 32) to[D + e] = a.delta[(t * a.hv + h) * D + row0 + e];
    }
    if (warp == 0) {
        // the sums of log a over what follows a token on the path (la[0]: over all of it), by doubling
        for (int j = lane; j < n; j += 32)
            if (on >> j & 1)
                la[__popcll(on & ((1ull << j) - 1))] = {clamp_log_a(a.log_a[static_cast<int64_t>(first + j) * a.hv + h]), 0.0f};
        if (lane == 0) la[np] = {0.0f, 0.0f};
        __syncwarp();
        for (int step = 1; step < np; step <<= 1) {
            Sum2 x[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int j = lane + 32 * m;
                if (j < np) x[m] = j + step < np ? sum2(la[j], la[j + step]) : la[j];
            }
            __syncwarp();
#pragma unroll
            for (int m = 0; m < 2; ++m)
                if (lane + 32 * m < np) la[lane + 32 * m] = x[m];
            __syncwarp();
        }
        for (int j = lane; j <= np; j += 32) w[j] = expf(la[j].hi + la[j].lo);
    }
    __syncthreads();
    const float grow = np ? w[0] : 1.0f;
    float f[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[j][e] = __uint_as_float(v[j][e]) * grow;
    for (int t = 0; t < np; ++t) {
        const float* from = cm + t * (D + ROWS);
        const float4 x = *reinterpret_cast<const float4*>(from + col), y = *reinterpret_cast<const float4*>(from + col + 4);
        const float k[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        const float after = w[t + 1];
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const float u = from[D + row + j * STEP] * after;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[j][e] = fmaf(u, k[e], f[j][e]);
        }
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = __float_as_uint(f[j][e]);
        if (GDN_IN_RANGE(g_draft_error, s < a.d.n_seqs && h < a.hv && row + j * STEP < D - row0))
            store_state<WIDE>(a.state_out + base + j * STEP * D, v[j]);
    }
}

template <int D, int CH, bool WIDE>
static cudaError_t commit_launch(const CommitArgs& a, cudaStream_t st) {
    constexpr int STEP = CM_THREADS / (D / 8), PARTS = D / (STEP * CH);
    constexpr int TOKEN = (D + STEP * CH) * 4;
    static PerDeviceOnce once;
    once.run([](int) { cudaFuncSetAttribute(commit_kernel<D, CH, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, GDN_MAX_NEW * TOKEN); });
    const int conv_blocks = a.tail_in ? (a.c_conv + CM_CHANNELS * CM_THREADS - 1) / (CM_CHANNELS * CM_THREADS) : 0;
    return launch_dependent(commit_kernel<D, CH, WIDE>, dim3(a.hv * PARTS + conv_blocks, a.d.n_seqs), dim3(CM_THREADS),
                            static_cast<size_t>(a.d.max_new * TOKEN), st, a);
}

cudaError_t launch_delta_commit(const gdn_layer& L, const DraftTokens& d, const uint16_t* qkv, const float* log_a, const float* delta,
                                const int32_t* node, const float* state_in, float* state_out, const uint16_t* qkvz, int64_t ld_qkvz,
                                const float* tail_in, float* tail_out, cudaStream_t st) {
    CommitArgs a;
    a.d = d;
    a.qkv = qkv;
    a.log_a = log_a;
    a.delta = delta;
    a.node = node;
    a.state_in = state_in;
    a.state_out = state_out;
    a.qkvz = qkvz;
    a.ld_qkvz = ld_qkvz;
    a.tail_in = tail_in;
    a.tail_out = tail_out;
    a.hv = L.n_v_heads;
    a.ratio = L.n_v_heads / L.n_qk_heads;
    a.c_qk = L.n_qk_heads * L.dk;
    a.c_conv = 2 * a.c_qk + L.n_v_heads * L.dv;
    const bool wide = on_32_bytes(state_in) && on_32_bytes(state_out);
    if (L.dk == 64) return wide ? commit_launch<64, 2, true>(a, st) : commit_launch<64, 2, false>(a, st);
    // 32 rows of a head to a block while there are few heads, else 64 (paths of up to 32 tokens, us with 32 and with 64: 32
    // heads 3.1 and 3.8, 160 5.8 and 6.4, 192 7.0 and 6.8, 224 8.6 and 7.9, 512 18.3 and 16.9, 2048 60 and 53; 128 rows leave
    // an SM two blocks: 68)
    if (a.hv * d.n_seqs < 192) return wide ? commit_launch<128, 2, true>(a, st) : commit_launch<128, 2, false>(a, st);
    return wide ? commit_launch<128, 4, true>(a, st) : commit_launch<128, 4, false>(a, st);
}

int* draft_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_draft_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

int* draft_skipped_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_draft_skipped) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdn
