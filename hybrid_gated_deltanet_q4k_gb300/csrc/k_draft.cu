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
    int c_conv, n_heads, n_qk_norm, n_q, hv, head_blocks;
    bool wide;             // rows of qkvz start on 16 bytes
    float eps, q_scale;
};

constexpr int CT_WARPS = 8;
constexpr int CT_TOKENS = 32;              // most tokens of a block

// Block (token run, head group, sequence): a warp per head, a thread for 8 of its
// channels, so that 2 (d = 128) or 4 tokens run side by side, CT_STEP of each in
// flight.  The taps' weights stay in registers; a raw input is read by up to four
// tokens, from L1 after the first.  The last slice of y computes the gates.
template <int D>
__global__ void __launch_bounds__(CT_WARPS * 32, 2) conv_tree_kernel(const __grid_constant__ ConvTreeArgs a) {
    constexpr int LANES = D / 8, SIDE = 32 / LANES, STEP = 2;
    __shared__ int at[CT_TOKENS][4];       // rows of the taps from the sequence's first, oldest first; -1, -2, -3: the conv state
    __shared__ float tail[CT_WARPS * D * 3];
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.z, tid = threadIdx.x;
    int first;
    const int n = draft_range(a.d, s, first, g_draft_skipped);
    const int i0 = blockIdx.x * CT_TOKENS, i1 = min(n, i0 + CT_TOKENS);
    if (i0 >= i1) return;
    if (static_cast<int>(blockIdx.y) == a.head_blocks) {
        for (int e = tid; e < (i1 - i0) * a.hv; e += blockDim.x) {
            const int64_t t = first + i0 + e / a.hv;
            const int h = e % a.hv;
            if (GDN_IN_RANGE(g_draft_error, t < a.d.n_tokens))
                gate_values(a.ba[t * a.ld_ba + h], a.ba[t * a.ld_ba + a.hv + h], a.A_log[h], a.dt_bias[h], a.log_a[t * a.hv + h],
                            a.b[t * a.hv + h]);
        }
        return;
    }
    const int head0 = blockIdx.y * CT_WARPS, heads = min(CT_WARPS, a.n_heads - head0);
    const int head = head0 + (tid >> 5), lane = tid & 31, sub = lane % LANES, side = lane / LANES;
    float w[8][4];
    const int c0 = head * D + 8 * sub;
    if (head < a.n_heads) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float4 v = *reinterpret_cast<const float4*>(a.conv_w + static_cast<int64_t>(c0 + e) * 4);
            w[e][0] = v.x; w[e][1] = v.y; w[e][2] = v.z; w[e][3] = v.w;
        }
    }
    if (tid < i1 - i0) {
        int x = i0 + tid;
        at[tid][3] = x;
#pragma unroll
        for (int m = 2; m >= 0; --m) {
            x = x < 0 ? x - 1 : draft_parent(draft_ancestors(a.d, first, x));
            at[tid][m] = x;
        }
    }
    const float* old = a.tail + (static_cast<int64_t>(s) * a.c_conv + head0 * D) * 3;
    for (int e = tid; e < heads * D * 3; e += blockDim.x) tail[e] = old[e];
    __syncthreads();
    if (head >= a.n_heads) return;
    const bool norm = head < a.n_qk_norm;
    const float mul = head < a.n_q ? a.q_scale : 1.0f;
    const float* mine = tail + ((tid >> 5) * D + 8 * sub) * 3;
    const uint16_t* src = a.qkvz + static_cast<int64_t>(first) * a.ld_qkvz + c0;
    bool over = false;
    for (int i = i0 + side; i - side < i1; i += SIDE * STEP) {
        uint4 x[STEP][4];
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
            const int r = min(i + k * SIDE, i1 - 1) - i0;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int64_t row = max(at[r][m], 0);
                if (a.wide) {
                    x[k][m] = *reinterpret_cast<const uint4*>(src + row * a.ld_qkvz);
                } else {
                    const uint2 lo = *reinterpret_cast<const uint2*>(src + row * a.ld_qkvz), hi = *reinterpret_cast<const uint2*>(src + row * a.ld_qkvz + 4);
                    x[k][m] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
            const int r = min(i + k * SIDE, i1 - 1) - i0;
            float y[8], ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t u = reinterpret_cast<const uint32_t*>(&x[k][m])[e >> 1];
                    v[m] = __uint_as_float(e & 1 ? u & 0xffff0000u : u << 16);
                }
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    if (at[r][m] < 0) v[m] = mine[3 * e + 3 + at[r][m]];
                y[e] = conv4_silu(make_float4(w[e][0], w[e][1], w[e][2], w[e][3]), v[0], v[1], v[2], v[3]);
                ss = fmaf(y[e], y[e], ss);
            }
            if (norm) {
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float f = rsqrtf(ss + a.eps) * mul;
                over |= !(ss <= 3.0e38f);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= f;
            }
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf_nan(top, fabsf(y[e]));
            over |= !(top <= 65504.0f);
            const int64_t row = first + i + k * SIDE;
            if (i + k * SIDE < i1 && GDN_IN_RANGE(g_draft_error, row < a.d.n_tokens && c0 + 8 <= a.c_conv))
                *reinterpret_cast<uint4*>(a.out + row * a.c_conv + c0) =
                    make_uint4(f16x2_bits(y[0], y[1]), f16x2_bits(y[2], y[3]), f16x2_bits(y[4], y[5]), f16x2_bits(y[6], y[7]));
        }
    }
    if (over) atomicCAS(&g_draft_error, 0, static_cast<int>(ERR_RANGE));
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
    a.head_blocks = (a.n_heads + CT_WARPS - 1) / CT_WARPS;
    a.eps = L.eps_l2;
    a.q_scale = L.q_scale;
    a.wide = reinterpret_cast<uintptr_t>(qkvz) % 16 == 0 && ld_qkvz % 8 == 0;
    const dim3 grid((d.max_new + CT_TOKENS - 1) / CT_TOKENS, a.head_blocks + (L.gate_log_a ? 0 : 1), d.n_seqs);
    return launch_dependent(L.dk == 128 ? conv_tree_kernel<128> : conv_tree_kernel<64>, grid, dim3(CT_WARPS * 32), 0, st, a);
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
    int hv, ratio, c_qk, c_conv;
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

// Shared memory of delta_tree_kernel for np tokens (a multiple of 8) and a
// number of warps: byte offsets.
constexpr int DT_STAGE = 336;               // floats per warp, see the kernel
template <int D>
struct DeltaTreeSmem {
    int k, q, kk, qk, u, stage, anc, uni, g, up, eg, b, end;
    __host__ __device__ DeltaTreeSmem(int np, int warps) {
        k = 0;                              // fp16 rows in units of 16 bytes, unit x of row r at x ^ 4 (r & 1)
        q = k + np * D * 2;
        kk = q + np * D * 2;                // [j][i]: -e^{g_i - g_j} k_j . k_i, 0 where j is no ancestor of i
        qk = kk + np * np * 4;              // [j][i]: e^{g_i - g_j} k_j . q_i, where j is one or i itself
        u = qk + np * np * 4;               // per warp [token][16 rows]: v, then u
        stage = u + warps * np * 64;        // per warp: S_0 k and S_0 q of 8 tokens
        anc = stage + warps * DT_STAGE * 4;
        uni = anc + np * 8;                 // per block of 8 tokens: their ancestors before the block
        g = uni + 64;
        up = g + np * 8;
        eg = up + np * 4;
        b = eg + np * 4;
        end = b + np * 4;
    }
};

// A warp holds 16 rows of S_0 for the whole kernel; the rows of u and o follow
// from them alone, so the CTA's warps meet only for what all rows share, the
// decayed products of keys and queries.  S_0 is read once, 32 bytes a thread
// and row at a time, straight into operands of the tensor cores (the k index is
// permuted alike in both operands: thread t of a quad holds columns 8t .. 8t+7
// of each 32): each row times a power of two, split into two fp16 numbers, the
// second taken 2^11 times as large, so that 22 bits of it and more count.  Keys
// and queries are fp16 as they come.
//
// Tokens go in blocks of 8: the products with S_0 by mma, then what the block's
// ancestors before it add (one pass over the union of their bits), then the
// block itself, token by token.  Lane r and lane 16 + r work on row r, the
// first for u, the second for o.  A u that is not finite is kept out of the
// sums (0 times it would reach tokens that do not descend from it) and marks
// its descendants.
template <int D>
__global__ void __launch_bounds__(256, 2) delta_tree_kernel(const __grid_constant__ DeltaTreeArgs a) {
    constexpr int KB = D / 32;              // blocks of 32 columns
    constexpr int UNITS = D / 8;            // 16-byte units of a row of keys
    extern __shared__ __align__(16) unsigned char raw[];
    pdl_wait();
    pdl_trigger();
    const int warps = blockDim.x >> 5, parts = D / (16 * warps);
    const int h = blockIdx.x / parts, part = blockIdx.x % parts, s = blockIdx.y, hk = h / a.ratio;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    int first;
    const int n = draft_range(a.d, s, first, g_draft_skipped);
    if (n == 0) return;
    const int np = (n + 7) & ~7;
    const DeltaTreeSmem<D> at(np, warps);
    const int r0 = (part * warps + warp) * 16;              // the warp's rows
    uint32_t w0[KB][8], w1[KB][8];                          // rows g and g + 8
    {
        const float* S = a.state + ((static_cast<int64_t>(s) * a.hv + h) * D + r0 + g) * D + 8 * t;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            load32(S + 32 * b, w0[b]);
            load32(S + 8 * D + 32 * b, w1[b]);
        }
    }
    uint4* ks = reinterpret_cast<uint4*>(raw + at.k);
    uint4* qs = reinterpret_cast<uint4*>(raw + at.q);
    float* kk = reinterpret_cast<float*>(raw + at.kk);
    float* qk = reinterpret_cast<float*>(raw + at.qk);
    float* us = reinterpret_cast<float*>(raw + at.u) + warp * np * 16;
    float* stage = reinterpret_cast<float*>(raw + at.stage) + warp * DT_STAGE;
    uint64_t* anc = reinterpret_cast<uint64_t*>(raw + at.anc);
    uint64_t* uni = reinterpret_cast<uint64_t*>(raw + at.uni);
    Sum2* gs = reinterpret_cast<Sum2*>(raw + at.g);
    int* ups = reinterpret_cast<int*>(raw + at.up);
    float* eg = reinterpret_cast<float*>(raw + at.eg);
    float* bs = reinterpret_cast<float*>(raw + at.b);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int e = tid; e < np * UNITS; e += blockDim.x) {
        const int i = e / UNITS, x = e % UNITS;
        const uint16_t* row = a.qkv + static_cast<int64_t>(first + i) * a.c_conv + hk * D + 8 * x;
        const int to = i * UNITS + (x ^ (4 * (i & 1)));
        qs[to] = i < n ? *reinterpret_cast<const uint4*>(row) : zero;
        ks[to] = i < n ? *reinterpret_cast<const uint4*>(row + a.c_qk) : zero;
    }
    for (int e = lane; e < 2 * np; e += 32) {               // v of the warp's rows, 8 at a time
        const int i = e >> 1, r = 8 * (e & 1);
        const uint4 v = i < n ? *reinterpret_cast<const uint4*>(a.qkv + static_cast<int64_t>(first + i) * a.c_conv + 2 * a.c_qk + h * D + r0 + r)
                              : zero;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[m]));
            us[i * 16 + r + 2 * m] = f.x;
            us[i * 16 + r + 2 * m + 1] = f.y;
        }
    }
    if (warp == 0) {
        // sums along the paths by doubling: after a round that looked 2^m tokens
        // back, a token holds the sum of the nearest 2^(m + 1) of its path
        Sum2 sum[2];
        int up[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int i = lane + 32 * m;
            const bool in = i < n;
            const uint64_t x = in ? draft_ancestors(a.d, first, i) : 0ull;
            sum[m] = {in ? clamp_log_a(a.log_a[static_cast<int64_t>(first + i) * a.hv + h]) : 0.0f, 0.0f};
            up[m] = draft_parent(x);
            if (i < np) {
                anc[i] = x;
                bs[i] = in ? a.b[static_cast<int64_t>(first + i) * a.hv + h] : 0.0f;
                gs[i] = sum[m];
                ups[i] = up[m];
            }
        }
        __syncwarp();
        for (int step = 1; step < n; step <<= 1) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
                if (up[m] >= 0) {
                    sum[m] = sum2(sum[m], gs[up[m]]);
                    up[m] = ups[up[m]];
                }
            __syncwarp();
#pragma unroll
            for (int m = 0; m < 2; ++m)
                if (lane + 32 * m < np) {
                    gs[lane + 32 * m] = sum[m];
                    ups[lane + 32 * m] = up[m];
                }
            __syncwarp();
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
            if (lane + 32 * m < np) eg[lane + 32 * m] = expf(sum[m].hi + sum[m].lo);
        if (lane < np / 8) {
            uint64_t x = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) x |= anc[8 * lane + c];
            uni[lane] = x & ((1ull << 8 * lane) - 1);
        }
    }
    __syncthreads();
    const int sw = t ^ (4 * (g & 1));       // the unit of columns 8t .. 8t+7 in rows of g's parity
    const int nb = np / 8;
    // products of the tokens, 16 tokens j by 8 tokens i, with keys and with queries
    for (int x = warp; x < ((np + 15) / 16) * nb * 2; x += warps) {
        const int side = x & 1, bi = (x >> 1) % nb, jt = (x >> 1) / nb;
        if (16 * jt > 8 * bi + 7) continue;
        float c[4] = {};
        const uint4* other = side ? qs : ks;
        const int j0 = 16 * jt + g;
        const bool second = 16 * jt + 8 < np;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            const int unit = (4 * b) ^ sw;
            const uint4 x0 = ks[j0 * UNITS + unit], x1 = second ? ks[(j0 + 8) * UNITS + unit] : zero;
            const uint4 y = other[(8 * bi + g) * UNITS + unit];
            mma_f16(c, x0.x, x1.x, x0.y, x1.y, y.x, y.y);
            mma_f16(c, x0.z, x1.z, x0.w, x1.w, y.z, y.w);
        }
        float* out = side ? qk : kk;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int j = j0 + 8 * (m >> 1), i = 8 * bi + 2 * t + (m & 1);
            if (j >= np) continue;
            const bool on = (anc[i] >> j & 1) || (side && i == j);
            const float w = expf((gs[i].hi - gs[j].hi) + (gs[i].lo - gs[j].lo));
            out[j * np + i] = on ? (side ? w : -w) * c[m] : 0.0f;
        }
    }
    // S_0's operands: row maxima to [2^13, 2^14), then high and low parts
    uint32_t h0[KB][4], h1[KB][4], l0[KB][4], l1[KB][4];
    float back[2];
    {
        const auto split = [&](const uint32_t (&w)[KB][8], uint32_t (&hi)[KB][4], uint32_t (&lo)[KB][4], float& undo) {
            uint32_t top = 0;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, w[b][e] & 0x7fffffffu);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t e8 = min(max(top >> 23, 14u), 254u);
            const float scale = __uint_as_float((267u - e8) << 23);
            undo = __uint_as_float((e8 - 13u) << 23);
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = __uint_as_float(w[b][2 * e]) * scale, y = __uint_as_float(w[b][2 * e + 1]) * scale;
                    const __half2 hh = __floats2half2_rn(x, y);
                    const float2 f = __half22float2(hh);
                    hi[b][e] = *reinterpret_cast<const uint32_t*>(&hh);
                    lo[b][e] = f16x2_bits((x - f.x) * 2048.0f, (y - f.y) * 2048.0f);
                }
        };
        split(w0, h0, l0, back[0]);
        split(w1, h1, l1, back[1]);
    }
    __syncthreads();
    const int row = lane & 15, side = lane >> 4;
    const float* coef = side ? qk : kk;
    uint64_t bad = 0;                       // tokens whose u in this row is not finite
    bool over = false;
    float* du = a.delta + (static_cast<int64_t>(first) * a.hv + h) * D + r0 + row;
    uint16_t* dof = a.o + (static_cast<int64_t>(first) * a.hv + h) * D + r0 + row;
    for (int bi = 0; bi < nb; ++bi) {
#pragma unroll
        for (int sd = 0; sd < 2; ++sd) {
            float c[4] = {}, d[4] = {};
            const uint4* other = sd ? qs : ks;
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                const uint4 y = other[(8 * bi + g) * UNITS + ((4 * b) ^ sw)];
                mma_f16(c, h0[b][0], h1[b][0], h0[b][1], h1[b][1], y.x, y.y);
                mma_f16(d, l0[b][0], l1[b][0], l0[b][1], l1[b][1], y.x, y.y);
                mma_f16(c, h0[b][2], h1[b][2], h0[b][3], h1[b][3], y.z, y.w);
                mma_f16(d, l0[b][2], l1[b][2], l0[b][3], l1[b][3], y.z, y.w);
            }
            // token c of the block at 20 c: the writers' banks differ, and so do the two halves of the readers'
#pragma unroll
            for (int m = 0; m < 4; ++m)
                stage[176 * sd + 20 * (2 * t + (m & 1)) + g + 8 * (m >> 1)] = fmaf(d[m], 0x1p-11f, c[m]) * back[m >> 1];
        }
        __syncwarp();
        float acc[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float x = stage[176 * side + 20 * c + row] * eg[8 * bi + c];
            acc[c] = side ? x : us[(8 * bi + c) * 16 + row] - x;
        }
        for (uint64_t m = uni[bi]; m; m &= m - 1) {
            const int j = __ffsll(static_cast<long long>(m)) - 1;
            const float u = us[j * 16 + row];
            const float4 x = *reinterpret_cast<const float4*>(coef + j * np + 8 * bi);
            const float4 y = *reinterpret_cast<const float4*>(coef + j * np + 8 * bi + 4);
            acc[0] = fmaf(x.x, u, acc[0]);
            acc[1] = fmaf(x.y, u, acc[1]);
            acc[2] = fmaf(x.z, u, acc[2]);
            acc[3] = fmaf(x.w, u, acc[3]);
            acc[4] = fmaf(y.x, u, acc[4]);
            acc[5] = fmaf(y.y, u, acc[5]);
            acc[6] = fmaf(y.z, u, acc[6]);
            acc[7] = fmaf(y.w, u, acc[7]);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int i = 8 * bi + c;
            float u = acc[c] * bs[i];
            if (bad & anc[i]) u = __uint_as_float(0x7fffffffu);
            u = __shfl_sync(0xffffffffu, u, row);
            const bool fine = fabsf(u) <= 3.402823466e38f;
            const float v = fine ? u : 0.0f;
            if (!fine) bad |= 1ull << i;
            const float* cr = coef + i * np + 8 * bi;
#pragma unroll
            for (int e = c; e < 8; ++e) acc[e] = fmaf(cr[e], v, acc[e]);
            if (side == 0) us[i * 16 + row] = v;
            if (i < n && GDN_IN_RANGE(g_draft_error, first + i < a.d.n_tokens)) {
                const int64_t to = static_cast<int64_t>(i) * a.hv * D;
                if (side == 0) {
                    du[to] = u;
                } else {
                    const float o = bad & (anc[i] | 1ull << i) ? __uint_as_float(0x7fffffffu) : acc[c];
                    over |= !(fabsf(o) <= 65504.0f);
                    dof[to] = __half_as_ushort(__float2half_rn(o));
                }
            }
        }
        __syncwarp();
    }
    if (over) atomicCAS(&g_draft_error, 0, static_cast<int>(ERR_RANGE));
}

template <int D>
static cudaError_t delta_tree_launch(const DeltaTreeArgs& a, cudaStream_t st) {
    const int np = (a.d.max_new + 7) & ~7;
    static PerDeviceOnce once;
    once.run([](int) {
        cudaFuncSetAttribute(delta_tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, DeltaTreeSmem<D>(GDN_MAX_NEW, 8).end);
    });
    // the whole head in a CTA, or its rows in several where that leaves SMs without one
    int warps = D / 16;
    while (warps > 2 && a.hv * a.d.n_seqs * (D / 16 / warps) < 152) warps >>= 1;
    return launch_dependent(delta_tree_kernel<D>, dim3(a.hv * (D / 16 / warps), a.d.n_seqs), dim3(32 * warps),
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
    a.c_conv = 2 * a.c_qk + L.n_v_heads * L.dv;
    return L.dk == 128 ? delta_tree_launch<128>(a, st) : delta_tree_launch<64>(a, st);
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
    const uint16_t* qkvz;    // null: no conv state
    int64_t ld_qkvz;
    const float* tail_in;
    float* tail_out;
    int hv, ratio, c_qk, c_conv;
};

constexpr int CM_THREADS = 256;

// The accepted token of sequence s, -1 where there is none; n: its tokens.
__device__ __forceinline__ int commit_node(const CommitArgs& a, int s, int n) {
    const int node = a.node[s];
    if (node >= -1 && node < n) return node;
    atomicCAS(&g_draft_skipped, 0, static_cast<int>(ERR_INDEX));
    return -1;
}

// Block (rows of a value head, sequence): a thread has 8 columns of CH rows, all
// of them loaded before it is known what is accepted (the loads are what bounds
// the kernel); then a rank-1 update per token of the path, from shared memory.
// Blocks past the heads: the conv state of CM_THREADS channels.
template <int D, int CH>
__global__ void __launch_bounds__(CM_THREADS, 2) commit_kernel(const __grid_constant__ CommitArgs a) {
    constexpr int COLS = D / 8, STEP = CM_THREADS / COLS, PARTS = D / (STEP * CH);
    extern __shared__ __align__(16) float cm[];        // k [path][D], then u of the block's rows [path][STEP * CH]
    __shared__ int path[GDN_MAX_NEW];
    __shared__ Sum2 la[GDN_MAX_NEW + 1];
    __shared__ float w[GDN_MAX_NEW + 1];
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    int first;
    if (static_cast<int>(blockIdx.x) >= a.hv * PARTS) {
        const int n = draft_range(a.d, s, first, g_draft_skipped), node = commit_node(a, s, n);
        const int c = (blockIdx.x - a.hv * PARTS) * CM_THREADS + tid;
        if (c >= a.c_conv) return;
        const float* in = a.tail_in + (static_cast<int64_t>(s) * a.c_conv + c) * 3;
        float x[3];
        int at = node;
#pragma unroll
        for (int m = 2; m >= 0; --m) {
            // at: a token, or -1, -2, -3: the old state from its newest entry on
            x[m] = at < 0 ? in[3 + at] : bf16_bits_to_float(a.qkvz[static_cast<int64_t>(first + at) * a.ld_qkvz + c]);
            at = at < 0 ? at - 1 : draft_parent(draft_ancestors(a.d, first, at));
        }
        float* out = a.tail_out + (static_cast<int64_t>(s) * a.c_conv + c) * 3;
#pragma unroll
        for (int m = 0; m < 3; ++m) out[m] = x[m];
        return;
    }
    const int h = blockIdx.x / PARTS, row0 = blockIdx.x % PARTS * (STEP * CH), hk = h / a.ratio;
    const int col = tid % COLS * 8, row = tid / COLS;
    const int64_t base = ((static_cast<int64_t>(s) * a.hv + h) * D + row0 + row) * D + col;
    uint32_t v[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) load32(a.state_in + base + j * STEP * D, v[j]);
    const int n = draft_range(a.d, s, first, g_draft_skipped), node = commit_node(a, s, n);
    const uint64_t on = node < 0 ? 0ull : draft_ancestors(a.d, first, node) | 1ull << node;
    const int np = __popcll(on);
    if (tid < 32) {
        // the sums of log a over what follows a token on the path (la[0]: over all of it), by doubling
        for (int j = lane; j < n; j += 32)
            if (on >> j & 1) {
                const int at = __popcll(on & ((1ull << j) - 1));
                path[at] = j;
                la[at] = {clamp_log_a(a.log_a[static_cast<int64_t>(first + j) * a.hv + h]), 0.0f};
            }
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
    float* ks = cm;
    float* us = cm + np * D;
    for (int e = tid; e < np * COLS; e += CM_THREADS) {
        const int64_t t = first + path[e / COLS];
        const uint4 x = *reinterpret_cast<const uint4*>(a.qkv + t * a.c_conv + a.c_qk + hk * D + e % COLS * 8);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[m]));
            *reinterpret_cast<float2*>(ks + e * 8 + 2 * m) = f;
        }
    }
    for (int e = tid; e < np * STEP * CH; e += CM_THREADS) {
        const int j = e / (STEP * CH), r = e % (STEP * CH);
        us[e] = w[j + 1] * a.delta[((first + path[j]) * static_cast<int64_t>(a.hv) + h) * D + row0 + r];
    }
    __syncthreads();
    const float grow = np ? w[0] : 1.0f;
    float f[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[j][e] = __uint_as_float(v[j][e]) * grow;
    for (int t = 0; t < np; ++t) {
        const float4 x = *reinterpret_cast<const float4*>(ks + t * D + col), y = *reinterpret_cast<const float4*>(ks + t * D + col + 4);
        const float k[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const float u = us[t * STEP * CH + row + j * STEP];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[j][e] = fmaf(u, k[e], f[j][e]);
        }
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = __float_as_uint(f[j][e]);
        store32(a.state_out + base + j * STEP * D, v[j]);
    }
}

template <int D, int CH>
static cudaError_t commit_launch(const CommitArgs& a, cudaStream_t st) {
    constexpr int STEP = CM_THREADS / (D / 8), PARTS = D / (STEP * CH);
    constexpr int TOKEN = (D + STEP * CH) * 4;
    static PerDeviceOnce once;
    once.run([](int) { cudaFuncSetAttribute(commit_kernel<D, CH>, cudaFuncAttributeMaxDynamicSharedMemorySize, GDN_MAX_NEW * TOKEN); });
    const int conv_blocks = a.qkvz ? (a.c_conv + CM_THREADS - 1) / CM_THREADS : 0;
    return launch_dependent(commit_kernel<D, CH>, dim3(a.hv * PARTS + conv_blocks, a.d.n_seqs), dim3(CM_THREADS),
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
    // a quarter of a head's rows to a block where whole heads leave SMs without one
    if (L.dk == 64) return commit_launch<64, 2>(a, st);
    return a.hv * d.n_seqs < 2 * 152 ? commit_launch<128, 2>(a, st) : commit_launch<128, 8>(a, st);
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
