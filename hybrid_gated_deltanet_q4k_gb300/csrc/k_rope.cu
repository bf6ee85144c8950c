// Rotary positions of the full-attention layers' queries and keys.
//
// Pair i of a head turns by pos * f_i: (a, b) -> amp (a cos - b sin, a sin + b
// cos).  The table holds f_i / 2 pi as a 64-bit fraction of a turn, so the
// product pos * step wraps modulo one turn by itself: the angle of position
// 2^31 is reduced exactly, with no 64-bit floating point and no argument
// reduction, and its top 32 bits go to sincospif (absolute error below 3e-7).
//
// Bound by memory: every element is read and written once (in place, only the
// rotated ones).  A CTA takes a run of (token, head) rows and computes the
// sines and cosines of its tokens once, into shared memory, for all of their
// heads, while its loads are under way.  A prompt of 32768 tokens, 16 + 4 heads
// of 256 with 64 rotated: 98 us, 6.85 TB/s, the rate of a copy; 5001 tokens out
// of a fused projection, 32 + 8 heads of 128 rotated whole: 20 us, 5.2 TB/s.
#include "common.cuh"

namespace gdn {

static __device__ int g_rope_error;   // index checks of the debug build

struct RopeArgs {
    const int32_t* pos;
    int64_t n;
    int d, hq, hk;
    const uint16_t* q;
    uint16_t* qo;
    const uint16_t* k;
    uint16_t* ko;
    int64_t ld_q, ld_qo, ld_k, ld_ko;
    int q_copy, k_copy;   // 1: pass-through elements are copied (0: in place)
};

constexpr int ROPE_THREADS = 256;

__device__ __forceinline__ float2 rope_cs(uint64_t step, int pos, float amp) {
    const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31
    return make_float2(c * amp, s * amp);
}

__device__ __forceinline__ void rope_pair(uint16_t a, uint16_t b, float2 cs, uint16_t& x, uint16_t& y) {
    const float fa = bf16_bits_to_float(a), fb = bf16_bits_to_float(b);
    x = float_to_bf16_bits(fa * cs.x - fb * cs.y);
    y = float_to_bf16_bits(fa * cs.y + fb * cs.x);
}

// Where pair p of a token has its sine and cosine in the table: eight threads
// read sixteen bytes each of pairs 8c + 2e, 64 bytes apart, which the exchange
// of e puts into different banks.
__device__ __forceinline__ int rope_at(int c, int e) { return 8 * c + 2 * (e ^ ((c >> 1) & 3)); }

// Rows whose parts are whole 16-byte pieces: a unit is 16 elements of a row,
// eight pairs (half layout: 8 elements at 8c and 8 at rot/2 + 8c; interleaved:
// 16 together) or 16 that pass through.  blockDim = (units of a row, rows);
// each thread takes K rows, all loads first.  WIDE: every row starts on 32
// bytes, and 16 elements that lie together move in one access.
template <int K, bool WIDE>
__global__ void __launch_bounds__(ROPE_THREADS, 4)
rope_vec_kernel(const __grid_constant__ gdn_rope_table t, const __grid_constant__ RopeArgs a) {
    extern __shared__ float2 table[];   // [tokens of the run][rot / 2]
    pdl_wait();
    pdl_trigger();
    const int half = t.rot / 2, heads = a.hq + a.hk, c = threadIdx.x;
    const int64_t rows = a.n * heads, r0 = static_cast<int64_t>(blockIdx.x) * (blockDim.y * K);
    const int64_t t0 = r0 / heads;
    const int first = static_cast<int>(r0 - t0 * heads), n_rows = static_cast<int>(min(static_cast<int64_t>(blockDim.y) * K, rows - r0));
    const int toks = (first + n_rows - 1) / heads + 1;
    const bool turns = c < t.rot / 16, split = turns && t.layout == GDN_ROPE_HALF;
    const int ea = split ? 8 * c : 16 * c, eb = split ? half + 8 * c : ea + 8;
    uint32_t v[K][8];
    int tk[K], hd[K];   // the row's token in the run (-1: nothing to do) and head
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = k * blockDim.y + threadIdx.y;
        tk[k] = -1;
        if (i >= n_rows) continue;
        const int r = first + i, tl = r / heads, h = r - tl * heads;
        const bool is_q = h < a.hq;
        if (!turns && !(is_q ? a.q_copy : a.k_copy)) continue;
        const int64_t tok = t0 + tl;
        if (!GDN_IN_RANGE(g_rope_error, tok < a.n && ea + 8 <= a.d && eb + 8 <= a.d)) continue;
        tk[k] = tl;
        hd[k] = h;
        const uint16_t* src = is_q ? a.q + tok * a.ld_q + h * a.d : a.k + tok * a.ld_k + (h - a.hq) * a.d;
        if (WIDE && !split) {
            load32(src + ea, v[k]);
        } else {
            const uint4 va = *reinterpret_cast<const uint4*>(src + ea), vb = *reinterpret_cast<const uint4*>(src + eb);
            v[k][0] = va.x, v[k][1] = va.y, v[k][2] = va.z, v[k][3] = va.w;
            v[k][4] = vb.x, v[k][5] = vb.y, v[k][6] = vb.z, v[k][7] = vb.w;
        }
    }
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < toks * half; i += blockDim.x * blockDim.y) {
        const int tok = i / half, p = i - tok * half;
        table[tok * half + rope_at(p / 8, p % 8 / 2) + p % 2] = rope_cs(t.step[p], a.pos[t0 + tok], t.amp);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (tk[k] < 0) continue;
        uint32_t(&x)[8] = v[k];
        if (turns) {
            const float2* cs = table + tk[k] * half;
            if (split) {   // x[e] and x[4 + e] hold pairs 2e, 2e + 1
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 w = *reinterpret_cast<const float4*>(cs + rope_at(c, e));
                    uint16_t a0, a1, b0, b1;
                    rope_pair(static_cast<uint16_t>(x[e]), static_cast<uint16_t>(x[4 + e]), make_float2(w.x, w.y), a0, b0);
                    rope_pair(static_cast<uint16_t>(x[e] >> 16), static_cast<uint16_t>(x[4 + e] >> 16), make_float2(w.z, w.w), a1, b1);
                    x[e] = a0 | (static_cast<uint32_t>(a1) << 16);
                    x[4 + e] = b0 | (static_cast<uint32_t>(b1) << 16);
                }
            } else {       // x[e] is pair e
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 w = *reinterpret_cast<const float4*>(cs + rope_at(c, e / 2));
                    uint16_t a0, b0;
                    rope_pair(static_cast<uint16_t>(x[e]), static_cast<uint16_t>(x[e] >> 16), make_float2(w.x, w.y), a0, b0);
                    x[e] = a0 | (static_cast<uint32_t>(b0) << 16);
                    rope_pair(static_cast<uint16_t>(x[e + 1]), static_cast<uint16_t>(x[e + 1] >> 16), make_float2(w.z, w.w), a0, b0);
                    x[e + 1] = a0 | (static_cast<uint32_t>(b0) << 16);
                }
            }
        }
        const int64_t tok = t0 + tk[k];
        const int h = hd[k];
        uint16_t* dst = h < a.hq ? a.qo + tok * a.ld_qo + h * a.d : a.ko + tok * a.ld_ko + (h - a.hq) * a.d;
        if (WIDE && !split) {
            store32(dst + ea, x);
        } else {
            *reinterpret_cast<uint4*>(dst + ea) = make_uint4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<uint4*>(dst + eb) = make_uint4(x[4], x[5], x[6], x[7]);
        }
    }
}

// Any even sizes and any alignment: one thread per pair or pass-through
// element, a CTA per token.
__global__ void __launch_bounds__(ROPE_THREADS)
rope_kernel(const __grid_constant__ gdn_rope_table t, const __grid_constant__ RopeArgs a) {
    __shared__ float2 cs[GDN_ROPE_MAX_PAIRS];
    pdl_wait();
    pdl_trigger();
    const int64_t tok = blockIdx.x;
    const int half = t.rot / 2, per = half + a.d - t.rot;
    const int pos = a.pos[tok];
    for (int i = threadIdx.x; i < half; i += ROPE_THREADS) cs[i] = rope_cs(t.step[i], pos, t.amp);
    __syncthreads();
    for (int u = threadIdx.x; u < (a.hq + a.hk) * per; u += ROPE_THREADS) {
        const int h = u / per, i = u - h * per;
        const bool is_q = h < a.hq;
        const uint16_t* src = is_q ? a.q + tok * a.ld_q + h * a.d : a.k + tok * a.ld_k + (h - a.hq) * a.d;
        uint16_t* dst = is_q ? a.qo + tok * a.ld_qo + h * a.d : a.ko + tok * a.ld_ko + (h - a.hq) * a.d;
        if (!GDN_IN_RANGE(g_rope_error, tok < a.n && h < a.hq + a.hk)) continue;
        if (i < half) {
            const int ia = t.layout == GDN_ROPE_HALF ? i : 2 * i, ib = t.layout == GDN_ROPE_HALF ? i + half : 2 * i + 1;
            uint16_t x, y;
            rope_pair(src[ia], src[ib], cs[i], x, y);
            dst[ia] = x;
            dst[ib] = y;
        } else if (is_q ? a.q_copy : a.k_copy) {
            dst[t.rot + i - half] = src[t.rot + i - half];
        }
    }
}

cudaError_t launch_rope(const gdn_rope_table& t, const int32_t* pos, int64_t n, int d, const uint16_t* q, int64_t ld_q,
                        int hq, uint16_t* qo, int64_t ld_qo, const uint16_t* k, int64_t ld_k, int hk, uint16_t* ko,
                        int64_t ld_ko, cudaStream_t st) {
    const RopeArgs a{pos, n, d, hq, hk, q, qo, k, ko, ld_q, ld_qo, ld_k, ld_ko, q != qo, k != ko};
    uintptr_t at = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(qo) | static_cast<uintptr_t>(2 * (ld_q | ld_qo));
    if (hk) at |= reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(ko) | static_cast<uintptr_t>(2 * (ld_k | ld_ko));
    const int units = d / 16;
    if (t.rot % 16 || d % 16 || at % 16) {
        return launch_dependent(rope_kernel, dim3(static_cast<unsigned>(n)), dim3(ROPE_THREADS), 0, st, t, a);
    }
    const dim3 block(static_cast<unsigned>(units), static_cast<unsigned>(ROPE_THREADS / units));
    const int64_t rows = n * (hq + hk);
    auto smem = [&](int kk) { return ((block.y * kk - 1) / (hq + hk) + 2) * (t.rot / 2) * sizeof(float2); };
    auto grid = [&](int kk) { return static_cast<unsigned>((rows + block.y * kk - 1) / (block.y * kk)); };
    const bool wide = at % 32 == 0;
    const auto launch = [&](void (*kernel)(const gdn_rope_table, const RopeArgs), int kk) {
        return launch_dependent(kernel, dim3(grid(kk)), block, smem(kk), st, t, a);
    };
    // rows a thread: as many as keep four blocks per SM busy (all loads of a thread are in flight at once)
    if (smem(4) <= 40960 && grid(4) >= 608) return launch(wide ? rope_vec_kernel<4, true> : rope_vec_kernel<4, false>, 4);
    if (smem(2) <= 40960 && grid(2) >= 608) return launch(wide ? rope_vec_kernel<2, true> : rope_vec_kernel<2, false>, 2);
    return launch(wide ? rope_vec_kernel<1, true> : rope_vec_kernel<1, false>, 1);
}

int* rope_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_rope_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdn
