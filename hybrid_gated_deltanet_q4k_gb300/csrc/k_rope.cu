// Rotary positions of the full-attention layers' queries and keys.
//
// Pair i of a head turns by pos * f_i: (a, b) -> amp (a cos - b sin, a sin + b
// cos).  The table holds f_i / 2 pi as a 64-bit fraction of a turn, so the
// product pos * step wraps modulo one turn by itself: the angle of position
// 2^31 is reduced exactly, with no 64-bit floating point and no argument
// reduction, and its top 32 bits go to sincospif (absolute error below 3e-7).
//
// Bound by memory: every element is read and written once (in place, only the
// rotated ones).  One CTA per token computes the token's rot/2 sines and
// cosines once into shared memory for all of its heads.
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

// One thread per pair or pass-through element.
__global__ void __launch_bounds__(ROPE_THREADS)
rope_kernel(const __grid_constant__ gdn_rope_table t, const __grid_constant__ RopeArgs a) {
    __shared__ float2 cs[GDN_ROPE_MAX_PAIRS];
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
    rope_kernel<<<static_cast<unsigned>(n), ROPE_THREADS, 0, st>>>(t, a);
    return cudaGetLastError();
}

int read_and_clear_rope_error() {
    int v = 0, z = 0;
    cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(int));
    if (v) cudaMemcpyToSymbol(g_rope_error, &z, sizeof(int));
    return v;
}

}  // namespace gdn
