// The paged key/value cache: rows quantised as they are stored, and read back.
//
// A row is one (token, head): int8 codes with scale amax/127, or e4m3 codes
// with scale amax/448, in the IEEE fp32 steps of the activation quantiser
// (scale = fl(amax / T), code = rne(fl(x / scale))).  Bound by memory: a store
// reads 2 bytes per element and writes 1 (2 for bf16), a fetch the reverse.
#include "common.cuh"
#include "qk_decode.cuh"

#include <cuda_fp8.h>

namespace gdn {

static __device__ int g_kv_error;   // a row or slot out of range

struct KvArgs {
    int heads, page;
    int64_t n_slots;     // n_pages * page
    void *ck, *cv;
    float *sk, *sv;
    uint16_t *k, *v;     // read only in a store
    int64_t ld_k, ld_v, n_rows;
    const int32_t* rows;
    const int64_t* slots;
    int64_t n;
};

constexpr int KV_THREADS = 256;

// The code of x by the IEEE divide (scale 0 or a NaN quotient: 0).
__device__ __forceinline__ uint8_t e4m3_code(float x, float s) {
    const float y = s == 0.0f ? 0.0f : __fdiv_rn(x, s);
    return y != y ? 0 : static_cast<uint8_t>(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3));
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// One warp per row.
template <int D, int T>
__global__ void __launch_bounds__(KV_THREADS) kv_write_kernel(const __grid_constant__ KvArgs a) {
    const int64_t r = (static_cast<int64_t>(blockIdx.x) * KV_THREADS + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t tok = r / (2 * a.heads);
    if (tok >= a.n) return;
    const int hs = static_cast<int>(r - tok * 2 * a.heads), h = hs >> 1, side = hs & 1;
    const int64_t row = a.rows ? a.rows[tok] : tok, slot = a.slots[tok];
    if (slot < 0) return;
    if (row < 0 || row >= a.n_rows || slot >= a.n_slots) {
        if (lane == 0) atomicCAS(&g_kv_error, 0, static_cast<int>(ERR_INDEX));
        return;
    }
    const uint16_t* src = (side ? a.v + row * a.ld_v : a.k + row * a.ld_k) + h * D;
    const int64_t cr = ((slot / a.page) * a.heads + h) * a.page + slot % a.page;
    float x[D / 32], amax = 0.0f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
        x[e] = bf16_bits_to_float(src[lane + 32 * e]);
        amax = fmaxf(amax, fabsf(x[e]));
    }
    void* c = side ? a.cv : a.ck;
    if (T == GDN_KV_BF16) {
#pragma unroll
        for (int e = 0; e < D / 32; ++e) static_cast<uint16_t*>(c)[cr * D + lane + 32 * e] = src[lane + 32 * e];
        return;
    }
    amax = warp_max(amax);
    const float s = __fdiv_rn(amax, T == GDN_KV_I8 ? 127.0f : 448.0f);
    if (lane == 0) (side ? a.sv : a.sk)[cr] = s;
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
        static_cast<uint8_t*>(c)[cr * D + lane + 32 * e] =
            T == GDN_KV_I8 ? static_cast<uint8_t>(static_cast<int8_t>(qcode_value(qcode_exact(x[e], s)))) : e4m3_code(x[e], s);
}

template <int D, int T>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const __grid_constant__ KvArgs a) {
    const int64_t r = (static_cast<int64_t>(blockIdx.x) * KV_THREADS + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t tok = r / (2 * a.heads);
    if (tok >= a.n) return;
    const int hs = static_cast<int>(r - tok * 2 * a.heads), h = hs >> 1, side = hs & 1;
    const int64_t slot = a.slots[tok];
    uint16_t* dst = (side ? a.v + tok * a.ld_v : a.k + tok * a.ld_k) + h * D;
    if (slot < 0 || slot >= a.n_slots) {
        if (slot >= 0 && lane == 0) atomicCAS(&g_kv_error, 0, static_cast<int>(ERR_INDEX));
#pragma unroll
        for (int e = 0; e < D / 32; ++e) dst[lane + 32 * e] = 0;
        return;
    }
    const int64_t cr = ((slot / a.page) * a.heads + h) * a.page + slot % a.page;
    const void* c = side ? a.cv : a.ck;
    const float s = T == GDN_KV_BF16 ? 1.0f : (side ? a.sv : a.sk)[cr];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
        const int64_t i = cr * D + lane + 32 * e;
        if (T == GDN_KV_BF16)
            dst[lane + 32 * e] = static_cast<const uint16_t*>(c)[i];
        else
            dst[lane + 32 * e] = float_to_bf16_bits(
                s * (T == GDN_KV_I8 ? static_cast<float>(static_cast<const int8_t*>(c)[i])
                                    : e4m3_value(static_cast<const uint8_t*>(c)[i])));
    }
}

static KvArgs kv_args(const gdn_kv_cache& c, const int64_t* slots, int64_t n) {
    KvArgs a{};
    a.heads = c.n_kv_heads;
    a.page = c.page_tokens;
    a.n_slots = c.n_pages * c.page_tokens;
    a.ck = c.k;
    a.cv = c.v;
    a.sk = c.k_scale;
    a.sv = c.v_scale;
    a.slots = slots;
    a.n = n;
    return a;
}

template <int D, int T>
static cudaError_t kv_launch(bool write, const KvArgs& a, cudaStream_t st) {
    const int64_t warps = a.n * 2 * a.heads;
    const unsigned grid = static_cast<unsigned>((warps + KV_THREADS / 32 - 1) / (KV_THREADS / 32));
    if (write)
        kv_write_kernel<D, T><<<grid, KV_THREADS, 0, st>>>(a);
    else
        kv_read_kernel<D, T><<<grid, KV_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

template <int D>
static cudaError_t kv_launch_t(int dtype, bool write, const KvArgs& a, cudaStream_t st) {
    if (dtype == GDN_KV_BF16) return kv_launch<D, GDN_KV_BF16>(write, a, st);
    if (dtype == GDN_KV_I8) return kv_launch<D, GDN_KV_I8>(write, a, st);
    return kv_launch<D, GDN_KV_E4M3>(write, a, st);
}

static cudaError_t kv_launch_d(const gdn_kv_cache& c, bool write, const KvArgs& a, cudaStream_t st) {
    if (c.head_dim == 64) return kv_launch_t<64>(c.dtype, write, a, st);
    if (c.head_dim == 128) return kv_launch_t<128>(c.dtype, write, a, st);
    return kv_launch_t<256>(c.dtype, write, a, st);
}

cudaError_t launch_kv_write(const gdn_kv_cache& c, const uint16_t* k, int64_t ld_k, const uint16_t* v, int64_t ld_v,
                            int64_t n_rows, const int32_t* rows, const int64_t* slots, int64_t n, cudaStream_t st) {
    KvArgs a = kv_args(c, slots, n);
    a.k = const_cast<uint16_t*>(k);
    a.v = const_cast<uint16_t*>(v);
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.n_rows = n_rows;
    a.rows = rows;
    return kv_launch_d(c, true, a, st);
}

cudaError_t launch_kv_read(const gdn_kv_cache& c, const int64_t* slots, int64_t n, uint16_t* k, int64_t ld_k, uint16_t* v,
                           int64_t ld_v, cudaStream_t st) {
    KvArgs a = kv_args(c, slots, n);
    a.k = k;
    a.v = v;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    return kv_launch_d(c, false, a, st);
}

int read_and_clear_kv_error() {
    int v = 0, z = 0;
    cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(int));
    if (v) cudaMemcpyToSymbol(g_kv_error, &z, sizeof(int));
    return v;
}

}  // namespace gdn
