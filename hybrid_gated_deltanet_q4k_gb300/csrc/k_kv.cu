// The paged key/value cache: rows quantised as they are stored, and read back.
//
// A row is one (token, head): int8 codes with scale amax/127, or e4m3 codes
// with scale amax/448, in the IEEE fp32 steps of the activation quantiser
// (scale = fl(amax / T), code = rne(fl(x / scale))).  Bound by memory: a store
// reads 2 bytes per element and writes 1 (2 for bf16), a fetch the reverse.
#include "common.cuh"
#include "qk_decode.cuh"

namespace gdn {

static __device__ int g_kv_error;   // a row or slot out of range

struct KvArgs {
    int heads, page, page_shift;
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
constexpr int KV_ITER = 4;   // rows a thread has in flight

// Eight bf16 values at p: one 16-byte access, or eight where the caller's rows
// are not 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
    if constexpr (VEC) return *reinterpret_cast<const uint4*>(p);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = p[2 * e] | (static_cast<uint32_t>(p[2 * e + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool VEC>
__device__ __forceinline__ void store8(uint16_t* p, uint4 v) {
    if constexpr (VEC) {
        *reinterpret_cast<uint4*>(p) = v;
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            p[2 * e] = static_cast<uint16_t>(w[e]);
            p[2 * e + 1] = static_cast<uint16_t>(w[e] >> 16);
        }
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight e4m3 codes of x / s (the IEEE quotient, rounded to nearest even; scale
// 0 or a NaN quotient: 0).  As the int8 quantiser does, the quotient is first
// taken as x * fl(1/s), within 3 units of the last place of fl(x/s): the two
// can round apart only next to a border, where the 20 bits that e4m3 drops are
// about one half, or below the smallest normal code; then all eight divide.
__device__ __forceinline__ uint2 e4m3_codes8(const float (&x)[8], const QScale& q) {
    float y[8];
    bool redo = !q.fast;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        y[e] = __fmul_rn(x[e], q.rs);
        const uint32_t b = __float_as_uint(y[e]) & 0x7fffffffu;
        redo |= (((b + 8u) ^ 0x80000u) & 0xfffffu) <= 16u || (b < 0x3c800000u && b != 0u) || b >= 0x7f800000u;
    }
    if (redo) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = q.s == 0.0f ? 0.0f : __fdiv_rn(x[e], q.s);
            y[e] = d != d ? 0.0f : d;
        }
    }
    return make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16), e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
}

__device__ __forceinline__ void e4m3_pair(uint32_t w, float& lo, float& hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    lo = f.x;
    hi = f.y;
}

// D/8 threads per row, each eight of its elements; blockIdx.y is the side (keys
// or values).  A thread takes KV_ITER rows a block's width apart, all loads
// before the first use.
template <int D, int T, bool VEC>
__global__ void __launch_bounds__(KV_THREADS) kv_write_kernel(const __grid_constant__ KvArgs a) {
    constexpr int G = D / 8, RB = KV_THREADS / G;
    pdl_wait();
    pdl_trigger();
    const int sub = threadIdx.x % G, side = blockIdx.y;
    const uint16_t* src = side ? a.v : a.k;
    const int64_t ld = side ? a.ld_v : a.ld_k, n_rows = a.n * a.heads;
    void* codes = side ? a.cv : a.ck;
    uint4 w[KV_ITER];
    int64_t to[KV_ITER];     // cache row, -1: none
#pragma unroll
    for (int i = 0; i < KV_ITER; ++i) {
        const int64_t r = static_cast<int64_t>(blockIdx.x) * (RB * KV_ITER) + i * RB + threadIdx.x / G;
        to[i] = -1;
        w[i] = make_uint4(0, 0, 0, 0);
        if (r >= n_rows) continue;
        const int64_t tok = r / a.heads;
        const int h = static_cast<int>(r - tok * a.heads);
        const int64_t row = a.rows ? a.rows[tok] : tok, slot = a.slots[tok];
        if (slot < 0) continue;
        if (row < 0 || row >= a.n_rows || slot >= a.n_slots) {
            if (sub == 0) atomicCAS(&g_kv_error, 0, static_cast<int>(ERR_INDEX));
            continue;
        }
        to[i] = ((slot >> a.page_shift) * a.heads + h) * a.page + (slot & (a.page - 1));
        w[i] = load8<VEC>(src + row * ld + h * D + 8 * sub);
    }
#pragma unroll
    for (int i = 0; i < KV_ITER; ++i) {
        if constexpr (T == GDN_KV_BF16) {
            if (to[i] >= 0) store8<true>(static_cast<uint16_t*>(codes) + to[i] * D + 8 * sub, w[i]);
        } else {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            float x[8], amax = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(u[e] << 16);
                x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
                amax = fmaxf(amax, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
            }
#pragma unroll
            for (int s = G / 2; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
            QScale q = make_qscale(amax);
            if constexpr (T == GDN_KV_E4M3) {
                q.s = __fdiv_rn(amax, 448.0f);
                q.rs = __frcp_rn(q.s);
                q.fast = q.s >= 1e-30f && q.s <= 1e30f;
            }
            uint2 c;
            if constexpr (T == GDN_KV_I8) {
                float t[8];
                quantise8(x, q, t);
                c = make_uint2(codes_to_i8x4(t[0], t[1], t[2], t[3]), codes_to_i8x4(t[4], t[5], t[6], t[7]));
            } else {
                c = e4m3_codes8(x, q);
            }
            if (to[i] >= 0) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(codes) + to[i] * D + 8 * sub) = c;
                if (sub == 0) (side ? a.sv : a.sk)[to[i]] = q.s;
            }
        }
    }
}

template <int D, int T, bool VEC>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const __grid_constant__ KvArgs a) {
    constexpr int G = D / 8, RB = KV_THREADS / G;
    pdl_wait();
    pdl_trigger();
    const int sub = threadIdx.x % G, side = blockIdx.y;
    const void* codes = side ? a.cv : a.ck;
    const float* scales = side ? a.sv : a.sk;
    const int64_t ld = side ? a.ld_v : a.ld_k, n_rows = a.n * a.heads;
    uint4 w[KV_ITER];
    float s[KV_ITER];
    uint16_t* dst[KV_ITER];
#pragma unroll
    for (int i = 0; i < KV_ITER; ++i) {
        const int64_t r = static_cast<int64_t>(blockIdx.x) * (RB * KV_ITER) + i * RB + threadIdx.x / G;
        dst[i] = nullptr;
        w[i] = make_uint4(0, 0, 0, 0);
        s[i] = 0.0f;
        if (r >= n_rows) continue;
        const int64_t tok = r / a.heads;
        const int h = static_cast<int>(r - tok * a.heads);
        dst[i] = (side ? a.v : a.k) + tok * ld + h * D + 8 * sub;
        const int64_t slot = a.slots[tok];
        if (slot < 0 || slot >= a.n_slots) {   // zeros
            if (slot >= 0 && sub == 0) atomicCAS(&g_kv_error, 0, static_cast<int>(ERR_INDEX));
            continue;
        }
        const int64_t from = ((slot >> a.page_shift) * a.heads + h) * a.page + (slot & (a.page - 1));
        if constexpr (T == GDN_KV_BF16) {
            w[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(codes) + from * D + 8 * sub);
        } else {
            const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(codes) + from * D + 8 * sub);
            w[i].x = c.x;
            w[i].y = c.y;
            s[i] = scales[from];
        }
    }
#pragma unroll
    for (int i = 0; i < KV_ITER; ++i) {
        if (!dst[i]) continue;
        if constexpr (T != GDN_KV_BF16) {
            const uint32_t u[2] = {w[i].x, w[i].y};
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t c = u[e >> 2] >> (8 * (e & 3));
                if constexpr (T == GDN_KV_I8)
                    x[e] = static_cast<float>(static_cast<int8_t>(c));
                else if (e % 2 == 0)
                    e4m3_pair(c & 0xffffu, x[e], x[e + 1]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(x[e], s[i]);
            w[i] = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
        }
        store8<VEC>(dst[i], w[i]);
    }
}

static KvArgs kv_args(const gdn_kv_cache& c, const int64_t* slots, int64_t n) {
    KvArgs a{};
    a.heads = c.n_kv_heads;
    a.page = c.page_tokens;
    a.page_shift = c.page_tokens == 16 ? 4 : c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : 7;
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
    constexpr int ROWS = KV_THREADS / (D / 8) * KV_ITER;
    const dim3 grid(static_cast<unsigned>((a.n * a.heads + ROWS - 1) / ROWS), 2);
    const bool vec = a.ld_k % 8 == 0 && a.ld_v % 8 == 0 && reinterpret_cast<uintptr_t>(a.k) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.v) % 16 == 0;
    auto kernel = write ? (vec ? kv_write_kernel<D, T, true> : kv_write_kernel<D, T, false>)
                        : (vec ? kv_read_kernel<D, T, true> : kv_read_kernel<D, T, false>);
    return launch_dependent(kernel, grid, dim3(KV_THREADS), 0, st, a);
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
