// The paged key/value cache: rows quantised as they are stored, and read back.
//
// A row is one (token, head): int8 codes with scale amax/127, or e4m3 codes
// with scale amax/448, in the IEEE fp32 steps of the activation quantiser
// (scale = fl(amax / T), code = rne(fl(x / scale))).  Bound by memory: a store
// reads 2 bytes per element and writes 1 (2 for bf16), a fetch the reverse.  32768
// tokens of 4 heads of 256 stored as e4m3 and fetched: 68 us together, 6.0 TB/s;
// 100003 tokens fetched from int8 pages: 105 us, 5.9 TB/s.
#include "common.cuh"
#include "qk_decode.cuh"

namespace gdn {

static __device__ int g_kv_error;   // a row or slot out of range

struct KvArgs {
    int heads, page, page_shift;
    uint32_t heads_inv;  // floor(2^32 / heads) + 1, or 0 for one head
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

// Sixteen bf16 values.  Rows that start on 32 bytes move in one access a thread,
// which keeps a warp's accesses to whole sectors; on 16 bytes in two; any others
// value by value.
struct KvVals {
    uint32_t w[8];
};
template <int BYTES>
__device__ __forceinline__ KvVals load16(const uint16_t* p) {
    KvVals r;
    if constexpr (BYTES == 32) {
        load32(p, r.w);
    } else if constexpr (BYTES == 16) {
        const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8);
        r = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.w[e] = p[2 * e] | (static_cast<uint32_t>(p[2 * e + 1]) << 16);
    }
    return r;
}
template <int BYTES>
__device__ __forceinline__ void store16(uint16_t* p, const KvVals& r) {
    if constexpr (BYTES == 32) {
        store32(p, r.w);
    } else if constexpr (BYTES == 16) {
        *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        *reinterpret_cast<uint4*>(p + 8) = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[2 * e] = static_cast<uint16_t>(r.w[e]);
            p[2 * e + 1] = static_cast<uint16_t>(r.w[e] >> 16);
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

// The row's scale and what the quotients need of it.
struct KvScale {
    float s, rs;
};

// Eight codes of x / s: int8, or e4m3 rounded to nearest even (scale 0 or a NaN
// quotient: 0).  The quotient is x * fl(1/s) corrected once by its residual
// (P. Markstein, 1990): y = fl(y0 + fl(x - y0 s) fl(1/s)) is within 2^-22 of a
// unit of the last place of x / s, rounded once.  That rounds to the same code
// as fl(x/s) does: between them lies the middle m of two codes only where x / s
// comes within 2^-22 ulp of m +- ulp/2.  With x = X 2^i (bf16, 8 bits) and
// s = S 2^j (24 bits) that asks for S within 8 of a multiple of 2^20 (e4m3, m of
// 5 bits) or of 2^17 (int8, 8 bits), but S is an 8-bit number over 7 or 127
// rounded, whose digits repeat with a period of 3 or 7 and so hold no run of
// that many zeros or ones, or it is such a multiple itself and x / s is not that
// near without being there.  No step underflows for s >= 2^-60, which is 2^-71
// for the smallest x with a code other than 0.  Otherwise, and where x holds a
// NaN, all eight divide.
template <int T>
__device__ __forceinline__ uint2 kv_codes8(const float (&x)[8], KvScale q) {
    const F2 rs = f2(q.rs, q.rs), ns = f2(-q.s, -q.s);
    float y[8];
    F2 sum;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const F2 x2 = f2(x[e], x[e + 1]), y0 = f2_mul(x2, rs);
        F2 y2 = f2_fma(f2_fma(y0, ns, x2), rs, y0);
        sum = e == 0 ? y2 : f2_add(sum, y2);
        if constexpr (T == GDN_KV_I8) y2 = f2_add(y2, f2(QCODE_MAGIC, QCODE_MAGIC));
        f2_split(y2, y[e], y[e + 1]);
    }
    float a, b;
    f2_split(sum, a, b);
    a += b;
    if (!(q.s >= 0x1p-60f && q.s <= 1e30f) || a != a) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float d = q.s == 0.0f ? 0.0f : __fdiv_rn(x[e], q.s);
            d = d != d ? 0.0f : d;
            y[e] = T == GDN_KV_I8 ? __fadd_rn(fminf(fmaxf(d, -127.0f), 127.0f), QCODE_MAGIC) : d;
        }
    }
    if constexpr (T == GDN_KV_I8)
        return make_uint2(codes_to_i8x4(y[0], y[1], y[2], y[3]), codes_to_i8x4(y[4], y[5], y[6], y[7]));
    return make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16), e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }

// The largest |x| of each of two rows' sixteen bf16, side by side.
__device__ __forceinline__ __nv_bfloat162 kv_amax2(const KvVals& u, const KvVals& v) {
    const auto row = [](const KvVals& a) {
        __nv_bfloat162 m = as_bf162(a.w[0] & 0x7fff7fffu);
#pragma unroll
        for (int e = 1; e < 8; ++e) m = __hmax2(m, as_bf162(a.w[e] & 0x7fff7fffu));
        return *reinterpret_cast<const uint32_t*>(&m);
    };
    const uint32_t a = row(u), b = row(v);
    return __hmax2(as_bf162(__byte_perm(a, b, 0x5410)), as_bf162(__byte_perm(a, b, 0x7632)));
}

__device__ __forceinline__ void e4m3_pair(uint32_t w, float& lo, float& hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    lo = f.x;
    hi = f.y;
}

// D/16 threads per row, each sixteen of its elements; blockIdx.y is the side
// (keys or values).  Nothing orders two rows of one slot, which the contract
// excludes: one winner would take a word per slot and two more launches.  A thread takes KV_ITER rows a block's width apart, all
// indices before the first row's load, all loads before the first use.  The
// block's first token is divided out once; from there a row is a small number
// (under 256 heads + 256 rows), whose product with heads_inv has the quotient in
// its upper word.
template <int D>
struct KvRows {
    static constexpr int G = D / 16, RB = KV_THREADS / G;
    int64_t tok0, left;   // first token, rows from its first head to the end
    uint32_t r0;
    int h;
    __device__ __forceinline__ explicit KvRows(const KvArgs& a) {
        const int64_t base = static_cast<int64_t>(blockIdx.x) * (RB * KV_ITER);
        tok0 = base / a.heads;
        left = (a.n - tok0) * a.heads;
        r0 = static_cast<uint32_t>(base - tok0 * a.heads) + threadIdx.x / G;
    }
    // row i's token, or false past the end; sets its head
    __device__ __forceinline__ bool token(const KvArgs& a, int i, int64_t& tok) {
        const uint32_t r = r0 + i * RB, t = a.heads_inv ? __umulhi(r, a.heads_inv) : r;
        h = static_cast<int>(r - t * a.heads);
        tok = tok0 + t;
        return r < left;
    }
};

template <int D, int T, int BYTES>
__global__ void __launch_bounds__(KV_THREADS, 4) kv_write_kernel(const __grid_constant__ KvArgs a) {
    using R = KvRows<D>;
    pdl_wait();
    pdl_trigger();
    const int sub = threadIdx.x % R::G, side = blockIdx.y;
    const uint16_t* src = (side ? a.v : a.k) + 16 * sub;
    const int64_t ld = side ? a.ld_v : a.ld_k;
    void* codes = side ? a.cv : a.ck;
    KvVals w[KV_ITER];
    int64_t to[KV_ITER], row[KV_ITER];     // slot, then cache row, -1: none; the caller's row
    int head[KV_ITER];
    R rows(a);
#pragma unroll
    for (int i = 0; i < KV_ITER; ++i) {
        int64_t tok;
        const bool in = rows.token(a, i, tok);
        head[i] = rows.h;
        to[i] = in ? a.slots[tok] : -1;
        row[i] = !in ? -1 : a.rows ? a.rows[tok] : tok;
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < KV_ITER; ++i) {
        const bool ok = row[i] >= 0 && row[i] < a.n_rows;
        w[i] = KvVals{};
        if (ok) w[i] = load16<BYTES>(src + row[i] * ld + head[i] * D);   // does not wait for the slot
        bad |= to[i] >= 0 && (!ok || to[i] >= a.n_slots);
        to[i] = ok && to[i] >= 0 && to[i] < a.n_slots ? ((to[i] >> a.page_shift) * a.heads + head[i]) * a.page + (to[i] & (a.page - 1)) : -1;
    }
    if (bad) atomicCAS(&g_kv_error, 0, static_cast<int>(ERR_INDEX));
    if constexpr (T == GDN_KV_BF16) {
#pragma unroll
        for (int i = 0; i < KV_ITER; ++i)
            if (to[i] >= 0) store16<32>(static_cast<uint16_t*>(codes) + to[i] * D + 16 * sub, w[i]);
    } else {
        // the four maxima, two to a register; then lane i of a row's threads
        // divides for row i, and the others take its results
        static_assert(KV_ITER == 4 && R::G >= KV_ITER);
        __nv_bfloat162 m[2] = {kv_amax2(w[0], w[1]), kv_amax2(w[2], w[3])};
#pragma unroll
        for (int s = R::G / 2; s > 0; s >>= 1)
#pragma unroll
            for (int j = 0; j < 2; ++j) m[j] = __hmax2(m[j], __shfl_xor_sync(0xffffffffu, m[j], s));
        const float2 m01 = __bfloat1622float2(m[0]), m23 = __bfloat1622float2(m[1]);
        const float mine = sub & 2 ? (sub & 1 ? m23.y : m23.x) : (sub & 1 ? m01.y : m01.x);
        const float s = __fdiv_rn(fmaxf(mine, 0.0f), T == GDN_KV_I8 ? 127.0f : 448.0f), rs = __frcp_rn(s);   // a row of NaN: 0
#pragma unroll
        for (int i = 0; i < KV_ITER; ++i) {
            const KvScale q = {__shfl_sync(0xffffffffu, s, i, R::G), __shfl_sync(0xffffffffu, rs, i, R::G)};
            uint2 c[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] = __uint_as_float(w[i].w[4 * p + e] << 16);
                    x[2 * e + 1] = __uint_as_float(w[i].w[4 * p + e] & 0xffff0000u);
                }
                c[p] = kv_codes8<T>(x, q);
            }
            if (to[i] >= 0) {
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(codes) + to[i] * D + 16 * sub) = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
                if (sub == 0) (side ? a.sv : a.sk)[to[i]] = q.s;
            }
        }
    }
}

template <int D, int T, int BYTES>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const __grid_constant__ KvArgs a) {
    using R = KvRows<D>;
    pdl_wait();
    pdl_trigger();
    const int sub = threadIdx.x % R::G, side = blockIdx.y;
    const void* codes = side ? a.cv : a.ck;
    const float* scales = side ? a.sv : a.sk;
    const int64_t ld = side ? a.ld_v : a.ld_k;
    uint16_t* out = (side ? a.v : a.k) + 16 * sub;
    KvVals w[KV_ITER];
    float s[KV_ITER];
    int64_t from[KV_ITER], dst[KV_ITER];
    int head[KV_ITER];
    R rows(a);
#pragma unroll
    for (int i = 0; i < KV_ITER; ++i) {
        int64_t tok;
        const bool in = rows.token(a, i, tok);
        head[i] = rows.h;
        from[i] = in ? a.slots[tok] : -1;
        dst[i] = in ? tok * ld + rows.h * D : -1;
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < KV_ITER; ++i) {
        w[i] = KvVals{};   // zeros where there is no slot
        s[i] = 0.0f;
        bad |= from[i] >= a.n_slots;
        if (from[i] < 0 || from[i] >= a.n_slots) continue;
        const int64_t c = ((from[i] >> a.page_shift) * a.heads + head[i]) * a.page + (from[i] & (a.page - 1));
        if constexpr (T == GDN_KV_BF16) {
            w[i] = load16<32>(static_cast<const uint16_t*>(codes) + c * D + 16 * sub);
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(codes) + c * D + 16 * sub);
            w[i].w[0] = v.x;
            w[i].w[1] = v.y;
            w[i].w[2] = v.z;
            w[i].w[3] = v.w;
            s[i] = scales[c];
        }
    }
    if (bad) atomicCAS(&g_kv_error, 0, static_cast<int>(ERR_INDEX));
#pragma unroll
    for (int i = 0; i < KV_ITER; ++i) {
        if constexpr (T != GDN_KV_BF16) {
            const F2 s2 = f2(s[i], s[i]);
            KvVals r;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t u = w[i].w[e >> 1];
                float lo, hi;
                if constexpr (T == GDN_KV_I8) {
                    // the code's offset byte in the low byte of 2^23, which is then taken off again
                    const uint32_t b = u ^ 0x80808080u;
                    lo = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7540 | (2 * e & 3)));
                    hi = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7540 | (2 * e + 1 & 3)));
                    f2_split(f2_mul(f2_sub(f2(lo, hi), f2(8388736.0f, 8388736.0f)), s2), lo, hi);
                } else {
                    e4m3_pair((u >> (16 * (e & 1))) & 0xffffu, lo, hi);
                    f2_split(f2_mul(f2(lo, hi), s2), lo, hi);
                }
                r.w[e] = bf16_pair(lo, hi);
            }
            w[i] = r;
        }
        if (dst[i] >= 0) store16<BYTES>(out + dst[i], w[i]);
    }
}

static KvArgs kv_args(const gdn_kv_cache& c, const int64_t* slots, int64_t n) {
    KvArgs a{};
    a.heads = c.n_kv_heads;
    a.heads_inv = c.n_kv_heads == 1 ? 0u : 0xffffffffu / c.n_kv_heads + 1u;
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
    constexpr int ROWS = KvRows<D>::RB * KV_ITER;
    const int64_t blocks = (a.n * a.heads + ROWS - 1) / ROWS;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;   // more rows than any memory holds
    const dim3 grid(static_cast<unsigned>(blocks), 2);
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) | static_cast<uintptr_t>(2 * (a.ld_k | a.ld_v));
    auto kernel = at % 32 == 0   ? (write ? kv_write_kernel<D, T, 32> : kv_read_kernel<D, T, 32>)
                  : at % 16 == 0 ? (write ? kv_write_kernel<D, T, 16> : kv_read_kernel<D, T, 16>)
                                 : (write ? kv_write_kernel<D, T, 2> : kv_read_kernel<D, T, 2>);
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

int* kv_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_kv_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdn
