// Attention of new tokens (one, a chain, or a tree of drafts) over the paged
// key/value cache.
//
// One CTA per (new token, query head); each warp takes every eighth key with
// its own running maximum and sum, and the warps' results are joined in shared
// memory.  Everything in fp32 on the CUDA cores.
#include "common.cuh"

#include <cuda_fp8.h>

namespace gdn {

static __device__ int g_attn_cache_error;

struct AttCacheArgs {
    const void *k, *v;
    const float *sk, *sv;
    int64_t n_pages;
    int heads, page, ratio, hq;
    const uint16_t* q;
    uint16_t* o;
    int64_t ld_q, ld_o, ld_table, n_tokens;
    const int32_t *cu, *table, *lens;
    const uint64_t* tree;
    int n_seqs, max_q, max_blocks;
    float scale;
};

constexpr int AC_WARPS = 8;

template <int T>
__device__ __forceinline__ float kv_value(const void* p, int64_t i) {
    if (T == GDN_KV_BF16) return bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
    if (T == GDN_KV_I8) return static_cast<float>(static_cast<const int8_t*>(p)[i]);
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[i], __NV_E4M3)));
}

// First and last + 1 new token of sequence s, forced into range.
__device__ __forceinline__ int2 new_tokens(const AttCacheArgs& a, int s) {
    int2 r = a.cu ? make_int2(a.cu[s], a.cu[s + 1]) : make_int2(s * a.max_q, (s + 1) * a.max_q);
    if (r.x < 0 || r.y < r.x || r.y > a.n_tokens || r.y - r.x > a.max_q) {
        atomicCAS(&g_attn_cache_error, 0, static_cast<int>(ERR_INDEX));
        r = make_int2(0, 0);
    }
    return r;
}

template <int D, int T>
__global__ void __launch_bounds__(32 * AC_WARPS) attn_cache_kernel(const __grid_constant__ AttCacheArgs a) {
    constexpr int E = D / 32;
    __shared__ float sm_m[AC_WARPS], sm_l[AC_WARPS], sm_o[AC_WARPS][D];
    const int h = blockIdx.x % a.hq, s = blockIdx.y, i = blockIdx.x / a.hq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = h / a.ratio;
    const int2 nt = new_tokens(a, s);
    if (i >= nt.y - nt.x) return;
    const int tok = nt.x + i;
    int64_t len = a.lens[s];
    if (len < 0 || len > static_cast<int64_t>(a.max_blocks) * a.page) {
        atomicCAS(&g_attn_cache_error, 0, static_cast<int>(ERR_INDEX));
        len = len < 0 ? 0 : static_cast<int64_t>(a.max_blocks) * a.page;
    }
    const int64_t ctx = len - (nt.y - nt.x);
    const uint64_t mask = a.tree ? a.tree[tok] : (i == 63 ? ~0ull : (1ull << (i + 1)) - 1);
    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = bf16_bits_to_float(a.q[tok * a.ld_q + h * D + lane + 32 * e]) * a.scale;
        o[e] = 0.0f;
    }
    for (int64_t j = warp; j < len; j += AC_WARPS) {
        if (j >= ctx && !((mask >> (j - ctx)) & 1)) continue;
        const int64_t page = a.table[s * a.ld_table + j / a.page];
        if (page < 0 || page >= a.n_pages) {
            atomicCAS(&g_attn_cache_error, 0, static_cast<int>(ERR_INDEX));
            continue;
        }
        const int64_t row = (page * a.heads + g) * a.page + j % a.page;
        float x = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) x = fmaf(q[e], kv_value<T>(a.k, row * D + lane + 32 * e), x);
        x = warp_sum(x);
        if (T != GDN_KV_BF16) x *= a.sk[row];
        const float mn = fmaxf(m, x), c = expf(m - mn), p = expf(x - mn), pv = T == GDN_KV_BF16 ? p : p * a.sv[row];
        m = mn;
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(pv, kv_value<T>(a.v, row * D + lane + 32 * e), o[e] * c);
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane + 32 * e] = o[e];
    __syncthreads();
    float mm = -INFINITY;
    for (int w = 0; w < AC_WARPS; ++w) mm = fmaxf(mm, sm_m[w]);
    for (int e = threadIdx.x; e < D; e += 32 * AC_WARPS) {
        float lt = 0.0f, ot = 0.0f;
        for (int w = 0; w < AC_WARPS; ++w)
            if (sm_l[w] != 0.0f) {
                const float c = expf(sm_m[w] - mm);
                lt += c * sm_l[w];
                ot += c * sm_o[w][e];
            }
        a.o[tok * a.ld_o + h * D + e] = float_to_bf16_bits(lt == 0.0f ? 0.0f : ot / lt);
    }
}

size_t attn_cache_workspace_bytes(const gdn_kv_cache&, int64_t, int) { return 256; }

template <int D>
static cudaError_t attn_cache_launch(int dtype, const AttCacheArgs& a, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(a.max_q * a.hq), static_cast<unsigned>(a.n_seqs));
    if (dtype == GDN_KV_BF16)
        attn_cache_kernel<D, GDN_KV_BF16><<<grid, 32 * AC_WARPS, 0, st>>>(a);
    else if (dtype == GDN_KV_I8)
        attn_cache_kernel<D, GDN_KV_I8><<<grid, 32 * AC_WARPS, 0, st>>>(a);
    else
        attn_cache_kernel<D, GDN_KV_E4M3><<<grid, 32 * AC_WARPS, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_attn_cache(const gdn_kv_cache& c, const uint16_t* q, int64_t ld_q, const int32_t* cu, int64_t n_tokens,
                              int max_q, const uint64_t* tree, const int32_t* table, int64_t ld_table, int max_blocks,
                              const int32_t* lens, int n_seqs, int hq, float scale, uint16_t* o, int64_t ld_o, void*, cudaStream_t st) {
    AttCacheArgs a{};
    a.k = c.k;
    a.v = c.v;
    a.sk = c.k_scale;
    a.sv = c.v_scale;
    a.n_pages = c.n_pages;
    a.heads = c.n_kv_heads;
    a.page = c.page_tokens;
    a.ratio = hq / c.n_kv_heads;
    a.hq = hq;
    a.q = q;
    a.o = o;
    a.ld_q = ld_q;
    a.ld_o = ld_o;
    a.ld_table = ld_table;
    a.max_blocks = max_blocks;
    a.n_tokens = n_tokens;
    a.cu = cu;
    a.table = table;
    a.lens = lens;
    a.tree = tree;
    a.n_seqs = n_seqs;
    a.max_q = max_q;
    a.scale = scale;
    if (c.head_dim == 64) return attn_cache_launch<64>(c.dtype, a, st);
    if (c.head_dim == 128) return attn_cache_launch<128>(c.dtype, a, st);
    return attn_cache_launch<256>(c.dtype, a, st);
}

int read_and_clear_attn_cache_error() {
    int v = 0, z = 0;
    cudaMemcpyFromSymbol(&v, g_attn_cache_error, sizeof(int));
    if (v) cudaMemcpyToSymbol(g_attn_cache_error, &z, sizeof(int));
    return v;
}

}  // namespace gdn
