// Block tables and slots of a paged cache, kept on the device: pages for the
// new tokens of every sequence from a stack of free ones, each token's slot and
// position, and the pages past a sequence's length back onto the stack.
#include "common.cuh"

namespace gdn {

static __device__ int g_pages_skipped;    // a length, page or number of the caller's, out of range

struct PagesArgs {
    gdn_kv_pages p;
    const int32_t* lens;       // trim: the lengths to keep
    const int32_t* n_new;
    const uint64_t* tree;
    int n_seqs;
    int max_tokens;
    int32_t* lens_out;
    int32_t* cu;
    int32_t* positions;
    int64_t* slots;
};

constexpr int PG_THREADS = GDN_MAX_SEQS;   // a thread per sequence where the tables change

__device__ __forceinline__ void pages_bad() { atomicCAS(&g_pages_skipped, 0, static_cast<int>(ERR_INDEX)); }

// An input held to [lo, hi].
__device__ __forceinline__ int pages_held(int x, int lo, int hi) {
    if (x >= lo && x <= hi) return x;
    pages_bad();
    return x < lo ? lo : hi;
}

// Inclusive sums over the block's threads.
__device__ __forceinline__ int64_t pages_scan(int64_t x) {
    __shared__ int64_t warp_total[PG_THREADS / 32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_total[w] = x;
    __syncthreads();
    for (int i = 0; i < w; ++i) x += warp_total[i];
    return x;
}

__global__ void __launch_bounds__(PG_THREADS) pages_extend_kernel(const __grid_constant__ PagesArgs a) {
    const int s = threadIdx.x;
    const bool in = s < a.n_seqs;
    const int64_t room = static_cast<int64_t>(a.p.max_blocks) * a.p.page_tokens;
    const int len = in ? pages_held(a.lens[s], 0, 0x7fffffff) : 0;
    const int n = in ? pages_held(a.n_new[s], 0, 0x7fffffff) : 0;
    const int had = in ? pages_held(a.p.n_blocks[s], 0, a.p.max_blocks) : 0;
    const int free = pages_held(*a.p.n_free, 0, static_cast<int>(a.p.n_pages));
    const int64_t end = pages_scan(n), total = static_cast<int64_t>(len) + n;
    const int64_t lo = end - n < a.max_tokens ? end - n : a.max_tokens, hi = end < a.max_tokens ? end : a.max_tokens;
    bool fits = total <= room && end <= a.max_tokens;
    if (in && !fits) pages_bad();
    int64_t need = fits ? (total + a.p.page_tokens - 1) / a.p.page_tokens - had : 0;
    if (need < 0) need = 0;
    const int64_t upto = pages_scan(need);
    const bool got = fits && (need == 0 || upto <= free);
    if (!got) need = 0;
    const int64_t used = pages_scan(need);
    if (in) {
        int32_t* row = a.p.block_table + s * a.p.ld_table;
        const int64_t top = free - 1 - (upto - need);          // of the stack, when it is this sequence's turn
        for (int64_t b = 0; b < need; ++b) row[had + b] = a.p.free_pages[top - b];
        a.p.n_blocks[s] = had + static_cast<int>(need);
        a.lens_out[s] = got ? static_cast<int>(total) : len;
        if (s == 0) a.cu[0] = 0;
        a.cu[s + 1] = static_cast<int>(hi);
    }
    __syncthreads();
    if (threadIdx.x == a.n_seqs - 1) *a.p.n_free = free - static_cast<int>(used);
    if (!in) return;
    for (int64_t t = lo; t < hi; ++t) {
        const int64_t i = t - lo, at = len + i;
        int64_t slot = -1;
        if (got) {
            const int page = a.p.block_table[s * a.p.ld_table + at / a.p.page_tokens];
            if (page >= 0 && page < a.p.n_pages) slot = static_cast<int64_t>(page) * a.p.page_tokens + at % a.p.page_tokens;
            else pages_bad();
        }
        int64_t pos = at;
        if (a.tree && i < 64) pos = len + __popcll(a.tree[t] & ((1ull << i) - 1));
        if (a.tree && i >= 64) pages_bad();
        a.slots[t] = slot;
        a.positions[t] = static_cast<int>(pos);
    }
}

// The rows behind the last sequence's.
__global__ void pages_rest_kernel(const __grid_constant__ PagesArgs a) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (t >= a.cu[a.n_seqs] && t < a.max_tokens) {
        a.slots[t] = -1;
        a.positions[t] = 0;
    }
}

__global__ void __launch_bounds__(PG_THREADS) pages_trim_kernel(const __grid_constant__ PagesArgs a) {
    const int s = threadIdx.x;
    const bool in = s < a.n_seqs;
    const int len = in ? pages_held(a.lens[s], 0, 0x7fffffff) : 0;
    const int had = in ? pages_held(a.p.n_blocks[s], 0, a.p.max_blocks) : 0;
    const int free = pages_held(*a.p.n_free, 0, static_cast<int>(a.p.n_pages));
    const int64_t want = (static_cast<int64_t>(len) + a.p.page_tokens - 1) / a.p.page_tokens;
    const int keep = want < had ? static_cast<int>(want) : had;
    const int64_t upto = pages_scan(had - keep);
    __shared__ int64_t total;
    if (s == PG_THREADS - 1) total = upto;
    __syncthreads();
    const int64_t after = free + total;
    if (in) {
        for (int b = keep; b < had; ++b) {
            const int64_t at = after - 1 - (upto - (had - keep)) - (b - keep);
            if (at < a.p.n_pages) a.p.free_pages[at] = a.p.block_table[s * a.p.ld_table + b];
            else pages_bad();
        }
        a.p.n_blocks[s] = keep;
    }
    if (s == 0) *a.p.n_free = static_cast<int>(after < a.p.n_pages ? after : a.p.n_pages);
}

cudaError_t launch_kv_extend(const gdn_kv_pages& p, const int32_t* lens, const int32_t* n_new, int n_seqs, const uint64_t* tree,
                             int64_t max_tokens, int32_t* lens_out, int32_t* cu, int32_t* positions, int64_t* slots, cudaStream_t st) {
    PagesArgs a{};
    a.p = p;
    a.lens = lens;
    a.n_new = n_new;
    a.tree = tree;
    a.n_seqs = n_seqs;
    a.max_tokens = static_cast<int>(max_tokens);
    a.lens_out = lens_out;
    a.cu = cu;
    a.positions = positions;
    a.slots = slots;
    pages_extend_kernel<<<1, PG_THREADS, 0, st>>>(a);
    if (max_tokens) pages_rest_kernel<<<static_cast<unsigned>((max_tokens + 255) / 256), 256, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_trim(const gdn_kv_pages& p, const int32_t* keep, int n_seqs, cudaStream_t st) {
    PagesArgs a{};
    a.p = p;
    a.lens = keep;
    a.n_seqs = n_seqs;
    pages_trim_kernel<<<1, PG_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

int* pages_skipped_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_pages_skipped) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdn
