// Block tables and slots of a paged cache, kept on the device: pages for the
// new tokens of every sequence from a stack of free ones, each token's slot and
// position, and the pages past a sequence's length back onto the stack.
//
// Who gets which page follows from sums over the sequences (at most
// GDN_MAX_SEQS), which every CTA takes for itself: a thread per sequence and
// two scans.  From there tokens and pages are independent: each finds its
// sequence by bisection of the sums in shared memory.  What is read by all
// (lengths, pages held, the stack's height) is written last: by the one CTA, or by
// a second launch that waits for the first.  A trim and an extension of 64 trees of
// up to 32 tokens: 8 us, two launches and their chains of loads; of 256 prompts
// (1.05 million tokens, 65 thousand pages): 20 us, four launches.
#include "common.cuh"

namespace gdn {

static __device__ int g_pages_error;      // debug: a store's index
static __device__ int g_pages_skipped;    // a length, page or number of the caller's, out of range

struct PagesArgs {
    gdn_kv_pages p;
    const int32_t* lens;       // trim: the lengths to keep
    const int32_t* n_new;
    const uint64_t* tree;
    int n_seqs;
    int page_shift;
    int max_tokens;
    int32_t* lens_out;
    int32_t* cu;
    int32_t* positions;
    int64_t* slots;
};

constexpr int PG_THREADS = 512;
constexpr int PG_STEP = 4;
static_assert(PG_THREADS >= GDN_MAX_SEQS, "a thread per sequence");

__device__ __forceinline__ void pages_bad() { atomicCAS(&g_pages_skipped, 0, static_cast<int>(ERR_INDEX)); }

// An input held to [lo, hi].
__device__ __forceinline__ int pages_held(int x, int lo, int hi) {
    if (x >= lo && x <= hi) return x;
    pages_bad();
    return x < lo ? lo : hi;
}

// Inclusive sums of x over the first GDN_MAX_SEQS threads.
__device__ __forceinline__ int64_t pages_scan(int64_t x, int64_t* warp_total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31 && w < GDN_MAX_SEQS / 32) warp_total[w] = x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < GDN_MAX_SEQS / 32; ++i) x += i < w ? warp_total[i] : 0;
    return x;
}

// The last i < n with first[i] <= x.
__device__ __forceinline__ int pages_find(const int* first, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

struct ExtendSums {
    int first[GDN_MAX_SEQS];   // token rows of the sequences, within max_tokens
    int page[GDN_MAX_SEQS];    // pages asked for by the sequences before
    int len[GDN_MAX_SEQS];
    int had[GDN_MAX_SEQS];     // pages held; negative: the sequence gets nothing
    int64_t warp_total[2][GDN_MAX_SEQS / 32];
    int used, total;
};

// tokens: this launch writes slots, positions and the block table; last: it
// ends with what the other CTAs read.
__global__ void __launch_bounds__(PG_THREADS) pages_extend_kernel(const __grid_constant__ PagesArgs a, bool tokens, bool last) {
    __shared__ ExtendSums sm;
    pdl_wait();
    pdl_trigger();
    const int s = threadIdx.x, shift = a.page_shift;
    const bool in = s < a.n_seqs;
    const int64_t room = static_cast<int64_t>(a.p.max_blocks) << shift;
    const int len = in ? pages_held(a.lens[s], 0, 0x7fffffff) : 0;
    const int n = in ? pages_held(a.n_new[s], 0, 0x7fffffff) : 0;
    const int had = in ? pages_held(a.p.n_blocks[s], 0, a.p.max_blocks) : 0;
    const int free = pages_held(*a.p.n_free, 0, static_cast<int>(a.p.n_pages));
    if (s == 0) sm.used = 0;
    const int64_t end = pages_scan(n, sm.warp_total[0]), total = static_cast<int64_t>(len) + n;
    const int lo = static_cast<int>(end - n < a.max_tokens ? end - n : a.max_tokens);
    const int hi = static_cast<int>(end < a.max_tokens ? end : a.max_tokens);
    const bool fits = total <= room && end <= a.max_tokens;
    if (in && !fits) pages_bad();
    int64_t need = fits ? ((total + (1 << shift) - 1) >> shift) - had : 0;
    if (need < 0) need = 0;
    const int64_t upto = pages_scan(need, sm.warp_total[1]);
    // once the stack did not reach, it does not reach for any later one that asks
    const bool got = fits && (need == 0 || upto <= free);
    if (in) {
        sm.first[s] = lo;
        sm.page[s] = static_cast<int>(upto - need < 0x7fffffff ? upto - need : 0x7fffffff);
        sm.len[s] = len;
        sm.had[s] = got ? had : -1;
        if (got && need) atomicMax(&sm.used, static_cast<int>(upto));
        if (s == a.n_seqs - 1) sm.total = hi;
    }
    __syncthreads();
    const int used = sm.used;
    if (tokens) {
        const int64_t step = static_cast<int64_t>(gridDim.x) * PG_THREADS;
        // PG_STEP at a time, so that their bisections and loads overlap
        for (int64_t k0 = blockIdx.x * PG_THREADS + s; k0 < used; k0 += PG_STEP * step) {
            int page[PG_STEP];
            int64_t to[PG_STEP];
#pragma unroll
            for (int e = 0; e < PG_STEP; ++e) {
                const int k = static_cast<int>(k0 + e * step < used ? k0 + e * step : k0), q = pages_find(sm.page, a.n_seqs, k);
                const int b = sm.had[q] + (k - sm.page[q]);
                page[e] = a.p.free_pages[free - 1 - k];
                to[e] = GDN_IN_RANGE(g_pages_error, sm.had[q] >= 0 && b < a.p.max_blocks) ? q * a.p.ld_table + b : -1;
            }
#pragma unroll
            for (int e = 0; e < PG_STEP; ++e)
                if (to[e] >= 0) a.p.block_table[to[e]] = page[e];
        }
        for (int64_t t0 = blockIdx.x * PG_THREADS + s; t0 < a.max_tokens; t0 += PG_STEP * step) {
            int64_t slot[PG_STEP];
            int pos[PG_STEP], page[PG_STEP];
#pragma unroll
            for (int e = 0; e < PG_STEP; ++e) {
                const int64_t t = t0 + e * step;
                slot[e] = -1;
                pos[e] = 0;
                page[e] = -1;
                if (t >= sm.total) continue;
                const int q = pages_find(sm.first, a.n_seqs, static_cast<int>(t)), i = static_cast<int>(t) - sm.first[q], h = sm.had[q];
                const int64_t at = static_cast<int64_t>(sm.len[q]) + i;
                if (h >= 0) {
                    // a new block's page is where the loop above takes it from
                    const int b = static_cast<int>(at >> shift);
                    page[e] = b < h ? a.p.block_table[q * a.p.ld_table + b] : a.p.free_pages[free - 1 - (sm.page[q] + b - h)];
                    slot[e] = at & ((1 << shift) - 1);
                }
                pos[e] = static_cast<int>(at);
                if (a.tree) {
                    if (i < 64) pos[e] = sm.len[q] + __popcll(a.tree[t] & ((1ull << i) - 1));
                    else pages_bad();
                }
            }
#pragma unroll
            for (int e = 0; e < PG_STEP; ++e) {
                const int64_t t = t0 + e * step;
                if (t >= a.max_tokens) break;
                if (slot[e] >= 0) {
                    if (page[e] >= 0 && page[e] < a.p.n_pages) {
                        slot[e] += static_cast<int64_t>(page[e]) << shift;
                    } else {
                        slot[e] = -1;
                        pages_bad();
                    }
                }
                a.slots[t] = slot[e];
                a.positions[t] = pos[e];
            }
        }
    }
    if (!last) return;
    __syncthreads();
    if (in) {
        a.p.n_blocks[s] = had + (got ? static_cast<int>(need) : 0);
        a.lens_out[s] = got ? static_cast<int>(total) : len;
        if (s == 0) {
            a.cu[0] = 0;
            *a.p.n_free = free - used;
        }
        a.cu[s + 1] = hi;
    }
}

__global__ void __launch_bounds__(PG_THREADS) pages_trim_kernel(const __grid_constant__ PagesArgs a, bool pages, bool last) {
    __shared__ int first[GDN_MAX_SEQS], held[GDN_MAX_SEQS];
    __shared__ int64_t warp_total[GDN_MAX_SEQS / 32];
    __shared__ int64_t sum;
    pdl_wait();
    pdl_trigger();
    const int s = threadIdx.x;
    const bool in = s < a.n_seqs;
    const int len = in ? pages_held(a.lens[s], 0, 0x7fffffff) : 0;
    const int had = in ? pages_held(a.p.n_blocks[s], 0, a.p.max_blocks) : 0;
    const int free = pages_held(*a.p.n_free, 0, static_cast<int>(a.p.n_pages));
    const int64_t want = (static_cast<int64_t>(len) + (1 << a.page_shift) - 1) >> a.page_shift;
    const int keep = want < had ? static_cast<int>(want) : had;
    const int64_t upto = pages_scan(had - keep, warp_total);
    if (in) {
        first[s] = static_cast<int>(upto - (had - keep) < 0x7fffffff ? upto - (had - keep) : 0x7fffffff);
        held[s] = keep;
        if (s == a.n_seqs - 1) sum = upto;
    }
    __syncthreads();
    // more than the cache has pages is a mistake of the caller's; the stack ends there
    const int64_t after = free + sum;
    if (after > a.p.n_pages) pages_bad();
    const int back = static_cast<int>(sum < 0x7fffffff ? sum : 0x7fffffff);
    const int64_t step = static_cast<int64_t>(gridDim.x) * PG_THREADS;
    for (int64_t k0 = blockIdx.x * PG_THREADS + s; pages && k0 < back; k0 += PG_STEP * step) {
        int page[PG_STEP];
#pragma unroll
        for (int e = 0; e < PG_STEP; ++e) {
            const int k = static_cast<int>(k0 + e * step < back ? k0 + e * step : k0), q = pages_find(first, a.n_seqs, k);
            page[e] = a.p.block_table[q * a.p.ld_table + held[q] + (k - first[q])];
        }
#pragma unroll
        for (int e = 0; e < PG_STEP; ++e) {
            const int64_t k = k0 + e * step, to = after - 1 - k;
            if (k < back && to < a.p.n_pages) a.p.free_pages[to] = page[e];
        }
    }
    if (!last) return;
    __syncthreads();
    if (in) a.p.n_blocks[s] = keep;
    if (s == 0) *a.p.n_free = static_cast<int>(after < a.p.n_pages ? after : a.p.n_pages);
}

static PagesArgs pages_args(const gdn_kv_pages& p, const int32_t* lens, int n_seqs) {
    PagesArgs a{};
    a.p = p;
    a.lens = lens;
    a.n_seqs = n_seqs;
    a.page_shift = p.page_tokens == 16 ? 4 : p.page_tokens == 32 ? 5 : p.page_tokens == 64 ? 6 : 7;
    return a;
}

cudaError_t launch_kv_extend(const gdn_kv_pages& p, const int32_t* lens, const int32_t* n_new, int n_seqs, const uint64_t* tree,
                             int64_t max_tokens, int32_t* lens_out, int32_t* cu, int32_t* positions, int64_t* slots, cudaStream_t st) {
    PagesArgs a = pages_args(p, lens, n_seqs);
    a.n_new = n_new;
    a.tree = tree;
    a.max_tokens = static_cast<int>(max_tokens);
    a.lens_out = lens_out;
    a.cu = cu;
    a.positions = positions;
    a.slots = slots;
    // one CTA where its threads have a few tokens each, else all SMs and a second launch for what they read (64 sequences,
    // 2048 tokens: 6.3 us in one, 8.3 in two; 4096: 8.3 and 7.8; one sequence 3.9 and 5.9, 4.9 and 6.0, of 16384 11 and 6)
    if (max_tokens <= PG_STEP * PG_THREADS) return launch_dependent(pages_extend_kernel, dim3(1), dim3(PG_THREADS), 0, st, a, true, true);
    const int64_t want = (max_tokens + PG_STEP * PG_THREADS - 1) / (PG_STEP * PG_THREADS);
    const cudaError_t e = launch_dependent(pages_extend_kernel, dim3(static_cast<unsigned>(want < 304 ? want : 304)), dim3(PG_THREADS), 0, st,
                                           a, true, false);
    return e != cudaSuccess ? e : launch_dependent(pages_extend_kernel, dim3(1), dim3(PG_THREADS), 0, st, a, false, true);
}

cudaError_t launch_kv_trim(const gdn_kv_pages& p, const int32_t* keep, int n_seqs, cudaStream_t st) {
    const PagesArgs a = pages_args(p, keep, n_seqs);
    // As above, where many pages may come back: only the table's width says so here.  In a step of drafts few do, and two
    // launches then cost more (64 pages of 64 sequences 3.2 us in one, 4.7 in two, at any width; 5120 of 256 7.2 and 5.1);
    // but one CTA takes 25 us for 32768 pages and 89 for 102400, where two launches take 5 and 7, so the width is a bound
    // on that (58 us for 65536).
    const int64_t most = static_cast<int64_t>(n_seqs) * p.max_blocks;
    if (most <= 128 * PG_THREADS) return launch_dependent(pages_trim_kernel, dim3(1), dim3(PG_THREADS), 0, st, a, true, true);
    const int64_t want = (most + 4 * PG_STEP * PG_THREADS - 1) / (4 * PG_STEP * PG_THREADS);
    const cudaError_t e = launch_dependent(pages_trim_kernel, dim3(static_cast<unsigned>(want < 304 ? want : 304)), dim3(PG_THREADS), 0, st, a,
                                           true, false);
    return e != cudaSuccess ? e : launch_dependent(pages_trim_kernel, dim3(1), dim3(PG_THREADS), 0, st, a, false, true);
}

int* pages_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_pages_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

int* pages_skipped_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_pages_skipped) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdn
