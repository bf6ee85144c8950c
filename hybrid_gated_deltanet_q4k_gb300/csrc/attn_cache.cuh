// What the two kernels of the cache attention share: the call's arguments, the
// sequences as read on the device, the partition into runs, and code helpers.
#pragma once

#include "common.cuh"
#include "tma.cuh"

#include <cuda_fp8.h>

#include <mutex>

namespace gdn {

// Of each translation unit: a wait that ran out (or an index check of the debug
// build), and an index held in device memory that was out of range.  Two words,
// so that a skipped index does not hide that the results are not valid.
static __device__ int g_attn_cache_error, g_attn_cache_skipped;

constexpr int AC_BLOCK = 128;           // keys of a block
constexpr int AC_MAX_RUNS = 152;        // one CTA per SM
constexpr int AC_JOIN_THREADS = 256;
constexpr float AC_MARGIN = 4.0f;
constexpr float AC_LIFT = 11.0f;        // fp16 probabilities times 2^11
// The least log2 of a value's scale that the running maximum knows: a smaller
// scale (a row of zeros has 0) counts as 2^-80 there, and as it is in the
// probability.  A key adds 2^(x - m) to the sum, and while only such keys have
// been seen m is as low as x - 80: up to 2^(4 + 11 + 80), which 2^30 keys do not
// bring past fp32.  AC_VS_FLOOR keeps the logarithm of a scale of 0 finite.
constexpr float AC_VS_MIN = -80.0f, AC_VS_TINY = 0x1p-80f, AC_VS_FLOOR = 1e-44f;
// The least exponent of a row of q that its power of two still lifts to 2^14: 2^(14 +
// 112) and its inverse are normal numbers, and so are 2^(14 - 127) and its inverse.
constexpr int AC_Q_MIN = -112;
constexpr float LOG2E = 1.4426950408889634f;

struct AttCacheArgs {
    int64_t n_pages;
    int heads, page, page_shift, ratio, hq;
    const void* v;
    const float *sk, *sv;
    const uint16_t* q;
    uint16_t* o;
    int64_t ld_q, ld_o, ld_table, n_tokens;
    const int32_t *cu, *table, *lens;
    const uint64_t* tree;
    int n_seqs, max_q, max_blocks;
    int runs, ranks;    // runs of blocks, and row tiles of a pair (a CTA per run and rank of rows)
    int start;          // blocks that each pair counts more than it has
    int box;            // keys of one copy
    int wide;           // rows of q and o start on 32 bytes (kernel for many rows)
    float sl2;          // scale * log2(e)
    float* part;        // partial accumulators [runs * ranks][2][rows][D]
    float2* part_ml;    // and their maxima and sums [runs * ranks][2][rows]
    uint64_t wait_ns;   // the limit of a wait
    int withhold;       // test: the first copy of a CTA is never issued, so that a wait for it runs out
};

// A sequence as the kernels see it, its device-held numbers forced into range.
struct AcSeq {
    int tok, nq, len;
};
__device__ __forceinline__ AcSeq ac_seq(const AttCacheArgs& a, int s, bool report) {
    AcSeq r;
    const int lo = a.cu ? a.cu[s] : s * a.max_q, hi = a.cu ? a.cu[s + 1] : lo + a.max_q;
    const int64_t cap = static_cast<int64_t>(a.max_blocks) * a.page;
    const int len = a.lens[s];
    const bool ok = lo >= 0 && hi >= lo && hi <= a.n_tokens && hi - lo <= a.max_q;
    r.tok = ok ? lo : 0;
    r.nq = ok ? hi - lo : 0;
    r.len = len < 0 ? 0 : len > cap ? static_cast<int>(cap) : len;
    if (report && (!ok || r.len != len)) atomicExch(&g_attn_cache_skipped, static_cast<int>(ERR_INDEX));
    return r;
}
// Blocks of each of its pairs (at least one where there is a row to write), and as they count.
__device__ __forceinline__ int ac_blocks(const AcSeq& s) { return s.len == 0 ? 1 : (s.len - 1) / AC_BLOCK + 1; }

// The counted blocks before each sequence (of one head), pre[0 .. n_seqs], and
// the sequences, by all threads of a CTA.
static_assert(GDN_MAX_SEQS <= AC_JOIN_THREADS, "a thread per sequence");
__device__ __forceinline__ void ac_prefix(const AttCacheArgs& a, int64_t* pre, AcSeq* seq, int64_t* wsum, bool report) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = (a.n_seqs + 31) / 32;
    int64_t v = 0;
    if (t < a.n_seqs) {
        const AcSeq q = ac_seq(a, t, report);
        seq[t] = q;
        v = q.nq == 0 ? 0 : ac_blocks(q) + a.start;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (warps > 1) {
        if (lane == 31 && warp < warps) wsum[warp] = v;
        __syncthreads();
        for (int w = 0; w < min(warp, warps); ++w) v += wsum[w];
    }
    if (t < a.n_seqs) pre[t + 1] = v;
    if (t == 0) pre[0] = 0;
    __syncthreads();
}
// Blocks per run, from the total over all pairs.
__device__ __forceinline__ int64_t ac_run_blocks(const AttCacheArgs& a, int64_t total) {
    return total < a.runs ? 1 : (total + a.runs - 1) / a.runs;
}

// One run's share of a pair: its blocks [b0, b1) of `blocks`.
struct AcPiece {
    AcSeq q;
    int s, head, b0, b1, blocks;
};
// The piece at counted block `at` (moved past it) of a run that ends at `end`;
// false at the end.  s: the sequence to look from.
__device__ __forceinline__ bool ac_next(const AttCacheArgs& a, const int64_t* pre, const AcSeq* seq, int64_t& at, int64_t end,
                                        int& s, AcPiece& p) {
    while (at < end) {
        while (pre[s + 1] * a.heads <= at) ++s;
        const int counted = static_cast<int>(pre[s + 1] - pre[s]);
        p.head = static_cast<int>((at - pre[s] * a.heads) / counted);
        const int64_t first = pre[s] * a.heads + static_cast<int64_t>(p.head) * counted;
        p.q = seq[s];
        p.s = s;
        p.blocks = counted - a.start;
        p.b0 = max(static_cast<int>(at - first) - a.start, 0);
        p.b1 = end - first < counted ? max(static_cast<int>(end - first) - a.start, 0) : p.blocks;
        at = first + counted < end ? first + counted : end;
        if (p.b0 < p.b1) return true;   // not only the blocks that count for the start
    }
    return false;
}
// The sequence of counted block `at`: the last s with pre[s] * heads <= at.
__device__ __forceinline__ int ac_seq_of(const AttCacheArgs& a, const int64_t* pre, int64_t at) {
    int s = 0;
    for (int hi = a.n_seqs - 1; s < hi;) {
        const int mid = (s + hi + 1) >> 1;
        if (pre[mid] * a.heads <= at) s = mid; else hi = mid - 1;
    }
    return s;
}

// Two codes of w (bytes I and J) as fp16 values; int8 codes come with the top bit flipped.
template <int T, int I, int J>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
    if constexpr (T == GDN_KV_I8) {
        const uint32_t b = __byte_perm(w, 0x64646464u, 0x4040u | (J << 8) | I);   // 1024 + (code + 128)
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&b), __half2half2(__ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const uint32_t b = __byte_perm(w, 0, (J << 4) | I);
        uint32_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
        return r;
    }
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
        : "memory");
}

// ------------------------------------------------------------ host

inline PFN_cuTensorMapEncodeTiled_v12000 ac_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// The pages as [n_pages * heads][slabs][page rows][slab bytes]; a box is
// the rows that a tile has in one page, in some of the slabs.  The page index
// is its own dimension, so no coordinate grows with the cache's bytes.
inline bool ac_map(CUtensorMap* map, const void* ptr, const gdn_kv_cache& c, int box_rows, int box_slabs) {
    auto enc = ac_map_encoder();
    if (!enc) return false;
    const bool wide = c.dtype == GDN_KV_BF16;
    const int row = c.head_dim * (wide ? 2 : 1), slab = row < 128 ? row : 128;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(wide ? slab / 2 : slab), static_cast<cuuint64_t>(c.page_tokens),
                          static_cast<cuuint64_t>(row / slab), static_cast<cuuint64_t>(c.n_pages * c.n_kv_heads)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(slab),
                             static_cast<cuuint64_t>(row) * c.page_tokens};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(dims[0]), static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_slabs), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, wide ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, slab == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdn
