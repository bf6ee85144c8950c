// Attention of new tokens (one, a chain, or a tree of drafts) over the paged
// key/value cache.
//
// The rows of a (sequence, key/value head) are its new tokens times the query
// heads that share the head: row r is token r / ratio, head r % ratio.  Every
// cached key and value of the head is read once for all of them, so a few rows
// are bound by memory: 2 D bytes of 8-bit cache (4 D of bf16) per key against
// 4 D flops per row and key.
//
// Work is cut into blocks of 128 keys, numbered through all (sequence, head)
// pairs, and each CTA takes one contiguous run of them: every SM gets the same
// bytes whatever the lengths are, with nothing planned on the host (lengths
// and offsets are read on the device, so a captured graph may be replayed with
// others).  A pair that lies in one run is written at once; the others leave
// (maximum, sum, fp32 accumulator) partials that a second kernel joins.
//
// Inside a CTA each of the eight warps walks every eighth tile of 16 keys on
// its own: its lane 0 copies the tile's keys and values by TMA into the warp's
// own ring, the warp multiplies them on the tensor cores (m16n8k16) with the
// scores and probabilities never leaving registers, and keeps its own running
// maximum, sum and accumulator; there is no barrier between warps until the
// end of a pair, where the eight results are joined in shared memory.
//
// 8-bit codes become fp16 in registers (exact), with the row scales kept out
// of the products: a key's scale multiplies its score, and a value's scale
// goes into the exponent of its probability, p' = 2^(x + log2 vs - m), which
// enters the product as fp16; the softmax sum adds p = 2^(x - m) in fp32.
// Scores x are in units of log 2.  A maximum is raised only past a margin of
// 2^8, so the accumulators are seldom rescaled; fp16 probabilities carry a
// factor 2^7 (at most 2^15 with the margin).  Those below 2^-14, where fp16
// loses bits, matter only to elements that are zero in every more probable
// row; a tile that has one multiplies the rounding errors p' - fp16(p') in
// bf16, whose exponents reach as far as fp32's, in a second pass.  q goes to fp16 times a power of two per row that puts its largest
// element in [2^14, 2^15): elements below 2^-38 of it are lost.
#include "common.cuh"
#include "tma.cuh"

#include <cuda_fp8.h>

#include <mutex>

namespace gdn {

static __device__ int g_attn_cache_error;

constexpr int AC_WARPS = 8;
constexpr int AC_THREADS = 32 * AC_WARPS;
constexpr int AC_TILE = 16;             // keys per tile
constexpr int AC_BLOCK = AC_WARPS;      // tiles of a block: one per warp
constexpr int AC_MAX_RUNS = 152;        // one CTA per SM
constexpr int AC_RING = 128 * 1024;     // bytes of tiles in flight per CTA
constexpr float AC_MARGIN = 8.0f;
constexpr float AC_LIFT = 7.0f;         // fp16 probabilities times 2^7
constexpr float LOG2E = 1.4426950408889634f;

struct AttCacheArgs {
    int64_t n_pages;
    int heads, page, page_shift, ratio, hq;
    const float *sk, *sv;
    const uint16_t* q;
    uint16_t* o;
    int64_t ld_q, ld_o, ld_table, n_tokens;
    const int32_t *cu, *table, *lens;
    const uint64_t* tree;
    int n_seqs, max_q, max_blocks;
    int runs, ranks;    // runs of tiles, and row tiles of a pair (a CTA per run and rank)
    float sl2;          // scale * log2(e)
    float* part;        // [runs * ranks][2][rows][D + 2] partials
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
    if (report && (!ok || r.len != len)) atomicCAS(&g_attn_cache_error, 0, static_cast<int>(ERR_INDEX));
    return r;
}
// Blocks of each of its pairs: at least one where there is a row to write.
__device__ __forceinline__ int64_t ac_blocks(const AcSeq& s) {
    constexpr int KEYS = AC_BLOCK * AC_TILE;
    return s.nq == 0 ? 0 : s.len == 0 ? 1 : (static_cast<int64_t>(s.len) + KEYS - 1) / KEYS;
}

// The blocks before each sequence (of one head): pre[0 .. n_seqs], by all AC_THREADS threads.
static_assert(GDN_MAX_SEQS <= AC_THREADS, "a thread per sequence");
__device__ __forceinline__ void ac_prefix(const AttCacheArgs& a, int64_t* pre, int64_t* wsum, bool report) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int64_t v = t < a.n_seqs ? ac_blocks(ac_seq(a, t, report)) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += wsum[w];
    if (t < a.n_seqs) pre[t + 1] = v;
    if (t == 0) pre[0] = 0;
    __syncthreads();
}
// Blocks per run, from the total over all pairs.
__device__ __forceinline__ int64_t ac_run_blocks(const AttCacheArgs& a, int64_t total) {
    return total < a.runs ? 1 : (total + a.runs - 1) / a.runs;
}

// ------------------------------------------------------------ tensor-core steps

template <int T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (T == GDN_KV_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
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

// ------------------------------------------------------------ shared memory

// A row of a tile is cut into slabs of 128 bytes (one of 64 for 8-bit heads of
// 64), each slab [16 keys][128 bytes] with the TMA's 128-byte (64-byte)
// swizzle, so that eight keys' 16-byte pieces fall into different banks.
template <int D, int T, int MT>
struct AcSmem {
    static constexpr int ES = T == GDN_KV_BF16 ? 2 : 1;
    static constexpr int ROW = D * ES;
    static constexpr int SLAB = ROW < 128 ? ROW : 128;      // bytes of a row in one slab
    static constexpr int NSLAB = ROW / SLAB;
    static constexpr int HALF = AC_TILE * ROW;              // the keys, or the values, of a tile
    static constexpr int ST = AC_RING / AC_WARPS / (2 * HALF);   // tiles in flight per warp
    static constexpr int ROWS = 16 * MT;
    static constexpr int OLD = D + 8;                       // padded rows of the joined accumulators
    static constexpr int JOIN = AC_WARPS * ROWS * OLD * 4;
    static constexpr int R0 = 0;                            // ring; the accumulators at the end of a pair
    static constexpr int S0 = AC_RING > JOIN ? AC_RING : JOIN;   // row scales of the tiles in flight: [warp][stage][2][16]
    static constexpr int M0 = S0 + AC_WARPS * ST * 2 * AC_TILE * 4;   // maxima and sums: [warp][rows][2]
    static constexpr int P0 = M0 + AC_WARPS * ROWS * 2 * 4;      // blocks before each sequence
    static constexpr int W0 = P0 + (GDN_MAX_SEQS + 2) * 8;
    static constexpr int F0 = W0 + AC_WARPS * 8;                 // pages in range: [warp][stage]
    static constexpr int Q0 = (F0 + AC_WARPS * ST * 4 + 15) & ~15;   // q fragments [row tile][step][lane] x 16 bytes
    static constexpr int B0 = Q0 + MT * (D / 16) * 512;          // mbarriers [warp][stage][keys, values]
    static constexpr int BYTES = B0 + AC_WARPS * ST * 2 * 8;
    static_assert(BYTES + 1024 <= 227 * 1024, "shared memory of a CTA");
};

// Byte offset of 16-byte piece c of key r in a tile.
template <class L>
__device__ __forceinline__ uint32_t ac_piece(int r, int c) {
    if constexpr (L::SLAB == 128)
        return static_cast<uint32_t>((c >> 3) * (AC_TILE * 128) + r * 128 + (((c ^ r) & 7) << 4));
    else
        return static_cast<uint32_t>(r * 64 + (((c ^ (r >> 1)) & 3) << 4));
}

// ------------------------------------------------------------ the kernel

template <int D, int T, int MT>
__global__ void __launch_bounds__(AC_THREADS, 1)
attn_cache_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ AttCacheArgs a) {
    using L = AcSmem<D, T, MT>;
    constexpr int NT = D / 8;             // output column tiles
    constexpr int KT = D / 16;            // 16-wide steps of a row
    constexpr bool Q8 = T != GDN_KV_BF16;
    extern __shared__ __align__(1024) unsigned char smb[];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smb) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    int64_t* pre = reinterpret_cast<int64_t*>(base + L::P0);
    float* join = reinterpret_cast<float*>(base + L::R0);
    float2* ml = reinterpret_cast<float2*>(base + L::M0);
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + L::B0) + warp * L::ST * 2;
    unsigned char* ring = base + L::R0 + warp * L::ST * 2 * L::HALF;
    float* scales = reinterpret_cast<float*>(base + L::S0) + warp * L::ST * 2 * AC_TILE;
    int* page_in = reinterpret_cast<int*>(base + L::F0) + warp * L::ST;
    uint4* qsm = reinterpret_cast<uint4*>(base + L::Q0);

    pdl_trigger();
    if (lane == 0) {
        for (int i = 0; i < L::ST * 2; ++i) mbar_init_cta(bars + i, 1);
        mbar_init_fence();
    }
    const int run = blockIdx.x / a.ranks, rank = blockIdx.x % a.ranks;
    ac_prefix(a, pre, reinterpret_cast<int64_t*>(base + L::W0), blockIdx.x == 0);
    const int64_t total = pre[a.n_seqs] * a.heads, per = ac_run_blocks(a, total);
    int64_t at = run * per;
    const int64_t end = at + per < total ? at + per : total;
    if (at >= end) return;

    // the sequence of the first block: the last s with pre[s] * heads <= at
    int s = 0;
    for (int hi = a.n_seqs - 1; s < hi;) {
        const int mid = (s + hi + 1) >> 1;
        if (pre[mid] * a.heads <= at) s = mid; else hi = mid - 1;
    }
    uint32_t uses = 0;          // tiles this warp has taken: stage uses % ST, phase uses / ST
    bool dead = false;          // a wait ran out

    while (at < end) {
        while (pre[s + 1] * a.heads <= at) ++s;
        const AcSeq q = ac_seq(a, s, false);
        const int blocks = static_cast<int>(pre[s + 1] - pre[s]);
        const int head = static_cast<int>((at - pre[s] * a.heads) / blocks);
        const int64_t first = pre[s] * a.heads + static_cast<int64_t>(head) * blocks;
        const int b0 = static_cast<int>(at - first);
        const int b1 = end - first < blocks ? static_cast<int>(end - first) : blocks;
        at = first + b1;
        const int t0 = b0 * AC_BLOCK, t1 = min(b1 * AC_BLOCK, max(1, (q.len + AC_TILE - 1) / AC_TILE));   // tiles
        const int row0 = rank * L::ROWS, rows = min(q.nq * a.ratio - row0, L::ROWS);
        if (rows <= 0) continue;
        const int ctx = q.len - q.nq;      // keys every row sees
        const int32_t* table = a.table + s * a.ld_table;

        // ---- copies: tile u of the piece goes to stage uses % ST
        const int mine = t1 - t0 - warp > 0 ? (t1 - t0 - warp + AC_WARPS - 1) / AC_WARPS : 0;   // tiles of this warp
        auto page_of = [&](int i) {
            return table[min(((t0 + warp + i * AC_WARPS) * AC_TILE) >> a.page_shift, a.max_blocks - 1)];
        };
        auto issue = [&](int i, int page, int half) {   // lane 0
            const int tile = t0 + warp + i * AC_WARPS, st = static_cast<int>((uses + i) % L::ST);
            const int row = (tile * AC_TILE) & (a.page - 1);
            const bool in = page >= 0 && page < a.n_pages;
            const int p = in ? page : 0;                // an unseen page: any rows, all of them masked
            page_in[st] = in;
            uint64_t* bar = bars + st * 2 + half;
            mbar_expect_tx(bar, L::HALF + (Q8 ? AC_TILE * 4 : 0));
            tma_load_4d(ring + (st * 2 + half) * L::HALF, half ? &mv : &mk, bar, 0, row, 0, p * a.heads + head);
            if constexpr (Q8)
                bulk_load_1d(scales + (st * 2 + half) * AC_TILE,
                             (half ? a.sv : a.sk) + (static_cast<int64_t>(p) * a.heads + head) * a.page + row, AC_TILE * 4, bar);
        };
        if (lane == 0 && !dead) {
            for (int i = 0; i < L::ST && i < mine; ++i) {
                const int p = page_of(i);
                issue(i, p, 0);
                issue(i, p, 1);
            }
        }
        int page_next = L::ST < mine ? page_of(L::ST) : 0;   // read one tile ahead of its copies

        // ---- q fragments: rows 16 mt + g and + 8, the same for every warp, in
        // shared memory (in registers they would spill).  The d elements a
        // thread holds at step kt are those its key fragments hold.
        float qs[MT][2];
        uint64_t seen[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t qf[KT][4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int r = 16 * mt + 8 * hh + g, rr = row0 + r, i = rr / a.ratio;
                const bool on = r < rows;
                const uint16_t* src = a.q + static_cast<int64_t>(q.tok + (on ? i : 0)) * a.ld_q +
                                      (head * a.ratio + (on ? rr - i * a.ratio : 0)) * D;
                seen[mt][hh] = !on ? 0 : a.tree ? a.tree[q.tok + i] : i >= 63 ? ~0ull : (1ull << (i + 1)) - 1;
                if constexpr (!Q8) {
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        qf[kt][hh] = on ? *reinterpret_cast<const uint32_t*>(src + 16 * kt + 2 * t) : 0u;
                        qf[kt][2 + hh] = on ? *reinterpret_cast<const uint32_t*>(src + 16 * kt + 8 + 2 * t) : 0u;
                    }
                    qs[mt][hh] = a.sl2;
                } else {
                    float amax = 0.0f;
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        const uint2 w = on ? *reinterpret_cast<const uint2*>(src + 16 * kt + 4 * t) : make_uint2(0u, 0u);
                        qf[kt][hh] = w.x;
                        qf[kt][2 + hh] = w.y;
                        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(__uint_as_float(w.x << 16)), fabsf(__uint_as_float(w.x & 0xffff0000u))),
                                                 fmaxf(fabsf(__uint_as_float(w.y << 16)), fabsf(__uint_as_float(w.y & 0xffff0000u)))));
                    }
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                    // 2^e with amax 2^e in [2^14, 2^15): exact both ways within the exponents that keep 2^e finite
                    const int ex = min(max(static_cast<int>((__float_as_uint(amax) >> 23) & 255) - 127, -100), 100);
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - ex) << 23);
                    qs[mt][hh] = a.sl2 * __uint_as_float(static_cast<uint32_t>(127 - 14 + ex) << 23);
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const uint32_t w = qf[kt][e + hh];
                            qf[kt][e + hh] = f16x2_bits(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
                        }
                }
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
                if (kt % AC_WARPS == warp)
                    qsm[(mt * KT + kt) * 32 + lane] = make_uint4(qf[kt][0], qf[kt][1], qf[kt][2], qf[kt][3]);
        }
        __syncthreads();

        float o[MT][NT][4], m[MT][2], l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.0f;
        }

#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            const int st = static_cast<int>((uses + i) % L::ST);
            const uint32_t par = ((uses + i) / L::ST) & 1;
            const int key0 = (t0 + warp + i * AC_WARPS) * AC_TILE;
            int lim = q.len - key0;   // keys of this tile below `lim` exist
            const uint32_t kb = smem_addr(ring + st * 2 * L::HALF), vb = kb + L::HALF;

            if (!dead && !mbar_wait_bounded(bars + st * 2, par, &g_attn_cache_error, ERR_WAIT_TIMEOUT)) dead = true;
            dead = __any_sync(0xffffffffu, dead);
            if (dead) break;
            if (!page_in[st]) {
                if (lane == 0 && lim > 0) atomicCAS(&g_attn_cache_error, 0, static_cast<int>(ERR_INDEX));
                lim = 0;
            }
            const bool edge = key0 + AC_TILE > ctx || lim < AC_TILE;   // some row may not see some key

            // ---- scores
            auto qfrag = [&](int mt, int kt, uint32_t (&f)[4]) {
                const uint4 w = qsm[(mt * KT + kt) * 32 + lane];
                f[0] = w.x;
                f[1] = w.y;
                f[2] = w.z;
                f[3] = w.w;
            };
            float sc[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[mt][n][e] = 0.0f;
            if constexpr (!Q8) {
                // matrices: keys 0-7 and 8-15, each by the two 8-wide halves of the step
                const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    uint32_t b[4];
                    ldsm_x4(kb + ac_piece<L>(kr, 2 * kt + kc), b);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t f[4];
                        qfrag(mt, kt, f);
                        mma16816<T>(sc[mt][0], f, b[0], b[1]);
                        mma16816<T>(sc[mt][1], f, b[2], b[3]);
                    }
                }
            } else {
                // matrices: keys 0-7 and 8-15 of 16 codes, then of the next 16; a thread gets codes 4t .. 4t+3
                const int kr = (lane & 7) + (((lane >> 3) & 1) << 3), kc = lane >> 4;
#pragma unroll
                for (int kt = 0; kt < KT; kt += 2) {
                    uint32_t b[4];
                    ldsm_x4(kb + ac_piece<L>(kr, kt + kc), b);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t k0[2], k1[2];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const uint32_t w = T == GDN_KV_I8 ? b[2 * u + n] ^ 0x80808080u : b[2 * u + n];
                            k0[n] = codes_f16<T, 0, 1>(w);
                            k1[n] = codes_f16<T, 2, 3>(w);
                        }
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t f[4];
                            qfrag(mt, kt + u, f);
                            mma16816<T>(sc[mt][0], f, k0[0], k1[0]);
                            mma16816<T>(sc[mt][1], f, k0[1], k1[1]);
                        }
                    }
                }
            }
            // scores to units of log 2; keys 2t, 2t+1, 8+2t, 9+2t of this thread
            float kv[2][2], lv[2][2];
            if constexpr (Q8) {
                const float* ks = scales + st * 2 * AC_TILE;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 x = *reinterpret_cast<const float2*>(ks + 8 * n + 2 * t);
                    kv[n][0] = x.x;
                    kv[n][1] = x.y;
                }
            }
            __syncwarp();
            const bool more = i + L::ST < mine;
            if (lane == 0 && more) issue(i + L::ST, page_next, 0);

            if (!mbar_wait_bounded(bars + st * 2 + 1, par, &g_attn_cache_error, ERR_WAIT_TIMEOUT)) dead = true;
            dead = __any_sync(0xffffffffu, dead);
            if (dead) break;
            if constexpr (Q8) {
                const float* vs = scales + (st * 2 + 1) * AC_TILE;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 x = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * t);
                    // a scale below 2^-110 counts as that (a row of zeros has scale 0 and codes 0)
                    lv[n][0] = lg2(fmaxf_nan(x.x, 7.7e-34f));
                    lv[n][1] = lg2(fmaxf_nan(x.y, 7.7e-34f));
                }
            }

            // ---- softmax of the tile
            uint32_t pf[MT][4];
            bool faint = false;      // an fp16 probability that lost bits
            float pk[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = sc[mt][n][e] * qs[mt][e >> 1];
                        if constexpr (Q8) x *= kv[n][e & 1];
                        if (edge) {
                            const int j = 8 * n + 2 * t + (e & 1), d = key0 + j - ctx;
                            if (j >= lim || (d >= 0 && !((seen[mt][e >> 1] >> (d & 63)) & 1))) x = -INFINITY;
                        }
                        sc[mt][n][e] = x;
                    }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = sc[mt][e >> 1][2 * hh + (e & 1)];
                        y[e] = x;
                        if constexpr (Q8)
                            if (x != -INFINITY) y[e] = x + lv[e >> 1][e & 1];
                    }
                    float bm = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2));
                    const float old = m[mt][hh];
                    const bool up = bm > old + AC_MARGIN || (old == -INFINITY && bm > old);
                    if (__any_sync(0xffffffffu, up)) {
                        const float mn = up ? bm : old, c = old == -INFINITY ? 0.0f : ex2_ftz(old - mn);
                        m[mt][hh] = mn;
                        l[mt][hh] *= c;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            o[mt][n][2 * hh] *= c;
                            o[mt][n][2 * hh + 1] *= c;
                        }
                    }
                    const float mm = m[mt][hh] == -INFINITY ? 0.0f : m[mt][hh];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = sc[mt][e >> 1][2 * hh + (e & 1)];
                        if constexpr (Q8) {
                            const float p = ex2_ftz(y[e] - mm + AC_LIFT);
                            pk[mt][e >> 1][2 * hh + (e & 1)] = p;
                            faint |= p != 0.0f && p < 6.1035156e-5f;
                            l[mt][hh] += ex2_ftz(x - mm + AC_LIFT);
                        } else {
                            pk[mt][e >> 1][2 * hh + (e & 1)] = ex2_ftz(y[e] - mm);
                        }
                    }
                }
                // the first product's accumulators are the second one's A fragments
                if constexpr (Q8) {
                    pf[mt][0] = f16x2_bits(pk[mt][0][0], pk[mt][0][1]);
                    pf[mt][1] = f16x2_bits(pk[mt][0][2], pk[mt][0][3]);
                    pf[mt][2] = f16x2_bits(pk[mt][1][0], pk[mt][1][1]);
                    pf[mt][3] = f16x2_bits(pk[mt][1][2], pk[mt][1][3]);
                } else {
                    pf[mt][0] = bf16x2(pk[mt][0][0], pk[mt][0][1]);
                    pf[mt][1] = bf16x2(pk[mt][0][2], pk[mt][0][3]);
                    pf[mt][2] = bf16x2(pk[mt][1][0], pk[mt][1][1]);
                    pf[mt][3] = bf16x2(pk[mt][1][2], pk[mt][1][3]);
                    // the sum takes the probabilities as rounded, so their rounding cancels where few keys matter
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        l[mt][e & 1] += __uint_as_float(pf[mt][e] << 16) + __uint_as_float(pf[mt][e] & 0xffff0000u);
                }
            }

            // ---- values: column tiles 2c and 2c+1 of each 16 columns
            const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), vc = lane >> 4;
            constexpr int STEP = Q8 ? 4 : 2;     // column tiles per ldmatrix
            uint32_t odd = 0;                    // a value that is not finite at the edge
            uint32_t km[2] = {~0u, ~0u};         // halves of the fragments whose keys exist
            if (edge) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    km[n] = (8 * n + 2 * t < lim ? 0xffffu : 0u) | (8 * n + 2 * t + 1 < lim ? 0xffff0000u : 0u);
            }
            // fragment register of keys 2t, 2t+1 (n = 0) or 8+2t, 9+2t: what does not exist, and
            // what is not finite (its rows see it below), is taken as zero
            auto clean = [&](uint32_t w, int n) {
                constexpr uint32_t EXP = Q8 ? 0x7c00u : 0x7f80u;
                w &= km[n];
                if (T != GDN_KV_I8) {
                    if ((w & EXP) == EXP) {
                        w &= 0xffff0000u;
                        odd = 1;
                    }
                    if ((w & (EXP << 16)) == (EXP << 16)) {
                        w &= 0xffffu;
                        odd = 1;
                    }
                }
                return w;
            };
            auto values = [&](int n, uint32_t (&f)[STEP][2]) {   // fragments of column tiles n .. n + STEP - 1
                uint32_t b[4];
                ldsm_x4_trans(vb + ac_piece<L>(vr, (Q8 ? n / 2 : n) + vc), b);
                if constexpr (Q8) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t w = T == GDN_KV_I8 ? b[u] ^ 0x80808080u : b[u];
                        f[(u >> 1) * 2][u & 1] = codes_f16<T, 0, 2>(w);
                        f[(u >> 1) * 2 + 1][u & 1] = codes_f16<T, 1, 3>(w);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < 4; ++u) f[u >> 1][u & 1] = b[u];
                }
                if (edge) {
#pragma unroll
                    for (int u = 0; u < STEP; ++u) {
                        f[u][0] = clean(f[u][0], 0);
                        f[u][1] = clean(f[u][1], 1);
                    }
                }
            };
#pragma unroll
            for (int n = 0; n < NT; n += STEP) {
                uint32_t f[STEP][2];
                values(n, f);
#pragma unroll
                for (int u = 0; u < STEP; ++u)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) mma16816<T>(o[mt][n + u], pf[mt], f[u][0], f[u][1]);
            }
            if constexpr (Q8) {
                if (__any_sync(0xffffffffu, faint)) {
                    uint32_t rf[MT][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&pf[mt][e]));
                            const float* p = &pk[mt][e >> 1][2 * (e & 1)];
                            rf[mt][e] = bf16x2(p[0] - r.x, p[1] - r.y);
                        }
#pragma unroll
                    for (int n = 0; n < NT; n += STEP) {
                        uint32_t f[STEP][2];
                        values(n, f);
#pragma unroll
                        for (int u = 0; u < STEP; ++u) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&f[u][e]));
                                f[u][e] = bf16x2(c.x, c.y);
                            }
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) mma16816<GDN_KV_BF16>(o[mt][n + u], rf[mt], f[u][0], f[u][1]);
                        }
                    }
                }
            }
            if (T != GDN_KV_I8 && edge && __any_sync(0xffffffffu, odd)) {
                // rows that see such a key add its term by themselves
                const unsigned char* vt = ring + (st * 2 + 1) * L::HALF;
#pragma unroll 1
                for (int j = 0; j < min(lim, AC_TILE); ++j) {
                    const int d = key0 + j - ctx, src = (lane & ~3) | ((j & 7) >> 1);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const float p0 = __shfl_sync(0xffffffffu, j < 8 ? pk[mt][0][2 * hh] : pk[mt][1][2 * hh], src);
                            const float p1 = __shfl_sync(0xffffffffu, j < 8 ? pk[mt][0][2 * hh + 1] : pk[mt][1][2 * hh + 1], src);
                            const bool see = d < 0 || ((seen[mt][hh] >> (d & 63)) & 1);
                            if (!see) continue;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    float v;
                                    if constexpr (Q8) {
                                        const int col = 16 * (n >> 1) + 4 * t + 2 * e + (n & 1);
                                        v = __half2float(__half(__nv_cvt_fp8_to_halfraw(vt[ac_piece<L>(j, col >> 4) + (col & 15)], __NV_E4M3)));
                                    } else {
                                        const int col = 8 * n + 2 * t + e;
                                        v = bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(vt + ac_piece<L>(j, col >> 3) + 2 * (col & 7)));
                                    }
                                    if (!(fabsf(v) < INFINITY)) o[mt][n][2 * hh + e] += (j & 1 ? p1 : p0) * v;
                                }
                        }
                }
            }
            __syncwarp();
            if (lane == 0 && more) issue(i + L::ST, page_next, 1);
            if (i + L::ST + 1 < mine) page_next = page_of(i + L::ST + 1);
        }
        uses += mine;

        // ---- join the warps
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                l[mt][hh] += __shfl_xor_sync(0xffffffffu, l[mt][hh], 1);
                l[mt][hh] += __shfl_xor_sync(0xffffffffu, l[mt][hh], 2);
                if (t == 0) ml[warp * L::ROWS + 16 * mt + 8 * hh + g] = make_float2(m[mt][hh], l[mt][hh]);
            }
        __syncthreads();   // every warp is done with its ring
        const int live = min(t1 - t0, AC_WARPS);
        if (warp < live) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int r = 16 * mt + 8 * hh + g;
                    if (r >= rows) continue;
                    float* dst = join + (warp * L::ROWS + r) * L::OLD;
                    if constexpr (Q8) {
#pragma unroll
                        for (int n = 0; n < NT; n += 2)
                            *reinterpret_cast<float4*>(dst + 8 * n + 4 * t) =
                                make_float4(o[mt][n][2 * hh], o[mt][n + 1][2 * hh], o[mt][n][2 * hh + 1], o[mt][n + 1][2 * hh + 1]);
                    } else {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            *reinterpret_cast<float2*>(dst + 8 * n + 2 * t) = make_float2(o[mt][n][2 * hh], o[mt][n][2 * hh + 1]);
                    }
                }
        }
        __syncthreads();
        const bool whole = b0 == 0 && b1 == blocks;
        float* part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (b0 > 0 ? 0 : 1)) * L::ROWS * (D + 2);
        for (int e = tid; e < rows * (D / 2); e += AC_THREADS) {
            const int r = e / (D / 2), c = (e % (D / 2)) * 2;
            float mx = -INFINITY;
            for (int w = 0; w < live; ++w) mx = fmaxf_nan(mx, ml[w * L::ROWS + r].x);
            float lt = 0.0f, x = 0.0f, y = 0.0f;
            for (int w = 0; w < live; ++w) {
                const float2 v = ml[w * L::ROWS + r];
                // weight 0, not left out: a NaN (of a score, or 0 times an infinite value) stays
                const float f = v.x == -INFINITY ? 0.0f : ex2_ftz(v.x - mx);
                const float2 ov = *reinterpret_cast<const float2*>(join + (w * L::ROWS + r) * L::OLD + c);
                lt = fmaf(f, v.y, lt);
                x = fmaf(f, ov.x, x);
                y = fmaf(f, ov.y, y);
            }
            if (whole) {
                const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
                const int rr = row0 + r, i = rr / a.ratio;
                if (GDN_IN_RANGE(g_attn_cache_error, q.tok + i < a.n_tokens && head * a.ratio + rr - i * a.ratio < a.hq))
                    *reinterpret_cast<uint32_t*>(a.o + (q.tok + i) * a.ld_o + (head * a.ratio + rr - i * a.ratio) * D + c) =
                        bf16x2(x * inv, y * inv);
            } else {
                *reinterpret_cast<float2*>(part + r * (D + 2) + 2 + c) = make_float2(x, y);
                if (c == 0) *reinterpret_cast<float2*>(part + r * (D + 2)) = make_float2(mx, lt);
            }
        }
        fence_proxy_async_smem();   // the ring was written here; copies come next
        __syncthreads();
    }
    if (dead) {
        // a wait ran out: let copies already issued land (bounded) before the shared memory is released
        for (int i = 0; i < L::ST * 2; ++i)
            for (uint32_t par = 0; par < 2; ++par) mbar_wait_bounded(bars + i, par, nullptr, 0, 20000000ull);
    }
}

// Joins the partials of the pairs that lie in more than one run.  D/4 threads
// per row, a block for 1024/D rows of one pair.
template <int D, int ROWS>
__global__ void __launch_bounds__(AC_THREADS) attn_cache_join_kernel(const __grid_constant__ AttCacheArgs a) {
    __shared__ int64_t pre[GDN_MAX_SEQS + 2], wsum[AC_WARPS];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = blockIdx.x / a.heads, head = blockIdx.x % a.heads;
    ac_prefix(a, pre, wsum, false);
    const int64_t total = pre[a.n_seqs] * a.heads, per = ac_run_blocks(a, total), blocks = pre[s + 1] - pre[s];
    const int64_t first = pre[s] * a.heads + head * blocks;
    if (blocks == 0 || first / per == (first + blocks - 1) / per) return;   // written by its one run
    const AcSeq q = ac_seq(a, s, false);
    const int rr = blockIdx.y * (1024 / D) + threadIdx.x / (D / 4), c = (threadIdx.x % (D / 4)) * 4;
    if (rr >= q.nq * a.ratio) return;
    const int rank = rr / ROWS, r = rr % ROWS;
    const int c0 = static_cast<int>(first / per), c1 = static_cast<int>((first + blocks - 1) / per);
    auto piece = [&](int run) {
        const int which = run * per > first ? 0 : 1;
        return a.part + ((static_cast<int64_t>(run) * a.ranks + rank) * 2 + which) * ROWS * (D + 2) + r * (D + 2);
    };
    float mx = -INFINITY;
    for (int run = c0; run <= c1; ++run) mx = fmaxf_nan(mx, piece(run)[0]);
    float lt = 0.0f, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int run = c0; run <= c1; ++run) {
        const float* p = piece(run);
        const float f = p[0] == -INFINITY ? 0.0f : ex2_ftz(p[0] - mx);
        lt = fmaf(f, p[1], lt);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const float2 v = *reinterpret_cast<const float2*>(p + 2 + c + e);
            x[e] = fmaf(f, v.x, x[e]);
            x[e + 1] = fmaf(f, v.y, x[e + 1]);
        }
    }
    const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
    const int i = rr / a.ratio;
    if (GDN_IN_RANGE(g_attn_cache_error, q.tok + i < a.n_tokens && head * a.ratio + rr - i * a.ratio < a.hq))
        *reinterpret_cast<uint2*>(a.o + (q.tok + i) * a.ld_o + (head * a.ratio + rr - i * a.ratio) * D + c) =
            make_uint2(bf16x2(x[0] * inv, x[1] * inv), bf16x2(x[2] * inv, x[3] * inv));
}

// ------------------------------------------------------------ host

static PFN_cuTensorMapEncodeTiled_v12000 ac_map_encoder() {
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

// The pages as [n_pages * heads][slabs][page rows][slab bytes]; a box is the
// 16 rows of a tile in all slabs.  The page index is its own dimension, so no
// coordinate grows with the cache's bytes.
static bool ac_map(CUtensorMap* map, const void* ptr, const gdn_kv_cache& c) {
    auto enc = ac_map_encoder();
    if (!enc) return false;
    const bool wide = c.dtype == GDN_KV_BF16;
    const int row = c.head_dim * (wide ? 2 : 1), slab = row < 128 ? row : 128;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(wide ? slab / 2 : slab), static_cast<cuuint64_t>(c.page_tokens),
                          static_cast<cuuint64_t>(row / slab), static_cast<cuuint64_t>(c.n_pages * c.n_kv_heads)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(slab),
                             static_cast<cuuint64_t>(row) * c.page_tokens};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(dims[0]), AC_TILE, static_cast<cuuint32_t>(dims[2]), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, wide ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, slab == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of one CTA: 16, 32 or 64, as many as the accumulators of a warp leave
// room for (4096 fp32 at most).
static int ac_rows(int d, int64_t rows) {
    const int most = 4096 / d;
    return rows <= 16 || most == 16 ? 16 : rows <= 32 || most == 32 ? 32 : 64;
}

size_t attn_cache_workspace_bytes(const gdn_kv_cache& c, int64_t n_tokens, int hq) {
    (void)n_tokens;
    (void)hq;
    const int rows = 4096 / c.head_dim;
    return static_cast<size_t>(AC_MAX_RUNS) * 2 * rows * (c.head_dim + 2) * 4;
}

template <int D, int T, int MT>
static cudaError_t ac_launch(const gdn_kv_cache& c, AttCacheArgs& a, cudaStream_t st) {
    using L = AcSmem<D, T, MT>;
    static PerDeviceOnce once;
    if (once.run([](int) {
            cudaFuncSetAttribute(attn_cache_kernel<D, T, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES + 1024);
        }) < 0)
        return cudaErrorInvalidDevice;
    CUtensorMap mk, mv;
    if (!ac_map(&mk, c.k, c) || !ac_map(&mv, c.v, c)) return cudaErrorInvalidValue;
    const int rows = a.max_q * a.ratio;
    a.ranks = (rows + L::ROWS - 1) / L::ROWS;
    a.runs = AC_MAX_RUNS / a.ranks;
    attn_cache_kernel<D, T, MT><<<static_cast<unsigned>(a.runs * a.ranks), AC_THREADS, L::BYTES + 1024, st>>>(mk, mv, a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n_seqs * a.heads), static_cast<unsigned>((rows + 1024 / D - 1) / (1024 / D)), 1);
    cfg.blockDim = dim3(AC_THREADS, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_cache_join_kernel<D, L::ROWS>, a);
}

template <int D, int MT>
static cudaError_t ac_launch_t(const gdn_kv_cache& c, AttCacheArgs& a, cudaStream_t st) {
    if (c.dtype == GDN_KV_BF16) return ac_launch<D, GDN_KV_BF16, MT>(c, a, st);
    if (c.dtype == GDN_KV_I8) return ac_launch<D, GDN_KV_I8, MT>(c, a, st);
    return ac_launch<D, GDN_KV_E4M3, MT>(c, a, st);
}

cudaError_t launch_attn_cache(const gdn_kv_cache& c, const uint16_t* q, int64_t ld_q, const int32_t* cu, int64_t n_tokens,
                              int max_q, const uint64_t* tree, const int32_t* table, int64_t ld_table, int max_blocks,
                              const int32_t* lens, int n_seqs, int hq, float scale, uint16_t* o, int64_t ld_o,
                              void* workspace, cudaStream_t st) {
    AttCacheArgs a{};
    a.n_pages = c.n_pages;
    a.heads = c.n_kv_heads;
    a.page = c.page_tokens;
    a.page_shift = c.page_tokens == 16 ? 4 : c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : 7;
    a.ratio = hq / c.n_kv_heads;
    a.hq = hq;
    a.sk = c.k_scale;
    a.sv = c.v_scale;
    a.q = q;
    a.o = o;
    a.ld_q = ld_q;
    a.ld_o = ld_o;
    a.ld_table = ld_table;
    a.n_tokens = n_tokens;
    a.cu = cu;
    a.table = table;
    a.lens = lens;
    a.tree = tree;
    a.n_seqs = n_seqs;
    a.max_q = max_q;
    a.max_blocks = max_blocks;
    a.sl2 = scale * LOG2E;
    a.part = static_cast<float*>(workspace);
    const int rows = ac_rows(c.head_dim, static_cast<int64_t>(max_q) * a.ratio);
    if (c.head_dim == 256) return ac_launch_t<256, 1>(c, a, st);
    if (c.head_dim == 128) return rows == 16 ? ac_launch_t<128, 1>(c, a, st) : ac_launch_t<128, 2>(c, a, st);
    return rows == 16 ? ac_launch_t<64, 1>(c, a, st) : rows == 32 ? ac_launch_t<64, 2>(c, a, st) : ac_launch_t<64, 4>(c, a, st);
}

int read_and_clear_attn_cache_error() {
    int v = 0, z = 0;
    cudaMemcpyFromSymbol(&v, g_attn_cache_error, sizeof(int));
    if (v) cudaMemcpyToSymbol(g_attn_cache_error, &z, sizeof(int));
    return v;
}

}  // namespace gdn
