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
// others).  Each pair counts some blocks more than it has, for the time that
// starting and joining it takes.  A pair that lies in one run is written at
// once; the others leave (maximum, sum, fp32 accumulator) partials that a
// second kernel joins.
//
// Inside a CTA each warp walks every 8th or 16th tile (16 to 64 keys) on its own:
// its lane 0 copies the tile's keys and values by TMA into the warp's own ring,
// the warp multiplies them on the tensor cores and keeps its own running
// maximum, sum and accumulator; there is no barrier between warps until the
// end of a pair, where their results are joined in shared memory.  The
// products are m16n8k16 with the cache as the 16-wide operand and eight rows as
// the other, S^T = K Q^T and O^T = V^T P^T: one new token of up to eight query
// heads then takes half the instructions and accumulators of the form with the
// rows on the wide side, which leaves registers for 16 warps.  The scores never
// leave registers: a transpose of 8 x 8 tiles (movmatrix) turns them into the
// second product's operand.
//
// 8-bit codes become fp16 in registers (exact), with the row scales kept out
// of the products: a key's scale multiplies its score, and a value's scale
// goes into the exponent of its probability, p' = 2^(x + log2 vs - m), which
// enters the product as fp16; the softmax sum adds p = 2^(x - m) in fp32.
// Scores x are in units of log 2.  A maximum is raised only past a margin of
// 2^4, so the accumulators are seldom rescaled; fp16 probabilities carry a
// factor 2^11 (at most 2^15 with the margin).  Those below 2^-14, where fp16
// loses bits (2^-25 of the largest), matter only to elements that are zero in
// every more probable row; a tile that has one multiplies the rounding errors
// p' - fp16(p') in bf16, whose exponents reach as far as fp32's, in a second
// pass, and leaves out the first where fp16 holds nothing.  q goes to fp16 times
// a power of two per row that puts its largest element in [2^14, 2^15): elements
// below 2^-38 of it are lost.  A scale counts as 2^-80 at least where the maximum
// is raised (AC_VS_MIN).
//
// Measured (us; bytes of the cache over the time): one token over 131072 int8
// keys, 16 over 4 heads of 256: 54, 5.0 TB/s, of which the join is 5; 48
// sequences of 1 to 16384 e4m3 keys: 134, 6.0 TB/s, bound by memory; 16 chains of
// up to four tokens over 300 to 12000 int8 keys, 32 over 8 heads of 128: 66, 3.0
// TB/s, where nothing is saturated (issue slots 43 %, tensor pipe 20 %): 16 rows'
// accumulators leave registers for two warps a scheduler, too few for the latency
// of loads, conversions and products in turn (one token each, eight rows: 48).
// 777 bf16 keys of one sequence: 10, the latencies of two kernels.
#include "attn_cache.cuh"

#include <algorithm>

namespace gdn {

constexpr int AC_RING = 192 * 1024;     // bytes of tiles in flight per CTA

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

// Whole warp: an 8 x 8 matrix of 16-bit values, two of row lane / 4 per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// ------------------------------------------------------------ shared memory

// A run's place, the piece it is at and that piece's rows.
struct AcRun {
    int64_t at, end;
    AcPiece pc;
    int s, rows;
};

// A row of a tile is cut into slabs of 128 bytes (one of 64 for 8-bit heads of
// 64), each slab [keys][128 bytes] with the TMA's 128-byte (64-byte) swizzle,
// so that eight keys' 16-byte pieces fall into different banks.
template <int D, int T, int NR>
struct AcSmem {
    static constexpr int ES = T == GDN_KV_BF16 ? 2 : 1;
    static constexpr int ROW = D * ES;
    static constexpr int SLAB = ROW < 128 ? ROW : 128;      // bytes of a row in one slab
    static constexpr int NSLAB = ROW / SLAB;
    static constexpr int SUB = ROW >= 256 ? 1 : 256 / ROW;  // 16-key steps of a tile: 4 KB or more, so that a
    static constexpr int KEYS = 16 * SUB;                   // tile's waits and copies are worth their instructions
    static constexpr int HALF = KEYS * ROW;                 // the keys, or the values, of a tile
    static constexpr int TILES = AC_BLOCK / KEYS;           // tiles of a block
    // blocks' worth of starting and joining a pair: 48 sequences of 1 .. 16384 keys, 8-bit heads of 256, take 155 us
    // counted as 512 / ROW blocks, 145 as 768, 135 as 1152 and 138 as 2304; 16 chains of heads of 128 72, 70, 69 and 77
    static constexpr int START = 1152 / ROW;
    // 16 warps where 128 registers hold the accumulators (one row tile, two of
    // heads of 64) and a warp's share of the ring a tile and a half.  Two row
    // tiles of heads of 64, e4m3: 49 us for six sequences of up to 24000 keys,
    // with 8 warps 59; of heads of 128, int8: 82 us, with 8 warps 65
    static constexpr int WARPS = (NR == 1 || D * NR <= 128) && 16 * 3 * HALF <= AC_RING ? 16 : 8;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int NS = AC_RING / WARPS / HALF < 8 ? AC_RING / WARPS / HALF : 8;   // half tiles in flight per warp
    static constexpr int ROWS = 8 * NR;
    static constexpr int OLD = D + 4;                       // padded rows of the joined accumulators: a warp's pieces in different banks
    static constexpr int QR = (ROWS + WARPS - 1) / WARPS;   // rows of q that a warp prepares
    static constexpr int R0 = 0;                            // ring [warp][slot]; the accumulators at the end of a pair
    static constexpr int S0 = AC_RING;                      // row scales of the half tiles: [warp][slot][keys]
    static constexpr int M0 = S0 + WARPS * NS * KEYS * 4;        // maxima and sums: [warp][rows][2]
    static constexpr int P0 = M0 + WARPS * ROWS * 2 * 4;         // blocks before each sequence
    static constexpr int T0 = P0 + (GDN_MAX_SEQS + 2) * 8;       // the sequences
    static constexpr int W0 = T0 + GDN_MAX_SEQS * 12;
    static constexpr int F0 = W0 + WARPS * 8;                    // pages in range, a bit per copy: [warp][slot]
    static constexpr int N0 = F0 + WARPS * NS * 4;               // mask word of each row
    static constexpr int X0 = N0 + ROWS * 8;                     // score factor of each row
    static constexpr int J0 = (X0 + ROWS * 4 + 7) & ~7;          // maximum and sum of each row
    static constexpr int H0 = J0 + ROWS * 8;                     // where the run stands while a piece's tiles pass
    static constexpr int Q0 = (H0 + static_cast<int>(sizeof(AcRun)) + 15) & ~15;        // q fragments [row tile][step][lane] x 8 bytes
    static constexpr int B0 = Q0 + NR * (D / 16) * 256;          // mbarriers [warp][slot]
    static constexpr int BYTES = B0 + WARPS * NS * 8;
    static_assert(WARPS * ROWS * OLD * 4 <= AC_RING, "the joined accumulators fit the ring");
    static_assert(SUB == 1 || NSLAB == 1, "copies of a tile follow each other");
    static_assert(BYTES + 1024 <= 227 * 1024, "shared memory of a CTA");
};

// Byte offset of 16-byte piece c of key r in a tile.
template <class L>
__device__ __forceinline__ uint32_t ac_piece(int r, int c) {
    if constexpr (L::SLAB == 128)
        return static_cast<uint32_t>((c >> 3) * (L::KEYS * 128) + r * 128 + (((c ^ r) & 7) << 4));
    else
        return static_cast<uint32_t>(r * 64 + (((c ^ (r >> 1)) & 3) << 4));
}

// ------------------------------------------------------------ the kernel

// A truth value that is known to the compiler.
template <bool V>
struct Flag {
    __device__ constexpr operator bool() const { return V; }
};

// NR tiles of eight rows per CTA.
template <int D, int T, int NR>
__global__ void __launch_bounds__(AcSmem<D, T, NR>::THREADS, 1)
attn_cache_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ AttCacheArgs a) {
    using L = AcSmem<D, T, NR>;
    constexpr int KT = D / 16;            // 16-wide steps of a row
    constexpr int SUB = L::SUB;
    constexpr bool Q8 = T != GDN_KV_BF16;
    extern __shared__ __align__(1024) unsigned char smb[];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smb) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    int64_t* pre = reinterpret_cast<int64_t*>(base + L::P0);
    AcSeq* seq = reinterpret_cast<AcSeq*>(base + L::T0);
    float* join = reinterpret_cast<float*>(base + L::R0);
    float2* ml = reinterpret_cast<float2*>(base + L::M0);
    uint64_t* seen = reinterpret_cast<uint64_t*>(base + L::N0);
    float* row_factor = reinterpret_cast<float*>(base + L::X0);
    float2* total_ml = reinterpret_cast<float2*>(base + L::J0);
    uint2* qsm = reinterpret_cast<uint2*>(base + L::Q0);
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + L::B0) + warp * L::NS;
    unsigned char* ring = base + L::R0 + warp * L::NS * L::HALF;
    float* scales = reinterpret_cast<float*>(base + L::S0) + warp * L::NS * L::KEYS;
    uint32_t* page_in = reinterpret_cast<uint32_t*>(base + L::F0) + warp * L::NS;

    if (lane == 0) {
        for (int i = 0; i < L::NS; ++i) mbar_init_cta(bars + i, 1);
        mbar_init_fence();
    }
    pdl_wait();
    pdl_trigger();   // after the wait: what precedes this kernel is complete when the next one's CTAs start
    const int run = blockIdx.x / a.ranks, rank = blockIdx.x % a.ranks;
    ac_prefix(a, pre, seq, reinterpret_cast<int64_t*>(base + L::W0), blockIdx.x == 0);
    const int64_t total = pre[a.n_seqs] * a.heads, per = ac_run_blocks(a, total);
    // in registers only between the tile loops, which have none to spare
    AcRun at{};
    at.at = run * per;
    at.end = at.at + per < total ? at.at + per : total;
    if (at.at >= at.end) return;
    at.s = ac_seq_of(a, pre, at.at);
    volatile AcRun* kept = reinterpret_cast<volatile AcRun*>(base + L::H0);
    int slot = 0;               // the next half tile of this warp's ring and its phase
    uint32_t par = 0;
    bool dead = false;          // a wait ran out

    // the lanes' rows of the ldmatrix operands: keys (lane & 7) + 8 ((lane >> 3) & 1), piece + (lane >> 4);
    // bf16 values swap the two
    const int kr = (lane & 7) + (((lane >> 3) & 1) << 3), kc = lane >> 4;
    const int vr = Q8 ? kr : (lane & 7) + ((lane >> 4) << 3), vc = Q8 ? kc : (lane >> 3) & 1;
    // piece c + kc (c even) of 16 keys at `b`: the swizzle is one exclusive or on the address
    const uint32_t koff = ac_piece<L>(kr, kc), voff = ac_piece<L>(vr, vc);
    auto piece_at = [](uint32_t b, int c) { return (b ^ ((c & 7) << 4)) + (c >> 3) * (L::KEYS * 128); };

    // The run's next piece that has rows of this rank, its first pages and its
    // rows of q (lane's share of rows warp, warp + WARPS, ..): asked for before
    // the piece before it is joined, so that its copies start without a wait.
    constexpr int QE = D / 32;            // elements of a row of q in a lane
    constexpr int PG = (L::NS + 1) / 2;   // tiles whose keys the ring takes
    const int row0 = rank * L::ROWS;
    const int copies = L::KEYS / a.box, mycopy = lane < copies ? lane * a.box : 0;
    int pg[PG];
    uint32_t qw[L::QR][QE / 2];
    auto last_tile = [](const AcPiece& p) { return min(p.b1 * L::TILES, p.q.len == 0 ? 1 : (p.q.len - 1) / L::KEYS + 1); };
    auto tiles_of_warp = [&](int t0, int t1) { return t1 - t0 - warp > 0 ? (t1 - t0 - warp + L::WARPS - 1) / L::WARPS : 0; };
    auto page_of = [&](const int32_t* table, int t0, int i) {
        return table[min(((t0 + warp + i * L::WARPS) * L::KEYS + mycopy) >> a.page_shift, a.max_blocks - 1)];
    };
    auto next = [&] {
        do {
            if (!ac_next(a, pre, seq, at.at, at.end, at.s, at.pc)) return false;
            at.rows = min(at.pc.q.nq * a.ratio - row0, L::ROWS);
        } while (at.rows <= 0);
        const int t0 = at.pc.b0 * L::TILES, n = tiles_of_warp(t0, last_tile(at.pc));
#pragma unroll
        for (int i = 0; i < PG; ++i) pg[i] = page_of(a.table + at.pc.s * a.ld_table, t0, min(i, max(n - 1, 0)));
#pragma unroll
        for (int x = 0; x < L::QR; ++x) {
            const int r = warp + x * L::WARPS, rr = row0 + r, i = rr / a.ratio;
#pragma unroll
            for (int e = 0; e < QE / 2; ++e) qw[x][e] = 0;
            if (r < at.rows) {
                const uint16_t* src = a.q + static_cast<int64_t>(at.pc.q.tok + i) * a.ld_q +
                                      (at.pc.head * a.ratio + rr - i * a.ratio) * D + lane * QE;
                if constexpr (QE == 8) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src);
                    qw[x][0] = v.x, qw[x][1] = v.y, qw[x][2] = v.z, qw[x][3] = v.w;
                } else if constexpr (QE == 4) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    qw[x][0] = v.x, qw[x][1] = v.y;
                } else {
                    qw[x][0] = *reinterpret_cast<const uint32_t*>(src);
                }
            }
        }
        return true;
    };

    bool more = next();
    while (more) {
        const AcSeq q = at.pc.q;
        const int head = at.pc.head, t0 = at.pc.b0 * L::TILES;
        const int mine = tiles_of_warp(t0, last_tile(at.pc));   // tiles of this warp
        const int ctx = q.len - q.nq;      // keys every row sees
        const int32_t* table = a.table + at.pc.s * a.ld_table;
        if (tid == 0) {
            kept->at = at.at;
            kept->end = at.end;
            kept->s = at.s;
            kept->rows = at.rows;
            kept->pc.s = at.pc.s;
            kept->pc.b0 = at.pc.b0;
            kept->pc.b1 = at.pc.b1;
            kept->pc.blocks = at.pc.blocks;
            kept->pc.q.tok = q.tok;
            kept->pc.q.len = q.len;
        }

        // ---- copies: half tile j (keys of tile j / 2, then its values)
        // follows j - NS in its slot.  A tile may lie in several pages: lane p
        // copies the rows of the p-th.
        auto issue = [&](int j, int sl, int page) {   // whole warp
            const int row = ((t0 + warp + (j >> 1) * L::WARPS) * L::KEYS + mycopy) & (a.page - 1);
            const bool in = page >= 0 && page < a.n_pages, val = j & 1;
            const int pair = (in ? page : 0) * a.heads + head;   // an unseen page: any rows, all of them masked
            const uint32_t ok = __ballot_sync(0xffffffffu, in);
            if (lane < copies) {
                if (lane == 0) {
                    page_in[sl] = ok;
                    mbar_expect_tx(bars + sl, L::HALF + (Q8 ? L::KEYS * 4 : 0));
                }
                tma_load_4d(ring + sl * L::HALF + mycopy * L::SLAB, val ? &mv : &mk, bars + sl, 0, row, 0, pair);
                if constexpr (Q8)
                    bulk_load_1d(scales + sl * L::KEYS + mycopy, (val ? a.sv : a.sk) + static_cast<int64_t>(pair) * a.page + row,
                                 a.box * 4, bars + sl);
            }
        };
        if (!dead) {
            int sl = slot;
#pragma unroll
            for (int j = 0; j < L::NS; ++j)
                if (j < 2 * mine) {
                    if (!(a.withhold && warp == 0 && j == 0)) issue(j, sl, pg[j >> 1]);
                    sl = sl + 1 == L::NS ? 0 : sl + 1;
                }
        }
        // pages of the tiles whose keys (a) and values (b) the next two free slots take
        int page_a = page_of(table, t0, min(L::NS / 2, max(mine - 1, 0))), page_b = page_of(table, t0, min((L::NS + 1) / 2, max(mine - 1, 0)));

        // ---- q fragments, the same for every warp, in shared memory: a thread's
        // d elements at step kt are those its key fragments hold (row 8 nr + g:
        // elements 4t .. 4t + 3 of 16, or 2t, 2t + 1, 2t + 8, 2t + 9 of bf16)
#pragma unroll
        for (int x = 0; x < L::QR; ++x) {
            const int r = warp + x * L::WARPS;
            if (r >= L::ROWS) break;
            float factor = a.sl2;
            unsigned char* dst = reinterpret_cast<unsigned char*>(qsm + ((r >> 3) * KT + lane * QE / 16) * 32 + 4 * (r & 7));
            const int e0 = lane * QE & 15;
            if constexpr (!Q8) {
#pragma unroll
                for (int e = 0; e < QE / 2; ++e)
                    *reinterpret_cast<uint32_t*>(dst + ((e0 & 7) + 2 * e) / 2 * 8 + (e0 >> 3) * 4) = qw[x][e];
            } else {
                float amax = 0.0f;
#pragma unroll
                for (int e = 0; e < QE / 2; ++e)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qw[x][e] << 16)), fabsf(__uint_as_float(qw[x][e] & 0xffff0000u))));
                amax = warp_max(amax);
                // 2^e with amax 2^e in [2^14, 2^15): exact both ways (below 2^AC_Q_MIN 2^e is that of 2^AC_Q_MIN)
                const int ex = min(max(static_cast<int>((__float_as_uint(amax) >> 23) & 255) - 127, AC_Q_MIN), 127);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - ex) << 23);
                factor *= __uint_as_float(static_cast<uint32_t>(127 - 14 + ex) << 23);
#pragma unroll
                for (int e = 0; e < QE / 2; ++e)
                    *reinterpret_cast<uint32_t*>(dst + (e0 + 2 * e) * 2) =
                        f16x2_bits(__uint_as_float(qw[x][e] << 16) * up, __uint_as_float(qw[x][e] & 0xffff0000u) * up);
            }
            if (lane == 0) {
                const int i = (row0 + r) / a.ratio;
                row_factor[r] = factor;
                seen[r] = r >= at.rows ? 0 : a.tree ? a.tree[q.tok + i] : i >= 63 ? ~0ull : (1ull << (i + 1)) - 1;
            }
        }
        __syncthreads();

        // ---- this thread's rows of the scores: 8 nr + 2t and + 1
        float m[NR][2], l[NR][2], o[NR][KT][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            m[nr][0] = m[nr][1] = -INFINITY;
            l[nr][0] = l[nr][1] = 0.0f;
#pragma unroll
            for (int c = 0; c < KT; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nr][c][e] = 0.0f;
        }

#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            const int key0 = (t0 + warp + i * L::WARPS) * L::KEYS;
            const uint32_t kb = smem_addr(ring + slot * L::HALF) + koff;

            if (!dead && !mbar_wait_bounded(bars + slot, par, &g_attn_cache_error, ERR_WAIT_TIMEOUT, a.wait_ns)) dead = true;
            dead = __any_sync(0xffffffffu, dead);
            if (dead) break;
            const uint32_t ok = page_in[slot] | (~0u << copies);
            const bool edge_tile = key0 + L::KEYS > ctx || ok != ~0u;
            if (ok != ~0u && lane < copies && !((ok >> lane) & 1) && key0 + mycopy < q.len)
                atomicExch(&g_attn_cache_skipped, static_cast<int>(ERR_INDEX));
            // keys of 16-key step u below limit(u) exist; those of an unseen page do not
            auto limit = [&](int u) {
                return (ok >> (16 * u / a.box)) & 1 ? q.len - key0 - 16 * u : 0;
            };

            // ---- scores of keys g and g + 8 (of each 16) for this thread's rows
            float y[SUB][NR][4], kv[SUB][2];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[u][nr][e] = 0.0f;
                const uint32_t ku = kb + u * (16 * L::SLAB);
                if constexpr (!Q8) {
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        uint32_t f[4];
                        ldsm_x4(piece_at(ku, 2 * kt), f);
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) {
                            const uint2 b = qsm[(nr * KT + kt) * 32 + lane];
                            mma16816<T>(y[u][nr], f, b.x, b.y);
                        }
                    }
                } else {
                    // 16 codes of eight keys per register set: a thread gets codes 4t .. 4t+3 of key g
#pragma unroll
                    for (int kt = 0; kt < KT; kt += 2) {
                        uint32_t w[4];
                        ldsm_x4(piece_at(ku, kt), w);
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            const uint32_t x = T == GDN_KV_I8 ? w[2 * v] ^ 0x80808080u : w[2 * v];
                            const uint32_t z = T == GDN_KV_I8 ? w[2 * v + 1] ^ 0x80808080u : w[2 * v + 1];
                            const uint32_t f[4] = {codes_f16<T, 0, 1>(x), codes_f16<T, 0, 1>(z), codes_f16<T, 2, 3>(x),
                                                   codes_f16<T, 2, 3>(z)};
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr) {
                                const uint2 b = qsm[(nr * KT + kt + v) * 32 + lane];
                                mma16816<T>(y[u][nr], f, b.x, b.y);
                            }
                        }
                    }
                }
                if constexpr (Q8) {
                    kv[u][0] = scales[slot * L::KEYS + 16 * u + g];
                    kv[u][1] = scales[slot * L::KEYS + 16 * u + 8 + g];
                }
            }
            __syncwarp();
            if (2 * i + L::NS < 2 * mine) issue(2 * i + L::NS, slot, page_a);
            if (++slot == L::NS) {
                slot = 0;
                par ^= 1;
            }
            const uint32_t vb = smem_addr(ring + slot * L::HALF) + voff;

            if (!mbar_wait_bounded(bars + slot, par, &g_attn_cache_error, ERR_WAIT_TIMEOUT, a.wait_ns)) dead = true;
            dead = __any_sync(0xffffffffu, dead);
            if (dead) break;

            // The rest of the tile; edge: some row may not see some key.
            auto finish = [&](auto edge) {
                // ---- softmax of the tile: y = x + log2 of the value's scale
                bool up = false;
                float lv[SUB][2];
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // a row of zeros has scale 0 and codes 0
                        lv[u][h] = Q8 ? lg2(fmaxf_nan(scales[slot * L::KEYS + 16 * u + 8 * h + g], AC_VS_FLOOR)) : 0.0f;
                        up |= lv[u][h] < AC_VS_MIN;
                    }
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
                        const float2 qs = *reinterpret_cast<const float2*>(row_factor + 8 * nr + 2 * t);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float f = e & 1 ? qs.y : qs.x;
                            y[u][nr][e] = Q8 ? fmaf(y[u][nr][e], f * kv[u][e >> 1], lv[u][e >> 1]) : y[u][nr][e] * f;
                        }
                        if (edge) {
                            const int lim = limit(u);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = 8 * (e >> 1) + g, d = key0 + 16 * u + j - ctx;
                                if (j >= lim || (d >= 0 && !((seen[8 * nr + 2 * t + (e & 1)] >> (d & 63)) & 1))) y[u][nr][e] = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) up |= y[u][nr][e] > m[nr][e & 1] + AC_MARGIN;   // from -inf: any finite score
                    }
                    if (edge) {      // a scale that is no number has reached the rows that see its key in y
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (!(fabsf(lv[u][h]) < INFINITY)) lv[u][h] = 0.0f;
                    }
                }
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float bm = -INFINITY;
#pragma unroll
                            for (int u = 0; u < SUB; ++u)
#pragma unroll
                                for (int h = 0; h < 2; ++h)   // a scale counts as 2^AC_VS_MIN at least
                                    bm = fmaxf(bm, Q8 ? y[u][nr][2 * h + e] + fmaxf(AC_VS_MIN - lv[u][h], 0.0f) : y[u][nr][2 * h + e]);
                            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
                            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
                            bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
                            const float old = m[nr][e], mn = fmaxf(old, bm);
                            const float c = old == -INFINITY ? 0.0f : ex2_ftz(old - mn);
                            m[nr][e] = mn;
                            l[nr][e] *= c;
#pragma unroll
                            for (int k = 0; k < KT; ++k) {
                                o[nr][k][e] *= c;
                                o[nr][k][2 + e] *= c;
                            }
                        }
                }

#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    uint32_t pf[NR][2];      // probabilities of (key g, rows 2t, 2t+1) and (key g + 8, ..)
                    float pk[NR][4];
                    bool faint = false;      // an fp16 probability that lost bits
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float mm = m[nr][e & 1] == -INFINITY ? 0.0f : Q8 ? m[nr][e & 1] - AC_LIFT : m[nr][e & 1];
                            const float x = y[u][nr][e] - mm, p = ex2_ftz(x);
                            pk[nr][e] = p;
                            if constexpr (Q8) {
                                faint |= p != 0.0f && p < 6.1035156e-5f;
                                l[nr][e & 1] += ex2_ftz(x - lv[u][e >> 1]);
                            }
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if constexpr (Q8) {
                                pf[nr][h] = f16x2_bits(pk[nr][2 * h], pk[nr][2 * h + 1]);
                            } else {
                                pf[nr][h] = bf16x2(pk[nr][2 * h], pk[nr][2 * h + 1]);
                                // the sum takes the probabilities as rounded, so their rounding cancels where few keys matter
                                l[nr][0] += __uint_as_float(pf[nr][h] << 16);
                                l[nr][1] += __uint_as_float(pf[nr][h] & 0xffff0000u);
                            }
                        }
                    }

                    // ---- values
                    const uint32_t vu = vb + u * (16 * L::SLAB);
                    uint32_t odd = 0;                    // a value that is not finite at the edge
                    uint32_t km[2] = {~0u, ~0u};         // halves of the fragments whose keys (2t, 2t+1; + 8) exist
                    if (edge) {
                        const int lim = limit(u);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            km[h] = (8 * h + 2 * t < lim ? 0xffffu : 0u) | (8 * h + 2 * t + 1 < lim ? 0xffff0000u : 0u);
                    }
                    // what does not exist, and what is not finite (its rows see it below), is taken as zero
                    auto clean = [&](uint32_t w, int h) {
                        constexpr uint32_t EXP = Q8 ? 0x7c00u : 0x7f80u;
                        w &= km[h];
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
                    // fragments of columns 16c .. 16c + 15 (8-bit: and of the next 16)
                    constexpr int STEP = Q8 ? 2 : 1;
                    auto values = [&](int c, uint32_t (&f)[STEP][4]) {
                        uint32_t w[4];
                        ldsm_x4_trans(piece_at(vu, Q8 ? c : 2 * c), w);
                        if constexpr (Q8) {
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                const uint32_t x = T == GDN_KV_I8 ? w[2 * v] ^ 0x80808080u : w[2 * v];
                                const uint32_t z = T == GDN_KV_I8 ? w[2 * v + 1] ^ 0x80808080u : w[2 * v + 1];
                                f[v][0] = codes_f16<T, 0, 2>(x);     // columns 2g of keys 0-7, 2g + 1, then keys 8-15
                                f[v][1] = codes_f16<T, 1, 3>(x);
                                f[v][2] = codes_f16<T, 0, 2>(z);
                                f[v][3] = codes_f16<T, 1, 3>(z);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[0][e] = w[e];
                        }
                        if (edge) {
#pragma unroll
                            for (int v = 0; v < STEP; ++v)
#pragma unroll
                                for (int e = 0; e < 4; ++e) f[v][e] = clean(f[v][e], e >> 1);
                        }
                    };
                    // the second product's operand: (keys 2t, 2t+1; row g)
                    uint32_t pt[NR][2];
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int h = 0; h < 2; ++h) pt[nr][h] = transpose8(pf[nr][h]);
                    bool first_pass = true;
                    if constexpr (Q8) {
                        faint = __any_sync(0xffffffffu, faint);
                        if (faint) {         // does fp16 hold anything of these keys?
                            uint32_t any = 0;
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr) any |= pt[nr][0] | pt[nr][1];
                            first_pass = __any_sync(0xffffffffu, any != 0);
                        }
                    }
                    if (first_pass) {
#pragma unroll
                        for (int c = 0; c < KT; c += STEP) {
                            uint32_t f[STEP][4];
                            values(c, f);
#pragma unroll
                            for (int v = 0; v < STEP; ++v)
#pragma unroll
                                for (int nr = 0; nr < NR; ++nr) mma16816<T>(o[nr][c + v], f[v], pt[nr][0], pt[nr][1]);
                        }
                    }
                    if constexpr (Q8) {
                        if (faint) {
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&pf[nr][h]));
                                    pt[nr][h] = transpose8(bf16x2(pk[nr][2 * h] - r.x, pk[nr][2 * h + 1] - r.y));
                                }
#pragma unroll
                            for (int c = 0; c < KT; c += STEP) {
                                uint32_t f[STEP][4];
                                values(c, f);
#pragma unroll
                                for (int v = 0; v < STEP; ++v) {
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f[v][e]));
                                        f[v][e] = bf16x2(x.x, x.y);
                                    }
#pragma unroll
                                    for (int nr = 0; nr < NR; ++nr)
                                        mma16816<GDN_KV_BF16>(o[nr][c + v], f[v], pt[nr][0], pt[nr][1]);
                                }
                            }
                        }
                    }
                    if (T != GDN_KV_I8 && edge && __any_sync(0xffffffffu, odd)) {
                        // rows that see such a key add its term by themselves
                        const unsigned char* vt = ring + slot * L::HALF;
#pragma unroll 1
                        for (int j = 0; j < min(limit(u), 16); ++j) {
                            const int d = key0 + 16 * u + j - ctx, src = ((j & 7) << 2) | t;
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float p = __shfl_sync(0xffffffffu, j < 8 ? pk[nr][e] : pk[nr][2 + e], src);
                                    if (d >= 0 && !((seen[8 * nr + 2 * t + e] >> (d & 63)) & 1)) continue;
#pragma unroll
                                    for (int c = 0; c < KT; ++c)
#pragma unroll
                                        for (int h = 0; h < 2; ++h) {
                                            const int col = 16 * c + (Q8 ? 2 * g + h : 8 * h + g), key = 16 * u + j;
                                            float v;
                                            if constexpr (Q8)
                                                v = __half2float(__half(__nv_cvt_fp8_to_halfraw(vt[ac_piece<L>(key, col >> 4) + (col & 15)], __NV_E4M3)));
                                            else
                                                v = bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(vt + ac_piece<L>(key, col >> 3) + 2 * (col & 7)));
                                            if (!(fabsf(v) < INFINITY)) o[nr][c][2 * h + e] += p * v;
                                        }
                                }
                        }
                    }
                }
            };
            if constexpr (T == GDN_KV_I8) {
                // two copies of the code, so that the plain tiles do without the tests (for the
                // other types, whose edge tiles look for values that are not finite, two copies spill)
                if (edge_tile)
                    finish(Flag<true>{});
                else
                    finish(Flag<false>{});
            } else {
                finish(edge_tile);
            }
            __syncwarp();
            if (2 * i + 1 + L::NS < 2 * mine) issue(2 * i + 1 + L::NS, slot, page_b);
            if (++slot == L::NS) {
                slot = 0;
                par ^= 1;
            }
            const int page = page_of(table, t0, min(i + 1 + (L::NS + 1) / 2, mine - 1));
            page_a = L::NS % 2 ? page_b : page;
            page_b = page;
        }

        // ---- join the warps
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 4);
                l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 8);
                l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 16);
                if (g == 0) ml[warp * L::ROWS + 8 * nr + 2 * t + e] = make_float2(m[nr][e], l[nr][e]);
            }
        __syncthreads();   // every warp is done with its ring
        at.at = kept->at;
        at.end = kept->end;
        at.s = kept->s;
        at.pc.b0 = kept->pc.b0;
        at.pc.b1 = kept->pc.b1;
        at.pc.q.len = kept->pc.q.len;
        const int b0 = at.pc.b0, live = min(last_tile(at.pc) - b0 * L::TILES, L::WARPS), rows = kept->rows, tok = kept->pc.q.tok;
        const bool whole = b0 == 0 && at.pc.b1 == kept->pc.blocks;
        // a thread per row and warp: what the warp's accumulator counts for, and the row's maximum and sum
        if (tid < L::ROWS * L::WARPS) {
            const int w = tid % L::WARPS, r = tid / L::WARPS;
            const float2 v = w < live ? ml[w * L::ROWS + r] : make_float2(-INFINITY, 0.0f);
            float mx = v.x;
#pragma unroll
            for (int x = L::WARPS / 2; x > 0; x >>= 1) mx = fmaxf_nan(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            // weight 0, not left out: a NaN (of a score, or 0 times an infinite value) stays
            const float f = v.x == -INFINITY ? 0.0f : ex2_ftz(v.x - mx);
            float lt = f * v.y;
#pragma unroll
            for (int x = L::WARPS / 2; x > 0; x >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, x);
            ml[w * L::ROWS + r].x = f;
            if (w == 0) total_ml[r] = make_float2(mx, lt);
        }
        if (warp < live) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * nr + 2 * t + e;
                    if (r >= rows) continue;
                    float* dst = join + (warp * L::ROWS + r) * L::OLD;
#pragma unroll
                    for (int c = 0; c < KT; ++c) {
                        if constexpr (Q8) {
                            *reinterpret_cast<float2*>(dst + 16 * c + 2 * g) = make_float2(o[nr][c][e], o[nr][c][2 + e]);
                        } else {
                            dst[16 * c + g] = o[nr][c][e];
                            dst[16 * c + 8 + g] = o[nr][c][2 + e];
                        }
                    }
                }
        }
        more = next();     // its loads fly while this piece is joined
        __syncthreads();
        const int64_t part0 = (static_cast<int64_t>(blockIdx.x) * 2 + (b0 > 0 ? 0 : 1)) * L::ROWS;
        for (int e = tid; e < rows * (D / 4); e += L::THREADS) {
            const int r = e / (D / 4), c = (e % (D / 4)) * 4;
            const float* from = join + r * L::OLD + c;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
            for (int w = 0; w < live; ++w) {
                const float f = ml[w * L::ROWS + r].x;
                const float4 v = *reinterpret_cast<const float4*>(from + w * (L::ROWS * L::OLD));
                x.x = fmaf(f, v.x, x.x);
                x.y = fmaf(f, v.y, x.y);
                x.z = fmaf(f, v.z, x.z);
                x.w = fmaf(f, v.w, x.w);
            }
            const float2 tot = total_ml[r];
            if (whole) {
                const float inv = tot.y == 0.0f ? 0.0f : 1.0f / tot.y;
                const int rr = row0 + r, i = rr / a.ratio;
                if (GDN_IN_RANGE(g_attn_cache_error, tok + i < a.n_tokens && head * a.ratio + rr - i * a.ratio < a.hq))
                    *reinterpret_cast<uint2*>(a.o + static_cast<int64_t>(tok + i) * a.ld_o + (head * a.ratio + rr - i * a.ratio) * D + c) =
                        make_uint2(bf16x2(x.x * inv, x.y * inv), bf16x2(x.z * inv, x.w * inv));
            } else {
                *reinterpret_cast<float4*>(a.part + (part0 + r) * D + c) = x;
                if (c == 0) a.part_ml[part0 + r] = tot;
            }
        }
        fence_proxy_async_smem();   // the ring was written here; copies come next
        __syncthreads();
    }
    if (dead) {
        // a wait ran out: let copies already issued land (bounded) before the shared memory is released
        for (int i = 0; i < L::NS; ++i)
            for (uint32_t p = 0; p < 2; ++p) mbar_wait_bounded(bars + i, p, nullptr, 0, 20000000ull);
    }
}

// Joins the partials of the pairs that lie in more than one run.  blockIdx.x is
// the pair.  Few partials: a warp per row, no barrier.  Many (one long
// sequence): a block per row, the partials dealt over its warps, since one
// row's chain of loads would take longer than its bytes.
template <int D>
__global__ void __launch_bounds__(AC_JOIN_THREADS, D == 256 ? 3 : 4)
attn_cache_join_kernel(const __grid_constant__ AttCacheArgs a, int rank_rows) {
    constexpr int WARPS = AC_JOIN_THREADS / 32, E = D / 32;   // each lane E columns, 2 at a time
    __shared__ int64_t pre[GDN_MAX_SEQS + 2], wsum[WARPS];
    __shared__ AcSeq seq[GDN_MAX_SEQS];
    __shared__ float2 acc[WARPS][D / 2];
    const int s = blockIdx.x / a.heads, head = blockIdx.x % a.heads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ac_prefix(a, pre, seq, wsum, false);     // inputs of the call: complete before the kernel that is waited for began
    pdl_wait();
    const int64_t total = pre[a.n_seqs] * a.heads, per = ac_run_blocks(a, total), counted = pre[s + 1] - pre[s];
    // the pair's own blocks, after those that count for its start
    const int64_t first = pre[s] * a.heads + head * counted + a.start, last = first + counted - a.start - 1;
    if (counted == 0 || first / per == last / per) return;   // written by its one run
    const AcSeq q = seq[s];
    const int c0 = static_cast<int>(first / per), n = static_cast<int>(last / per) - c0 + 1;
    const bool many = n > 8;
    const int rows = q.nq * a.ratio;
    for (int rr = many ? blockIdx.y : blockIdx.y * WARPS + warp; rr < rows; rr += many ? gridDim.y : gridDim.y * WARPS) {
        const int rank = rr / rank_rows, r = rr - rank * rank_rows;
        auto piece = [&](int k) {
            return ((static_cast<int64_t>(c0 + k) * a.ranks + rank) * 2 + (k > 0 ? 0 : 1)) * rank_rows + r;
        };
        // the first accumulators are asked for before the maxima that weigh them
        const int k_first = many ? warp : 0, k_step = many ? WARPS : 1;
        float2 ahead[4][E / 2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k_first + j * k_step;
            if (k >= n) continue;
            const float2* p = reinterpret_cast<const float2*>(a.part + piece(k) * D) + lane;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) ahead[j][e] = p[32 * e];
        }
        // maximum over all partials; each lane's weight and share of the sum (partials lane, lane + 32, ..)
        float mx = -INFINITY;
        for (int k = lane; k < n; k += 32) mx = fmaxf_nan(mx, a.part_ml[piece(k)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float lt = 0.0f;
        float2 x[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) x[e] = make_float2(0.0f, 0.0f);
        for (int k0 = 0; k0 < n; k0 += 32) {
            float w = 0.0f;
            if (k0 + lane < n) {
                const float2 v = a.part_ml[piece(k0 + lane)];
                // weight 0, not left out: a NaN (of a score, or 0 times an infinite value) stays
                w = v.x == -INFINITY ? 0.0f : ex2_ftz(v.x - mx);
                lt = fmaf(w, v.y, lt);
            }
            if (k0 == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = k_first + j * k_step;
                    const float f = __shfl_sync(0xffffffffu, w, k & 31);
                    if (k >= n) continue;
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        x[e].x = fmaf(f, ahead[j][e].x, x[e].x);
                        x[e].y = fmaf(f, ahead[j][e].y, x[e].y);
                    }
                }
            }
#pragma unroll 2
            for (int k = k_first + (k0 == 0 ? 4 * k_step : 0); k < min(n - k0, 32); k += k_step) {
                const float f = __shfl_sync(0xffffffffu, w, k);
                const float2* p = reinterpret_cast<const float2*>(a.part + piece(k0 + k) * D) + lane;
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const float2 v = p[32 * e];
                    x[e].x = fmaf(f, v.x, x[e].x);
                    x[e].y = fmaf(f, v.y, x[e].y);
                }
            }
        }
        lt = warp_sum(lt);
        if (many) {
#pragma unroll
            for (int e = 0; e < E / 2; ++e) acc[warp][lane + 32 * e] = x[e];
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    for (int w = 1; w < WARPS; ++w) {
                        x[e].x += acc[w][lane + 32 * e].x;
                        x[e].y += acc[w][lane + 32 * e].y;
                    }
            }
            __syncthreads();
            if (warp > 0) continue;
        }
        const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
        const int i = rr / a.ratio;
        if (GDN_IN_RANGE(g_attn_cache_error, q.tok + i < a.n_tokens && head * a.ratio + rr - i * a.ratio < a.hq)) {
            uint32_t* out = reinterpret_cast<uint32_t*>(a.o + (q.tok + i) * a.ld_o + (head * a.ratio + rr - i * a.ratio) * D) + lane;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) out[32 * e] = bf16x2(x[e].x * inv, x[e].y * inv);
        }
    }
}

// ------------------------------------------------------------ host

cudaError_t launch_attn_tree(const gdn_kv_cache& c, AttCacheArgs& a, cudaStream_t st);   // k_attn_tree.cu
constexpr int AC_TREE_TILE = 128;       // its rows per CTA

// The kernel for many rows from this many rows of a pair on (max_q times the
// heads of a key/value head), for every type and head size.  Six sequences of
// 4000 to 24000 keys, this kernel and the other, us, heads of 256 / 128 / 64: 32
// rows bf16 81 and 82 / 99 and 90 / 57 and 59, int8 81 and 104 / 93 and 150 / 57
// and 110, e4m3 93 and 109 / 125 and 152 / 85 and 110; 48 rows bf16 113 and 86 /
// 173 and 92 / 93 and 59, int8 113 and 107 / 163 and 149 / 92 and 112, e4m3 131
// and 111 / 226 and 152 / 142 and 112.  So one threshold costs bf16 heads of 128 a
// tenth from 20 to 32 rows and int8 heads of 64 a fifth from 33 to 64.  Up to 32
// rows this kernel reads the cache once (twice for heads of 256), the other up to
// 128.
constexpr int AC_TREE_ROWS = 33;

size_t attn_cache_workspace_bytes(const gdn_kv_cache& c, int64_t n_tokens, int hq) {
    // partials of the rows of one CTA: 4096 / D at most in the kernel for few rows
    const int rows = n_tokens * (hq / c.n_kv_heads) >= AC_TREE_ROWS ? AC_TREE_TILE : 4096 / c.head_dim;
    return static_cast<size_t>(AC_MAX_RUNS) * 2 * rows * (c.head_dim * 4 + 8);
}

template <int D>
static cudaError_t ac_join(const AttCacheArgs& a, int rank_rows, cudaStream_t st) {
    // a warp per row, and up to a block per row while that is two blocks per SM
    const int rows = a.max_q * a.ratio, pairs = a.n_seqs * a.heads;
    const int y = std::max((rows + AC_JOIN_THREADS / 32 - 1) / (AC_JOIN_THREADS / 32), std::min(rows, 2 * AC_MAX_RUNS / pairs));
    return launch_dependent(attn_cache_join_kernel<D>, dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(y)),
                            dim3(AC_JOIN_THREADS), 0, st, a, rank_rows);
}

template <int D, int T, int NR>
static cudaError_t ac_launch(const gdn_kv_cache& c, AttCacheArgs& a, cudaStream_t st) {
    using L = AcSmem<D, T, NR>;
    static PerDeviceOnce once;
    if (once.run([](int) {
            cudaFuncSetAttribute(attn_cache_kernel<D, T, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES + 1024);
        }) < 0)
        return cudaErrorInvalidDevice;
    CUtensorMap mk, mv;
    a.box = c.page_tokens < L::KEYS ? c.page_tokens : L::KEYS;
    a.start = L::START;
    if (!ac_map(&mk, c.k, c, a.box, L::NSLAB) || !ac_map(&mv, c.v, c, a.box, L::NSLAB)) return cudaErrorInvalidValue;
    a.ranks = (a.max_q * a.ratio + L::ROWS - 1) / L::ROWS;
    a.runs = AC_MAX_RUNS / a.ranks;
    cudaError_t e = launch_dependent(attn_cache_kernel<D, T, NR>, dim3(static_cast<unsigned>(a.runs * a.ranks)), dim3(L::THREADS),
                                     L::BYTES + 1024, st, mk, mv, a);
    if (e != cudaSuccess) return e;
    return ac_join<D>(a, L::ROWS, st);
}

template <int D, int NR>
static cudaError_t ac_launch_t(const gdn_kv_cache& c, AttCacheArgs& a, cudaStream_t st) {
    if (c.dtype == GDN_KV_BF16) return ac_launch<D, GDN_KV_BF16, NR>(c, a, st);
    if (c.dtype == GDN_KV_I8) return ac_launch<D, GDN_KV_I8, NR>(c, a, st);
    return ac_launch<D, GDN_KV_E4M3, NR>(c, a, st);
}

cudaError_t launch_attn_cache(const gdn_kv_cache& c, const uint16_t* q, int64_t ld_q, const int32_t* cu, int64_t n_tokens,
                              int max_q, const uint64_t* tree, const int32_t* table, int64_t ld_table, int max_blocks,
                              const int32_t* lens, int n_seqs, int hq, float scale, uint16_t* o, int64_t ld_o,
                              void* workspace, cudaStream_t st, uint64_t fault_wait_ns) {
    AttCacheArgs a{};
    a.wait_ns = fault_wait_ns ? fault_wait_ns : 2000000000ull;
    a.withhold = fault_wait_ns != 0;
    a.n_pages = c.n_pages;
    a.heads = c.n_kv_heads;
    a.page = c.page_tokens;
    a.page_shift = c.page_tokens == 16 ? 4 : c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : 7;
    a.ratio = hq / c.n_kv_heads;
    a.hq = hq;
    a.v = c.v;
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
    a.max_q = max_q < n_tokens ? max_q : static_cast<int>(n_tokens);
    a.max_blocks = max_blocks;
    a.sl2 = scale * LOG2E;
    a.part_ml = static_cast<float2*>(workspace);
    const int rows = a.max_q * a.ratio;
    // maxima and sums first, then the accumulators
    const int part_rows = rows >= AC_TREE_ROWS ? AC_TREE_TILE : 4096 / c.head_dim;
    a.part = static_cast<float*>(workspace) + static_cast<int64_t>(AC_MAX_RUNS) * 2 * part_rows * 2;
    if (rows >= AC_TREE_ROWS) {
        const cudaError_t e = launch_attn_tree(c, a, st);
        if (e != cudaSuccess) return e;
        return c.head_dim == 64 ? ac_join<64>(a, AC_TREE_TILE, st) : c.head_dim == 128 ? ac_join<128>(a, AC_TREE_TILE, st) : ac_join<256>(a, AC_TREE_TILE, st);
    }
    if (c.head_dim == 256) return rows <= 8 ? ac_launch_t<256, 1>(c, a, st) : ac_launch_t<256, 2>(c, a, st);
    if (c.head_dim == 128)
        return rows <= 8 ? ac_launch_t<128, 1>(c, a, st) : rows <= 16 ? ac_launch_t<128, 2>(c, a, st) : ac_launch_t<128, 4>(c, a, st);
    return rows <= 8 ? ac_launch_t<64, 1>(c, a, st) : rows <= 16 ? ac_launch_t<64, 2>(c, a, st) : ac_launch_t<64, 4>(c, a, st);
}

int* attn_cache_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_attn_cache_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

int* attn_cache_skipped_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_attn_cache_skipped) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdn
