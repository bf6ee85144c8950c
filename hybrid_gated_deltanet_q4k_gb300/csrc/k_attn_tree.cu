// Cache attention of many rows (trees of drafts, long chains): the same
// operator, partition and partials as the kernel for few rows, on the
// fifth-generation tensor cores, 128 rows per CTA.
//
// With R rows of a (sequence, key/value head) pair every cached byte of an
// 8-bit cache is worth 4 R flops (of bf16, 2 R): from some tens of rows on the
// kernel for few rows, which reads the cache once per 8 to 32 rows, is bound by
// L2 and its own instructions, while 128 rows of one tcgen05 instruction cost
// the cache one read.  Pairs of more than 128 rows take several CTAs with the
// same run of blocks; they walk it at the same time, so the cache comes from L2
// for all but one.
//
// Per tile of 128 keys (row r = TMEM lane r):
//   S = Q K^T      M = 128, N = 128, K = D; Q in TMEM, K from shared memory; two
//                  S buffers (one for heads of 256, where TMEM has no more)
//   softmax        two threads per row, 64 scores each; P goes over the
//                  thread's own scores.  The running maximum is raised only
//                  past a margin: the two threads swap their maxima when one of
//                  their 32 rows asks for it, a vote in the barrier between them
//   O += P V       M = 128, N = D, K = 128; P from TMEM, V [key][d] as the
//                  MN-major operand, the image that the copy writes: no transpose
// The products are as wide as they go, for an instruction takes 65 cycles to
// issue here however little it multiplies (tiles of 64 keys were bound by that).
// The pages are bf16: TMA writes the operand images (128-byte swizzle).  8-bit
// codes go through a ring of raw tiles that four warps turn into fp16 images
// (exact); the row scales stay out of the products, as in the other kernel: a
// key's multiplies its scores, a value's goes into the exponent of p'.  fp16
// probabilities are p' 2^11, exact to 2^-11 down to 2^-25 of the largest and
// zero below 2^-36 of it.  The scales' logarithms are held twice: at least -80
// (AC_VS_MIN) for the maximum, and as they are for the probabilities where a tile
// has one far from 1.
//
// Warps: 0 copies, 1 allocates TMEM and issues the products, 2-9 softmax, and
// for 8-bit caches 10-13 convert.  Every wait is bounded; after one runs out the
// CTA stops issuing, lets copies and products finish and returns with the error
// word set.
//
// Measured: six trees of 28 to 63 tokens over 11674 to 24000 keys, 16 over 4
// heads of 256: bf16 139 us (585 TFLOP/s, 3.3 TB/s of cache), int8 222, e4m3 224.
// S, the softmax and P V of a tile of heads of 256 follow each other, because TMEM
// holds one S beside Q and O: of a tile's 4400 cycles the softmax waits 2800 for S
// (tensor pipe 41 %, issue slots 19 %).  8-bit tiles of heads of 256 add the
// conversion to that chain, for shared memory holds two images; those of 128 and
// 64 (32 over 8 heads: 250 and 193) wait for their four converting warps, one a
// scheduler (tensor pipe 18 and 11 %, issue slots 48 %).  A piece's start and end
// take 8 us of the 139, the join 9.
#include "attn_cache.cuh"
#include "tcgen05.cuh"

#include <type_traits>

namespace gdn {

constexpr int AT_ROWS = 128;
constexpr int AT_SM_WARPS = 8;
constexpr int AT_SM_THREADS = 32 * AT_SM_WARPS;

template <int D, int T>
struct AtSmem {
    static constexpr bool Q8 = T != GDN_KV_BF16;
    static constexpr int BN = 128;
    static constexpr int THREADS = 32 * (2 + AT_SM_WARPS + (Q8 ? 4 : 0));
    static constexpr int ROW = D * (Q8 ? 1 : 2);
    static constexpr int SLAB = ROW < 128 ? ROW : 128;      // bytes of a cached row in one slab of the copies
    static constexpr int NSLAB = ROW / SLAB;
    static constexpr int RAW = BN * ROW;                    // a tile as cached
    static constexpr int S16 = D / 64;                      // slabs of an operand image: [rows][64 x 16 bit]
    static constexpr int TILE = BN * D * 2;                 // a K or V image
    // S buffers in TMEM; images held at once (K and V of the tiles in turn); raw tiles in flight.  An odd
    // number of images needs the single S buffer (see the waits on ID).
    static constexpr int SB = D == 256 ? 1 : 2;
    static constexpr int NI = Q8 ? (D == 256 ? 2 : 4) : D == 256 ? 3 : D == 128 ? 6 : 8;
    static constexpr int RS = !Q8 ? 1 : D == 256 ? 2 : D == 128 ? 4 : 8;
    static constexpr int I0 = 0;
    static constexpr int R0 = I0 + NI * TILE;
    static constexpr int F0 = R0 + (Q8 ? RS * RAW : 0);     // key factors, log2 value scales, their inverses: [softmax warp][4][BN / 2]
    static constexpr int X0 = F0 + (Q8 ? AT_SM_WARPS * 4 * BN / 2 * 4 : 0);   // maxima of the halves; masks of zero weights [2][128]
    static constexpr int L0 = X0 + 2 * AT_ROWS * 8;         // row sums of each half
    static constexpr int P0 = L0 + 2 * AT_ROWS * 4;         // blocks before each sequence
    static constexpr int T0 = P0 + (GDN_MAX_SEQS + 2) * 8;  // the sequences
    static constexpr int W0 = T0 + GDN_MAX_SEQS * 12;
    static constexpr int B0 = W0 + 16 * 8;                  // mbarriers
    // Q in; P in, alternating; per image: full, and done (the product that reads it); raw tiles, full and empty
    static constexpr int QF = 0, PF = 1, FIN = 3, IF = 4, ID = IF + NI, RF = ID + NI, RE = RF + RS, NBAR = RE + RS;
    static constexpr int MISC = B0 + 8 * NBAR;              // TMEM base, abort flag, keys with values that are not finite, tiles of the piece
    static constexpr int BYTES = MISC + 32;
    // at least 120 KB, so that one CTA holds an SM (it allocates all TMEM columns)
    static constexpr int DYN = BYTES + 1024 > 120 * 1024 ? BYTES + 1024 : 120 * 1024;
    static_assert(DYN <= 227 * 1024, "shared memory of a CTA");
    // TMEM columns: S (BN each; the P of either half over the first half of its scores), Q, O
    static constexpr uint32_t QCOL = SB * BN, OCOL = QCOL + D / 2;
    static_assert(OCOL + D <= 512, "TMEM columns");
};

// Waits for a phase, asleep for up to 20 us at a time: warps that poll take
// issue slots and shared-memory cycles from the one that issues the products.
// Gives up after limit_ns with the error word set, and at once after any wait of
// the CTA has.
__device__ __forceinline__ bool at_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    auto sleep = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
            : "memory");
        return ok != 0;
    };
    if (sleep()) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!*abort) {
        if (sleep()) return true;
        if (globaltimer_ns() - t0 > limit_ns) {
            atomicCAS(&g_attn_cache_error, 0, static_cast<int>(ERR_WAIT_TIMEOUT));
            *abort = 1;
        }
    }
    return false;
}
__device__ __forceinline__ bool at_ready(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void at_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// One arrival for a warp whose lanes have all done their part.
__device__ __forceinline__ void at_arrive_warp(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) at_arrive(bar);
}
// All softmax threads; the two warps that share 32 rows (barriers 2 .. 5), as they are and with a vote.
__device__ __forceinline__ void at_bar_softmax() { asm volatile("bar.sync 1, %0;" ::"n"(AT_SM_THREADS) : "memory"); }
__device__ __forceinline__ void at_bar_rows(int quad) { asm volatile("bar.sync %0, 64;" ::"r"(2 + quad) : "memory"); }
__device__ __forceinline__ bool at_vote_rows(int quad, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %2, 0;\n\t"
        "bar.red.or.pred p, %1, 64, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r)
        : "r"(2 + quad), "r"(x ? 1u : 0u)
        : "memory");
    return r != 0;
}

template <int D, int T>
__global__ void __launch_bounds__(AtSmem<D, T>::THREADS, 1)
attn_tree_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                 const __grid_constant__ AttCacheArgs a) {
    using L = AtSmem<D, T>;
    constexpr int BN = L::BN, HN = BN / 2, SB = L::SB, NI = L::NI, RS = L::RS;
    constexpr bool Q8 = L::Q8;
    extern __shared__ __align__(1024) unsigned char smb[];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smb) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + L::B0);
    int64_t* pre = reinterpret_cast<int64_t*>(base + L::P0);
    AcSeq* seq = reinterpret_cast<AcSeq*>(base + L::T0);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(base + L::MISC);
    volatile int* abort = reinterpret_cast<volatile int*>(base + L::MISC + 4);
    unsigned long long* odd = reinterpret_cast<unsigned long long*>(base + L::MISC + 8);
    volatile int* piece_tiles = reinterpret_cast<volatile int*>(base + L::MISC + 16);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t sbase = smem_addr(base);

    if (tid == 0) {
        for (int i = 0; i < L::NBAR; ++i) {
            int n = 1;
            if (i == L::QF || i == L::PF || i == L::PF + 1) n = AT_SM_WARPS;
            if (Q8 && ((i >= L::IF && i < L::ID) || i >= L::RE)) n = 4;   // the converting warps
            mbar_init_cta(bars + i, n);
        }
        mbar_init_fence();
        *abort = 0;
        *odd = 0;
    }
    // TMEM is taken when the kernel before this one is through, and the next one may start when it is taken: a CTA that
    // held it while it waited could keep it from the kernel it waits for
    pdl_wait();
    if (warp == 1) t5::alloc(tslot, 512);
    t5::fence_before();
    ac_prefix(a, pre, seq, reinterpret_cast<int64_t*>(base + L::W0), blockIdx.x == 0);   // ends with a barrier
    pdl_trigger();
    t5::fence_after();
    const uint32_t tmem = *tslot;
    const int run = blockIdx.x / a.ranks, row0 = (blockIdx.x % a.ranks) * AT_ROWS;
    const int64_t total = pre[a.n_seqs] * a.heads, per = ac_run_blocks(a, total);
    int64_t at = run * per;
    const int64_t end = at + per < total ? at + per : total;
    int s = at < end ? ac_seq_of(a, pre, at) : 0;
    AcPiece pc;
    // every role walks the same pieces; a piece is `nb` tiles of BN keys from tile t0
    int t0 = 0, nb = 0, rows = 0;
    auto next = [&]() {
        while (ac_next(a, pre, seq, at, end, s, pc)) {
            rows = min(pc.q.nq * a.ratio - row0, AT_ROWS);
            if (rows <= 0) continue;
            t0 = pc.b0 * (AC_BLOCK / BN);
            nb = min(pc.b1 * (AC_BLOCK / BN), pc.q.len == 0 ? 1 : (pc.q.len - 1) / BN + 1) - t0;
            return true;
        }
        return false;
    };
    // copies of a tile: the rows of each of its pages, by slab; lane = page * NSLAB + slab
    const int copies = BN / a.box;
    uint32_t n = 0;   // tiles so far, over all pieces

    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        const int p = lane / L::NSLAB, slab = lane % L::NSLAB;
        const bool on = lane < copies * L::NSLAB;
        const int off = on ? p * a.box : 0;
        bool ok = true;
        while (ok && next()) {
            const int32_t* table = a.table + pc.s * a.ld_table;
            auto page_of = [&](int j) { return table[min(((t0 + j) * BN + off) >> a.page_shift, a.max_blocks - 1)]; };
            auto load = [&](const CUtensorMap* map, uint64_t* bar, int dst, int bytes, int j, int page) {
                const int row = ((t0 + j) * BN + off) & (a.page - 1);
                const int pg = page >= 0 && page < a.n_pages ? page : 0;   // an unseen page: any rows, all of them masked
                if (lane == 0) mbar_expect_tx(bar, bytes);
                if (on) tma_load_4d(base + dst + slab * (BN * L::SLAB) + off * L::SLAB, map, bar, 0, row, slab, pg * a.heads + pc.head);
            };
            int page = page_of(0);
            for (int j = 0; ok && j < nb; ++j) {
                const int ahead = page_of(min(j + 1, nb - 1));
                for (int v = 0; ok && v < 2; ++v) {      // keys, then values
                    const uint32_t m = 2 * n + v;
                    if constexpr (Q8) {
                        const uint32_t sl = m % RS;
                        if (m >= RS) ok = __all_sync(0xffffffffu, at_wait(bars + L::RE + sl, (m / RS - 1) & 1, abort, a.wait_ns));
                        if (ok && !(a.withhold && m == 0)) load(v ? &mv : &mk, bars + L::RF + sl, L::R0 + sl * L::RAW, L::RAW, j, page);
                    } else {
                        const uint32_t sl = m % NI;
                        if (m >= NI) ok = __all_sync(0xffffffffu, at_wait(bars + L::ID + sl, (m / NI - 1) & 1, abort, a.wait_ns));
                        if (ok && !(a.withhold && m == 0)) load(v ? &mv : &mk, bars + L::IF + sl, L::I0 + sl * L::TILE, L::TILE, j, page);
                    }
                }
                page = ahead;
                ++n;
            }
        }
    } else if (Q8 && warp >= 10) {
        // ------------------------------------------------------------ codes to fp16 images
        bool ok = true;
        const int ct = tid - 320;
        while (ok && next()) {
            for (int j = 0; ok && j < nb; ++j) {
                for (int v = 0; ok && v < 2; ++v) {
                    const uint32_t m = 2 * n + v, sl = m % RS, im = m % NI;
                    ok = at_wait(bars + L::RF + sl, (m / RS) & 1, abort, a.wait_ns);
                    if (ok && m >= NI) ok = at_wait(bars + L::ID + im, (m / NI - 1) & 1, abort, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const unsigned char* src = base + L::R0 + sl * L::RAW;
                    unsigned char* dst = base + L::I0 + im * L::TILE;
                    // 16 codes per step; consecutive threads take consecutive keys
#pragma unroll 4
                    for (int e = ct; e < BN * (D / 16); e += 128) {
                        const int key = e % BN, c = e / BN;
                        uint4 w;
                        if constexpr (L::SLAB == 128)
                            w = *reinterpret_cast<const uint4*>(src + (c >> 3) * (BN * 128) + key * 128 + (((c ^ key) & 7) << 4));
                        else
                            w = *reinterpret_cast<const uint4*>(src + key * 64 + (((c ^ (key >> 1)) & 3) << 4));
                        if constexpr (T == GDN_KV_I8) {
                            w.x ^= 0x80808080u;
                            w.y ^= 0x80808080u;
                            w.z ^= 0x80808080u;
                            w.w ^= 0x80808080u;
                        }
                        unsigned char* row = dst + (c >> 2) * (BN * 128) + key * 128;
                        const int c0 = (2 * c) & 7;
                        *reinterpret_cast<uint4*>(row + (((c0 ^ key) & 7) << 4)) =
                            make_uint4(codes_f16<T, 0, 1>(w.x), codes_f16<T, 2, 3>(w.x), codes_f16<T, 0, 1>(w.y), codes_f16<T, 2, 3>(w.y));
                        *reinterpret_cast<uint4*>(row + ((((c0 + 1) ^ key) & 7) << 4)) =
                            make_uint4(codes_f16<T, 0, 1>(w.z), codes_f16<T, 2, 3>(w.z), codes_f16<T, 0, 1>(w.w), codes_f16<T, 2, 3>(w.w));
                    }
                    fence_proxy_async_smem();
                    at_arrive_warp(bars + L::IF + im, lane);
                    at_arrive_warp(bars + L::RE + sl, lane);
                }
                ++n;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // S of a tile needs its K image and its buffer (P V of the tile SB before
        // has read P there); P V needs P and the V image.  The warp polls both and
        // one lane issues what is ready; a stall past the limit sets the error word.
        constexpr uint32_t FULL = 0xffffffffu;
        constexpr uint32_t IDS = Q8 ? t5::idesc_f16(AT_ROWS, BN) : t5::idesc_bf16(AT_ROWS, BN);
        constexpr uint32_t IDO = (Q8 ? t5::idesc_f16(AT_ROWS, D) : t5::idesc_bf16(AT_ROWS, D)) | (1u << 16);   // B MN-major
        const uint32_t one = lane == 0, tm = __reduce_max_sync(FULL, tmem);
        const uint64_t kd0 = t5::desc_sw128(sbase + L::I0), vd0 = t5::desc_sw128_mn(sbase + L::I0, BN * 128);
        bool ok = true;
        uint32_t piece = 0;
        uint32_t si = 0, sslot = 0, sphase = 0;    // tile, image and its phase of the next S
        uint32_t bslot = 1, bphase = 0;            // image and phase of P V of the tile SB before it
        uint32_t pi = 0, pslot = 1, pphase = 0;    // of the next P V
        auto two_on = [](uint32_t& slot, uint32_t& phase) {    // the image of the next tile
            slot += 2;
            if (slot >= NI) {
                slot -= NI;
                phase ^= 1;
            }
        };
        while (true) {
            // the softmax says how many tiles the piece has (0: no more pieces)
            ok = __all_sync(FULL, at_wait(bars + L::QF, piece & 1, abort, a.wait_ns));
            const int tiles = static_cast<int>(__reduce_max_sync(FULL, static_cast<uint32_t>(*piece_tiles)));
            if (!ok || tiles == 0) break;
            ++piece;
            int ns = 0, np = 0, spins = 0;
            uint64_t t_last = 0;
            while (ok && np < tiles) {
                // all four tests under one latency; what is ready of both is issued without another look
                const bool k = at_ready(bars + L::IF + sslot, sphase), b = at_ready(bars + L::ID + bslot, bphase);
                const bool p = at_ready(bars + L::PF + (pi & 1), (pi >> 1) & 1), v = at_ready(bars + L::IF + pslot, pphase);
                const bool s_on = __all_sync(FULL, ns < tiles && ns < np + SB && k && (ns < SB || b));
                const bool p_on = __all_sync(FULL, np < ns && p && v);
                if (s_on) {
                    t5::fence_after();
                    const uint64_t kd = kd0 + sslot * (L::TILE / 16);
                    const uint32_t to = tm + (SB == 2 ? (si & 1) * BN : 0);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        t5::mma_f16_ts_on(one, to, tm + L::QCOL + kk * 8, kd + ((kk >> 2) * (BN * 128) + (kk & 3) * 32) / 16, IDS,
                                          kk > 0 ? 1u : 0u);
                    t5::commit_on(one, bars + L::ID + sslot);
                    ++ns;
                    two_on(sslot, sphase);
                    if (++si > SB) two_on(bslot, bphase);
                }
                if (p_on) {
                    t5::fence_after();
                    const uint64_t vd = vd0 + pslot * (L::TILE / 16);
                    const uint32_t from = tm + (SB == 2 ? (pi & 1) * BN : 0);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        t5::mma_f16_ts_on(one, tm + L::OCOL, from + (kk >> 2) * HN + (kk & 3) * 8, vd + kk * (2048 / 16), IDO,
                                          (np > 0 || kk > 0) ? 1u : 0u);
                    t5::commit_on(one, bars + L::ID + pslot);
                    ++np;
                    ++pi;
                    two_on(pslot, pphase);
                }
                if (s_on || p_on) {
                    spins = 0;
                } else if (++spins >= 1024) {
                    const uint64_t now = globaltimer_ns();
                    if (spins == 1024) t_last = now;
                    if (__any_sync(FULL, *abort || now - t_last > a.wait_ns)) {
                        if (lane == 0 && !*abort) atomicCAS(&g_attn_cache_error, 0, static_cast<int>(ERR_WAIT_TIMEOUT));
                        __syncwarp();
                        *abort = 1;
                        ok = false;
                    }
                }
            }
        }
        // every product issued has completed before TMEM is released
        t5::commit_on(one, bars + L::FIN);
        mbar_wait_bounded(bars + L::FIN, 0, nullptr, 0, 200000000ull);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        // thread half `half` of a row: half of the keys of each tile, and of the columns of q and o
        const int quad = warp & 3, half = (warp - 2) >> 2, r = 32 * quad + lane, st = tid - 64;
        const uint32_t trow = tmem + (static_cast<uint32_t>(32 * quad) << 16);
        float* xmax = reinterpret_cast<float*>(base + L::X0);
        float* lsum = reinterpret_cast<float*>(base + L::L0);
        float* kfac = reinterpret_cast<float*>(base + L::F0) + (warp - 2) * 4 * HN;   // this warp's: HN key factors,
        float* vlog = kfac + HN;                          // log2 value scales, and the scales' inverses
        float* vinv = vlog + HN;
        float* vraw = vinv + HN;
        constexpr int CH = HN / 32;                       // 32 scores at a time
        bool ok = true;
        while (next()) {
            const AcSeq q = pc.q;
            const int ctx = q.len - q.nq, rr = row0 + r, tok = rr / a.ratio;
            const bool on = r < rows;
            const int hq = pc.head * a.ratio + rr - tok * a.ratio;
            const int32_t* table = a.table + pc.s * a.ld_table;
            const uint64_t seen = !on ? 0 : a.tree ? a.tree[q.tok + tok] : tok >= 63 ? ~0ull : (1ull << (tok + 1)) - 1;

            // ---- Q to TMEM: this thread half a row.  The last piece's products have read theirs.
            float factor = a.sl2;
            {
                const uint16_t* src = a.q + static_cast<int64_t>(q.tok + (on ? tok : 0)) * a.ld_q + (on ? hq : 0) * D + half * (D / 2);
                auto load = [&](int c, uint32_t (&w)[8]) {     // elements 16 c .. 16 c + 15
                    if (a.wide) {
                        load32(src + 16 * c, w);
                    } else {
                        const uint4 x = *reinterpret_cast<const uint4*>(src + 16 * c), y = *reinterpret_cast<const uint4*>(src + 16 * c + 8);
                        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
                        w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = on ? w[e] : 0u;
                };
                float up = 1.0f;
                if constexpr (Q8) {
                    float amax = 0.0f;
#pragma unroll 4
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t u[8];
                        load(c, u);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u))));
                    }
                    lsum[half * AT_ROWS + r] = amax;
                    at_bar_softmax();
                    amax = fmaxf(amax, lsum[(half ^ 1) * AT_ROWS + r]);
                    const int ex = min(max(static_cast<int>((__float_as_uint(amax) >> 23) & 255) - 127, AC_Q_MIN), 127);
                    up = __uint_as_float(static_cast<uint32_t>(127 + 14 - ex) << 23);
                    factor *= __uint_as_float(static_cast<uint32_t>(127 - 14 + ex) << 23);
                }
#pragma unroll
                for (int c = 0; c < D / 32; c += 2) {
                    uint32_t v[2][8], u[16];
                    load(c, v[0]);
                    load(c + 1, v[1]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) u[e] = v[e >> 3][e & 7];
                    if constexpr (Q8) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            u[e] = f16x2_bits(__uint_as_float(u[e] << 16) * up, __uint_as_float(u[e] & 0xffff0000u) * up);
                    }
                    t5::st16u(trow + L::QCOL + half * (D / 4) + 8 * c, u);
                }
                t5::fence_before();
                if (warp == 2 && lane == 0) *piece_tiles = nb;
                at_arrive_warp(bars + L::QF, lane);
            }

            // ---- do all pages of the piece lie in the cache?
            bool all_in = true;
            {
                const int lo = (t0 * BN) >> a.page_shift, hi = (min((t0 + nb) * BN, q.len) - 1) >> a.page_shift;
                for (int b = lo + lane; b <= hi; b += 32) {
                    const int pg = table[b];
                    all_in &= pg >= 0 && pg < a.n_pages;
                }
                all_in = __all_sync(0xffffffffu, all_in);
                if (!all_in && warp == 2 && lane == 0) atomicExch(&g_attn_cache_skipped, static_cast<int>(ERR_INDEX));
            }
            auto page_at = [&](int key) { return table[min(key >> a.page_shift, a.max_blocks - 1)]; };

            // ---- 8-bit: the scales of this half's keys (by lane), read a tile ahead, their pages two
            constexpr int KL = HN / 32;     // keys per lane
            float ksn[KL], vsn[KL];
            int pgn[KL];
            auto key_of = [&](int j, int x) { return (t0 + min(j, nb - 1)) * BN + half * HN + 32 * x + lane; };
            auto scales_of = [&](int j) {
#pragma unroll
                for (int x = 0; x < KL; ++x) {
                    const int pg = pgn[x] >= 0 && pgn[x] < a.n_pages ? pgn[x] : 0;
                    const int64_t row = (static_cast<int64_t>(pg) * a.heads + pc.head) * a.page + (key_of(j, x) & (a.page - 1));
                    ksn[x] = a.sk[row];
                    vsn[x] = a.sv[row];
                    pgn[x] = page_at(key_of(j + 1, x));
                }
            };
            if constexpr (Q8) {
#pragma unroll
                for (int x = 0; x < KL; ++x) pgn[x] = page_at(key_of(0, x));
                scales_of(0);
            }

            float m = -INFINITY, l = 0.0f;
            uint64_t none = 0;      // new keys this row sees with probability zero
            // A tile; EDGE: some row may not see some key.  Two copies of the code, since
            // the tests inside its loops would cost the plain tiles five times their exponentials.
            auto tile = [&](int j, auto edge_tag) {
                constexpr bool edge = decltype(edge_tag)::value;
                constexpr int KEEP = edge || Q8 ? 1 : CH;   // chunks of scores in registers (fewer: read twice)
                const uint32_t i = n + j;
                const int key0 = (t0 + j) * BN;
                bool wide = false;      // a value scale so far from 1 that its inverse will not do
                const uint32_t sbuf = trow + (SB == 2 ? (i & 1) * BN : 0) + half * HN;   // this half's scores
                auto exists = [&](int key) {
                    if (key0 + key >= q.len) return false;
                    if (all_in) return true;
                    const int pg = page_at(key0 + key);
                    return pg >= 0 && pg < a.n_pages;
                };
                if constexpr (Q8) {
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < KL; ++x) {
                        const float lv = lg2(fmaxf_nan(vsn[x], AC_VS_TINY));
                        kfac[32 * x + lane] = ksn[x];
                        vlog[32 * x + lane] = lv;
                        vinv[32 * x + lane] = ex2_ftz(-lv);
                        vraw[32 * x + lane] = lg2(fmaxf_nan(vsn[x], AC_VS_FLOOR));
                        wide |= !(fabsf(lv) <= 60.0f);
                    }
                    wide = __any_sync(0xffffffffu, wide);
                    __syncwarp();     // the tables are read by all lanes (a vote does not order memory)
                    scales_of(j + 1);
                }

                ok = __all_sync(0xffffffffu, ok && at_wait(bars + L::ID + 2 * i % NI, (2 * i / NI) & 1, abort, a.wait_ns));
                // 32 scores: raw for a bf16 cache (their factor is positive), else y = x + log2 of the value's scale
                float xs[KEEP][32];
                auto scores = [&](int ch, float (&x)[32], const float* vs) {
                    t5::ld32(sbuf + 32 * ch, x);
                    if constexpr (Q8) {
                        const F2 f = f2(factor, factor);
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 k4 = *reinterpret_cast<const float4*>(kfac + 32 * ch + c);
                            const float4 v4 = *reinterpret_cast<const float4*>(vs + 32 * ch + c);
                            f2_split(f2_fma(f2(x[c], x[c + 1]), f2_mul(f, f2(k4.x, k4.y)), f2(v4.x, v4.y)), x[c], x[c + 1]);
                            f2_split(f2_fma(f2(x[c + 2], x[c + 3]), f2_mul(f, f2(k4.z, k4.w)), f2(v4.z, v4.w)), x[c + 2], x[c + 3]);
                        }
                    }
                    if constexpr (edge) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const int key = half * HN + 32 * ch + c, d = key0 + key - ctx;
                            if (!exists(key) || (d >= 0 && !((seen >> (d & 63)) & 1))) x[c] = -INFINITY;
                        }
                    }
                };
                float bm = -INFINITY;
                if (ok) {
                    t5::fence_after();
#pragma unroll
                    for (int ch = 0; ch < CH; ++ch) {
                        float(&x)[32] = xs[KEEP == CH ? ch : 0];
                        scores(ch, x, vlog);
                        float b0 = fmaxf(x[0], x[1]), b1 = fmaxf(x[2], x[3]);
#pragma unroll
                        for (int c = 4; c < 32; c += 4) {
                            b0 = fmaxf(b0, fmaxf(x[c], x[c + 1]));
                            b1 = fmaxf(b1, fmaxf(x[c + 2], x[c + 3]));
                        }
                        bm = fmaxf(bm, fmaxf(b0, b1));
                    }
                    if constexpr (!Q8) bm *= factor;
                }
                if (at_vote_rows(quad, j == 0 || bm > m + AC_MARGIN)) {
                    // the row's maximum over both halves
                    xmax[half * AT_ROWS + r] = bm;
                    at_bar_rows(quad);
                    bm = fmaxf(bm, xmax[(half ^ 1) * AT_ROWS + r]);
                    at_bar_rows(quad);
                    if (j == 0) {
                        m = bm;
                    } else {
                        // O is rescaled once P V of tile i - 1 has finished
                        ok = __all_sync(0xffffffffu, ok && at_wait(bars + L::ID + (2 * i - 1) % NI, ((2 * i - 1) / NI) & 1, abort, a.wait_ns));
                        if (ok) {
                            const float mn = fmaxf(m, bm), f = m == -INFINITY ? 0.0f : ex2_ftz(m - mn);
                            m = mn;
                            l *= f;
                            t5::fence_after();
#pragma unroll 1
                            for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
                                float ov[32];
                                t5::ld32(trow + L::OCOL + c0, ov);
#pragma unroll
                                for (int e = 0; e < 32; ++e) ov[e] *= f;
                                t5::st32(trow + L::OCOL + c0, ov);
                            }
                        }
                    }
                }
                if (ok) {
                    const float mm = m == -INFINITY ? 0.0f : Q8 ? m - AC_LIFT : m;
                    const F2 nm = f2(-mm, -mm), ff = f2(factor, factor);
                    F2 l2 = f2(0.0f, 0.0f);
                    // P over this half's scores, and the row's sum: of 2^(x - m), which is p' times the inverse
                    // of the value's scale, or for scales far from 1 a power of its own
                    auto probabilities = [&](auto wide_tag) {
                        constexpr bool far = decltype(wide_tag)::value;
#pragma unroll
                        for (int ch = 0; ch < CH; ++ch) {
                            float(&x)[32] = xs[KEEP == CH ? ch : 0];
                            if (KEEP < CH) scores(ch, x, far ? vraw : vlog);
                            uint32_t pk[16];
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                float y0, y1;
                                f2_split(Q8 ? f2_add(f2(x[c], x[c + 1]), nm) : f2_fma(f2(x[c], x[c + 1]), ff, nm), y0, y1);
                                const float p0 = ex2_ftz(y0), p1 = ex2_ftz(y1);
                                if constexpr (Q8 && far) {
                                    const float2 lv = *reinterpret_cast<const float2*>(vraw + 32 * ch + c);
                                    float e0, e1;
                                    f2_split(f2_sub(f2(y0, y1), f2(lv.x, lv.y)), e0, e1);
                                    e0 = ex2_ftz(e0);
                                    e1 = ex2_ftz(e1);
                                    if constexpr (edge) {     // a scale that is no number reaches only the rows that see its key
                                        if (y0 == -INFINITY) e0 = 0.0f;
                                        if (y1 == -INFINITY) e1 = 0.0f;
                                    }
                                    l2 = f2_add(l2, f2(e0, e1));
                                } else if constexpr (Q8) {
                                    const float2 iv = *reinterpret_cast<const float2*>(vinv + 32 * ch + c);
                                    l2 = f2_fma(f2(p0, p1), f2(iv.x, iv.y), l2);
                                } else {
                                    l2 = f2_add(l2, f2(p0, p1));
                                }
                                if constexpr (Q8) {
                                    pk[c / 2] = f16x2_bits(p0, p1);
                                } else {
                                    const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
                                    pk[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
                                }
                                if constexpr (edge) {
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const int d = key0 + half * HN + 32 * ch + c + e - ctx;
                                        if (d >= 0 && d < 64 && (e ? p1 : p0) == 0.0f) none |= 1ull << d;
                                    }
                                }
                            }
                            t5::st16u(sbuf + 16 * ch, pk);   // over scores that have been read
                        }
                    };
                    if (Q8 && wide)
                        probabilities(std::true_type{});
                    else
                        probabilities(std::false_type{});
                    float s0, s1;
                    f2_split(l2, s0, s1);
                    l += s0 + s1;
                    if constexpr (edge) {
                        // values of keys that do not exist become zero, and so do those of
                        // new keys that are not finite: the rows that see them add them at the end
                        ok = __all_sync(0xffffffffu, at_wait(bars + L::IF + (2 * i + 1) % NI, ((2 * i + 1) / NI) & 1, abort, a.wait_ns));
                        unsigned char* vt = base + L::I0 + (2 * i + 1) % NI * L::TILE;
                        if (ok)
#pragma unroll 1
                            for (int e = st; e < BN * (D / 8); e += AT_SM_THREADS) {
                                const int key = e % BN, c = e / BN, d = key0 + key - ctx;
                                uint4* p = reinterpret_cast<uint4*>(vt + (c >> 3) * (BN * 128) + key * 128 + (((c ^ key) & 7) << 4));
                                if (!exists(key)) {
                                    *p = make_uint4(0u, 0u, 0u, 0u);
                                } else if (d >= 0 && T != GDN_KV_I8) {
                                    constexpr uint32_t EXP = Q8 ? 0x7c00u : 0x7f80u;
                                    uint32_t u[4] = {p->x, p->y, p->z, p->w}, any = 0;
#pragma unroll
                                    for (int h = 0; h < 4; ++h) {
                                        if ((u[h] & EXP) == EXP) u[h] &= 0xffff0000u, any = 1;
                                        if ((u[h] & (EXP << 16)) == (EXP << 16)) u[h] &= 0xffffu, any = 1;
                                    }
                                    if (any) {
                                        *p = make_uint4(u[0], u[1], u[2], u[3]);
                                        atomicOr(odd, 1ull << (d & 63));
                                    }
                                }
                            }
                        fence_proxy_async_smem();
                    }
                }
                t5::fence_before();
                at_arrive_warp(bars + L::PF + (i & 1), lane);
            };
            for (int j = 0; j < nb; ++j) {
                if ((t0 + j + 1) * BN > ctx || !all_in)
                    tile(j, std::true_type{});
                else
                    tile(j, std::false_type{});
            }
            n += nb;

            // ---- the piece's rows out
            const uint32_t i1 = n - 1;
            ok = __all_sync(0xffffffffu, ok && at_wait(bars + L::ID + (2 * i1 + 1) % NI, ((2 * i1 + 1) / NI) & 1, abort, a.wait_ns));
            lsum[half * AT_ROWS + r] = l;
            uint64_t* none_of = reinterpret_cast<uint64_t*>(xmax);   // the maxima have been read: every P is in
            none_of[half * AT_ROWS + r] = none;
            at_bar_softmax();
            const uint64_t odd_keys = *odd & seen;
            none |= none_of[(half ^ 1) * AT_ROWS + r];
            const float lt = lsum[r] + lsum[AT_ROWS + r];
            if (ok) {
                t5::fence_after();
                // half of the columns, 32 at a time, in whole sectors: 32 bytes a thread
                const bool whole = pc.b0 == 0 && pc.b1 == pc.blocks;
                const float inv = !whole ? 1.0f : lt == 0.0f ? 0.0f : 1.0f / lt;
                const int64_t part0 = (static_cast<int64_t>(blockIdx.x) * 2 + (pc.b0 > 0 ? 0 : 1)) * AT_ROWS + r;
                const bool out = on && GDN_IN_RANGE(g_attn_cache_error, q.tok + tok < a.n_tokens && hq < a.hq);
#pragma unroll 1
                for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
                    float ov[32];
                    t5::ld32(trow + L::OCOL + c0, ov);
                    if (odd_keys) {
                        // values that are not finite: infinite or NaN whatever their (positive) weight is
#pragma unroll 1
                        for (int d = 0; d < 64; ++d) {
                            if (!((odd_keys >> d) & 1)) continue;
                            const int key = ctx + d;
                            if (key < 0 || key < pc.b0 * AC_BLOCK || key >= pc.b1 * AC_BLOCK) continue;
                            const int pg = page_at(key);
                            if (pg < 0 || pg >= a.n_pages) continue;
                            const int64_t vr = ((static_cast<int64_t>(pg) * a.heads + pc.head) * a.page + (key & (a.page - 1))) * D + c0;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float v;
                                if constexpr (Q8)
                                    v = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(a.v)[vr + e], __NV_E4M3)));
                                else
                                    v = bf16_bits_to_float(static_cast<const uint16_t*>(a.v)[vr + e]);
                                if (!(fabsf(v) < INFINITY)) ov[e] += ((none >> d) & 1 ? 0.0f : 1.0f) * v;
                            }
                        }
                    }
                    if (whole && out) {
                        uint16_t* dst = a.o + static_cast<int64_t>(q.tok + tok) * a.ld_o + static_cast<int64_t>(hq) * D + c0;
#pragma unroll
                        for (int y = 0; y < 32; y += 16) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = bf16x2(ov[y + 2 * e] * inv, ov[y + 2 * e + 1] * inv);
                            if (a.wide) {
                                store32(dst + y, w);
                            } else {
                                *reinterpret_cast<uint4*>(dst + y) = make_uint4(w[0], w[1], w[2], w[3]);
                                *reinterpret_cast<uint4*>(dst + y + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    } else if (!whole && on) {
#pragma unroll
                        for (int y = 0; y < 32; y += 8) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(ov[y + e]);
                            store32(a.part + part0 * D + c0 + y, w);
                        }
                    }
                }
                if (!whole && on && half == 0) a.part_ml[part0] = make_float2(m, lt);
                t5::fence_before();
            }
            at_bar_softmax();           // every row has read what the others left it
            if (st == 0) *odd = 0;
        }
        if (warp == 2 && lane == 0) *piece_tiles = 0;
        at_arrive_warp(bars + L::QF, lane);
    }

    __syncthreads();   // the copies' warp may be through long before another one's wait runs out
    if (*abort && tid == 0) {
        // a wait ran out: let copies already issued land (bounded) before the shared memory is released
        constexpr int FIRST = Q8 ? L::RF : L::IF, N = Q8 ? RS : NI;
        for (int i = FIRST; i < FIRST + N; ++i)
            for (uint32_t par = 0; par < 2; ++par) mbar_wait_bounded(bars + i, par, nullptr, 0, 20000000ull);
    }
    t5::fence_before();
    __syncthreads();
    if (warp == 1) {
        t5::fence_after();
        t5::dealloc(tmem, 512);
    }
}

template <int D, int T>
static cudaError_t at_launch(const gdn_kv_cache& c, AttCacheArgs& a, cudaStream_t st) {
    using L = AtSmem<D, T>;
    static PerDeviceOnce once;
    if (once.run([](int) {
            cudaFuncSetAttribute(attn_tree_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::DYN);
        }) < 0)
        return cudaErrorInvalidDevice;
    CUtensorMap mk, mv;
    a.box = c.page_tokens < L::BN ? c.page_tokens : L::BN;
    // starting and ending a piece count as 12 blocks: 20 trees over up to 6000 keys, bf16 heads of 256, take 185 us with
    // 4, 153 with 8, 135 with 12 and 141 with 16; six over up to 24000 keys 153, 148, 143 and 145
    a.start = 12;
    if (!ac_map(&mk, c.k, c, a.box, 1) || !ac_map(&mv, c.v, c, a.box, 1)) return cudaErrorInvalidValue;
    a.ranks = (a.max_q * a.ratio + AT_ROWS - 1) / AT_ROWS;
    a.runs = AC_MAX_RUNS / a.ranks;
    a.wide = ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.o) | static_cast<uintptr_t>(2 * (a.ld_q | a.ld_o))) & 31) == 0;
    return launch_dependent(attn_tree_kernel<D, T>, dim3(static_cast<unsigned>(a.runs * a.ranks)), dim3(L::THREADS), L::DYN, st,
                            mk, mv, a);
}

template <int D>
static cudaError_t at_launch_t(const gdn_kv_cache& c, AttCacheArgs& a, cudaStream_t st) {
    if (c.dtype == GDN_KV_BF16) return at_launch<D, GDN_KV_BF16>(c, a, st);
    if (c.dtype == GDN_KV_I8) return at_launch<D, GDN_KV_I8>(c, a, st);
    return at_launch<D, GDN_KV_E4M3>(c, a, st);
}

// Fills in a.box, a.start, a.ranks and a.runs; the partials have AT_ROWS rows.
cudaError_t launch_attn_tree(const gdn_kv_cache& c, AttCacheArgs& a, cudaStream_t st) {
    if (c.head_dim == 64) return at_launch_t<64>(c, a, st);
    if (c.head_dim == 128) return at_launch_t<128>(c, a, st);
    return at_launch_t<256>(c, a, st);
}

int* attn_tree_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_attn_cache_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

int* attn_tree_skipped_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_attn_cache_skipped) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdn
