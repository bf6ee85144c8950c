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
// Per tile of 64 keys (row r = TMEM lane r):
//   S = Q K^T      M = 128, N = 64, K = D; Q in TMEM (from shared memory its
//                  reads alone would take three times the product), K shared;
//                  two S buffers
//   softmax        a thread per row; two groups of four warps take the tiles in
//                  turn, so that one's exponentials run beside the other's
//                  waits; P goes over its own S
//   O += P V       M = 128, N = D, K = 64; P from TMEM, V [key][d] as the
//                  MN-major operand, the image that the copy writes: no transpose
// The running maximum is raised only past a margin; the groups hand it on: a
// warp waits for the decision of the tile before (not for its exponentials)
// before it takes its own.
// The pages are bf16: TMA writes the operand images (128-byte swizzle).  8-bit
// codes go through a ring of raw tiles that four warps turn into fp16 images
// (exact); the row scales stay out of the products, as in the other kernel: a
// key's multiplies its scores, a value's goes into the exponent of p'.  fp16
// probabilities are p' 2^11, exact to 2^-11 down to 2^-25 of the largest and
// zero below 2^-36 of it.
//
// Warps: 0 copies the keys (8-bit: both), 1 allocates TMEM and issues the
// products (S of a tile two ahead of its P V), 2-5 and 6-9 softmax, 10 copies
// the values (8-bit: 10-13 convert).  Every wait is bounded; after one runs out the
// CTA stops issuing, lets copies and products finish and returns with the error
// word set.
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
    static constexpr int BN = 64;
    static constexpr int THREADS = 32 * (2 + AT_SM_WARPS + (Q8 ? 4 : 1));
    static constexpr int ROW = D * (Q8 ? 1 : 2);
    static constexpr int SLAB = ROW < 128 ? ROW : 128;      // bytes of a cached row in one slab of the copies
    static constexpr int NSLAB = ROW / SLAB;
    static constexpr int RAW = BN * ROW;                    // a tile as cached
    static constexpr int S16 = D / 64;                      // slabs of an operand image: [rows][64 x 16 bit]
    static constexpr int TILE = BN * D * 2;                 // a K or V image
    // images of K (and of V) held at once, raw tiles in flight
    static constexpr int ST = Q8 ? 2 : D == 256 ? 3 : 6;
    static constexpr int RS = !Q8 ? 1 : D == 256 ? 4 : 8;
    static constexpr int K0 = 0;
    static constexpr int V0 = K0 + ST * TILE;
    static constexpr int R0 = V0 + ST * TILE;
    static constexpr int F0 = R0 + (Q8 ? RS * RAW : 0);     // key factors and log2 value scales: [softmax warp][2][BN]
    static constexpr int X0 = F0 + (Q8 ? AT_SM_WARPS * 2 * BN * 4 : 0);   // maximum of each row; masks of zero weights [2][128]
    static constexpr int L0 = X0 + 2 * AT_ROWS * 8;         // row sums of each group
    static constexpr int E0 = L0 + 2 * AT_ROWS * 4;         // 16 columns on their way out: [softmax warp][32 rows][17]
    static constexpr int P0 = E0 + AT_SM_WARPS * 32 * 17 * 4;         // blocks before each sequence
    static constexpr int T0 = P0 + (GDN_MAX_SEQS + 2) * 8;  // the sequences
    static constexpr int W0 = T0 + GDN_MAX_SEQS * 12;
    static constexpr int B0 = W0 + 16 * 8;                  // mbarriers
    // Q in; P by buffer; decisions by group and 32 rows; per image slot: K and V full, S and P V done (which also
    // empties the slot); raw tiles, full and empty
    static constexpr int QF = 0, PF = 1, FIN = 3, DR = 4, KF = 12, VF = KF + ST, SF = VF + ST, PV = SF + ST, RF = PV + ST,
                         RE = RF + RS, NBAR = RE + RS;
    static constexpr int MISC = B0 + 8 * NBAR;              // TMEM base, abort flag, keys with values that are not finite, tiles of the piece
    static constexpr int BYTES = MISC + 32;
    // at least 120 KB, so that one CTA holds an SM (it allocates all TMEM columns)
    static constexpr int DYN = BYTES + 1024 > 120 * 1024 ? BYTES + 1024 : 120 * 1024;
    static_assert(DYN <= 227 * 1024, "shared memory of a CTA");
    // TMEM columns: two buffers of S (BN columns) with P over their first BN / 2, Q, O
    static constexpr uint32_t QCOL = 2 * BN, OCOL = 2 * BN + D / 2;
    static_assert(OCOL + D <= 512, "TMEM columns");
};

// Waits for a phase, asleep for up to 20 us at a time: warps that poll take
// issue slots and shared-memory cycles from the one that issues the products.
// Gives up after 2 s with the error word set, and at once after any wait of the
// CTA has.
__device__ __forceinline__ bool at_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
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
        if (globaltimer_ns() - t0 > 2000000000ull) {
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
// All softmax threads.
__device__ __forceinline__ void at_bar_softmax() { asm volatile("bar.sync 1, %0;" ::"n"(AT_SM_THREADS) : "memory"); }

template <int D, int T>
__global__ void __launch_bounds__(AtSmem<D, T>::THREADS, 1)
attn_tree_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                 const __grid_constant__ AttCacheArgs a) {
    using L = AtSmem<D, T>;
    constexpr int BN = L::BN, ST = L::ST, RS = L::RS;
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
            if (i == L::QF) n = AT_SM_WARPS;
            if (i == L::PF || i == L::PF + 1) n = AT_SM_WARPS / 2;
            if (Q8 && ((i >= L::KF && i < L::SF) || i >= L::RE)) n = 4;   // the converting warps
            mbar_init_cta(bars + i, n);
        }
        mbar_init_fence();
        *abort = 0;
        *odd = 0;
    }
    if (warp == 1) t5::alloc(tslot, 512);
    pdl_wait();
    pdl_trigger();
    t5::fence_before();
    ac_prefix(a, pre, seq, reinterpret_cast<int64_t*>(base + L::W0), blockIdx.x == 0);   // ends with a barrier
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

    if (warp == 0 || (!Q8 && warp == 10)) {
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
                if constexpr (Q8) {
                    // raw tiles: keys, then values
                    for (int v = 0; ok && v < 2; ++v) {
                        const uint32_t m = 2 * n + v, sl = m % RS;
                        if (m >= RS) ok = __all_sync(0xffffffffu, at_wait(bars + L::RE + sl, (m / RS - 1) & 1, abort));
                        if (ok) load(v ? &mv : &mk, bars + L::RF + sl, L::R0 + sl * L::RAW, L::RAW, j, page);
                    }
                } else {
                    const bool v = warp == 10;
                    const uint32_t sl = n % ST;
                    if (n >= ST) ok = __all_sync(0xffffffffu, at_wait(bars + (v ? L::PV : L::SF) + sl, (n / ST - 1) & 1, abort));
                    if (ok) load(v ? &mv : &mk, bars + (v ? L::VF : L::KF) + sl, (v ? L::V0 : L::K0) + sl * L::TILE, L::TILE, j, page);
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
                    const uint32_t m = 2 * n + v, sl = m % RS;
                    ok = at_wait(bars + L::RF + sl, (m / RS) & 1, abort);
                    if (ok && n >= ST) ok = at_wait(bars + (v ? L::PV : L::SF) + n % ST, (n / ST - 1) & 1, abort);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const unsigned char* src = base + L::R0 + sl * L::RAW;
                    unsigned char* dst = base + (v ? L::V0 : L::K0) + (n % ST) * L::TILE;
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
                    at_arrive_warp(bars + (v ? L::VF : L::KF) + n % ST, lane);
                    at_arrive_warp(bars + L::RE + sl, lane);
                }
                ++n;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // S of a tile needs its K image and its buffer (P V two tiles before has
        // read P there); P V needs P and the V image.  The warp polls both and one
        // lane issues what is ready; a stall past 2 s sets the error word.  All
        // lanes run the loop, on values that are uniform to the compiler (votes and
        // reductions): a single thread's loop took longer to issue the products
        // than they run.
        constexpr uint32_t FULL = 0xffffffffu;
        constexpr uint32_t IDS = Q8 ? t5::idesc_f16(AT_ROWS, BN) : t5::idesc_bf16(AT_ROWS, BN);
        constexpr uint32_t IDO = (Q8 ? t5::idesc_f16(AT_ROWS, D) : t5::idesc_bf16(AT_ROWS, D)) | (1u << 16);   // B MN-major
        const uint32_t one = lane == 0, tm = __reduce_max_sync(FULL, tmem);
        const uint64_t kd0 = t5::desc_sw128(sbase + L::K0), vd0 = t5::desc_sw128_mn(sbase + L::V0, BN * 128);
        bool ok = true;
        uint32_t piece = 0;
        uint32_t si = 0, sslot = 0, sphase = 0;    // tile, image slot and its phase of the next S
        uint32_t bslot = 0, bphase = 0;            // slot and phase of P V two tiles before it
        uint32_t pi = 0, pslot = 0, pphase = 0;    // of the next P V
        while (true) {
            // the softmax says how many tiles the piece has (0: no more pieces)
            ok = __all_sync(FULL, at_wait(bars + L::QF, piece & 1, abort));
            const int tiles = static_cast<int>(__reduce_max_sync(FULL, static_cast<uint32_t>(*piece_tiles)));
            if (!ok || tiles == 0) break;
            ++piece;
            int ns = 0, np = 0, spins = 0;
            uint64_t t_last = 0;
            while (ok && np < tiles) {
                // all four tests under one latency; what is ready of both is issued without another look
                const bool k = at_ready(bars + L::KF + sslot, sphase), b = at_ready(bars + L::PV + bslot, bphase);
                const bool p = at_ready(bars + L::PF + (pi & 1), (pi >> 1) & 1), v = at_ready(bars + L::VF + pslot, pphase);
                const bool s_on = __all_sync(FULL, ns < tiles && ns < np + 2 && k && (ns < 2 || b));
                const bool p_on = __all_sync(FULL, np < ns && p && v);
                if (s_on) {
                    t5::fence_after();
                    const uint64_t kd = kd0 + sslot * (L::TILE / 16);
                    const uint32_t to = tm + (si & 1) * BN;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        t5::mma_f16_ts_on(one, to, tm + L::QCOL + kk * 8, kd + ((kk >> 2) * (BN * 128) + (kk & 3) * 32) / 16, IDS,
                                          kk > 0 ? 1u : 0u);
                    t5::commit_on(one, bars + L::SF + sslot);
                    ++ns;
                    if (++sslot == ST) {
                        sslot = 0;
                        sphase ^= 1;
                    }
                    if (++si > 2 && ++bslot == ST) {
                        bslot = 0;
                        bphase ^= 1;
                    }
                }
                if (p_on) {
                    t5::fence_after();
                    const uint64_t vd = vd0 + pslot * (L::TILE / 16);
                    const uint32_t from = tm + (pi & 1) * BN;
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        t5::mma_f16_ts_on(one, tm + L::OCOL, from + kk * 8, vd + kk * (2048 / 16), IDO, (np > 0 || kk > 0) ? 1u : 0u);
                    t5::commit_on(one, bars + L::PV + pslot);
                    ++np;
                    ++pi;
                    if (++pslot == ST) {
                        pslot = 0;
                        pphase ^= 1;
                    }
                }
                if (s_on || p_on) {
                    spins = 0;
                } else if (++spins >= 1024) {
                    const uint64_t now = globaltimer_ns();
                    if (spins == 1024) t_last = now;
                    if (__any_sync(FULL, *abort || now - t_last > 2000000000ull)) {
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
        // group `half` takes the tiles of its parity (and half of the columns of q and o)
        const int quad = warp & 3, half = (warp - 2) >> 2, r = 32 * quad + lane, st = (tid - 64) & 127;
        const uint32_t trow = tmem + (static_cast<uint32_t>(32 * quad) << 16);
        float* row_max = reinterpret_cast<float*>(base + L::X0);
        float* lsum = reinterpret_cast<float*>(base + L::L0);
        float* kfac = reinterpret_cast<float*>(base + L::F0) + (warp - 2) * 2 * BN;   // this warp's: BN key factors, BN log2 value scales
        float* vlog = kfac + BN;
        constexpr int CH = BN / 32;                       // 32 scores at a time
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
                const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(q.tok + (on ? tok : 0)) * a.ld_q +
                                                                  (on ? hq : 0) * D + half * (D / 2));
                float up = 1.0f;
                if constexpr (Q8) {
                    float amax = 0.0f;
#pragma unroll 8
                    for (int c = 0; c < D / 16; ++c) {
                        const uint4 w = on ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u))));
                    }
                    lsum[half * AT_ROWS + r] = amax;
                    at_bar_softmax();
                    amax = fmaxf(amax, lsum[(half ^ 1) * AT_ROWS + r]);
                    const int ex = min(max(static_cast<int>((__float_as_uint(amax) >> 23) & 255) - 127, -100), 100);
                    up = __uint_as_float(static_cast<uint32_t>(127 + 14 - ex) << 23);
                    factor *= __uint_as_float(static_cast<uint32_t>(127 - 14 + ex) << 23);
                }
#pragma unroll
                for (int c = 0; c < D / 16; c += 4) {
                    uint32_t u[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 w = on ? src[c + e] : make_uint4(0u, 0u, 0u, 0u);
                        u[4 * e] = w.x;
                        u[4 * e + 1] = w.y;
                        u[4 * e + 2] = w.z;
                        u[4 * e + 3] = w.w;
                    }
                    if constexpr (Q8) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            u[e] = f16x2_bits(__uint_as_float(u[e] << 16) * up, __uint_as_float(u[e] & 0xffff0000u) * up);
                    }
                    t5::st16u(trow + L::QCOL + half * (D / 4) + 4 * c, u);
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
                if (!all_in && warp == 2 && lane == 0) atomicCAS(&g_attn_cache_error, 0, static_cast<int>(ERR_INDEX));
            }
            auto page_at = [&](int key) { return table[min(key >> a.page_shift, a.max_blocks - 1)]; };

            // ---- 8-bit: the scales of the tile's keys (by lane), read one of this group's tiles ahead, their pages two
            constexpr int KL = BN / 32;     // keys per lane
            float ksn[KL], vsn[KL];
            int pgn[KL];
            auto key_of = [&](int j, int x) { return (t0 + min(j, nb - 1)) * BN + 32 * x + lane; };
            auto scales_of = [&](int j) {
#pragma unroll
                for (int x = 0; x < KL; ++x) {
                    const int pg = pgn[x] >= 0 && pgn[x] < a.n_pages ? pgn[x] : 0;
                    const int64_t row = (static_cast<int64_t>(pg) * a.heads + pc.head) * a.page + (key_of(j, x) & (a.page - 1));
                    ksn[x] = a.sk[row];
                    vsn[x] = a.sv[row];
                    pgn[x] = page_at(key_of(j + 2, x));
                }
            };
            const int j0 = (n & 1) == static_cast<uint32_t>(half) ? 0 : 1;    // this group's first tile
            if constexpr (Q8) {
#pragma unroll
                for (int x = 0; x < KL; ++x) pgn[x] = page_at(key_of(j0, x));
                scales_of(j0);
            }

            float m = -INFINITY, l = 0.0f;
            uint64_t none = 0;      // new keys this row sees with probability zero
            // A tile; EDGE: some row may not see some key.  Two copies of the code, since
            // the tests inside its loops would cost the plain tiles five times their exponentials.
            auto tile = [&](int j, auto edge_tag) {
                constexpr bool edge = decltype(edge_tag)::value;
                constexpr int KEEP = edge || Q8 ? 1 : CH;   // scores in registers (fewer: the others are read twice)
                const uint32_t i = n + j;
                const int key0 = (t0 + j) * BN;
                const uint32_t sbuf = trow + (i & 1) * BN;
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
                        kfac[32 * x + lane] = ksn[x];
                        vlog[32 * x + lane] = lg2(fmaxf_nan(vsn[x], 7.7e-34f));
                    }
                    __syncwarp();
                    scales_of(j + 2);
                }

                ok = __all_sync(0xffffffffu, ok && at_wait(bars + L::SF + i % ST, (i / ST) & 1, abort));
                // 32 scores: raw for a bf16 cache (their factor is positive), else y = x + log2 of the value's scale
                float xs[KEEP][32];
                auto scores = [&](int ch, float (&x)[32]) {
                    t5::ld32(sbuf + 32 * ch, x);
                    if constexpr (Q8) {
                        const F2 f = f2(factor, factor);
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 k4 = *reinterpret_cast<const float4*>(kfac + 32 * ch + c);
                            const float4 v4 = *reinterpret_cast<const float4*>(vlog + 32 * ch + c);
                            f2_split(f2_fma(f2(x[c], x[c + 1]), f2_mul(f, f2(k4.x, k4.y)), f2(v4.x, v4.y)), x[c], x[c + 1]);
                            f2_split(f2_fma(f2(x[c + 2], x[c + 3]), f2_mul(f, f2(k4.z, k4.w)), f2(v4.z, v4.w)), x[c + 2], x[c + 3]);
                        }
                    }
                    if constexpr (edge) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const int key = 32 * ch + c, d = key0 + key - ctx;
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
                        scores(ch, x);
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
                // ---- the maximum after the tile before (the other group's), then this tile's
                if (j > 0) {
                    ok = __all_sync(0xffffffffu, ok && at_wait(bars + L::DR + 4 * (half ^ 1) + quad, ((i - 1) >> 1) & 1, abort));
                    const float mo = row_max[r];
                    if (__any_sync(0xffffffffu, mo != m)) {
                        l *= m == -INFINITY ? 0.0f : ex2_ftz(m - mo);
                        m = mo;
                    }
                    if (ok && __any_sync(0xffffffffu, bm > m + AC_MARGIN)) {
                        // O is rescaled once P V of tile i - 1 has finished
                        ok = __all_sync(0xffffffffu, at_wait(bars + L::PV + (i - 1) % ST, ((i - 1) / ST) & 1, abort));
                        if (ok) {
                            const float mn = fmaxf(m, bm), f = m == -INFINITY ? 0.0f : ex2_ftz(m - mn);
                            m = mn;
                            l *= f;
                            row_max[r] = m;
                            t5::fence_after();
#pragma unroll 1
                            for (int c0 = 0; c0 < D; c0 += 32) {
                                float ov[32];
                                t5::ld32(trow + L::OCOL + c0, ov);
#pragma unroll
                                for (int e = 0; e < 32; ++e) ov[e] *= f;
                                t5::st32(trow + L::OCOL + c0, ov);
                            }
                        }
                    }
                } else {
                    m = bm;
                    row_max[r] = m;
                }
                at_arrive_warp(bars + L::DR + 4 * half + quad, lane);
                if (ok) {
                    const float mm = m == -INFINITY ? 0.0f : Q8 ? m - AC_LIFT : m;
                    const F2 nm = f2(-mm, -mm), ff = f2(factor, factor);
                    F2 l2 = f2(0.0f, 0.0f);
#pragma unroll
                    for (int ch = 0; ch < CH; ++ch) {
                        float(&x)[32] = xs[KEEP == CH ? ch : 0];
                        if (KEEP < CH) scores(ch, x);
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            float y0, y1;
                            f2_split(Q8 ? f2_add(f2(x[c], x[c + 1]), nm) : f2_fma(f2(x[c], x[c + 1]), ff, nm), y0, y1);
                            const float p0 = ex2_ftz(y0), p1 = ex2_ftz(y1);
                            if constexpr (Q8) {
                                const float2 lv = *reinterpret_cast<const float2*>(vlog + 32 * ch + c);
                                float e0, e1;
                                f2_split(f2_sub(f2(y0, y1), f2(lv.x, lv.y)), e0, e1);
                                e0 = ex2_ftz(e0);
                                e1 = ex2_ftz(e1);
                                if constexpr (edge) {     // a scale that is no number reaches only the rows that see its key
                                    if (y0 == -INFINITY) e0 = 0.0f;
                                    if (y1 == -INFINITY) e1 = 0.0f;
                                }
                                l2 = f2_add(l2, f2(e0, e1));
                                pk[c / 2] = f16x2_bits(p0, p1);
                            } else {
                                l2 = f2_add(l2, f2(p0, p1));
                                const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
                                pk[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            if constexpr (edge) {
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int d = key0 + 32 * ch + c + e - ctx;
                                    if (d >= 0 && d < 64 && (e ? p1 : p0) == 0.0f) none |= 1ull << d;
                                }
                            }
                        }
                        t5::st16u(sbuf + 16 * ch, pk);   // over scores that have been read
                    }
                    float s0, s1;
                    f2_split(l2, s0, s1);
                    l += s0 + s1;
                    if constexpr (edge) {
                        // values of keys that do not exist become zero, and so do those of
                        // new keys that are not finite: the rows that see them add them at the end
                        ok = __all_sync(0xffffffffu, at_wait(bars + L::VF + i % ST, (i / ST) & 1, abort));
                        unsigned char* vt = base + L::V0 + (i % ST) * L::TILE;
                        if (ok)
#pragma unroll 1
                            for (int e = st; e < BN * (D / 8); e += AT_SM_THREADS / 2) {
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
            for (int j = j0; j < nb; j += 2) {
                if ((t0 + j + 1) * BN > ctx || !all_in)
                    tile(j, std::true_type{});
                else
                    tile(j, std::false_type{});
            }
            n += nb;

            // ---- the piece's rows out
            const uint32_t i1 = n - 1;
            // the last S first: the phase of P V before the last one, of the same barrier, is then over
            ok = __all_sync(0xffffffffu, ok && at_wait(bars + L::SF + i1 % ST, (i1 / ST) & 1, abort) &&
                                             at_wait(bars + L::PV + i1 % ST, (i1 / ST) & 1, abort));
            // the last decision, for the group that did not take it
            at_bar_softmax();
            const float mo = row_max[r];
            l *= m == -INFINITY ? 0.0f : ex2_ftz(m - mo);
            m = mo;
            lsum[half * AT_ROWS + r] = l;
            at_bar_softmax();
            uint64_t* none_of = reinterpret_cast<uint64_t*>(row_max);   // the maxima have been read
            none_of[half * AT_ROWS + r] = none;
            at_bar_softmax();
            const uint64_t odd_keys = *odd & seen;
            none |= none_of[(half ^ 1) * AT_ROWS + r];
            const float lt = lsum[r] + lsum[AT_ROWS + r];
            if (ok) {
                t5::fence_after();
                // Half of the columns, 16 at a time, through this warp's piece of shared
                // memory: a thread holds a row, and memory wants whole sectors of one.
                const bool whole = pc.b0 == 0 && pc.b1 == pc.blocks;
                const float inv = !whole ? 1.0f : lt == 0.0f ? 0.0f : 1.0f / lt;
                float* stage = reinterpret_cast<float*>(base + L::E0) + (warp - 2) * (32 * 17);
                const int64_t part0 = (static_cast<int64_t>(blockIdx.x) * 2 + (pc.b0 > 0 ? 0 : 1)) * AT_ROWS + 32 * quad;
#pragma unroll 1
                for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 16) {
                    float ov[16];
                    t5::ld16(trow + L::OCOL + c0, ov);
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
                            for (int e = 0; e < 16; ++e) {
                                float v;
                                if constexpr (Q8)
                                    v = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(a.v)[vr + e], __NV_E4M3)));
                                else
                                    v = bf16_bits_to_float(static_cast<const uint16_t*>(a.v)[vr + e]);
                                if (!(fabsf(v) < INFINITY)) ov[e] += ((none >> d) & 1 ? 0.0f : 1.0f) * v;
                            }
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 16; ++e) stage[lane * 17 + e] = ov[e] * inv;
                    __syncwarp();
                    if (whole) {
                        // four rows of 32 bytes at a time
#pragma unroll
                        for (int y = 0; y < 32; y += 4) {
                            const int rl = y + (lane >> 3), c = 2 * (lane & 7), orow = row0 + 32 * quad + rl, ot = orow / a.ratio;
                            if (32 * quad + rl < rows &&
                                GDN_IN_RANGE(g_attn_cache_error, q.tok + ot < a.n_tokens && pc.head * a.ratio + orow - ot * a.ratio < a.hq)) {
                                const __nv_bfloat162 b2 = __floats2bfloat162_rn(stage[rl * 17 + c], stage[rl * 17 + c + 1]);
                                *reinterpret_cast<uint32_t*>(a.o + (q.tok + ot) * a.ld_o + (pc.head * a.ratio + orow - ot * a.ratio) * D + c0 + c) =
                                    *reinterpret_cast<const uint32_t*>(&b2);
                            }
                        }
                    } else {
                        // two rows of 64 bytes at a time
#pragma unroll
                        for (int y = 0; y < 32; y += 2) {
                            const int rl = y + (lane >> 4), c = lane & 15;
                            if (32 * quad + rl < rows) a.part[(part0 + rl) * D + c0 + c] = stage[rl * 17 + c];
                        }
                    }
                }
                if (!whole && on && half == 0) a.part_ml[part0 + lane] = make_float2(m, lt);
                t5::fence_before();
            }
            at_bar_softmax();           // every row has read what the others left it
            if (st == 0) *odd = 0;
        }
        if (warp == 2 && lane == 0) *piece_tiles = 0;
        at_arrive_warp(bars + L::QF, lane);
    }

    if (*abort && tid == 0) {
        // a wait ran out: let copies already issued land (bounded) before the shared memory is released
        for (int i = L::KF; i < L::NBAR; ++i)
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
    a.start = 4;   // starting and ending a piece take about as long as four blocks
    if (!ac_map(&mk, c.k, c, a.box, 1) || !ac_map(&mv, c.v, c, a.box, 1)) return cudaErrorInvalidValue;
    a.ranks = (a.max_q * a.ratio + AT_ROWS - 1) / AT_ROWS;
    a.runs = AC_MAX_RUNS / a.ranks;
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

int read_and_clear_attn_tree_error() {
    int v = 0, z = 0;
    cudaMemcpyFromSymbol(&v, g_attn_cache_error, sizeof(int));
    if (v) cudaMemcpyToSymbol(g_attn_cache_error, &z, sizeof(int));
    return v;
}

}  // namespace gdn
