// Attention, forward: O = softmax(scale Q K^T) V over the key rows of each query
// row's sequence that a mode lets it see, one pass with a running maximum and sum.
//   kAll    cross attention: all of them
//   kBand   a window of positions around the row's own (cross.cuh)
//   kPaged  the same over a cache in pages, whose lengths the device holds
//
// A CTA takes a tile of 128 query rows of one key/value head and walks over
// key tiles of 64 (or 128): S = Q K^T and O += P V on the tensor cores
// (tcgen05), S, P and O in TMEM, P over its S as the TMEM operand of the second
// product, so that scores and probabilities never touch shared memory.  Two
// score tiles of 64 keys are in flight: while the softmax (four warps, a thread
// a row, no shuffles) works on one, the MMA warp multiplies the other's P and
// forms the scores after it.  Two CTAs (64-wide heads: four) share an SM, so one's
// start and end run beside the other's loop as well.  A CTA of two query tiles
// that read the keys together was slower at every size: its softmax warps all
// wait for one MMA warp (131072 keys: 242 us against 199; 8192 x 4096: 722, 682).
//
// Measured on one GB300: 2 x 8192 x 4096 tokens, 32 heads of 128 (bf16) 682 to 734
// us, 1500 to 1610 TFLOP/s, the tensor pipe 65 % active; what bounds it is the chain from
// scores to scores of a CTA (softmax 1500 cycles, its products 1024, hand-offs),
// of which two run at a time.  One token of 64 sequences against 2048 to 4096
// states: 68 us, 5.9 TB/s of 6.7.  64-wide heads: 510 us for 2 x 8192 x 4096
// tokens, issue slots 57 % used, the tensor pipe 41 %.
//
// The running maximum is lazy: O and the sum are rescaled only when a row's
// maximum grows by more than 2^8 over the reference in use, which any reference
// allows (O / sum does not depend on it); P then stays <= 2^8, far from the
// 16-bit types' limits.  P is rounded to 16 bits as an operand; the sum is
// taken of the unrounded fp32 values.
//
// Few query rows and many keys: the key tiles of a unit are split over the
// CTAs of a cluster, whose partial O, maximum and sum are joined through
// distributed shared memory in rank order: one launch, no workspace.  Windowed and
// paged ones with room for more than two such clusters a unit: up to 152 pieces
// of a unit, whose fp32 O, maximum and sum go to the workspace, and a second
// launch (k_xjoin) that adds them in their order.  Either way the same bits on
// every run.
#pragma once

#include <type_traits>

#include "cross.cuh"
#include "kernels.cuh"
#include "xtmap.cuh"

namespace sag {

namespace {

constexpr int kFwdThreads = 192, kFwdTma = 4, kFwdMma = 5;   // warps 0-3 softmax and epilogue, then TMA and MMA

// kKeys: keys of a tile, BUFS: score tiles in flight, CTAS: of an SM.  TMEM columns: S of tile i from (i % BUFS) * kKeys,
// P over it from column P_AT of it on, O from COL_O.  64-wide heads spend most of their time in the softmax, whose
// latencies more warps hide: four CTAs with one score tile each (128 columns) instead of two with two.  They have 80
// registers a thread, so a tile's scores are taken in halves, the first one twice.
template <int D, int kKeys>
struct FwdShape {
    static constexpr bool NARROW = D == 64;
    static constexpr int CTAS = NARROW ? 4 : 2;
    static constexpr int BUFS = NARROW ? 1 : 128 / kKeys, HALVES = kKeys / 64;
    static constexpr int P_AT = NARROW ? 32 : 0;
    static constexpr int COL_O = BUFS * kKeys, TMEM = 512 / CTAS;
    static constexpr bool MASK_AHEAD = kKeys == 64 && !NARROW;   // elsewhere registers are wanting
    static constexpr int KC = D / 64;
    static constexpr int Q_BYTES = KC * 16384;
    static constexpr int TILE = KC * kKeys * 128;
    static constexpr int STAGES = NARROW ? 4 : 81920 / TILE;      // K and V tiles
    static constexpr int OFF_RING = Q_BYTES;
    static constexpr int OFF_BAR = OFF_RING + STAGES * TILE;
    static constexpr int TOTAL = OFF_BAR + 256;
    // split units, over Q and the ring: float [128][XROW] of O (padded against bank conflicts), float2 [128]
    static constexpr int XROW = D + 4;
    static constexpr int OFF_ML = kXRows * XROW * 4;
    static_assert(OFF_ML + kXRows * 8 <= OFF_BAR, "the exchange overlays Q and the ring");
    static_assert(CTAS * (TOTAL + 1024) <= 228 * 1024, "shared memory of an SM");
};
// XF_S: scores of an even / odd tile formed, and P V of the tile two before complete; XF_P: P written.  Where CTAs take unit
// after unit, also XF_QE: Q has been read, and XF_O: the unit's last P V complete.  It is no phase of XF_S there: the next
// unit's scores may complete before a softmax warp looks, which would wait for a phase that is two behind (modelled in the tests).
enum { XF_Q = 0, XF_S = 1, XF_P = 3, XF_DRAIN = 5, XF_QE = 6, XF_O = 7, XF_FULL = 8 };

// Whether CTAs take unit after unit: with short loops, which 128-key tiles are not for, and registers for it (64-wide heads,
// four CTAs an SM, have none to spare: a window of 512 over 32768 tokens 497 us so, 399 with a unit a CTA).
__host__ __device__ constexpr bool x_walks(int mode, int d, int keys) { return mode != kAll && d == 128 && keys == 64; }

// What a CTA does for a query tile and key/value head.
struct XJob {
    XUnit u;
    BandKeys band;
    int tok0, cover;                    // first token, tokens that the outputs have
    int t0, n;                          // first tile of this CTA's share of the keys, and their number
    int whole, partial;                 // tiles of the share from `whole` on, before `partial`, lack no key
};
// The keys of a unit whose sequence, head and tile are known.
template <int kKeys, int kMode>
__device__ __forceinline__ void x_keys(const XArgs &A, int rank, int ways, XJob &w) {
    w.tok0 = w.u.tile * A.tpt;
    w.cover = A.s1_pad ? A.s1_pad : w.u.seq.qlen;
    if constexpr (kMode != kAll) w.band = BandKeys::of<kKeys, kMode == kPaged>(A, w.u.seq, w.tok0);
    else w.band = BandKeys{};
    const int nkt = kMode != kAll ? w.band.tiles : w.tok0 < w.u.seq.qlen ? (w.u.seq.klen + kKeys - 1) / kKeys : 0;
    x_share(nkt, rank, ways, &w.t0, &w.n);
    w.whole = kMode == kAll ? 0 : w.band.f0 - w.t0;
    w.partial = A.mask ? 0 : (kMode == kAll ? w.u.seq.klen / kKeys : w.band.f1) - w.t0;
}
template <int kKeys, int kMode>
__device__ __forceinline__ XJob x_job(const XArgs &A, int unit, int rank, int ways) {
    XJob w;
    w.u = x_decode<&SeqRow::qtile0, kMode == kAll ? kByHead : kDown>(A, unit);
    if (kMode == kPaged) w.u.seq.klen = min(max(__ldg(A.klens + w.u.b), 0), A.width * A.page);
    x_keys<kKeys, kMode>(A, rank, ways, w);
    return w;
}

// The next unit of a CTA that walks, as many tiles and heads on as the grid has CTAs: without divisions or loads, unless it
// is another sequence's.
struct XStep {
    int tiles, heads;
    __device__ __forceinline__ explicit XStep(const XArgs &A) : tiles(gridDim.x / A.n2), heads(gridDim.x - tiles * A.n2) {}
};
template <int kKeys, int kMode>
__device__ __forceinline__ XJob x_job_after(const XArgs &A, XJob w, const XStep &step, int unit, int rank, int ways) {
    int head = w.u.head + step.heads, tile = w.u.tile - step.tiles;
    if (head >= A.n2) {
        head -= A.n2;
        --tile;
    }
    if (tile < 0) return x_job<kKeys, kMode>(A, unit, rank, ways);
    w.u.head = head;
    w.u.tile = tile;
    x_keys<kKeys, kMode>(A, rank, ways, w);
    return w;
}

// Pages of a loop's tiles, for the lane whose load takes `shift` keys from a tile's first one on.  Lane l holds the table's
// entries `base` + l, and those 32 on, which are on their way since the last refill.
struct PageWalk {
    const int32_t *table;
    int base, cur, nxt;                 // the first entry at hand is the tile's first page
    int first, first_row;               // the tile's first page and row in it
    int page, row;                      // of this lane
    int by_page, by_row;
    __device__ __forceinline__ int load(const XArgs &A, int p) const { return p < A.width ? __ldg(table + p) : -1; }
    __device__ __forceinline__ static void on(const XArgs &A, int pages, int rows, int *page, int *row) {
        *page += pages;
        *row += rows;
        if (*row >= A.page) {
            *row -= A.page;
            ++*page;
        }
    }
    __device__ __forceinline__ PageWalk(const XArgs &A, int b, int key, int keys, int shift, int lane)
        : table(A.table + (int64_t)b * A.width), by_page(keys / A.page), by_row(keys % A.page) {
        first = key / A.page;
        first_row = key - first * A.page;
        page = (key + shift) / A.page;
        row = key + shift - page * A.page;
        base = first;
        cur = load(A, base + lane);
        nxt = load(A, base + 32 + lane);
    }
    __device__ __forceinline__ int id(const XArgs &A, int lane) {
        const int i = page - base;
        const int c = __shfl_sync(0xffffffffu, cur, i & 31);
        if (__all_sync(0xffffffffu, i < 32)) return c;
        const int n = __shfl_sync(0xffffffffu, nxt, i & 31);
        return i < 32 ? c : n;
    }
    __device__ __forceinline__ void next(const XArgs &A, int lane) {
        on(A, by_page, by_row, &first, &first_row);
        on(A, by_page, by_row, &page, &row);
        if (first >= base + 32) {
            base += 32;
            cur = nxt;
            nxt = load(A, base + 32 + lane);
        }
    }
};

// Parities by which the barriers of NB score buffers move on over n tiles, a bit a buffer.
template <int NB>
__device__ __forceinline__ uint32_t x_parity(int n) {
    return NB == 1 ? (uint32_t)n & 1u : (uint32_t)(((n + 1) / 2) & 1) | (uint32_t)((n / 2) & 1) << 1;
}

template <bool kFp16, int D, int kKeys, int kMode>
__global__ void __launch_bounds__(kFwdThreads, FwdShape<D, kKeys>::CTAS)
    k_xfwd(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
           const __grid_constant__ CUtensorMap map_v, const __grid_constant__ XArgs A) {
    using L = FwdShape<D, kKeys>;
    constexpr int NB = L::BUFS;
    constexpr int ST = L::STAGES;
    constexpr float kShift = kFp16 ? kFwdShiftF16 : 0.f;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    uint64_t *full = bars + XF_FULL, *empty = full + ST;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(empty + ST);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *bad_index = abort_flag + 1;            // paged: a page or a length out of range
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *bad_index = 0;
        // one arrival a softmax warp, one of everything else
        for (int i = 0; i < XF_FULL + 2 * ST; ++i) tc::mbar_init(&bars[i], i == XF_P || i == XF_P + 1 ? 4 : 1);
        tc::fence_mbar_init();
    }
    if (warp == kFwdMma) {
        tc::tmem_alloc(tmem_slot, L::TMEM);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == kFwdTma * 32) {
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_k);
        tc::prefetch_tmap(&map_v);
    }
    const int ns = A.nsplit;
    const int ways = kMode == kAll ? ns : ns * A.pieces; // CTAs of the unit: a cluster's, or pieces
    const int rank = blockIdx.x % ways;
    // windowed: CTAs that share no unit take one after the other, so that the next one's loads and first scores run beside
    // the last one's end (a window of 128 over 32768 tokens, 64 heads of 128: 376 us with a unit a CTA, 342 with this; 266
    // with the next unit stepped to instead of looked up, its divisions and loads gone, and a shorter end)
    const int unit0 = blockIdx.x / ways;
    auto next_unit = [&](int unit) { return x_walks(kMode, D, kKeys) && ways == 1 ? unit + (int)gridDim.x : 1 << 30; };
    XJob w = x_job<kKeys, kMode>(A, unit0, rank, ways);
    const XStep step(A);
    if (kMode != kAll && A.pieces > 1) grid_next();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sbase = tc::smem_u32(smem);
    const int G = A.group;
    auto first_key = [&](int i) { return w.band.base + (w.t0 + i) * kKeys; };
    auto fail = [&]() { *abort_flag = 1; };

    if (warp >= kFwdTma) {
        if (warp == kFwdTma) {
            // -------------------------------------------------- TMA producer
            if constexpr (kMode == kPaged) {
                // The whole warp: a lane issues one load, of `box` rows within a page.  A tile's rows outside the window are
                // not loaded: what the buffer held is masked out of the scores, and zeroed before P V.
                bool ok = true;
                int loads = 0, nonempty = 0;
                const int per = kKeys / A.box, box = lane % per, chunk = lane / per;
                for (int unit = unit0;;) {
                    if (const int given = __ldg(A.klens + w.u.b); given != w.u.seq.klen) *bad_index = 1;
                    PageWalk walk_k(A, w.u.b, first_key(0), kKeys, box * A.box, lane), walk_v = walk_k;
                    auto stage = [&](const CUtensorMap *map, PageWalk &walk, int key) {
                        const int s = loads % ST, use = loads / ST;
                        int id = walk.id(A, lane);
                        const int k = key + box * A.box, in_page = walk.row;
                        const bool on = chunk < L::KC && k < w.band.hi && k + A.box > w.band.lo;
                        if (on && (unsigned)id >= (unsigned)A.pages) {
                            *bad_index = 1;
                            id = 0;
                        }
                        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, on)) * A.box * 128;
                        if (use > 0 && !warp_wait(abort_flag, Phase{&empty[s], (uint32_t)(use - 1) & 1u})) return false;
                        if (lane == 0) tc::mbar_arrive_expect_tx(&full[s], bytes);
                        __syncwarp();
                        if (on)
                            tc::tma_load_4d(smem + L::OFF_RING + s * L::TILE + (chunk * kKeys + box * A.box) * 128, map, chunk * 64,
                                            w.u.head, in_page, id, &full[s]);
                        walk.next(A, lane);
                        ++loads;
                        return true;
                    };
                    if (w.n > 0) {
                        if (nonempty > 0) ok = warp_wait(abort_flag, Phase{&bars[XF_QE], (uint32_t)(nonempty - 1) & 1u});
                        if (!ok) break;
                        if (lane == 0) {
                            tc::mbar_arrive_expect_tx(&bars[XF_Q], (uint32_t)L::KC * A.tpt * G * 128);
                            for (int c = 0; c < L::KC; ++c)
                                tc::tma_load_3d(smem + c * 16384, &map_q, c * 64, w.u.head * G, w.u.seq.q0 + w.tok0, &bars[XF_Q]);
                        }
                        __syncwarp();
                        ++nonempty;
                    }
                    for (int i = -NB; i < w.n && ok; ++i) {      // the order of the MMA warp, as below
                        if (i >= 0) ok = stage(&map_v, walk_v, first_key(i));
                        if (ok && i + NB < w.n) ok = stage(&map_k, walk_k, first_key(i + NB));
                    }
                    unit = next_unit(unit);
                    if (!ok || !x_walks(kMode, D, kKeys) || unit >= A.units) break;
                    w = x_job_after<kKeys, kMode>(A, w, step, unit, rank, ways);
                }
                if (!ok) fail();
                if (lane == 0) {
                    bool drained = tc::drain_armed(&bars[XF_Q], nonempty, kXWaitNs);
                    for (int s = 0; s < ST; ++s)
                        drained = tc::drain_armed(&full[s], loads > s ? (loads - s - 1) / ST + 1 : 0, kXWaitNs) && drained;
                    if (!drained) fail();
                }
            } else if (lane == 0) {
                bool ok = true;
                int loads = 0, nonempty = 0;
                auto stage = [&](const CUtensorMap *map, int key) {
                    const int s = loads % ST, use = loads / ST;
                    if (use > 0 && !tc::mbar_wait(&empty[s], (use - 1) & 1, abort_flag, kXWaitNs)) return false;
                    tc::mbar_arrive_expect_tx(&full[s], L::TILE);
                    for (int c = 0; c < L::KC; ++c)
                        tc::tma_load_3d(smem + L::OFF_RING + s * L::TILE + c * kKeys * 128, map, c * 64, w.u.head,
                                        w.u.seq.k0 + key, &full[s]);
                    ++loads;
                    return true;
                };
                for (int unit = unit0;;) {
                    if (w.n > 0) {
                        if (nonempty > 0) ok = tc::mbar_wait(&bars[XF_QE], (nonempty - 1) & 1, abort_flag, kXWaitNs);
                        if (!ok) break;
                        tc::mbar_arrive_expect_tx(&bars[XF_Q], (uint32_t)L::KC * A.tpt * G * 128);
                        for (int c = 0; c < L::KC; ++c)
                            tc::tma_load_3d(smem + c * 16384, &map_q, c * 64, w.u.head * G, w.u.seq.q0 + w.tok0, &bars[XF_Q]);
                        ++nonempty;
                    }
                    // in the order the MMA warp takes them: the first K, then V i and K i + NB
                    for (int i = -NB; i < w.n && ok; ++i) {
                        if (i >= 0) ok = stage(&map_v, first_key(i));
                        if (ok && i + NB < w.n) ok = stage(&map_k, first_key(i + NB));
                    }
                    unit = next_unit(unit);
                    if (!ok || !x_walks(kMode, D, kKeys) || unit >= A.units) break;
                    w = x_job_after<kKeys, kMode>(A, w, step, unit, rank, ways);
                }
                if (!ok) fail();
                // every load issued must have landed before the CTA exits
                bool drained = tc::drain_armed(&bars[XF_Q], nonempty, kXWaitNs);
                for (int s = 0; s < ST; ++s)
                    drained = tc::drain_armed(&full[s], loads > s ? (loads - s - 1) / ST + 1 : 0, kXWaitNs) && drained;
                if (!drained) fail();
            }
        } else if (warp == kFwdMma) {
            // -------------------------------------------------- MMA issuer
            // The tensor pipe queues about four instructions (256 cycles),
            // which hides a wait, a commit or some arithmetic between two
            // products, but not all of a tile's together: they are spread.
            constexpr uint32_t id_s = tc::idesc_f16(kXRows, kKeys, !kFp16, false, false);
            constexpr uint32_t id_o = tc::idesc_f16(kXRows, D, !kFp16, false, true);
            const uint32_t ring = sbase + L::OFF_RING;
            bool ok = true;
            int base = 0, nonempty = 0;                  // loads and units before this unit
            uint32_t written_by = 0;                     // parities of XF_P before this unit, a bit a barrier
            for (int unit = unit0;;) {
                const int n = w.n;
                // load j of the unit: the first K tiles, then V i (behind min(i + NB, n) tiles of K) and K i + NB
                auto landed = [&](int j) { return Phase{&full[(base + j) % ST], (uint32_t)((base + j) / ST) & 1u}; };
                auto issue_s = [&](int i, int j) {
                    mma_abt<D, kKeys>(tmem + i % NB * kKeys, sbase, ring + (base + j) % ST * L::TILE, id_s);
                    tc::mma_commit_warp(&bars[XF_S + i % NB]);
                    tc::mma_commit_warp(&empty[(base + j) % ST]);
                    if (x_walks(kMode, D, kKeys) && i + 1 == n) tc::mma_commit_warp(&bars[XF_QE]);
                };
                for (int i = 0; i < NB && i < n && ok; ++i) {
                    ok = warp_wait(abort_flag, Phase{&bars[XF_Q], (uint32_t)nonempty & 1u}, landed(i));
                    tc::tc_fence_after();
                    if (ok) issue_s(i, i);
                }
                for (int i = 0; i < n && ok; ++i) {
                    const bool more = i + NB < n;
                    const int jv = i + (more ? i + NB : n);
                    const uint32_t vt = ring + (base + jv) % ST * L::TILE, acc = tmem + L::COL_O, pt = tmem + i % NB * kKeys + L::P_AT;
                    // P (its first half), V, and with the last half the K tile of the scores that follow
                    auto written = [&](int h) {
                        const int b = L::HALVES == 2 ? h : i % NB;
                        return Phase{&bars[XF_P + b], ((written_by >> b) ^ (uint32_t)(i / NB)) & 1u};
                    };
                    ok = L::HALVES == 1 && more ? warp_wait(abort_flag, written(0), landed(jv), landed(jv + 1))
                                                : warp_wait(abort_flag, written(0), landed(jv));
                    if (!ok) break;
                    tc::tc_fence_after();
                    mma_ab<kKeys, 32, 0, 4>(acc, pt, vt, id_o, i > 0);
                    if (L::HALVES == 2) {
                        ok = more ? warp_wait(abort_flag, written(1), landed(jv + 1)) : warp_wait(abort_flag, written(1));
                        if (!ok) break;
                        tc::tc_fence_after();
                        mma_ab<kKeys, 32, 4, kKeys / 16>(acc, pt, vt, id_o, true);
                    }
                    tc::mma_commit_warp(&empty[(base + jv) % ST]);
                    if (more) issue_s(i + NB, jv + 1);
                    else tc::mma_commit_warp(&bars[x_walks(kMode, D, kKeys) && i + 1 == n ? XF_O : XF_S + i % NB]);
                }
                unit = next_unit(unit);
                if (!ok || !x_walks(kMode, D, kKeys) || unit >= A.units) break;
                base += 2 * n;
                nonempty += n > 0;
                if (L::HALVES == 2) written_by ^= n & 1 ? 3u : 0u;
                else written_by ^= x_parity<NB>(n);
                w = x_job_after<kKeys, kMode>(A, w, step, unit, rank, ways);
            }
            if (!ok && lane == 0) fail();
            // every MMA issued must be complete before TMEM is freed
            tc::mma_commit_warp(&bars[XF_DRAIN]);
            if (!__all_sync(0xffffffffu, tc::mbar_wait_drain(&bars[XF_DRAIN], 0, kXWaitNs)) && lane == 0) fail();
        }
        if (ns > 1) {                                    // as below
            __syncthreads();
            cluster_sync();
            cluster_sync();
        }
    } else {
        const int r = warp * 32 + lane;                  // query row = TMEM lane
        const int r_tok = r / G, r_head = r - r_tok * G;
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        const uint32_t to = trow + L::COL_O;
        float m = -INFINITY, l = 0.f;                    // reference maximum (log2 units), sum
        const float kLn2 = 0.6931471805599453f;
        int base = 0;                                    // loads before this unit
        uint32_t formed_by = 0, ended = 0;               // parities of XF_S (a bit a barrier) and of XF_O before this unit
        for (int unit = unit0;;) {
        const int n = w.n, next = next_unit(unit);
        bool ok = true;
        auto wait = [&](int b, uint32_t parity) { return warp_wait(abort_flag, Phase{&bars[b], parity}); };
        // tile i's scores (or, behind the last two tiles, just the products before) are complete
        auto formed = [&](int i) { return wait(XF_S + i % NB, ((formed_by >> (i % NB)) ^ (uint32_t)(i / NB)) & 1u); };
        if (n > 0) {
            // -------------------------------------------------- softmax
            const float c = A.scale_log2;
            // One tile; a copy of its own for tiles with absent keys, whose
            // selects otherwise run for every tile.  Paired fp32 operations
            // (f32x2): half the instructions where issue slots are short,
            // 540 -> 507 us for 8192 x 4096 tokens of 64-wide heads.
            KeyLoad<kKeys / 32> keys{};                  // of the next tile that may lack keys
            // the row's keys, from the first tile's first one on
            const int row_p = w.tok0 + r_tok + w.u.seq.klen - w.u.seq.qlen - first_key(0);
            const int row_a = row_p - A.left, row_b = row_p + A.right + 1;
            auto tile = [&](auto masked, int i) -> bool {
                const bool lacking = masked;
                const uint32_t ts = trow + i % NB * kKeys;
                KeyBits<kKeys / 32> kb{};
                if (lacking) {
                    if (kMode == kAll || A.mask) {
                        if (!L::MASK_AHEAD) keys.start(A.mask, w.u.seq, first_key(i), lane);
                        kb = keys.finish();
                        if (L::MASK_AHEAD && i + 1 < n) keys.start(A.mask, w.u.seq, first_key(i + 1), lane);
                    } else {
                        kb.set_first(kKeys);
                    }
                    // rows that are not the sequence's may hold anything; paged: rows that no window holds were not loaded
                    if constexpr (kMode == kBand) kb.clip(0, w.u.seq.klen - first_key(i));
                    if constexpr (kMode == kPaged) kb.clip(w.band.lo - first_key(i), w.band.hi - first_key(i));
                    if (!kb.all()) {
                        const int jv = i + (i + NB < n ? i + NB : n);   // V's place in the ring, as in the MMA warp
                        if (!warp_wait(abort_flag, Phase{&full[(base + jv) % ST], (uint32_t)((base + jv) / ST) & 1u})) return false;
                        zero_rows<L::KC, kKeys / 32, 128>(smem + L::OFF_RING + (base + jv) % ST * L::TILE, kb, r);
                    }
                    if constexpr (kMode != kAll) kb.clip(row_a - i * kKeys, row_b - i * kKeys);
                }
                constexpr int kHeld = L::NARROW ? 32 : kKeys;           // scores held in registers at a time
                float x[kHeld];
                // columns `from` .. from + kHeld - 1
                auto scores = [&](int from) {
#pragma unroll
                    for (int j = 0; j < kHeld; j += 32) tmem_ld32(ts + from + j, reinterpret_cast<uint32_t *>(x) + j);
                    tc::tmem_wait_ld();
                    if (lacking) {
#pragma unroll
                        for (int j = 0; j < kHeld; ++j)
                            if (!((kb.w[(from + j) >> 5] >> (j & 31)) & 1u)) x[j] = -INFINITY;
                    }
                };
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int from = 0; from < kKeys; from += kHeld) {
                    scores(from);
#pragma unroll
                    for (int j = 0; j < kHeld; j += 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(fmaxf(mx[e], x[j + e]), x[j + 4 + e]);
                    }
                }
                const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                const bool grow = mt > m + 8.f;
                if (__any_sync(0xffffffffu, grow)) {
                    const float mnew = grow ? mt : m;
                    const float f = grow ? xex2(m - mnew) : 1.f;
                    l *= f;
                    m = mnew;
                    if (i > 0) {
                        if (!formed(i - 1 + NB)) return false;   // P V of the tile before is complete
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int j = 0; j < D; j += 16) {
                            uint32_t y[16];
                            tc::tmem_ld16(to + j, y);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                            tmem_st16(to + j, y);
                        }
                    }
                }
                const float from = m == -INFINITY ? 0.f : m - kShift;
                const float2 c2 = make_float2(c, c), b2 = make_float2(-from, -from);
                float2 sum[2] = {};
                // two rounded probabilities
                auto pair = [&](int j) {
                    float2 e = fma2(make_float2(x[j], x[j + 1]), c2, b2);
                    e = make_float2(xex2(e.x), xex2(e.y));
                    sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], e);
                    return xpack<kFp16>(e.x, e.y);
                };
                // the product two tiles before is complete, whether or not that was waited for: so no wait of the next unit finds
                // its barrier a phase behind
                if (x_walks(kMode, D, kKeys) && NB == 2 && n > 1 && i + 1 == n && !formed(n)) return false;
                auto written = [&](int which) {
                    tmem_wait_st();
                    tc::tc_fence_before();
                    warp_arrive(&bars[XF_P + which], lane);
                };
                if constexpr (L::NARROW) {
                    // the second half's scores are at hand, and P lies over them
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[j] = pair(2 * j);
                    tmem_st16(ts + 48, p);
                    scores(0);
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[j] = pair(2 * j);
                    tmem_st16(ts + 32, p);
                    written(0);
                } else {
#pragma unroll
                    for (int h = 0; h < L::HALVES; ++h) {
                        uint32_t p[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) p[j] = pair(h * 64 + 2 * j);
                        tmem_st32(ts + h * 32, p);
                        written(L::HALVES == 2 ? h : i % NB);
                    }
                }
                const float2 both = add2(sum[0], sum[1]);
                l += both.x + both.y;
                return true;
            };
            if (L::MASK_AHEAD && w.partial < n && (kMode == kAll || A.mask))
                keys.start(A.mask, w.u.seq, first_key(w.partial > 0 ? w.partial : 0), lane);
            for (int i = 0; i < n && ok; ++i) {
                ok = formed(i);
                if (!ok) break;
                tc::tc_fence_after();
                // Short loops alternate between the two: with a copy of the code for each, more instructions are fetched than
                // found (a window of 128 over 32768 tokens, then: 342 us, with one copy 329).  Long ones hardly do (2 x 8192 causal
                // tokens, then: 781 us, with one copy 821).
                const bool lacking = i < w.whole || i >= w.partial;
                if constexpr (kMode != kAll && kKeys == 64) ok = tile(lacking, i);
                else ok = lacking ? tile(std::true_type{}, i) : tile(std::false_type{}, i);
            }
        }
        const int tok = w.tok0 + r_tok;
        const bool mine = r < A.tpt * G && tok < w.cover, pad = tok >= w.u.seq.qlen;
        const int64_t row = (int64_t)(w.u.seq.q0 + tok) * A.n1 + w.u.head * G + r_head;
        const bool more = x_walks(kMode, D, kKeys) && next < A.units;
        if (more) w = x_job_after<kKeys, kMode>(A, w, step, next, rank, ways);   // beside the last product
        if (n > 0) {
            if (ok) ok = x_walks(kMode, D, kKeys) ? wait(XF_O, ended) : formed(n - 1 + NB);
            ended ^= 1;
            if (!ok && lane == 0) fail();
            tc::tc_fence_after();
        }

            if (ways > 1 || !ok) break;                  // stored below
            // -------------------------------------------------- epilogue
            const bool some = l > 0.f || l != l;         // l is NaN when a score was
            const float inv = some ? 1.f / l : 0.f;
            RowStore<kFp16> rows;
            rows.rows(mine ? row * D : -1, lane);
            const uint32_t keep = n > 0 && some && !pad ? 0xffffffffu : 0u;
            // in a loop: instructions that run once a unit are fetched each time (a window of 128 over 32768 tokens: 270 us
            // unrolled, 263 so; 64 wide 404, 412; cross attention of 2 x 8192 x 4096 tokens 691, 694).  The next columns' loads
            // ahead of these spill registers (window 512: 507, 580).
#pragma unroll(L::NARROW || kMode == kAll ? 4 : 1)
            for (int j = 0; j < D; j += 32) {
                float y[32];
                if (n > 0) {
                    tmem_ld32(to + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                }
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 v = mul2(make_float2(y[2 * e], y[2 * e + 1]), make_float2(inv, inv));
                    p[e] = xpack<kFp16>(v.x, v.y) & keep;
                }
                rows.store_packed(A.o, p, j, lane);
            }
            if (mine) A.lse[row] = pad ? 0.f : some ? (m - kShift) * kLn2 + logf(l) : -INFINITY;
            if (!more) break;
            tc::tc_fence_before();                       // O has been read before the next unit's products may follow
            unit = next;
            base += 2 * n;
            formed_by ^= x_parity<NB>(n) ^ (NB == 2 && n > 1 ? 1u << (n % NB) : 0u);
            m = -INFINITY;
            l = 0.f;
        }
        const int n = w.n;
        if (kMode != kAll && A.pieces > 1) {
            // a piece's rows as they are, for k_xjoin
            if (r < A.tpt * G && w.tok0 + r / G < w.u.seq.qlen) {
                A.part_ml[(int64_t)blockIdx.x * kXRows + r] = make_float2(m, l);
            }
            if (n > 0) {
#pragma unroll 1
                for (int j = 0; j < D; j += 32) {
                    float y[32];
                    tmem_ld32(to + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                    if (r < A.tpt * G && w.tok0 + r / G < w.u.seq.qlen) {
                        float *at = A.parts + ((int64_t)blockIdx.x * kXRows + r) * D + j;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(at + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                    }
                }
            }
        } else if (ns > 1) {
            // partial O, maximum and sum of every rank into its shared memory, then each rank joins its share of the rows
            float2 *ml = reinterpret_cast<float2 *>(smem + L::OFF_ML);
            float *xo = reinterpret_cast<float *>(smem);
            __syncthreads();                             // all loads and products on this memory are complete
            ml[r] = make_float2(m, l);
            if (n > 0) {
#pragma unroll
                for (int j = 0; j < D; j += 32) {
                    float y[32];
                    tmem_ld32(to + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4 *>(xo + r * L::XROW + j + e) =
                            make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                }
            }
            cluster_sync();
            const int mine = min(A.tpt * G, (w.cover - w.tok0) * G);
            auto join = [&](auto np) {
                // A remote read takes 600 cycles, so a warp has eight (row, rank) pairs' reads in flight while it adds the
                // eight before up, and what a row needs besides is formed for all rows of a round at once, by lanes NP i + p
                // for row i and rank p.  (A row after the other, a full tile took 14000 cycles.)  A rank that saw nothing has
                // (-inf, 0) and no O.
                constexpr int NP = decltype(np)::value;  // ranks, up to a power of two
                constexpr int RG = 32 / NP, RS = 8 / NP; // rows of a round of the warp, and of eight reads
                constexpr int E = D / 64;                // float2 a lane and row
                uint32_t at[NP];
#pragma unroll
                for (int p = 0; p < NP; ++p) at[p] = peer_addr(tc::smem_u32(xo + lane * 2), p < ns ? p : 0);
                for (int first = rank + ns * warp; first < mine; first += ns * 4 * RG) {
                    auto row_of = [&](int i) { return first + i * ns * 4; };
                    float2 y[2][RS][NP][E];
                    auto read = [&](int sub) {
#pragma unroll
                        for (int a = 0; a < RS; ++a) {
                            const uint32_t off = min(row_of(sub * RS + a), mine - 1) * (L::XROW * 4);
#pragma unroll
                            for (int p = 0; p < NP; ++p)
                                if (p < ns)
#pragma unroll
                                    for (int e = 0; e < E; ++e) y[sub & 1][a][p][e] = peer_ld2(at[p] + off + e * 256);
                        }
                    };
                    const int k = row_of(lane / NP), p_lane = lane % NP, group = lane & ~(NP - 1), tok = w.tok0 + k / G;
                    const bool pad = tok >= w.u.seq.qlen;
                    float2 v = make_float2(-INFINITY, 0.f);
                    if (p_lane < ns && k < mine && !pad) v = peer_ld2(peer_addr(tc::smem_u32(ml + k), p_lane));
                    read(0);
                    // place of the row; negative: none
                    const int row = k < mine ? (w.u.seq.q0 + tok) * A.n1 + w.u.head * G + k % G : -1;
                    float top = v.x;
#pragma unroll
                    for (int o = NP / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // A rank that saw something counts even where its weight underflows: 0 times its NaN is NaN, as in an
                    // undivided loop.  (A rank of NaN scores alone has -inf and NaN.)
                    const float weight = v.y == 0.f ? -1.f : xex2(v.x - top);           // -1: saw nothing
                    float sum = 0.f;
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const float wp = __shfl_sync(0xffffffffu, weight, group + p), lp = __shfl_sync(0xffffffffu, v.y, group + p);
                        if (wp != -1.f) sum += lp * wp;
                    }
                    const bool some = sum > 0.f || sum != sum;
                    const float inv = some ? 1.f / sum : 0.f;
                    if (p_lane == 0 && row >= 0) A.lse[row] = pad ? 0.f : some ? (top - kShift) * kLn2 + logf(sum) : -INFINITY;
#pragma unroll
                    for (int sub = 0; sub < 4; ++sub) {
                        if (row_of(sub * RS) >= mine) break;             // the same for the warp
                        if (sub < 3) read(sub + 1);
#pragma unroll
                        for (int a = 0; a < RS; ++a) {
                            const int from = (sub * RS + a) * NP;
                            float2 acc[E] = {};
#pragma unroll
                            for (int p = 0; p < NP; ++p) {
                                const float wp = __shfl_sync(0xffffffffu, weight, from + p);
                                if (p >= ns || wp == -1.f) continue;
#pragma unroll
                                for (int e = 0; e < E; ++e) {
                                    acc[e].x += y[sub & 1][a][p][e].x * wp;
                                    acc[e].y += y[sub & 1][a][p][e].y * wp;
                                }
                            }
                            const int to = __shfl_sync(0xffffffffu, row, from);
                            const float f = __shfl_sync(0xffffffffu, inv, from);
                            if (to < 0) continue;
#pragma unroll
                            for (int e = 0; e < E; ++e)          // (f = 0 where no rank saw anything, and so is the sum)
                                *reinterpret_cast<uint32_t *>(A.o + (int64_t)to * D + e * 64 + lane * 2) =
                                    xpack<kFp16>(acc[e].x * f, acc[e].y * f);
                        }
                    }
                }
            };
            if (ns == 2) join(std::integral_constant<int, 2>{});
            else if (ns <= 4) join(std::integral_constant<int, 4>{});
            else join(std::integral_constant<int, 8>{});
            cluster_sync();                              // peers are done with this CTA's shared memory
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kFwdMma) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, L::TMEM);
    }
    if (threadIdx.x == 0) {
        A.status[blockIdx.x] = *abort_flag ? SAG_ERR_TIMEOUT : kMode == kPaged && *bad_index ? SAG_ERR_INDEX : SAG_OK;
        if (blockIdx.x == 0) *A.count = A.n_status;
    }
}

// Joins the pieces of units: a block a row; its warps take every sixteenth piece and are added up in their order.  All
// maxima and sums are read at once, and a warp's first eight pieces' rows beside them (one token over 131072 states: 48.4 us;
// eight warps, and rows after sums: 50.3).
constexpr int kJoinWarps = 16, kMaxJoin = 512;           // pieces of a unit at most
template <bool kFp16, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) k_xjoin(const __grid_constant__ XArgs A) {
    constexpr float kShift = kFp16 ? kFwdShiftF16 : 0.f;
    constexpr int E = D / 32;
    __shared__ float acc_of[kJoinWarps][D], weight_of[kMaxJoin], red[2][kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / A.join_rows, k = blockIdx.x % A.join_rows;
    const XUnit u = x_decode<&SeqRow::qtile0, kDown>(A, unit);
    const int tok = u.tile * A.tpt + k / A.group;
    const int64_t row = (int64_t)(u.seq.q0 + tok) * A.n1 + u.head * A.group + k % A.group;
    grid_wait();                                         // the pieces
    if (tok >= (A.s1_pad ? A.s1_pad : u.seq.qlen)) return;
    const bool pad = tok >= u.seq.qlen;
    const int pieces = pad ? 0 : A.pieces;
    const float2 *ml = A.part_ml + ((int64_t)unit * A.pieces * kXRows + k);
    const float *part = A.parts + ((int64_t)unit * A.pieces * kXRows + k) * D + lane * E;
    static_assert(kMaxFwdPieces <= kMaxJoin && kMaxJoin == kJoinWarps * 32, "a thread a piece");
    const float2 v = (int)threadIdx.x < pieces ? ml[(int64_t)threadIdx.x * kXRows] : make_float2(-INFINITY, 0.f);
    float y[8][E];
    auto read = [&](int p0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = p0 + i * kJoinWarps;
#pragma unroll
            for (int e = 0; e < E; ++e) y[i][e] = 0.f;
            if (p >= pieces) continue;
            const float *at = part + (int64_t)p * kXRows * D;
            if constexpr (E == 4) *reinterpret_cast<float4 *>(y[i]) = *reinterpret_cast<const float4 *>(at);
            else *reinterpret_cast<float2 *>(y[i]) = *reinterpret_cast<const float2 *>(at);
        }
    };
    read(warp);
    float top = v.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) red[0][warp] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, red[0][i]);
    // a piece that saw nothing does not count (its O was not written); one whose weight underflows does: 0 times NaN is NaN
    const bool saw = v.y != 0.f;
    const float weight = saw ? xex2(v.x - top) : 0.f;
    float sum = saw ? v.y * weight : 0.f;
    weight_of[threadIdx.x] = saw ? weight : -1.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) sum += red[1][i];
    float acc[E] = {};
    for (int p0 = warp; p0 < pieces; p0 += 8 * kJoinWarps) {
        if (p0 != warp) read(p0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = p0 + i * kJoinWarps;
            const float w = p < pieces ? weight_of[p] : -1.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (w != -1.f) acc[e] += y[i][e] * w;    // (else what was read is no sum)
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc_of[warp][lane * E + e] = acc[e];
    __syncthreads();
    const bool some = sum > 0.f || sum != sum;
    const float inv = some ? 1.f / sum : 0.f;
    if (threadIdx.x < D) {
        float sums = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) sums += acc_of[w][threadIdx.x];
        A.o[row * D + threadIdx.x] = some ? f_to_u16<kFp16>(sums * inv) : (uint16_t)0;
    }
    if (threadIdx.x == 0) A.lse[row] = pad ? 0.f : some ? (top - kShift) * 0.6931471805599453f + logf(sum) : -INFINITY;
}

}  // namespace
}  // namespace sag
