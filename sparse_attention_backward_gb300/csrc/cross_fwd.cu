// Cross attention, forward: O = softmax(scale Q K^T) V over the key rows of
// each query row's sequence, one pass with a running maximum and sum.
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
// distributed shared memory in rank order: one launch, no workspace, the same
// bits on every run.
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
// XF_S: scores of an even / odd tile formed, and P V of the tile two before complete; XF_P: P written
enum { XF_Q = 0, XF_S = 1, XF_P = 3, XF_DRAIN = 5, XF_FULL = 6 };

template <bool kFp16, int D, int kKeys>
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort_flag = 0;
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
    const int ns = A.nsplit, rank = blockIdx.x % ns;
    const XUnit u = x_decode<&SeqRow::qtile0>(A, blockIdx.x / A.nsplit);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sbase = tc::smem_u32(smem);
    const int G = A.group, tok0 = u.tile * A.tpt;
    const int cover = A.s1_pad ? A.s1_pad : u.seq.qlen;
    const int nkt = tok0 < u.seq.qlen ? (u.seq.klen + kKeys - 1) / kKeys : 0;
    int t0, n;
    x_share(nkt, rank, ns, &t0, &n);
    const int partial = A.mask ? 0 : u.seq.klen / kKeys - t0;    // tiles from this one on may lack keys
    auto fail = [&]() { *abort_flag = 1; };

    if (warp >= kFwdTma) {
        if (warp == kFwdTma) {
            // -------------------------------------------------- TMA producer
            if (lane == 0 && n > 0) {
                bool ok = true;
                int loads = 0;
                auto stage = [&](const CUtensorMap *map, int key) {
                    const int s = loads % ST, use = loads / ST;
                    if (use > 0 && !tc::mbar_wait(&empty[s], (use - 1) & 1, abort_flag, kXWaitNs)) return false;
                    tc::mbar_arrive_expect_tx(&full[s], L::TILE);
                    for (int c = 0; c < L::KC; ++c)
                        tc::tma_load_3d(smem + L::OFF_RING + s * L::TILE + c * kKeys * 128, map, c * 64, u.head,
                                        u.seq.k0 + key, &full[s]);
                    ++loads;
                    return true;
                };
                tc::mbar_arrive_expect_tx(&bars[XF_Q], (uint32_t)L::KC * A.tpt * G * 128);
                for (int c = 0; c < L::KC; ++c)
                    tc::tma_load_3d(smem + c * 16384, &map_q, c * 64, u.head * G, u.seq.q0 + tok0, &bars[XF_Q]);
                // in the order the MMA warp takes them: the first K, then V i and K i + NB
                for (int i = -NB; i < n && ok; ++i) {
                    if (i >= 0) ok = stage(&map_v, (t0 + i) * kKeys);
                    if (ok && i + NB < n) ok = stage(&map_k, (t0 + i + NB) * kKeys);
                }
                if (!ok) fail();
                // every load issued must have landed before the CTA exits
                bool drained = tc::drain_armed(&bars[XF_Q], 1, kXWaitNs);
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
            // load j of the ring: the first K tiles, then V i (behind min(i + NB, n) tiles of K) and K i + NB
            auto landed = [&](int j) { return Phase{&full[j % ST], (uint32_t)(j / ST) & 1u}; };
            auto issue_s = [&](int i, int j) {
                mma_abt<D, kKeys>(tmem + i % NB * kKeys, sbase, ring + j % ST * L::TILE, id_s);
                tc::mma_commit_warp(&bars[XF_S + i % NB]);
                tc::mma_commit_warp(&empty[j % ST]);
            };
            bool ok = true;
            for (int i = 0; i < NB && i < n && ok; ++i) {
                ok = warp_wait(abort_flag, Phase{&bars[XF_Q], 0}, landed(i));
                tc::tc_fence_after();
                if (ok) issue_s(i, i);
            }
            for (int i = 0; i < n && ok; ++i) {
                const bool more = i + NB < n;
                const int jv = i + (more ? i + NB : n);
                const uint32_t vt = ring + jv % ST * L::TILE, acc = tmem + L::COL_O, pt = tmem + i % NB * kKeys + L::P_AT;
                // P (its first half), V, and with the last half the K tile of the scores that follow
                auto written = [&](int h) {
                    return L::HALVES == 2 ? Phase{&bars[XF_P + h], (uint32_t)i & 1u}
                                          : Phase{&bars[XF_P + i % NB], (uint32_t)(i / NB) & 1u};
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
                tc::mma_commit_warp(&empty[jv % ST]);
                if (more) issue_s(i + NB, jv + 1);
                else tc::mma_commit_warp(&bars[XF_S + i % NB]);
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
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        const uint32_t to = trow + L::COL_O;
        float m = -INFINITY, l = 0.f;                    // reference maximum (log2 units), sum
        if (n > 0) {
            // -------------------------------------------------- softmax
            const float c = A.scale_log2;
            auto wait = [&](int b, uint32_t parity) {
                return warp_wait(abort_flag, Phase{&bars[b], parity});
            };
            // tile i's scores (or, behind the last two tiles, just the products before) are complete
            auto formed = [&](int i) { return wait(XF_S + i % NB, (uint32_t)(i / NB) & 1u); };
            // One tile; a copy of its own for tiles with absent keys, whose
            // selects otherwise run for every tile.  Paired fp32 operations
            // (f32x2): half the instructions where issue slots are short,
            // 540 -> 507 us for 8192 x 4096 tokens of 64-wide heads.
            KeyLoad<kKeys / 32> keys{};                  // of the next tile that may lack keys
            auto tile = [&](auto masked, int i) -> bool {
                const uint32_t ts = trow + i % NB * kKeys;
                KeyBits<kKeys / 32> kb{};
                if constexpr (decltype(masked)::value) {
                    if (!L::MASK_AHEAD) keys.start(A.mask, u.seq, (t0 + i) * kKeys, lane);
                    kb = keys.finish();
                    if (L::MASK_AHEAD && i + 1 < n) keys.start(A.mask, u.seq, (t0 + i + 1) * kKeys, lane);
                    if (!kb.all()) {
                        const int jv = i + (i + NB < n ? i + NB : n);   // V's place in the ring, as in the MMA warp
                        if (!warp_wait(abort_flag, Phase{&full[jv % ST], (uint32_t)(jv / ST) & 1u})) return false;
                        zero_rows<L::KC, kKeys / 32, 128>(smem + L::OFF_RING + jv % ST * L::TILE, kb, r);
                    }
                }
                constexpr int kHeld = L::NARROW ? 32 : kKeys;           // scores held in registers at a time
                float x[kHeld];
                // columns `from` .. from + kHeld - 1
                auto scores = [&](int from) {
#pragma unroll
                    for (int j = 0; j < kHeld; j += 32) tmem_ld32(ts + from + j, reinterpret_cast<uint32_t *>(x) + j);
                    tc::tmem_wait_ld();
                    if constexpr (decltype(masked)::value) {
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
                const float base = m == -INFINITY ? 0.f : m - kShift;
                const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
                float2 sum[2] = {};
                // two rounded probabilities
                auto pair = [&](int j) {
                    float2 e = fma2(make_float2(x[j], x[j + 1]), c2, b2);
                    e = make_float2(xex2(e.x), xex2(e.y));
                    sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], e);
                    return xpack<kFp16>(e.x, e.y);
                };
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
            if (L::MASK_AHEAD && partial < n) keys.start(A.mask, u.seq, (t0 + (partial > 0 ? partial : 0)) * kKeys, lane);
            bool ok = true;
            for (int i = 0; i < n && ok; ++i) {
                ok = formed(i);
                if (!ok) break;
                tc::tc_fence_after();
                ok = i < partial ? tile(std::false_type{}, i) : tile(std::true_type{}, i);
            }
            if (ok) ok = formed(n - 1 + NB);
            if (!ok && lane == 0) fail();
            tc::tc_fence_after();
        }

        // ------------------------------------------------------ epilogue
        const float kLn2 = 0.6931471805599453f;
        if (ns == 1) {
            const int tok = tok0 + r / G;
            const bool mine = r < A.tpt * G && tok < cover;
            const bool pad = tok >= u.seq.qlen;
            const int64_t row = (int64_t)(u.seq.q0 + tok) * A.n1 + u.head * G + r % G;
            const bool some = l > 0.f || l != l;         // l is NaN when a score was
            const float inv = some ? 1.f / l : 0.f;
            RowStore<kFp16> rows;
            rows.rows(mine ? row * D : -1, lane);
#pragma unroll
            for (int j = 0; j < D; j += 32) {
                float y[32];
                if (n > 0) {
                    tmem_ld32(to + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = some && !pad ? y[e] * inv : 0.f;
                rows.store(A.o, y, j, lane);
            }
            if (mine) A.lse[row] = pad ? 0.f : some ? (m - kShift) * kLn2 + logf(l) : -INFINITY;
        } else {
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
            constexpr int E = D / 64;                    // float2 a lane and row
            for (int k = rank + ns * warp; k < A.tpt * G; k += ns * 4) {
                const int tok = tok0 + k / G;
                if (tok >= cover) break;
                const int64_t row = (int64_t)(u.seq.q0 + tok) * A.n1 + u.head * G + k % G;
                const bool pad = tok >= u.seq.qlen;
                // lane p holds rank p's maximum and sum; a rank that saw nothing has (-inf, 0) and no O
                float2 v = make_float2(-INFINITY, 0.f);
                if (!pad && lane < ns) v = peer_ld2(peer_addr(tc::smem_u32(ml + k), lane));
                float2 y[kMaxSplit][E], acc[E] = {};
#pragma unroll
                for (int p = 0; p < kMaxSplit; ++p)
                    if (p < ns) {
                        const uint32_t a = peer_addr(tc::smem_u32(xo + k * L::XROW + lane * 2), p);
#pragma unroll
                        for (int e = 0; e < E; ++e) y[p][e] = peer_ld2(a + e * 256);
                    }
                float top = v.x;
#pragma unroll
                for (int o = kMaxSplit / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                top = __shfl_sync(0xffffffffu, top, 0);
                // A rank that saw something counts even where its weight underflows: 0 times its NaN is NaN, as in an undivided
                // loop.  (A rank of NaN scores alone has -inf and NaN.)
                const float w = v.y == 0.f ? 0.f : xex2(v.x - top);
                float sum = 0.f;
#pragma unroll
                for (int p = 0; p < kMaxSplit; ++p) {
                    const float wp = __shfl_sync(0xffffffffu, w, p), lp = __shfl_sync(0xffffffffu, v.y, p);
                    if (lp == 0.f) continue;
                    sum += lp * wp;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        acc[e].x += y[p][e].x * wp;
                        acc[e].y += y[p][e].y * wp;
                    }
                }
                const bool some = sum > 0.f || sum != sum;
                const float inv = some ? 1.f / sum : 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    *reinterpret_cast<uint32_t *>(A.o + row * D + e * 64 + lane * 2) =
                        some ? xpack<kFp16>(acc[e].x * inv, acc[e].y * inv) : 0u;
                if (lane == 0) A.lse[row] = pad ? 0.f : some ? (top - kShift) * kLn2 + logf(sum) : -INFINITY;
            }
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
        A.status[blockIdx.x] = *abort_flag ? SAG_ERR_TIMEOUT : SAG_OK;
        if (blockIdx.x == 0) *A.count = A.n_status;
    }
}

template <bool kFp16, int D, int kKeys>
cudaError_t launch(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!x_map_q(&mq, io.query, d, a, d.q_stride) || !x_map_k(&mk, io.key, io.query, d, d.k_stride, kKeys) ||
        !x_map_k(&mv, io.value, io.query, d, d.v_stride, kKeys))
        return cudaErrorInvalidValue;
    return x_launch(k_xfwd<kFp16, D, kKeys>, a.ctas, kFwdThreads, a.nsplit, FwdShape<D, kKeys>::TOTAL, false, s, mq,
                    mk, mv, a);
}

}  // namespace

// Tiles of 128 keys take 64 cycles a step for their scores where two of 64 take 96 (M = 128 rows re-read per instruction),
// but leave one score tile in flight instead of two.  They are taken for 128-wide heads where products dominate: full
// query tiles and long loops.  Measured, 64 against 128: 8192 x 4096 tokens 825 / 742 us, 130 x 131072 233 / 205;
// 1024 x 1024 33 / 35, 2048 x 512 70 / 74, one token x 4096 69 / 74 us; 64-wide heads 582 / 596 us.  (Sharing a row of 128
// keys between two threads, for a shorter softmax, was slower: 792 us for the first, and 235 for the second.)
cudaError_t launch_xfwd(const XArgs &a, const sca_io &io, const sca_desc &d, bool long_loops, cudaStream_t s) {
    const bool fp16 = d.dtype == SAG_FP16;
    if (d.d == 128 && long_loops)
        return fp16 ? launch<true, 128, 128>(a, io, d, s) : launch<false, 128, 128>(a, io, d, s);
    if (d.d == 128) return fp16 ? launch<true, 128, 64>(a, io, d, s) : launch<false, 128, 64>(a, io, d, s);
    return fp16 ? launch<true, 64, 64>(a, io, d, s) : launch<false, 64, 64>(a, io, d, s);
}

}  // namespace sag
