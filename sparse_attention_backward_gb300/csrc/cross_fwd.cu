// Cross attention, forward: O = softmax(scale Q K^T) V over the key rows of
// each query row's sequence, one pass with a running maximum and sum.
//
// A CTA takes 256 query rows (two tiles) of one key/value head and walks over
// the key tiles: S = Q K^T and O += P V on the tensor cores (tcgen05), S, P and
// O in TMEM, P written over S as the TMEM operand of the second product, so
// that scores and probabilities never touch shared memory.  The two tiles
// alternate: while one tile's softmax runs on its four warps (a thread a row,
// no shuffles), the MMA warp does the other tile's products.
//
// The running maximum is lazy: O and the sum are rescaled only when a row's
// maximum grows by more than 2^8 over the reference in use, which any reference
// allows (O / sum does not depend on it); P then stays <= 2^8, far from the
// 16-bit types' limits.  The rescaling happens in the row's own thread, when
// the score tile has arrived: the earlier P V is complete then, since both
// were issued in order by one thread.  P is rounded to 16 bits as an operand;
// the sum is taken of the unrounded fp32 values.
//
// Few query rows and many keys: the key tiles of a unit are split over the
// CTAs of a cluster, whose partial O, maximum and sum are joined through
// distributed shared memory in rank order: one launch, no workspace, the same
// bits on every run.
#include "cross.cuh"
#include "kernels.cuh"
#include "tmap.cuh"
#include "xtmap.cuh"

namespace sag {

namespace {

// warps 0-3 and 4-7: softmax and epilogue of the two tiles, 8: TMA, 9: MMA, 10-11: none (a warpgroup's registers are
// handed over as a whole: 2 * 208 + 88 = 3 * 168, what the block is launched with)
constexpr int kFwdThreads = 384;

template <int D>
struct FwdSmem {
    static constexpr int KC = D / 64;
    static constexpr int TILE = KC * 16384;
    static constexpr int STAGES = 131072 / TILE;
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_ML = OFF_RING + STAGES * TILE;       // float2 [2][128]
    static constexpr int OFF_BAR = OFF_ML + 2048;
    static constexpr int TOTAL = OFF_BAR + 256;
    static constexpr int XROW = D + 4;                            // exchange rows, padded against bank conflicts
    static_assert(2 * kXRows * XROW * 4 <= OFF_ML, "the exchange overlays Q and the ring");
};
// XF_P: per tile, one barrier for each half of its probabilities
enum { XF_Q = 0, XF_S = 1, XF_P = 3, XF_DRAIN = 7, XF_FULL = 8 };

template <bool kFp16, int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
    k_xfwd(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
           const __grid_constant__ CUtensorMap map_v, const __grid_constant__ XArgs A) {
    using L = FwdSmem<D>;
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
        tc::mbar_init(&bars[XF_Q], 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars[XF_S + i], 1);
            tc::mbar_init(&bars[XF_P + 2 * i], 128);
            tc::mbar_init(&bars[XF_P + 2 * i + 1], 128);
        }
        tc::mbar_init(&bars[XF_DRAIN], 1);
        for (int i = 0; i < ST; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        tc::fence_mbar_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 256) {
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_k);
        tc::prefetch_tmap(&map_v);
    }
    const int ns = A.nsplit, rank = blockIdx.x % ns;
    const XUnit u = x_decode<&SeqRow::qtile0>(A, blockIdx.x / ns);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sbase = tc::smem_u32(smem);
    const int G = A.group;
    const int cover = A.s1_pad ? A.s1_pad : u.seq.qlen;
    const int tok0[2] = {u.tile * 2 * A.tpt, (u.tile * 2 + 1) * A.tpt};
    const bool active[2] = {tok0[0] < u.seq.qlen, tok0[1] < u.seq.qlen};
    const int nkt = active[0] ? (u.seq.klen + kXRows - 1) / kXRows : 0;
    const int t0 = (int)((int64_t)nkt * rank / ns), n = (int)((int64_t)nkt * (rank + 1) / ns) - t0;
    auto fail = [&]() { *abort_flag = 1; };

    // The softmax warps take registers from the others.  The two sides share no code up to the end of the kernel: what
    // both run must fit the smaller number.
    if (warp >= 8) {
    regs_fewer<88>();
    if (warp == 8) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0 && n > 0) {
            bool ok = true;
            const uint32_t qbytes = (uint32_t)L::KC * A.tpt * G * 128;
            int loads = 0;
            auto stage = [&](const CUtensorMap *map, int key) {
                const int s = loads % ST, use = loads / ST;
                if (use > 0 && !tc::mbar_wait(&empty[s], (use - 1) & 1, abort_flag, kXWaitNs)) return false;
                tc::mbar_arrive_expect_tx(&full[s], L::TILE);
                for (int c = 0; c < L::KC; ++c)
                    tc::tma_load_3d(smem + L::OFF_RING + s * L::TILE + c * 16384, map, c * 64, u.head, u.seq.k0 + key,
                                    &full[s]);
                ++loads;
                return true;
            };
            tc::mbar_arrive_expect_tx(&bars[XF_Q], qbytes * (active[1] ? 2 : 1));
            for (int sl = 0; sl < 2; ++sl)
                if (active[sl])
                    for (int c = 0; c < L::KC; ++c)
                        tc::tma_load_3d(smem + sl * L::TILE + c * 16384, &map_q, c * 64, u.head * G, u.seq.q0 + tok0[sl],
                                        &bars[XF_Q]);
            for (int i = 0; i < n && ok; ++i) {
                const int key = (t0 + i) * kXRows;
                ok = stage(&map_k, key) && stage(&map_v, key);
            }
            if (!ok) fail();
            // every load issued must have landed before the CTA exits
            bool drained = tc::drain_armed(&bars[XF_Q], 1, kXWaitNs);
            for (int s = 0; s < ST; ++s)
                drained = tc::drain_armed(&full[s], loads > s ? (loads - s - 1) / ST + 1 : 0, kXWaitNs) && drained;
            if (!drained) fail();
        }
    } else if (warp == 9) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t id_s = tc::idesc_f16(kXRows, kXRows, !kFp16, false, false);
        constexpr uint32_t id_o = tc::idesc_f16(kXRows, D, !kFp16, false, true);
        auto wait = [&](uint64_t *b, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, tc::mbar_wait(b, parity, abort_flag, kXWaitNs));
        };
        const uint32_t ring = sbase + L::OFF_RING;
        KeyBits next = key_bits(A.mask, u.seq, t0 * kXRows, lane);
        bool ok = n == 0 || wait(&bars[XF_Q], 0);
        if (ok && n > 0) ok = wait(&full[0], 0);
        if (ok && n > 0) {
            tc::tc_fence_after();
            for (int sl = 0; sl < 2; ++sl)
                if (active[sl]) {
                    mma_abt<D>(tmem + sl * 128, sbase + sl * L::TILE, ring, id_s);
                    tc::mma_commit_warp(&bars[XF_S + sl]);
                }
            tc::mma_commit_warp(&empty[0]);
        }
        for (int i = 0; i < n && ok; ++i) {
            const int sv = (2 * i + 1) % ST, uv = (2 * i + 1) / ST;
            const int sk = (2 * i + 2) % ST, uk = (2 * i + 2) / ST;
            if (!wait(&full[sv], uv & 1)) { ok = false; break; }
            const KeyBits kb = next;
            if (i + 1 < n) next = key_bits(A.mask, u.seq, (t0 + i + 1) * kXRows, lane);
            if (!kb.all()) zero_rows<L::KC>(smem + L::OFF_RING + sv * L::TILE, kb, lane);
            const bool more = i + 1 < n;
            for (int sl = 0; sl < 2; ++sl) {
                if (!active[sl]) continue;
                // the first half of the keys while the softmax forms the second half's probabilities
                if (!wait(&bars[XF_P + 2 * sl], i & 1)) { ok = false; break; }
                tc::tc_fence_after();
                mma_ab<32, 0, 4>(tmem + 256 + sl * 128, tmem + sl * 128, ring + sv * L::TILE, id_o, i > 0);
                if (!wait(&bars[XF_P + 2 * sl + 1], i & 1)) { ok = false; break; }
                tc::tc_fence_after();
                mma_ab<32, 4, 8>(tmem + 256 + sl * 128, tmem + sl * 128, ring + sv * L::TILE, id_o, true);
                if (more) {
                    if (sl == 0 && !wait(&full[sk], uk & 1)) { ok = false; break; }
                    tc::tc_fence_after();
                    mma_abt<D>(tmem + sl * 128, sbase + sl * L::TILE, ring + sk * L::TILE, id_s);
                }
                tc::mma_commit_warp(&bars[XF_S + sl]);
            }
            if (!ok) break;
            tc::mma_commit_warp(&empty[sv]);
            if (more) tc::mma_commit_warp(&empty[sk]);
        }
        if (!ok && lane == 0) fail();
        // every MMA issued must be complete before TMEM is freed
        tc::mma_commit_warp(&bars[XF_DRAIN]);
        if (!__all_sync(0xffffffffu, tc::mbar_wait_drain(&bars[XF_DRAIN], 0, kXWaitNs)) && lane == 0) fail();
    }

    if (ns > 1) {                                        // as below
        __syncthreads();
        cluster_sync();
        cluster_sync();
    }
    } else {
    regs_more<208>();
    const int sl = warp >> 2;                            // softmax warps: their tile
    const int r = (warp & 3) * 32 + lane;                // query row = TMEM lane
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float m = -INFINITY, l = 0.f;                        // reference maximum (log2 units), sum
    if (active[sl] && n > 0) {
        // ------------------------------------------------------ softmax
        const float c = A.scale_log2;
        const uint32_t ts = trow + sl * 128, to = trow + 256 + sl * 128;
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const KeyBits kb = key_bits(A.mask, u.seq, (t0 + i) * kXRows, lane);
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[XF_S + sl], i & 1, abort_flag, kXWaitNs));
            if (!ok) break;
            tc::tc_fence_after();
            float x[128];
            for (int j = 0; j < 4; ++j) tmem_ld32(ts + j * 32, reinterpret_cast<uint32_t *>(x) + j * 32);
            tc::tmem_wait_ld();
            if (!kb.all()) {
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    if (!((kb.w[j >> 5] >> (j & 31)) & 1u)) x[j] = -INFINITY;
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int j = 4; j < 124; j += 8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(fmaxf(mx[e], x[j + e]), x[j + 4 + e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[124 + e]);
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            const bool grow = mt > m + 8.f;
            if (__any_sync(0xffffffffu, grow)) {
                const float mnew = grow ? mt : m;
                const float f = grow ? xex2(m - mnew) : 1.f;
                l *= f;
                m = mnew;
                if (i > 0) {
#pragma unroll
                    for (int j = 0; j < D; j += 32) {
                        float y[32];
                        tmem_ld32(to + j, reinterpret_cast<uint32_t *>(y));
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] *= f;
                        tmem_st32(to + j, reinterpret_cast<const uint32_t *>(y));
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : m - kShift;
            const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
            float2 s4[4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float2 e = fma2(make_float2(x[h * 64 + 2 * j], x[h * 64 + 2 * j + 1]), c2, b2);
                    e.x = xex2(e.x);
                    e.y = xex2(e.y);
                    s4[j & 3] = add2(s4[j & 3], e);
                    p[j] = xpack<kFp16>(e.x, e.y);
                }
                tmem_st32(ts + h * 32, p);
                tmem_wait_st();
                tc::tc_fence_before();
                tc::mbar_arrive(&bars[XF_P + 2 * sl + h]);
            }
            const float2 s2 = add2(add2(s4[0], s4[1]), add2(s4[2], s4[3]));
            l += s2.x + s2.y;
        }
        if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[XF_S + sl], n & 1, abort_flag, kXWaitNs));
        if (!ok && lane == 0) fail();
        tc::tc_fence_after();
    }

    // ---------------------------------------------------------- epilogue
    const float kLn2 = 0.6931471805599453f;
    if (ns == 1) {
        {
            const int tok = tok0[sl] + r / G;
            const bool mine = r < A.tpt * G && tok < cover;
            const bool pad = tok >= u.seq.qlen;
            const int64_t row = (int64_t)(u.seq.q0 + tok) * A.n1 + u.head * G + r % G;
            const bool some = l > 0.f || l != l;         // l is NaN when a score was
            const float inv = some ? 1.f / l : 0.f;
            const bool have = active[sl] && n > 0;
#pragma unroll
            for (int j = 0; j < D; j += 32) {
                float y[32];
                if (have) {
                    tmem_ld32(trow + 256 + sl * 128 + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = some && !pad ? y[e] * inv : 0.f;
                if (mine) store_row<kFp16, 32>(A.o + row * D + j, y);
            }
            if (mine) A.lse[row] = pad ? 0.f : some ? (m - kShift) * kLn2 + logf(l) : -INFINITY;
        }
    } else {
        // partial O, maximum and sum of every rank into its shared memory, then each rank joins its share of the rows
        float2 *ml = reinterpret_cast<float2 *>(smem + L::OFF_ML);
        float *xo = reinterpret_cast<float *>(smem);
        __syncthreads();                                 // all loads and products on this memory are complete
        if (active[sl]) {
            ml[sl * 128 + r] = make_float2(m, l);
            if (n > 0) {
#pragma unroll
                for (int j = 0; j < D; j += 32) {
                    float y[32];
                    tmem_ld32(trow + 256 + sl * 128 + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4 *>(xo + (sl * 128 + r) * L::XROW + j + e) =
                            make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                }
            }
        }
        cluster_sync();
        {
            constexpr int E = D / 64;                    // float2 a lane and row
            for (int k = rank + ns * warp; k < 2 * kXRows; k += ns * 8) {
                const int ks = k / kXRows, kr = k % kXRows, tok = tok0[ks] + kr / G;
                if (kr >= A.tpt * G || tok >= cover) continue;
                const int64_t row = (int64_t)(u.seq.q0 + tok) * A.n1 + u.head * G + kr % G;
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
                const float w = v.y == 0.f ? 0.f : xex2(v.x - top);
                float sum = 0.f;
#pragma unroll
                for (int p = 0; p < kMaxSplit; ++p) {
                    const float wp = __shfl_sync(0xffffffffu, w, p), lp = __shfl_sync(0xffffffffu, v.y, p);
                    if (wp == 0.f) continue;
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
        }
        cluster_sync();                                  // peers are done with this CTA's shared memory
    }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0) {
        A.status[blockIdx.x] = *abort_flag ? SAG_ERR_TIMEOUT : SAG_OK;
        if (blockIdx.x == 0) *A.count = A.n_status;
    }
}

template <bool kFp16, int D>
cudaError_t launch(const XArgs &a, const sca_io &io, const sca_desc &d, int units, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!x_map_q(&mq, io.query, d, a, d.q_stride) || !x_map_k(&mk, io.key, io.query, d, a, d.k_stride) ||
        !x_map_k(&mv, io.value, io.query, d, a, d.v_stride))
        return cudaErrorInvalidValue;
    return x_launch(k_xfwd<kFp16, D>, units * a.nsplit, kFwdThreads, a.nsplit, FwdSmem<D>::TOTAL, s, mq, mk, mv, a);
}

}  // namespace

cudaError_t launch_xfwd(const XArgs &a, const sca_io &io, const sca_desc &d, int units, cudaStream_t s) {
    const bool fp16 = d.dtype == SAG_FP16;
    if (d.d == 128) return fp16 ? launch<true, 128>(a, io, d, units, s) : launch<false, 128>(a, io, d, units, s);
    return fp16 ? launch<true, 64>(a, io, d, units, s) : launch<false, 64>(a, io, d, units, s);
}

}  // namespace sag
