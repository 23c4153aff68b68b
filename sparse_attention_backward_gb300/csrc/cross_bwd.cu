// Cross attention, gradient: three launches, no atomics, no fp32 accumulators
// in memory.
//
//   k_xpre  Delta = rowsum(dY * O) and lse in log2 units, packed by query tile
//   k_xdq   per query tile:  S = Q K^T, dP = dY V^T, dS = P (dP - Delta),  dQ += dS K      (over key tiles)
//   k_xdkv  per key tile:    S^T = K Q^T, dP^T = V dY^T,  dV += P^T dY,  dK += dS^T Q      (over query tiles)
//
// Scores and dP are formed twice (7 products instead of 5), which buys sums in
// a fixed order with every accumulator in TMEM for a tile's whole life: the
// alternative adds a 64 KB fp32 dQ partial to memory for each pair of tiles.
// P and dS go back to TMEM as 16-bit operands (over the S and dP columns they
// came from), so only the tiles themselves are read from shared memory.
//
// k_xdkv works on the transposed scores (lane = key): P^T and dS^T are then
// K-major TMEM operands as they stand.  Its two phases alternate with the MMA
// warp: exp beside dK and the next dP, dS beside dV and the next S.
//
// P and dS are rounded to the 16-bit type as operands; fp16 ones are scaled by
// powers of two first (cross.cuh), dS by one found from the largest norms of
// dY and V rows of the sequence and head: |dP - Delta| <= 2 |dY| |V|, so that
// neither a loss scale overflows nor a long softmax vanishes.
//
// Few tiles: a cluster's CTAs split the loop and join their accumulators
// through distributed shared memory, in rank order.
#include <type_traits>

#include "cross.cuh"
#include "kernels.cuh"
#include "xtmap.cuh"

namespace sag {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ k_xpre
template <bool kFp16, int D>
__global__ void __launch_bounds__(256) k_xpre(const __grid_constant__ XArgs A) {
    constexpr int LPR = D / 8;                           // lanes a row, 16 bytes each
    constexpr int RPW = 32 / LPR;
    __shared__ float red[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = lane % LPR;
    const int q_units = A.q_tiles * A.n2;
    float top = 0.f;
    int64_t slot;
    if ((int)blockIdx.x < q_units) {
        const XUnit u = x_decode<&SeqRow::qtile0>(A, blockIdx.x);
        slot = u.tile_id;
        float *st = A.stats + u.tile_id * 256;
        for (int r = warp * RPW + lane / LPR; r < kXRows; r += 8 * RPW) {
            const int tok = u.tile * A.tpt + r / A.group;
            const bool live = r < A.tpt * A.group && tok < u.seq.qlen;
            const int64_t row = (int64_t)(u.seq.q0 + tok) * A.n1 + u.head * A.group + r % A.group;
            float dot = 0.f, nrm = 0.f, lse = -INFINITY;
            if (live) {
                uint4 a = *reinterpret_cast<const uint4 *>(A.o_in + row * D + part * 8);
                uint4 b = *reinterpret_cast<const uint4 *>(A.dy + row * D + part * 8);
                lse = A.lse[row];
                const uint32_t *pa = &a.x, *pb = &b.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y0 = u16_to_f<kFp16>((uint16_t)pb[i]), y1 = u16_to_f<kFp16>((uint16_t)(pb[i] >> 16));
                    dot += u16_to_f<kFp16>((uint16_t)pa[i]) * y0 + u16_to_f<kFp16>((uint16_t)(pa[i] >> 16)) * y1;
                    nrm += y0 * y0 + y1 * y1;
                }
            }
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) {
                dot += __shfl_xor_sync(0xffffffffu, dot, o);
                nrm += __shfl_xor_sync(0xffffffffu, nrm, o);
            }
            if (part == 0) {
                const bool some = live && lse != -INFINITY;
                st[r] = some ? -lse * kLog2e : -INFINITY;   // makes P = 0 where there is nothing
                st[128 + r] = some ? -dot : 0.f;
            }
            if (nrm < INFINITY) top = fmaxf(top, nrm);
        }
    } else {
        // fp16 only: row norms of V
        const XUnit u = x_decode<&SeqRow::ktile0>(A, blockIdx.x - q_units);
        slot = q_units + u.tile_id;
        for (int r = warp * RPW + lane / LPR; r < kXRows; r += 8 * RPW) {
            const int key = u.tile * kXRows + r;
            const int64_t row = (int64_t)u.seq.k0 + key;
            float nrm = 0.f;
            if (key < u.seq.klen && (!A.mask || A.mask[row])) {
                uint4 a = *reinterpret_cast<const uint4 *>(A.v_in + row * A.v_stride + u.head * D + part * 8);
                const uint32_t *pa = &a.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y0 = u16_to_f<kFp16>((uint16_t)pa[i]), y1 = u16_to_f<kFp16>((uint16_t)(pa[i] >> 16));
                    nrm += y0 * y0 + y1 * y1;
                }
            }
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) nrm += __shfl_xor_sync(0xffffffffu, nrm, o);
            if (nrm < INFINITY) top = fmaxf(top, nrm);
        }
    }
    if constexpr (kFp16) {
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) red[warp] = top;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < 8; ++i) top = fmaxf(top, red[i]);
            A.norms[slot] = sqrtf(top);
        }
    }
}

// fp16: exponent e such that 2^e |dS| <= 2^15 for every dS of the sequence and head.  `red` is [kXThreads / 32] floats of
// shared memory; holds a __syncthreads.
__device__ __forceinline__ float ds_exponent(const XArgs &A, const SeqRow &a, const SeqRow &b, int head, float *red) {
    float ny = 0.f, nv = 0.f;
    for (int t = a.qtile0 + threadIdx.x; t < b.qtile0; t += kXThreads) ny = fmaxf(ny, A.norms[(int64_t)t * A.n2 + head]);
    for (int t = a.ktile0 + threadIdx.x; t < b.ktile0; t += kXThreads)
        nv = fmaxf(nv, A.norms[(int64_t)(A.q_tiles + t) * A.n2 + head]);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        ny = fmaxf(ny, __shfl_xor_sync(0xffffffffu, ny, o));
        nv = fmaxf(nv, __shfl_xor_sync(0xffffffffu, nv, o));
    }
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
        red[2 * warp] = ny;
        red[2 * warp + 1] = nv;
    }
    __syncthreads();
    ny = nv = 0.f;
    for (int i = 0; i < kXThreads / 32; ++i) {
        ny = fmaxf(ny, red[2 * i]);
        nv = fmaxf(nv, red[2 * i + 1]);
    }
    const float bound = 2.f * ny * nv;
    if (!(bound > 0.f) || !(bound < INFINITY)) return 0.f;
    return fminf(fmaxf(14.f - (float)ilogbf(bound), -40.f), 40.f);
}

// ------------------------------------------------------------------- shared
// Two resident tiles (X, Y) and two rings: tiles that live long (A: keys in k_xdq, queries in k_xdkv) and tiles that one
// product reads (B: values, or output gradients, which two read).
template <int D>
struct BwdSmem {
    static constexpr int KC = D / 64;
    static constexpr int TILE = KC * 16384;
    static constexpr int RA = D == 128 ? 3 : 4, RB = D == 128 ? 2 : 4;
    static constexpr int OFF_X = 0, OFF_Y = TILE, OFF_A = 2 * TILE, OFF_B = OFF_A + RA * TILE;
    static constexpr int OFF_STAT = OFF_B + RB * TILE;   // k_xdkv: [2][256] floats
    static constexpr int OFF_BAR = OFF_STAT + 2048;
    static constexpr int TOTAL = OFF_BAR + 512;
    static constexpr int XROW = D + 4;
    static_assert(2 * kXRows * XROW * 4 <= OFF_STAT, "the exchange overlays the tiles");
    static_assert(TOTAL <= 227 * 1024, "shared memory of one CTA");
};
// barriers
enum { XB_XY = 0, XB_S = 1, XB_DP = 3, XB_PF = 4, XB_DS = 5, XB_ACC = 6, XB_DRAIN = 7, XB_STF = 8, XB_STE = 10, XB_RING = 12 };

struct Ring {
    uint64_t *full, *empty;
    int n;
    __device__ __forceinline__ Phase landed(int i) const { return Phase{&full[i % n], (uint32_t)(i / n) & 1u}; }
};

__device__ __forceinline__ bool ring_wait_free(const Ring &r, int i, volatile int *abort) {
    return i < r.n || tc::mbar_wait(&r.empty[i % r.n], (i / r.n - 1) & 1, abort, kXWaitNs);
}
__device__ __forceinline__ bool ring_drain(const Ring &r, int loads) {
    bool ok = true;
    for (int s = 0; s < r.n; ++s) ok = tc::drain_armed(&r.full[s], loads > s ? (loads - s - 1) / r.n + 1 : 0, kXWaitNs) && ok;
    return ok;
}

// Joins the ranks' partial accumulators: `rows` rows of D columns each, in xo[row][XROW] of every rank; row k of this
// rank's share goes to out(k) (nullptr: not stored), scaled by mul(k).
template <bool kFp16, int D, class Out, class Mul>
__device__ __forceinline__ void join_rows(float *xo, int rows, int ns, int rank, int warp, int lane, Out &&out, Mul &&mul) {
    constexpr int E = D / 64;
    for (int k = rank + ns * warp; k < rows; k += ns * 8) {
        uint16_t *dst = out(k);
        if (!dst) continue;
        float2 y[kMaxSplit][E], acc[E] = {};
#pragma unroll
        for (int p = 0; p < kMaxSplit; ++p)
            if (p < ns) {
                const uint32_t a = peer_addr(tc::smem_u32(xo + k * (D + 4) + lane * 2), p);
#pragma unroll
                for (int e = 0; e < E; ++e) y[p][e] = peer_ld2(a + e * 256);
            }
#pragma unroll
        for (int p = 0; p < kMaxSplit; ++p)
            if (p < ns)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = add2(acc[e], y[p][e]);
        const float f = mul(k);
#pragma unroll
        for (int e = 0; e < E; ++e)
            *reinterpret_cast<uint32_t *>(dst + e * 64 + lane * 2) = xpack<kFp16>(acc[e].x * f, acc[e].y * f);
    }
}

// ------------------------------------------------------------------- k_xdq
// TMEM columns: S of even / odd key tiles at 0 / 128 (dS over them, the second half of K 64 columns on), dP 256, dQ 384.
template <bool kFp16, int D>
__global__ void __launch_bounds__(kXThreads, 1)
    k_xdq(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_dy,
          const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
          const __grid_constant__ XArgs A) {
    using L = BwdSmem<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    const Ring ra = {bars + XB_RING, bars + XB_RING + L::RA, L::RA};
    const Ring rb = {ra.empty + L::RA, ra.empty + L::RA + L::RB, L::RB};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rb.empty + L::RB);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < XB_RING; ++i) tc::mbar_init(&bars[i], i == XB_DS || i == XB_PF ? 8 : 1);   // one arrival a warp
        for (int i = 0; i < 2 * (L::RA + L::RB); ++i) tc::mbar_init(&ra.full[i], 1);
        tc::fence_mbar_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 256) {
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_dy);
        tc::prefetch_tmap(&map_k);
        tc::prefetch_tmap(&map_v);
    }
    const int ns = A.nsplit, rank = blockIdx.x % ns;
    const XUnit u = x_decode<&SeqRow::qtile0>(A, blockIdx.x / ns);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot, sbase = tc::smem_u32(smem);
    const int G = A.group, tok0 = u.tile * A.tpt;
    const int cover = A.s1_pad ? A.s1_pad : u.seq.qlen;
    const int nkt = tok0 < u.seq.qlen ? (u.seq.klen + kXRows - 1) / kXRows : 0;
    const int t0 = (int)((int64_t)nkt * rank / ns), n = (int)((int64_t)nkt * (rank + 1) / ns) - t0;
    const int partial = A.mask ? 0 : u.seq.klen / kXRows - t0;   // tiles from this one on may lack keys
    float up = 0.f;                                      // exponent that dS is scaled by
    if constexpr (kFp16) {
        up = ds_exponent(A, u.seq, seq_row(A.seq, u.b + 1), u.head, reinterpret_cast<float *>(smem + L::OFF_STAT));
    }
    auto fail = [&]() { *abort_flag = 1; };

    if (warp == 8) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0 && n > 0) {
            const uint32_t qbytes = (uint32_t)L::KC * A.tpt * G * 128;
            tc::mbar_arrive_expect_tx(&bars[XB_XY], 2 * qbytes);
            for (int c = 0; c < L::KC; ++c) {
                tc::tma_load_3d(smem + L::OFF_X + c * 16384, &map_q, c * 64, u.head * G, u.seq.q0 + tok0, &bars[XB_XY]);
                tc::tma_load_3d(smem + L::OFF_Y + c * 16384, &map_dy, c * 64, u.head * G, u.seq.q0 + tok0, &bars[XB_XY]);
            }
            int la = 0, lb = 0;
            auto load = [&](const Ring &r, int off, const CUtensorMap *map, int &i, int key) {
                if (!ring_wait_free(r, i, abort_flag)) return false;
                const int s = i % r.n;
                tc::mbar_arrive_expect_tx(&r.full[s], L::TILE);
                for (int c = 0; c < L::KC; ++c)
                    tc::tma_load_3d(smem + off + s * L::TILE + c * 16384, map, c * 64, u.head, u.seq.k0 + key, &r.full[s]);
                ++i;
                return true;
            };
            // keys run one tile ahead of values, as the MMA warp takes them
            bool ok = load(ra, L::OFF_A, &map_k, la, t0 * kXRows);
            for (int i = 0; i < n && ok; ++i) {
                ok = load(rb, L::OFF_B, &map_v, lb, (t0 + i) * kXRows);
                if (ok && i + 1 < n) ok = load(ra, L::OFF_A, &map_k, la, (t0 + i + 1) * kXRows);
            }
            if (!ok) fail();
            bool drained = tc::drain_armed(&bars[XB_XY], 1, kXWaitNs);
            drained = ring_drain(ra, la) && drained;
            drained = ring_drain(rb, lb) && drained;
            if (!drained) fail();
        }
    } else if (warp == 9) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t id_s = tc::idesc_f16(kXRows, kXRows, !kFp16, false, false);
        constexpr uint32_t id_q = tc::idesc_f16(kXRows, D, !kFp16, false, true);
        auto k_in = [&](int i) { return ra.landed(i); };
        auto v_in = [&](int i) { return rb.landed(i); };
        auto issue_s = [&](int i) {
            mma_abt<D, kXRows>(tmem + (i & 1) * 128, sbase + L::OFF_X, sbase + L::OFF_A + i % L::RA * L::TILE, id_s);
            tc::mma_commit_warp(&bars[XB_S + (i & 1)]);
        };
        auto issue_dp = [&](int i) {
            mma_abt<D, kXRows>(tmem + 256, sbase + L::OFF_Y, sbase + L::OFF_B + i % L::RB * L::TILE, id_s);
            tc::mma_commit_warp(&bars[XB_DP]);
            tc::mma_commit_warp(&rb.empty[i % L::RB]);
        };
        bool ok = true;
        if (n > 0) {
            ok = warp_wait(abort_flag, Phase{&bars[XB_XY], 0}, k_in(0));
            tc::tc_fence_after();
            if (ok) issue_s(0);
            ok = ok && warp_wait(abort_flag, v_in(0));
            if (ok) issue_dp(0);
            if (ok && n > 1) {
                ok = warp_wait(abort_flag, k_in(1));
                if (ok) issue_s(1);
            }
        }
        for (int i = 0; i < n && ok; ++i) {
            // the next dP once this one has been read, then this tile's dQ, then the scores two tiles on
            if (i + 1 < n) {
                ok = warp_wait(abort_flag, Phase{&bars[XB_PF], (uint32_t)i & 1u}, v_in(i + 1));
                if (!ok) break;
                tc::tc_fence_after();
                issue_dp(i + 1);
            }
            const Phase ds{&bars[XB_DS], (uint32_t)i & 1u};
            ok = i + 2 < n ? warp_wait(abort_flag, ds, k_in(i + 2)) : warp_wait(abort_flag, ds);
            if (!ok) break;
            const uint32_t kt = L::OFF_A + i % L::RA * L::TILE;
            if (i >= partial) {
                // S(i) has read this tile already (dS(i) follows from it), so its dead rows may go
                const KeyBits<4> kb = key_bits<4>(A.mask, u.seq, (t0 + i) * kXRows, lane);
                if (!kb.all()) zero_rows<L::KC>(smem + kt, kb, lane);
            }
            tc::tc_fence_after();
            mma_ab<kXRows, 64>(tmem + 384, tmem + (i & 1) * 128, sbase + kt, id_q, i > 0);
            tc::mma_commit_warp(&ra.empty[i % L::RA]);
            if (i + 2 < n) issue_s(i + 2);
        }
        if (!ok && lane == 0) fail();
        tc::mma_commit_warp(&bars[XB_ACC]);
        if (!__all_sync(0xffffffffu, tc::mbar_wait_drain(&bars[XB_ACC], 0, kXWaitNs)) && lane == 0) fail();
    }

    const int h = warp >> 2;                             // softmax warps: half of the columns
    const int r = (warp & 3) * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    if (warp < 8 && n > 0) {
        // ------------------------------------------------------ softmax
        const float *st = A.stats + u.tile_id * 256;
        const float c = A.scale_log2, nl = st[r] + up, nd = st[128 + r];
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const uint32_t ts = trow + (i & 1) * 128 + h * 64;
            ok = warp_wait(abort_flag, Phase{&bars[XB_S + (i & 1)], (uint32_t)(i >> 1) & 1u});
            if (!ok) break;
            tc::tc_fence_after();
            // dS over the scores; a copy of its own for tiles with absent keys
            auto tile = [&](auto masked) -> bool {
                float p[64];
                tmem_ld32(ts, reinterpret_cast<uint32_t *>(p));
                tmem_ld32(ts + 32, reinterpret_cast<uint32_t *>(p) + 32);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 64; ++j) p[j] = xex2(fmaf(p[j], c, nl));
                if (!warp_wait(abort_flag, Phase{&bars[XB_DP], (uint32_t)i & 1u})) return false;
                tc::tc_fence_after();
                float y[64];
                tmem_ld32(trow + 256 + h * 64, reinterpret_cast<uint32_t *>(y));
                tmem_ld32(trow + 256 + h * 64 + 32, reinterpret_cast<uint32_t *>(y) + 32);
                tc::tmem_wait_ld();
                tc::tc_fence_before();
                warp_arrive(&bars[XB_PF], lane);           // dP has been read
                KeyBits<4> kb{};
                if constexpr (decltype(masked)::value) kb = key_bits<4>(A.mask, u.seq, (t0 + i) * kXRows, lane);
                uint32_t q[32];
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float a = p[j] * (y[j] + nd), b = p[j + 1] * (y[j + 1] + nd);
                    if constexpr (decltype(masked)::value) {
                        const uint32_t w = h ? kb.w[2 + (j >> 5)] : kb.w[j >> 5];
                        if (!((w >> (j & 31)) & 1u)) a = 0.f;
                        if (!((w >> ((j + 1) & 31)) & 1u)) b = 0.f;
                    }
                    q[j / 2] = xpack<kFp16>(a, b);
                }
                tmem_st32(ts, q);
                tmem_wait_st();
                tc::tc_fence_before();
                warp_arrive(&bars[XB_DS], lane);
                return true;
            };
            ok = i < partial ? tile(std::false_type{}) : tile(std::true_type{});
            if (!ok) break;
        }
        if (ok) ok = warp_wait(abort_flag, Phase{&bars[XB_ACC], 0});
        if (!ok && lane == 0) fail();
        tc::tc_fence_after();
    }

    // ---------------------------------------------------------- epilogue
    const float f = A.scale * (kFp16 ? exp2f(-up) : 1.f);
    auto out = [&](int k) -> uint16_t * {
        const int tok = tok0 + k / G;
        if (k >= A.tpt * G || tok >= cover) return nullptr;
        return A.dq + ((int64_t)(u.seq.q0 + tok) * A.n1 + u.head * G + k % G) * D;
    };
    if (ns == 1) {
        if (warp < 8) {
            uint16_t *dst = out(r);
            const bool pad = n == 0 || tok0 + r / G >= u.seq.qlen;
#pragma unroll
            for (int j = 0; j < D / 2; j += 32) {
                float y[32];
                if (n > 0) {
                    tmem_ld32(trow + 384 + h * (D / 2) + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = pad ? 0.f : y[e] * f;
                if (dst) store_row<kFp16, 32>(dst + h * (D / 2) + j, y);
            }
        }
    } else {
        float *xo = reinterpret_cast<float *>(smem);
        __syncthreads();                                 // loads and products on this memory are complete
        if (warp < 8) {
            const bool pad = n == 0 || tok0 + r / G >= u.seq.qlen;
#pragma unroll
            for (int j = 0; j < D / 2; j += 32) {
                float y[32];
                if (n > 0) {
                    tmem_ld32(trow + 384 + h * (D / 2) + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(xo + r * L::XROW + h * (D / 2) + j + e) =
                        pad ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            }
        }
        cluster_sync();
        if (warp < 8) join_rows<kFp16, D>(xo, kXRows, ns, rank, warp, lane, out, [&](int) { return f; });
        cluster_sync();                                  // peers are done with this CTA's shared memory
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0) A.status[blockIdx.x] = *abort_flag ? SAG_ERR_TIMEOUT : SAG_OK;
}

// ------------------------------------------------------------------ k_xdkv
// TMEM columns: S^T 0 (P^T over it), dP^T 128 (dS^T over it), dV 256, dK 384.
template <bool kFp16, int D>
__global__ void __launch_bounds__(kXThreads, 1)
    k_xdkv(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_dy,
           const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
           const __grid_constant__ XArgs A) {
    using L = BwdSmem<D>;
    constexpr float kShift = kFp16 ? kGradShiftF16 : 0.f;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    const Ring ra = {bars + XB_RING, bars + XB_RING + L::RA, L::RA};
    const Ring rb = {ra.empty + L::RA, ra.empty + L::RA + L::RB, L::RB};
    const Ring rs = {bars + XB_STF, bars + XB_STE, 2};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rb.empty + L::RB);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < XB_RING; ++i)
            tc::mbar_init(&bars[i], i == XB_DS || i == XB_PF || i == XB_STE || i == XB_STE + 1 ? 8 : 1);   // one arrival a warp
        for (int i = 0; i < 2 * (L::RA + L::RB); ++i) tc::mbar_init(&ra.full[i], 1);
        tc::fence_mbar_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 256) {
        tc::prefetch_tmap(&map_q);
        tc::prefetch_tmap(&map_dy);
        tc::prefetch_tmap(&map_k);
        tc::prefetch_tmap(&map_v);
    }
    const int ns = A.nsplit, rank = blockIdx.x % ns;
    const XUnit u = x_decode<&SeqRow::ktile0>(A, blockIdx.x / ns);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot, sbase = tc::smem_u32(smem);
    const int G = A.group, key0 = u.tile * kXRows;
    const int cover = A.s2_pad ? A.s2_pad : u.seq.klen;
    const int nqt = key0 < u.seq.klen ? (u.seq.qlen + A.tpt - 1) / A.tpt : 0;
    const int t0 = (int)((int64_t)nqt * rank / ns), n = (int)((int64_t)nqt * (rank + 1) / ns) - t0;
    float up = 0.f;
    if constexpr (kFp16) {
        up = ds_exponent(A, u.seq, seq_row(A.seq, u.b + 1), u.head, reinterpret_cast<float *>(smem + L::OFF_STAT));
        __syncthreads();                                 // the scratch becomes the ring of statistics
    }
    auto fail = [&]() { *abort_flag = 1; };

    if (warp == 8) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0 && n > 0) {
            if (kFp16) tc::fence_proxy_async_smem();     // the scratch was written by plain stores
            tc::mbar_arrive_expect_tx(&bars[XB_XY], 2 * L::TILE);
            for (int c = 0; c < L::KC; ++c) {
                tc::tma_load_3d(smem + L::OFF_X + c * 16384, &map_k, c * 64, u.head, u.seq.k0 + key0, &bars[XB_XY]);
                tc::tma_load_3d(smem + L::OFF_Y + c * 16384, &map_v, c * 64, u.head, u.seq.k0 + key0, &bars[XB_XY]);
            }
            const uint32_t qbytes = (uint32_t)L::KC * A.tpt * G * 128;
            int la = 0, lb = 0, ls = 0;
            bool ok = true;
            auto load = [&](const Ring &r, int off, const CUtensorMap *map, int &i) {
                if (!ring_wait_free(r, i, abort_flag)) return false;
                const int s = i % r.n;
                tc::mbar_arrive_expect_tx(&r.full[s], qbytes);
                for (int c = 0; c < L::KC; ++c)
                    tc::tma_load_3d(smem + off + s * L::TILE + c * 16384, map, c * 64, u.head * G,
                                    u.seq.q0 + (t0 + i) * A.tpt, &r.full[s]);
                ++i;
                return true;
            };
            for (int i = 0; i < n && ok; ++i) {
                ok = load(ra, L::OFF_A, &map_q, la);
                if (ok) ok = ring_wait_free(rs, i, abort_flag);
                if (!ok) break;
                tc::mbar_arrive_expect_tx(&rs.full[i & 1], 1024);
                bulk_load(smem + L::OFF_STAT + (i & 1) * 1024,
                          A.stats + ((int64_t)(u.seq.qtile0 + t0 + i) * A.n2 + u.head) * 256, 1024, &rs.full[i & 1]);
                ++ls;
                ok = load(rb, L::OFF_B, &map_dy, lb);
            }
            if (!ok) fail();
            bool drained = tc::drain_armed(&bars[XB_XY], 1, kXWaitNs);
            drained = ring_drain(ra, la) && drained;
            drained = ring_drain(rb, lb) && drained;
            drained = ring_drain(rs, ls) && drained;
            if (!drained) fail();
        }
    } else if (warp == 9) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t id_s = tc::idesc_f16(kXRows, kXRows, !kFp16, false, false);
        constexpr uint32_t id_g = tc::idesc_f16(kXRows, D, !kFp16, false, true);
        // rows behind the sequence's (or the tile's) last one are zeroed in a tile that has landed
        auto clear = [&](int off, int s, int i) {
            const int left = u.seq.qlen - (t0 + i) * A.tpt;
            const int live = (left < A.tpt ? left : A.tpt) * G;
            if (live < kXRows) {
                KeyBits<4> kb;
                kb.set_first(live);
                zero_rows<L::KC>(smem + off + s * L::TILE, kb, lane);
            }
            tc::tc_fence_after();
        };
        auto issue_s = [&](int i) {
            clear(L::OFF_A, i % L::RA, i);
            mma_abt<D, kXRows>(tmem, sbase + L::OFF_X, sbase + L::OFF_A + (i % L::RA) * L::TILE, id_s);
            tc::mma_commit_warp(&bars[XB_S]);
        };
        auto issue_dp = [&](int i) {
            clear(L::OFF_B, i % L::RB, i);
            mma_abt<D, kXRows>(tmem + 128, sbase + L::OFF_Y, sbase + L::OFF_B + (i % L::RB) * L::TILE, id_s);
            tc::mma_commit_warp(&bars[XB_DP]);
        };
        bool ok = true;
        if (n > 0) {
            ok = warp_wait(abort_flag, Phase{&bars[XB_XY], 0}, ra.landed(0));
            if (ok) issue_s(0);
            ok = ok && warp_wait(abort_flag, rb.landed(0));
            if (ok) issue_dp(0);
        }
        for (int i = 0; i < n && ok; ++i) {
            const Phase p{&bars[XB_PF], (uint32_t)i & 1u}, ds{&bars[XB_DS], (uint32_t)i & 1u};
            const bool more = i + 1 < n;
            ok = more ? warp_wait(abort_flag, p, ra.landed(i + 1)) : warp_wait(abort_flag, p);
            if (!ok) break;
            tc::tc_fence_after();
            mma_ab<kXRows, 64>(tmem + 256, tmem, sbase + L::OFF_B + (i % L::RB) * L::TILE, id_g, i > 0);
            tc::mma_commit_warp(&rb.empty[i % L::RB]);
            if (more) issue_s(i + 1);
            ok = more ? warp_wait(abort_flag, ds, rb.landed(i + 1)) : warp_wait(abort_flag, ds);
            if (!ok) break;
            tc::tc_fence_after();
            mma_ab<kXRows, 64>(tmem + 384, tmem + 128, sbase + L::OFF_A + (i % L::RA) * L::TILE, id_g, i > 0);
            tc::mma_commit_warp(&ra.empty[i % L::RA]);
            if (more) issue_dp(i + 1);
        }
        if (!ok && lane == 0) fail();
        tc::mma_commit_warp(&bars[XB_ACC]);
        if (!__all_sync(0xffffffffu, tc::mbar_wait_drain(&bars[XB_ACC], 0, kXWaitNs)) && lane == 0) fail();
    }

    const int h = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                // key = TMEM lane
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    if (warp < 8 && n > 0) {
        // ------------------------------------------------------ softmax
        const float c = A.scale_log2;
        const bool live = key0 + r < u.seq.klen && (!A.mask || A.mask[(int64_t)u.seq.k0 + key0 + r]);
        const float k = kFp16 ? exp2f(up - kShift) : 1.f;
        // One query tile; a copy of its own for key tiles with absent keys.
        auto tile = [&](auto masked, int i) -> bool {
            constexpr bool kMasked = decltype(masked)::value;
            const float4 *st = reinterpret_cast<const float4 *>(smem + L::OFF_STAT + (i & 1) * 1024) + h * 16;
            float p[64];
            tmem_ld32(trow + h * 64, reinterpret_cast<uint32_t *>(p));
            tmem_ld32(trow + h * 64 + 32, reinterpret_cast<uint32_t *>(p) + 32);
            tc::tmem_wait_ld();
            uint32_t q[32];
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
                const float4 nl4 = st[j / 4];
                const float nl[4] = {nl4.x, nl4.y, nl4.z, nl4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = fmaf(p[j + e], c, nl[e]);
                    if (kFp16) x += kShift;
                    p[j + e] = xex2(x);
                    if (kMasked && !live) p[j + e] = 0.f;
                }
                q[j / 2] = xpack<kFp16>(p[j], p[j + 1]);
                q[j / 2 + 1] = xpack<kFp16>(p[j + 2], p[j + 3]);
            }
            tmem_st32(trow + h * 64, q);
            tmem_wait_st();
            tc::tc_fence_before();
            warp_arrive(&bars[XB_PF], lane);
            if (!warp_wait(abort_flag, Phase{&bars[XB_DP], (uint32_t)i & 1u})) return false;
            tc::tc_fence_after();
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                float y[32];
                tmem_ld32(trow + 128 + h * 64 + g * 32, reinterpret_cast<uint32_t *>(y));
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 nd4 = st[32 + (g * 32 + j) / 4];
                    const float nd[4] = {nd4.x, nd4.y, nd4.z, nd4.w};
                    float a[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        a[e] = y[j + e] + nd[e];
                        if (kFp16) a[e] *= k;
                        a[e] *= p[g * 32 + j + e];
                        if (kMasked && !live) a[e] = 0.f;
                    }
                    q[(g * 32 + j) / 2] = xpack<kFp16>(a[0], a[1]);
                    q[(g * 32 + j) / 2 + 1] = xpack<kFp16>(a[2], a[3]);
                }
            }
            tmem_st32(trow + 128 + h * 64, q);
            tmem_wait_st();
            tc::tc_fence_before();
            warp_arrive(&bars[XB_DS], lane);
            if (lane == 0) tc::mbar_arrive(&rs.empty[i & 1]);
            return true;
        };
        const bool all = __all_sync(0xffffffffu, live);
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            ok = warp_wait(abort_flag, rs.landed(i), Phase{&bars[XB_S], (uint32_t)i & 1u});
            if (!ok) break;
            tc::tc_fence_after();
            ok = all ? tile(std::false_type{}, i) : tile(std::true_type{}, i);
        }
        if (ok) ok = warp_wait(abort_flag, Phase{&bars[XB_ACC], 0});
        if (!ok && lane == 0) fail();
        tc::tc_fence_after();
    }

    // ---------------------------------------------------------- epilogue: warps 0-3 dV, warps 4-7 dK
    const float fv = kFp16 ? exp2f(-kShift) : 1.f, fk = A.scale * (kFp16 ? exp2f(-up) : 1.f);
    auto out = [&](int k) -> uint16_t * {
        const int key = key0 + k % kXRows;
        if (key >= cover) return nullptr;
        return (k < kXRows ? A.dv : A.dk) + (((int64_t)u.seq.k0 + key) * A.n2 + u.head) * D;
    };
    if (ns == 1) {
        if (warp < 8) {
            uint16_t *dst = out(h * kXRows + r);
            const float f = h ? fk : fv;
#pragma unroll
            for (int j = 0; j < D; j += 32) {
                float y[32];
                if (n > 0) {
                    tmem_ld32(trow + 256 + h * 128 + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = n > 0 ? y[e] * f : 0.f;
                if (dst) store_row<kFp16, 32>(dst + j, y);
            }
        }
    } else {
        float *xo = reinterpret_cast<float *>(smem);
        __syncthreads();                                 // loads and products on this memory are complete
        if (warp < 8) {
#pragma unroll
            for (int j = 0; j < D; j += 32) {
                float y[32];
                if (n > 0) {
                    tmem_ld32(trow + 256 + h * 128 + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(xo + (h * kXRows + r) * L::XROW + j + e) =
                        n > 0 ? make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        cluster_sync();
        if (warp < 8)
            join_rows<kFp16, D>(xo, 2 * kXRows, ns, rank, warp, lane, out, [&](int k) { return k < kXRows ? fv : fk; });
        cluster_sync();                                  // peers are done with this CTA's shared memory
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

struct BwdMaps {
    CUtensorMap q, dy, k, v;
};
bool maps(BwdMaps *m, const XArgs &a, const sca_io &io, const sca_desc &d) {
    return x_map_q(&m->q, io.query, d, a, d.q_stride, io.key) && x_map_q(&m->dy, io.attention_out_grad, d, a, 0, io.key) &&
           x_map_k(&m->k, io.key, io.query, d, d.k_stride, kXRows) &&
           x_map_k(&m->v, io.value, io.query, d, d.v_stride, kXRows);
}

template <bool kFp16, int D>
cudaError_t launch(const XArgs &a, const sca_io &io, const sca_desc &d, bool dkv, int units, cudaStream_t s) {
    BwdMaps m;
    if (!maps(&m, a, io, d)) return cudaErrorInvalidValue;
    return x_launch(dkv ? k_xdkv<kFp16, D> : k_xdq<kFp16, D>, units * a.nsplit, kXThreads, a.nsplit, BwdSmem<D>::TOTAL, s, m.q, m.dy,
                    m.k, m.v, a);
}

}  // namespace

cudaError_t launch_xpre(const XArgs &a, bool fp16, int d, cudaStream_t s) {
    const int64_t ctas = (int64_t)a.q_tiles * a.n2 + (fp16 ? (int64_t)a.k_tiles * a.n2 : 0);
    if (ctas == 0) return cudaSuccess;
    if (d == 128) {
        if (fp16) k_xpre<true, 128><<<(unsigned)ctas, 256, 0, s>>>(a);
        else k_xpre<false, 128><<<(unsigned)ctas, 256, 0, s>>>(a);
    } else {
        if (fp16) k_xpre<true, 64><<<(unsigned)ctas, 256, 0, s>>>(a);
        else k_xpre<false, 64><<<(unsigned)ctas, 256, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_xdq(const XArgs &a, const sca_io &io, const sca_desc &d, int units, cudaStream_t s) {
    const bool fp16 = d.dtype == SAG_FP16;
    if (d.d == 128) return fp16 ? launch<true, 128>(a, io, d, false, units, s) : launch<false, 128>(a, io, d, false, units, s);
    return fp16 ? launch<true, 64>(a, io, d, false, units, s) : launch<false, 64>(a, io, d, false, units, s);
}

cudaError_t launch_xdkv(const XArgs &a, const sca_io &io, const sca_desc &d, int units, cudaStream_t s) {
    const bool fp16 = d.dtype == SAG_FP16;
    if (d.d == 128) return fp16 ? launch<true, 128>(a, io, d, true, units, s) : launch<false, 128>(a, io, d, true, units, s);
    return fp16 ? launch<true, 64>(a, io, d, true, units, s) : launch<false, 64>(a, io, d, true, units, s);
}

}  // namespace sag
