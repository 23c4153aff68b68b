// Cross and windowed attention, gradient: three launches (four for windows in
// fp16, window_bwd.cu), no fp32 accumulators in memory (but for the sums of a cut
// unit's pieces), no atomics but a maximum, tickets and counters, so the same bits
// on every run.
//
//   k_xpre  Delta = rowsum(dY * O) and lse in log2 units, packed by query tile; zeros for absent states
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
// powers of two first (cross.cuh), so that neither a loss scale overflows nor a
// long softmax vanishes.  |dP - Delta| <= 2 |dY| max|V| gives the one of dS.  In
// k_xdq each query row has its own, from its dY: with one for the sequence, rows
// of small dY lost their bits to subnormals (30000 states, dY 2^-18 of the
// largest: dQ off by 12 %, now by 0.03 %; 1500 states: 0.6 %).  k_xdkv sums over
// the rows of a sequence, where the largest count most, and takes one exponent
// from the largest |dY|.  In a window the largest row need not be in a key's sum,
// nor the largest V in a row's: there each key and each query row has its own
// exponent, from what its window joins (k_wscale).
//
// A CTA (one per SM) walks over units, so that the next unit's tiles land and
// its first products run beside the last one's stores.  Few units: a cluster's
// CTAs split one unit's loop and join their accumulators through distributed
// shared memory, in rank order.  More: the units beyond full rounds of the SMs
// are cut into pieces, joined through the workspace in their order.  (Clusters
// there cost 2269 us against 2271 without and 2100 with pieces for the gradient
// below: a cluster's CTAs cannot take unit after unit.)
//
// Measured on one GB300, 2 x 8192 x 4096 tokens, 32 heads of 128 (bf16): k_xpre 50
// us (5.3 TB/s), k_xdq 906 us (the tensor pipe 75 % active), k_xdkv 1130 us (80 %):
// 1840 TFLOP/s of products, 0.92 of the measured bf16 rate (2000); call after call,
// at the power limit, 2.2 to 2.3 ms.
// 64-wide heads: 1530 us for the same tokens; a thread's chain of a tile bounds it
// (16 softmax warps of 32 columns instead of 8 of 64: 1620 us, 136 -> 150 us for
// 4 x 1000 x 1290 masked tokens).
#pragma once

#include <type_traits>

#include "cross.cuh"
#include "kernels.cuh"
#include "xtmap.cuh"

namespace sag {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ k_xpre
// kScaled: fp16 of windows, whose norms k_wscale takes
template <bool kFp16, int D, bool kScaled>
__global__ void __launch_bounds__(256) k_xpre(const __grid_constant__ XArgs A) {
    constexpr int LPR = D / 8;                           // lanes a row, 16 bytes each
    constexpr int RPW = 32 / LPR;
    constexpr int STEP = 8 * RPW, AHEAD = 4;             // rows of a step of the block, steps whose loads are in flight
    __shared__ float2 red[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = lane % LPR;
    if (blockIdx.x == 0) {
        if (threadIdx.x < 2) A.ticket[threadIdx.x] = 0;
        for (int i = threadIdx.x; i < A.n_arrived; i += 256) A.arrived[i] = 0;
    }
    grid_next();
    const int q_units = A.q_tiles * A.n2;
    float top = 0.f, far = 0.f;                          // largest squared norm, and |Delta|
    int64_t slot, tile_id;
    if ((int)blockIdx.x < q_units) {
        const XUnit u = x_decode<&SeqRow::qtile0>(A, blockIdx.x);
        slot = ((int64_t)u.b * A.n2 + u.head) * 2;
        tile_id = u.tile_id;
        float *st = A.stats + u.tile_id * 256;
        int r = warp * RPW + lane / LPR, tok = r / A.group, h = r - tok * A.group;
        const int step_tok = STEP / A.group, step_h = STEP - step_tok * A.group;
        const int row0 = u.seq.q0 + u.tile * A.tpt, most = min(A.tpt, u.seq.qlen - u.tile * A.tpt);
#pragma unroll
        for (int done = 0; done < kXRows / STEP; done += AHEAD) {
            uint4 a[AHEAD], b[AHEAD];
            float lses[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                a[k] = b[k] = make_uint4(0, 0, 0, 0);
                lses[k] = -INFINITY;
                if (tok < most) {
                    const int64_t row = (int64_t)(row0 + tok) * A.n1 + u.head * A.group + h;
                    a[k] = *reinterpret_cast<const uint4 *>(A.o_in + row * D + part * 8);
                    b[k] = *reinterpret_cast<const uint4 *>(A.dy + row * D + part * 8);
                    lses[k] = A.lse[row];
                }
                tok += step_tok;
                h += step_h;
                if (h >= A.group) {
                    h -= A.group;
                    ++tok;
                }
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const uint32_t *pa = &a[k].x, *pb = &b[k].x;
                float dot = 0.f, nrm = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y0 = u16_to_f<kFp16>((uint16_t)pb[i]), y1 = u16_to_f<kFp16>((uint16_t)(pb[i] >> 16));
                    dot += u16_to_f<kFp16>((uint16_t)pa[i]) * y0 + u16_to_f<kFp16>((uint16_t)(pa[i] >> 16)) * y1;
                    nrm += y0 * y0 + y1 * y1;
                }
#pragma unroll
                for (int o = LPR / 2; o; o >>= 1) {
                    dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    if constexpr (kFp16) nrm += __shfl_xor_sync(0xffffffffu, nrm, o);
                }
                if (part == 0) {
                    const bool some = lses[k] != -INFINITY;
                    st[r] = some ? -lses[k] * kLog2e : -INFINITY;   // makes P = 0 where there is nothing
                    st[128 + r] = some ? -dot : 0.f;
                    if constexpr (kFp16) A.row_norms[u.tile_id * kXRows + r] = nrm;
                }
                if (nrm < INFINITY) top = fmaxf(top, nrm);
                if (kScaled && fabsf(dot) < INFINITY) far = fmaxf(far, fabsf(dot));
                r += STEP;
            }
        }
    } else {
        // zeros for the gradients of absent states; fp16: row norms of V
        const XUnit u = x_decode<&SeqRow::ktile0>(A, blockIdx.x - q_units);
        slot = ((int64_t)u.b * A.n2 + u.head) * 2 + 1;
        tile_id = u.tile_id;
        const int cover = A.s2_pad ? A.s2_pad : u.seq.klen;
#pragma unroll
        for (int done = 0; done < kXRows / STEP; done += AHEAD) {
            uint4 a[AHEAD];
            bool there[AHEAD];
            const int key0 = u.tile * kXRows + done * STEP + warp * RPW + lane / LPR;
            const int64_t row0 = (int64_t)u.seq.k0 + key0;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                there[k] = key0 + k * STEP < u.seq.klen && (!A.mask || A.mask[row0 + k * STEP]);
            if constexpr (kFp16) {
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    a[k] = make_uint4(0, 0, 0, 0);
                    if (there[k])
                        a[k] = *reinterpret_cast<const uint4 *>(A.v_in + (row0 + k * STEP) * A.v_stride + u.head * D + part * 8);
                }
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (!there[k] && key0 + k * STEP < cover) {
                    const int64_t at = ((row0 + k * STEP) * A.n2 + u.head) * D + part * 8;
                    *reinterpret_cast<uint4 *>(A.dk + at) = *reinterpret_cast<uint4 *>(A.dv + at) = make_uint4(0, 0, 0, 0);
                }
                if constexpr (kFp16) {
                    float nrm = 0.f;
                    const uint32_t *pa = &a[k].x;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float y0 = u16_to_f<kFp16>((uint16_t)pa[i]), y1 = u16_to_f<kFp16>((uint16_t)(pa[i] >> 16));
                        nrm += y0 * y0 + y1 * y1;
                    }
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) nrm += __shfl_xor_sync(0xffffffffu, nrm, o);
                    if (nrm < INFINITY) top = fmaxf(top, nrm);
                    if (kScaled && part == 0)
                        A.key_norms[u.tile_id * kXRows + key0 - u.tile * kXRows + k * STEP] = nrm;
                }
            }
        }
    }
    if constexpr (kFp16) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if constexpr (kScaled) far = fmaxf(far, __shfl_xor_sync(0xffffffffu, far, o));
        }
        if (lane == 0) red[warp] = make_float2(top, far);
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < 8; ++i) {
                top = fmaxf(top, red[i].x);
                far = fmaxf(far, red[i].y);
            }
            if constexpr (kScaled) ((int)blockIdx.x < q_units ? A.q_tops : A.k_tops)[tile_id] = make_float2(top, far);
            else atomicMax(A.norms + slot, __float_as_uint(top));   // a maximum does not depend on the order
        }
    }
}

// fp16: exponent e such that 2^e |dS| <= 2^15 for every |dS| <= bound, or for every dS of rows of dY and V whose largest
// squared norms are given.
__device__ __forceinline__ float ds_exponent(float bound) {
    if (!(bound > 0.f) || !(bound < INFINITY)) return 0.f;
    return fminf(fmaxf(14.f - (float)ilogbf(bound), -40.f), 40.f);
}
__device__ __forceinline__ float ds_exponent(float dy, float v) { return ds_exponent(2.f * sqrtf(dy) * sqrtf(v)); }
__device__ __forceinline__ float2 ds_norms(const XArgs &A, int b, int head) {
    return *reinterpret_cast<const float2 *>(A.norms + ((int64_t)b * A.n2 + head) * 2);
}

// ------------------------------------------------------------------- shared
// Resident tiles (X, Y) of a unit and two rings: tiles that live long (A: keys in k_xdq, queries in k_xdkv) and tiles that one
// product reads (B: values, or output gradients, which two read).
template <int D>
struct BwdSmem {
    static constexpr int KC = D / 64;
    static constexpr int TILE = KC * 16384;
    static constexpr int RA = D == 128 ? 3 : 4, RB = D == 128 ? 2 : 4;
    static constexpr int RX = D == 128 ? 1 : 2;          // pairs of resident tiles: the next unit's land early (1588 -> 1540 us)
    static constexpr int OFF_Y = TILE, OFF_A = RX * 2 * TILE, OFF_B = OFF_A + RA * TILE;
    static constexpr int OFF_STAT = OFF_B + RB * TILE;   // k_xdkv: [2][256] floats
    static constexpr int OFF_BAR = OFF_STAT + 2048;
    static constexpr int TOTAL = OFF_BAR + 512;
    static constexpr int XROW = D + 4;
    static_assert(2 * kXRows * XROW * 4 <= OFF_STAT, "the exchange overlays the tiles");
    static_assert(TOTAL <= 227 * 1024, "shared memory of one CTA");
    // 512 bytes behind OFF_BAR: barriers, TMEM address, abort flag; from 320 on the two slots of units
};
// barriers; XB_XYE: the resident tiles may be overwritten; XB_UF, XB_UE: units handed out; XB_DS: two in k_xdq, where the
// softmax warps may be done with the next tile before the MMA warp looks for this one (modelled in the tests)
enum {
    XB_XY = 0, XB_XYE = XB_XY + 2, XB_S = XB_XYE + 2, XB_DP = XB_S + 2, XB_PF, XB_DS, XB_ACC = XB_DS + 2,
    XB_STF, XB_STE = XB_STF + 2, XB_UF = XB_STE + 2, XB_UE = XB_UF + 2, XB_RING = XB_UE + 2
};
// arrivals that complete a phase: one a softmax warp; every reader's for the units; one of everything else
__device__ __forceinline__ int bwd_arrivals(int i) {
    return i == XB_PF || i == XB_DS || i == XB_DS + 1 || i == XB_STE || i == XB_STE + 1 ? 8 : i == XB_UE || i == XB_UE + 1 ? 9 : 1;
}

// A unit as its roles need it, in shared memory.
struct alignas(16) Work {
    SeqRow seq;
    int32_t b, head;
    int32_t first;                      // k_xdq: first token, k_xdkv: first key, within the sequence
    int32_t t0, n;                      // this rank's first tile of the loop and their number; n < 0: no more units
    int32_t stat;                       // (tile of all sequences) * n2 + head
    int32_t piece;                      // number of the piece; -1: a whole unit, or a cluster's
    // windowed: first key of the loop's first tile (k_xdq), and the tiles [f0, f1) of this share that no window's edge crosses
    int32_t base, f0, f1;
};

// Work item -> unit, and the share of its loop.
struct Item {
    int unit, rank, ranks, piece;
    __device__ __forceinline__ Item(const XArgs &A, int item, int rank_, int ranks_)
        : unit(item), rank(rank_), ranks(ranks_), piece(-1) {
        if (item >= A.full) {
            piece = item - A.full;
            unit = A.full + piece / A.pieces;
            rank = piece % A.pieces;
            ranks = A.pieces;
        }
    }
    // of a loop of `tiles`; a piece always has some (only units of long, alike loops are cut), but for windowed attention,
    // whose units differ
    __device__ __forceinline__ void share(int tiles, Work *w) const {
        x_share(tiles, rank, ranks, &w->t0, &w->n);
        w->piece = piece;
    }
};

// A piece's sums: a thread's 32-bit accumulators of COLS columns go to the workspace; of each warp's rows, the warp that
// arrives last adds all pieces up in their order, so the order of arrival does not show in the result.
template <int COLS>
struct Pieces {
    float4 *mine;                       // [piece][warp][COLS / 4][lane]
    unsigned *arrived;
    int pieces, rank;
    __device__ __forceinline__ Pieces(const XArgs &A, int piece, int warp, int lane)
        : mine(reinterpret_cast<float4 *>(A.parts) + ((int64_t)piece * 8 + warp) * (COLS * 8) + lane),
          arrived(A.arrived + piece / A.pieces * 8 + warp), pieces(A.pieces), rank(piece % A.pieces) {}
    __device__ __forceinline__ void put(int j, const float *y) const {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            __stcg(mine + (j / 4 + e) * 32, make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]));
    }
    __device__ __forceinline__ bool last(int lane) const {
        __threadfence();
        __syncwarp();
        unsigned before = 0;
        if (lane == 0) before = atomicAdd(arrived, 1u);
        before = __shfl_sync(0xffffffffu, before, 0);
        __threadfence();
        return before + 1 == (unsigned)pieces;
    }
    __device__ __forceinline__ void sum(int j, float *y) const {
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = 0.f;
        const float4 *p = mine - (int64_t)rank * 8 * (COLS * 8) + j / 4 * 32;
        for (int k = 0; k < pieces; ++k, p += 8 * (COLS * 8)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float4 v = __ldcg(p + e * 32);
                y[4 * e] += v.x;
                y[4 * e + 1] += v.y;
                y[4 * e + 2] += v.z;
                y[4 * e + 3] += v.w;
            }
        }
    }
};

// Units of a CTA, one after the other: the first by its number, the others from a ticket counter, since units differ (short
// sequences, masked and padding tiles) and a fixed order left SMs idle: 142 us against 101 for k_xdkv of a padded batch.
// The producer takes and decodes a unit when it has issued the loads of the one before, and hands it to the MMA and softmax
// warps through two slots.  A split unit is its cluster's only one.
struct Units {
    Work *slot;
    uint64_t *full, *empty;
    // one thread; false: timeout
    template <class Decode>
    __device__ __forceinline__ bool take(const XArgs &A, int k, volatile int *abort, Work *w, Decode &&decode) const {
        if (k >= 2 && !tc::mbar_wait(&empty[k & 1], (k / 2 - 1) & 1, abort, kXWaitNs)) return false;
        int item = A.items;
        if (k == 0) item = blockIdx.x / A.nsplit;
        else if (A.ctas < A.items) item = (int)(gridDim.x + atomicAdd(A.ticket, 1u));
        if (item < A.items) *w = decode(item);
        else w->n = -1;
        slot[k & 1] = *w;
        tc::mbar_arrive(&full[k & 1]);
        return true;
    }
    // a warp; false: timeout
    __device__ __forceinline__ bool read(int k, volatile int *abort, int lane, Work *w) const {
        if (!warp_wait(abort, Phase{&full[k & 1], (uint32_t)(k >> 1) & 1u})) return false;
        *w = slot[k & 1];
        warp_arrive(&empty[k & 1], lane);
        return true;
    }
};

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

// Joins the ranks' partial accumulators: 128 rows of D columns each, in xo[row][XROW] of every rank; row k of this
// rank's share goes to dst + out(k) (negative: not stored), scaled by f.
template <bool kFp16, int D, class Out>
__device__ __forceinline__ void join_rows(float *xo, uint16_t *dst, int ns, int rank, int warp, int lane, Out &&out, float f) {
    constexpr int E = D / 64, R = 2;                     // float2 a lane and row; rows at a time, for the remote reads' latency
    for (int k0 = rank + ns * warp; k0 < kXRows; k0 += ns * 8 * R) {
        float2 y[R][kMaxSplit][E];
        int64_t at[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int k = k0 + i * ns * 8;
            at[i] = k < kXRows ? out(k) : -1;
            if (at[i] < 0) continue;
#pragma unroll
            for (int p = 0; p < kMaxSplit; ++p)
                if (p < ns) {
                    const uint32_t a = peer_addr(tc::smem_u32(xo + k * (D + 4) + lane * 2), p);
#pragma unroll
                    for (int e = 0; e < E; ++e) y[i][p][e] = peer_ld2(a + e * 256);
                }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (at[i] < 0) continue;
            float2 acc[E] = {};
#pragma unroll
            for (int p = 0; p < kMaxSplit; ++p)
                if (p < ns)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = add2(acc[e], y[i][p][e]);
#pragma unroll
            for (int e = 0; e < E; ++e)
                *reinterpret_cast<uint32_t *>(dst + at[i] + e * 64 + lane * 2) = xpack<kFp16>(acc[e].x * f, acc[e].y * f);
        }
    }
}

// ------------------------------------------------------------------- k_xdq
// TMEM columns: S of even / odd key tiles at 0 / 128 (dS over them, the second half of K 64 columns on), dP 256, dQ 384.
// Tiles are counted through all units (g): buffers and phases follow the count.
template <bool kFp16, int D, bool kBand>
__global__ void __launch_bounds__(kXThreads, 1)
    k_xdq(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_dy,
          const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
          const __grid_constant__ XArgs A) {
    using L = BwdSmem<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    const Ring rx = {bars + XB_XY, bars + XB_XYE, L::RX};
    const Ring ra = {bars + XB_RING, bars + XB_RING + L::RA, L::RA};
    const Ring rb = {ra.empty + L::RA, ra.empty + L::RA + L::RB, L::RB};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rb.empty + L::RB);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const Units units = {reinterpret_cast<Work *>(smem + L::OFF_BAR + 320), bars + XB_UF, bars + XB_UE};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < XB_RING + 2 * (L::RA + L::RB); ++i) tc::mbar_init(&bars[i], bwd_arrivals(i));
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
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot, sbase = tc::smem_u32(smem);
    if (!kBand || !A.late) grid_wait();                  // statistics and tickets of the kernel before
    const int ns = A.nsplit, rank = blockIdx.x % ns;
    const int G = A.group;
    grid_next();
    auto fail = [&]() { *abort_flag = 1; };
    auto first_key = [&](const Work &w, int i) { return kBand ? w.base + i * kXRows : (w.t0 + i) * kXRows; };
    auto decode = [&](int number) {
        const Item item(A, number, rank, ns);
        const XUnit u = x_decode<&SeqRow::qtile0, kBand ? kDown : kByHead>(A, item.unit);
        Work w{};
        w.seq = u.seq;
        w.b = u.b;
        w.head = u.head;
        w.first = u.tile * A.tpt;
        w.stat = (int32_t)u.tile_id;
        if constexpr (kBand) {
            const BandKeys band = BandKeys::of<kXRows, false>(A, u.seq, w.first);
            item.share(band.tiles, &w);
            w.base = band.base + w.t0 * kXRows;
            w.f0 = band.f0 - w.t0;
            w.f1 = band.f1 - w.t0;
        } else {
            item.share(w.first < u.seq.qlen ? (u.seq.klen + kXRows - 1) / kXRows : 0, &w);
        }
        return w;
    };

    if (warp == 8) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            const uint32_t qbytes = (uint32_t)L::KC * A.tpt * G * 128;
            int la = 0, lb = 0, lx = 0;                  // loads so far
            bool ok = true;
            for (int k = 0; ok; ++k) {
                Work w{};
                ok = units.take(A, k, abort_flag, &w, decode);
                if (!ok || w.n < 0) break;
                if (w.n == 0) continue;
                auto load = [&](const Ring &r, int off, const CUtensorMap *map, int &i, int key) {
                    if (!ring_wait_free(r, i, abort_flag)) return false;
                    const int s = i % r.n;
                    tc::mbar_arrive_expect_tx(&r.full[s], L::TILE);
                    for (int c = 0; c < L::KC; ++c)
                        tc::tma_load_3d(smem + off + s * L::TILE + c * 16384, map, c * 64, w.head, w.seq.k0 + key,
                                        &r.full[s]);
                    ++i;
                    return true;
                };
                ok = ring_wait_free(rx, lx, abort_flag);
                if (!ok) break;
                const int x = lx % L::RX;
                tc::mbar_arrive_expect_tx(&rx.full[x], 2 * qbytes);
                for (int c = 0; c < L::KC; ++c) {
                    const int row = w.seq.q0 + w.first;
                    tc::tma_load_3d(smem + x * 2 * L::TILE + c * 16384, &map_q, c * 64, w.head * G, row, &rx.full[x]);
                    tc::tma_load_3d(smem + x * 2 * L::TILE + L::OFF_Y + c * 16384, &map_dy, c * 64, w.head * G, row, &rx.full[x]);
                }
                ++lx;
                // keys run one tile ahead of values, as the MMA warp takes them
                ok = load(ra, L::OFF_A, &map_k, la, first_key(w, 0));
                for (int i = 0; i < w.n && ok; ++i) {
                    ok = load(rb, L::OFF_B, &map_v, lb, first_key(w, i));
                    if (ok && i + 1 < w.n) ok = load(ra, L::OFF_A, &map_k, la, first_key(w, i + 1));
                }
            }
            if (!ok) fail();
            bool drained = ring_drain(rx, lx);
            drained = ring_drain(ra, la) && drained;
            drained = ring_drain(rb, lb) && drained;
            if (!drained) fail();
        }
    } else if (warp == 9) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t id_s = tc::idesc_f16(kXRows, kXRows, !kFp16, false, false);
        constexpr uint32_t id_q = tc::idesc_f16(kXRows, D, !kFp16, false, true);
        bool ok = true;
        int g = 0, nonempty = 0;
        auto resident = [&]() { return sbase + nonempty % L::RX * 2 * L::TILE; };
        auto issue_s = [&](int g) {
            mma_abt<D, kXRows>(tmem + (g & 1) * 128, resident(), sbase + L::OFF_A + g % L::RA * L::TILE, id_s);
            tc::mma_commit_warp(&bars[XB_S + (g & 1)]);
        };
        auto issue_dp = [&](int g) {
            mma_abt<D, kXRows>(tmem + 256, resident() + L::OFF_Y, sbase + L::OFF_B + g % L::RB * L::TILE, id_s);
            tc::mma_commit_warp(&bars[XB_DP]);
            tc::mma_commit_warp(&rb.empty[g % L::RB]);
        };
        for (int k = 0; ok; ++k) {
            Work w;
            ok = units.read(k, abort_flag, lane, &w);
            if (!ok || w.n < 0) break;
            const int n = w.n;
            if (n == 0) continue;
            ok = warp_wait(abort_flag, rx.landed(nonempty), ra.landed(g));
            if (!ok) break;
            tc::tc_fence_after();
            issue_s(g);
            ok = warp_wait(abort_flag, rb.landed(g));
            if (!ok) break;
            issue_dp(g);
            if (n > 1) {
                ok = warp_wait(abort_flag, ra.landed(g + 1));
                if (!ok) break;
                issue_s(g + 1);
            } else {
                tc::mma_commit_warp(&rx.empty[nonempty % L::RX]);
            }
            for (int i = 0; i < n; ++i, ++g) {
                // the next dP once this one has been read, then this tile's dQ, then the scores two tiles on
                if (i + 1 < n) {
                    ok = warp_wait(abort_flag, Phase{&bars[XB_PF], (uint32_t)g & 1u}, rb.landed(g + 1));
                    if (!ok) break;
                    tc::tc_fence_after();
                    issue_dp(g + 1);
                    if (i + 2 == n) tc::mma_commit_warp(&rx.empty[nonempty % L::RX]);
                }
                const Phase ds{&bars[XB_DS + (g & 1)], (uint32_t)(g >> 1) & 1u};
                ok = i + 2 < n ? warp_wait(abort_flag, ds, ra.landed(g + 2)) : warp_wait(abort_flag, ds);
                if (!ok) break;
                const uint32_t kt = L::OFF_A + g % L::RA * L::TILE;
                tc::tc_fence_after();
                mma_ab<kXRows, 64>(tmem + 384, tmem + (g & 1) * 128, sbase + kt, id_q, i > 0);
                tc::mma_commit_warp(&ra.empty[g % L::RA]);
                if (i + 2 < n) issue_s(g + 2);
            }
            if (!ok) break;
            tc::mma_commit_warp(&bars[XB_ACC]);
            ++nonempty;
        }
        if (!ok && lane == 0) fail();
        // every MMA issued must be complete before TMEM is freed: one more phase of XB_ACC
        if (!ok) tc::mma_commit_warp(&bars[XB_ACC]);
        const int phases = nonempty + (ok ? 0 : 1);
        if (!__all_sync(0xffffffffu, tc::drain_armed(&bars[XB_ACC], phases, kXWaitNs)) && lane == 0) fail();
    }

    const int h = warp >> 2;                             // softmax warps: half of the columns
    const int r = (warp & 3) * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    Work w{};
    float up = 0.f;                                      // exponent that the row's dS is scaled by
    auto place = [&](int tok_in, int head_in) -> int64_t {   // place of a row (token and head in the tile) in dQ
        const int tok = w.first + tok_in;
        if (tok_in >= A.tpt || tok >= (A.s1_pad ? A.s1_pad : w.seq.qlen)) return -1;
        return ((int64_t)(w.seq.q0 + tok) * A.n1 + w.head * G + head_in) * D;
    };
    auto out = [&](int k) { return place(k / G, k % G); };
    const int my_tok = r / G, my_head = r % G;
    if (warp < 8) {
        bool ok = true;
        int g = 0, nonempty = 0;
        // the next unit's statistics are on their way while this one is stored
        float st_nl = 0.f, st_nd = 0.f;
        float2 norms{};
        auto begin = [&](int k) {
            ok = units.read(k, abort_flag, lane, &w);
            if (!ok || w.n < 0) return;
            st_nl = A.stats[(int64_t)w.stat * 256 + r];
            st_nd = A.stats[(int64_t)w.stat * 256 + 128 + r];
            if constexpr (kFp16 && kBand) norms.x = A.q_up[(int64_t)w.stat * kXRows + r];
            else if constexpr (kFp16)
                norms = make_float2(A.row_norms[(int64_t)w.stat * kXRows + r], ds_norms(A, w.b, w.head).y);
        };
        begin(0);
        for (int k = 0; ok && w.n >= 0; ++k) {
            const int n = w.n;
            if constexpr (kFp16) up = kBand ? norms.x : ds_exponent(norms.x, norms.y);
            const float nl = st_nl + up, nd = st_nd;
            if (n > 0) {
                // ---------------------------------------------- softmax
                const float c = A.scale_log2;
                // tiles from `whole` on, before `partial`, lack no key
                const int whole = kBand ? w.f0 : 0;
                const int partial = A.mask ? 0 : kBand ? w.f1 : w.seq.klen / kXRows - w.t0;
                KeyLoad<4> keys{};                       // of the next tile that may lack keys
                if (partial < n && (!kBand || A.mask)) keys.start(A.mask, w.seq, first_key(w, partial > 0 ? partial : 0), lane);
                // the row's keys, from the first tile's first one on
                const int row_p = w.first + my_tok + w.seq.klen - w.seq.qlen - w.base;
                // dS over the scores; a copy of its own for tiles with absent keys
                auto tile = [&](auto masked, int i) -> bool {
                    const uint32_t ts = trow + (g & 1) * 128 + h * 64;
                    float p[64];
                    tmem_ld32(ts, reinterpret_cast<uint32_t *>(p));
                    tmem_ld32(ts + 32, reinterpret_cast<uint32_t *>(p) + 32);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        const float2 e = fma2(make_float2(p[j], p[j + 1]), make_float2(c, c), make_float2(nl, nl));
                        p[j] = xex2(e.x);
                        p[j + 1] = xex2(e.y);
                    }
                    uint32_t bits[2] = {0xffffffffu, 0xffffffffu};
                    if constexpr (decltype(masked)::value) {
                        KeyBits<4> kb;
                        if (!kBand || A.mask) {
                            kb = keys.finish();
                            if (i + 1 < n) keys.start(A.mask, w.seq, first_key(w, i + 1), lane);
                        } else {
                            kb.set_first(kXRows);
                        }
                        if constexpr (kBand) kb.clip(0, w.seq.klen - w.base - i * kXRows);
                        // the scores have read this tile's keys, so the rows in it that are not the sequence's, which may hold
                        // anything, may go before dS K
                        if (!kb.all()) zero_rows<L::KC, 4, 256>(smem + L::OFF_A + g % L::RA * L::TILE, kb, threadIdx.x);
                        if constexpr (kBand) kb.clip(row_p - A.left - i * kXRows, row_p + A.right + 1 - i * kXRows);
                        bits[0] = h ? kb.w[2] : kb.w[0];
                        bits[1] = h ? kb.w[3] : kb.w[1];
                    }
                    if (!warp_wait(abort_flag, Phase{&bars[XB_DP], (uint32_t)g & 1u})) return false;
                    tc::tc_fence_after();
                    uint32_t q[32];
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        float y[32];
                        tmem_ld32(trow + 256 + h * 64 + f * 32, reinterpret_cast<uint32_t *>(y));
                        tc::tmem_wait_ld();
                        if (f) {
                            tc::tc_fence_before();
                            warp_arrive(&bars[XB_PF], lane);   // dP has been read
                        }
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float2 e = mul2(make_float2(p[f * 32 + j], p[f * 32 + j + 1]),
                                                  add2(make_float2(y[j], y[j + 1]), make_float2(nd, nd)));
                            float a = e.x, b = e.y;
                            if constexpr (decltype(masked)::value) {
                                if (!((bits[f] >> j) & 1u)) a = 0.f;
                                if (!((bits[f] >> (j + 1)) & 1u)) b = 0.f;
                            }
                            q[(f * 32 + j) / 2] = xpack<kFp16>(a, b);
                        }
                    }
                    tmem_st32(ts, q);
                    tmem_wait_st();
                    tc::tc_fence_before();
                    warp_arrive(&bars[XB_DS + (g & 1)], lane);
                    return true;
                };
                for (int i = 0; i < n && ok; ++i, ++g) {
                    ok = warp_wait(abort_flag, Phase{&bars[XB_S + (g & 1)], (uint32_t)(g >> 1) & 1u});
                    if (!ok) break;
                    tc::tc_fence_after();
                    ok = i >= whole && i < partial ? tile(std::false_type{}, i) : tile(std::true_type{}, i);
                }
            }
            // beside the last product: the places of this unit's rows, and the next unit (they took 600 of a unit's 5400 cycles
            // after it, with one tile a unit)
            const int piece = w.piece;
            const bool pad = (n == 0 && (!kBand || piece < 0)) || w.first + my_tok >= w.seq.qlen;   // (others have a piece's sums)
            RowStore<kFp16> rows;
            if (ns == 1 && ok) {
                rows.rows(place(my_tok, my_head), lane);
                begin(k + 1);
            }
            if (n > 0) {
                if (ok) ok = warp_wait(abort_flag, Phase{&bars[XB_ACC], (uint32_t)nonempty & 1u});
                ++nonempty;
                tc::tc_fence_after();
            }
            if (ns > 1 || !ok) break;                    // stored below
            // -------------------------------------------------- epilogue
            const float f = A.scale * (kFp16 ? exp2f(-up) : 1.f);
            auto sums = [&](int j, float *y) {
                if (n > 0) {
                    tmem_ld32(trow + 384 + h * (D / 2) + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = 0.f;
                }
            };
            auto store = [&](int j, float *y) {
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = pad ? 0.f : y[e] * f;
                rows.store(A.dq, y, h * (D / 2) + j, lane);
            };
            if (piece < 0) {
#pragma unroll 1
                for (int j = 0; j < D / 2; j += 32) {
                    float y[32];
                    sums(j, y);
                    store(j, y);
                }
            } else {
                const Pieces<D / 2> part(A, piece, warp, lane);
#pragma unroll 1
                for (int j = 0; j < D / 2; j += 32) {
                    float y[32];
                    sums(j, y);
                    part.put(j, y);
                }
                if (part.last(lane))
#pragma unroll 1
                    for (int j = 0; j < D / 2; j += 32) {
                        float y[32];
                        part.sum(j, y);
                        store(j, y);
                    }
            }
            tc::tc_fence_before();                       // read before the next unit's products may follow
        }
        if (!ok && lane == 0) fail();
    }
    if (ns > 1) {
        // the CTA's only unit: partial sums into shared memory, then each rank joins its share of the rows
        float *xo = reinterpret_cast<float *>(smem);
        __syncthreads();                                 // loads and products on this memory are complete
        if (warp < 8) {
            const bool pad = w.n == 0 || w.first + my_tok >= w.seq.qlen;
            const float down = kFp16 ? exp2f(-up) : 1.f; // of this row, undone before rows change threads
#pragma unroll
            for (int j = 0; j < D / 2; j += 32) {
                float y[32];
                if (w.n > 0) {
                    tmem_ld32(trow + 384 + h * (D / 2) + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(xo + r * L::XROW + h * (D / 2) + j + e) =
                        pad ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(y[e] * down, y[e + 1] * down, y[e + 2] * down, y[e + 3] * down);
            }
        }
        cluster_sync();
        if (warp < 8) join_rows<kFp16, D>(xo, A.dq, ns, rank, warp, lane, out, A.scale);
        cluster_sync();                                  // peers are done with this CTA's shared memory
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0) A.status[blockIdx.x] = *abort_flag ? SAG_ERR_TIMEOUT : SAG_OK;
    if (kBand && A.late) grid_wait();                    // what follows the call follows k_xdkv too
}

// ------------------------------------------------------------------ k_xdkv
// TMEM columns: S^T 0 (P^T over it), dP^T 128 (dS^T over it), dV 256, dK 384.
template <bool kFp16, int D, bool kBand>
__global__ void __launch_bounds__(kXThreads, 1)
    k_xdkv(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_dy,
           const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
           const __grid_constant__ XArgs A) {
    using L = BwdSmem<D>;
    constexpr float kShift = kFp16 ? kGradShiftF16 : 0.f;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    const Ring rx = {bars + XB_XY, bars + XB_XYE, L::RX};
    const Ring ra = {bars + XB_RING, bars + XB_RING + L::RA, L::RA};
    const Ring rb = {ra.empty + L::RA, ra.empty + L::RA + L::RB, L::RB};
    const Ring rs = {bars + XB_STF, bars + XB_STE, 2};
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rb.empty + L::RB);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const Units units = {reinterpret_cast<Work *>(smem + L::OFF_BAR + 320), bars + XB_UF, bars + XB_UE};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < XB_RING + 2 * (L::RA + L::RB); ++i) tc::mbar_init(&bars[i], bwd_arrivals(i));
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
    if (A.tpt * A.group < kXRows) {
        // groups that do not divide 128 leave rows that no load writes: they stay zero
        KeyBits<4> kb;
        kb.set_first(A.tpt * A.group);
        if (warp < 8)
            for (int i = 0; i < L::RA + L::RB; ++i)
                zero_rows<L::KC, 4, 256>(smem + L::OFF_A + i * L::TILE, kb, threadIdx.x);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot, sbase = tc::smem_u32(smem);
    grid_wait();                                         // statistics and tickets of the kernel before
    if (kBand) grid_next();
    const int ns = A.nsplit, rank = blockIdx.x % ns;
    const int G = A.group;
    auto fail = [&]() { *abort_flag = 1; };
    auto decode = [&](int number) {
        const Item item(A, number, rank, ns);
        const XUnit u = x_decode<&SeqRow::ktile0, kBand ? kAcross : kByHead>(A, item.unit);
        Work w{};
        w.seq = u.seq;
        w.b = u.b;
        w.head = u.head;
        w.first = u.tile * kXRows;
        w.stat = (int32_t)u.tile_id;
        if constexpr (kBand) {
            // queries that see any of the tile's keys, and the tiles of queries that all see all of them
            const int off = u.seq.klen - u.seq.qlen, last = min(w.first + kXRows, u.seq.klen) - 1;
            const int from = max(0, w.first - off - A.right), to = min(u.seq.qlen, last - off + A.left + 1);
            const bool any = w.first < u.seq.klen && to > from;
            w.base = any ? from / A.tpt : 0;
            item.share(any ? (to + A.tpt - 1) / A.tpt - w.base : 0, &w);
            w.t0 += w.base;
            w.f0 = (max(last - off - A.right, 0) + A.tpt - 1) / A.tpt - w.t0;
            w.f1 = max(w.first - off + A.left + 1, 0) / A.tpt - w.t0;
        } else {
            item.share(w.first < u.seq.klen ? (u.seq.qlen + A.tpt - 1) / A.tpt : 0, &w);
        }
        return w;
    };

    if (warp == 8) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            const uint32_t qbytes = (uint32_t)L::KC * A.tpt * G * 128;
            int la = 0, lb = 0, ls = 0, lx = 0;          // loads so far
            bool ok = true;
            for (int k = 0; ok; ++k) {
                Work w{};
                ok = units.take(A, k, abort_flag, &w, decode);
                if (!ok || w.n < 0) break;
                if (w.n == 0) continue;
                auto load = [&](const Ring &r, int off, const CUtensorMap *map, int &i, int tile) {
                    if (!ring_wait_free(r, i, abort_flag)) return false;
                    const int s = i % r.n;
                    tc::mbar_arrive_expect_tx(&r.full[s], qbytes);
                    for (int c = 0; c < L::KC; ++c)
                        tc::tma_load_3d(smem + off + s * L::TILE + c * 16384, map, c * 64, w.head * G,
                                        w.seq.q0 + tile * A.tpt, &r.full[s]);
                    ++i;
                    return true;
                };
                ok = ring_wait_free(rx, lx, abort_flag);
                if (!ok) break;
                const int x = lx % L::RX;
                tc::mbar_arrive_expect_tx(&rx.full[x], 2 * L::TILE);
                for (int c = 0; c < L::KC; ++c) {
                    const int row = w.seq.k0 + w.first;
                    tc::tma_load_3d(smem + x * 2 * L::TILE + c * 16384, &map_k, c * 64, w.head, row, &rx.full[x]);
                    tc::tma_load_3d(smem + x * 2 * L::TILE + L::OFF_Y + c * 16384, &map_v, c * 64, w.head, row, &rx.full[x]);
                }
                ++lx;
                for (int i = 0; i < w.n && ok; ++i) {
                    ok = load(ra, L::OFF_A, &map_q, la, w.t0 + i);
                    if (ok) ok = ring_wait_free(rs, ls, abort_flag);
                    if (!ok) break;
                    tc::mbar_arrive_expect_tx(&rs.full[ls & 1], 1024);
                    bulk_load(smem + L::OFF_STAT + (ls & 1) * 1024,
                              A.stats + ((int64_t)(w.seq.qtile0 + w.t0 + i) * A.n2 + w.head) * 256, 1024,
                              &rs.full[ls & 1]);
                    ++ls;
                    ok = load(rb, L::OFF_B, &map_dy, lb, w.t0 + i);
                }
            }
            if (!ok) fail();
            bool drained = ring_drain(rx, lx);
            drained = ring_drain(ra, la) && drained;
            drained = ring_drain(rb, lb) && drained;
            drained = ring_drain(rs, ls) && drained;
            if (!drained) fail();
        }
    } else if (warp == 9) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t id_s = tc::idesc_f16(kXRows, kXRows, !kFp16, false, false);
        constexpr uint32_t id_g = tc::idesc_f16(kXRows, D, !kFp16, false, true);
        bool ok = true;
        int g = 0, nonempty = 0;
        for (int k = 0; ok; ++k) {
            Work w;
            ok = units.read(k, abort_flag, lane, &w);
            if (!ok || w.n < 0) break;
            const int n = w.n;
            if (n == 0) continue;
            // rows behind the sequence's last one are zeroed in a tile that has landed
            auto clear = [&](int off, int s, int i) {
                const int left = w.seq.qlen - (w.t0 + i) * A.tpt;
                if (left < A.tpt) {
                    KeyBits<4> kb;
                    kb.set_first(left * G);
                    zero_rows<L::KC, 4, 32>(smem + off + s * L::TILE, kb, lane);
                    __syncwarp();
                }
                tc::tc_fence_after();
            };
            const uint32_t resident = sbase + nonempty % L::RX * 2 * L::TILE;
            auto issue_s = [&](int i, int gi) {
                clear(L::OFF_A, gi % L::RA, i);
                mma_abt<D, kXRows>(tmem, resident, sbase + L::OFF_A + (gi % L::RA) * L::TILE, id_s);
                tc::mma_commit_warp(&bars[XB_S]);
            };
            auto issue_dp = [&](int i, int gi) {
                clear(L::OFF_B, gi % L::RB, i);
                mma_abt<D, kXRows>(tmem + 128, resident + L::OFF_Y, sbase + L::OFF_B + (gi % L::RB) * L::TILE, id_s);
                tc::mma_commit_warp(&bars[XB_DP]);
                if (i + 1 == n) tc::mma_commit_warp(&rx.empty[nonempty % L::RX]);
            };
            ok = warp_wait(abort_flag, rx.landed(nonempty), ra.landed(g));
            if (!ok) break;
            issue_s(0, g);
            ok = warp_wait(abort_flag, rb.landed(g));
            if (!ok) break;
            issue_dp(0, g);
            for (int i = 0; i < n; ++i, ++g) {
                const Phase p{&bars[XB_PF], (uint32_t)g & 1u}, ds{&bars[XB_DS], (uint32_t)g & 1u};
                const bool more = i + 1 < n;
                ok = more ? warp_wait(abort_flag, p, ra.landed(g + 1)) : warp_wait(abort_flag, p);
                if (!ok) break;
                tc::tc_fence_after();
                mma_ab<kXRows, 64>(tmem + 256, tmem, sbase + L::OFF_B + (g % L::RB) * L::TILE, id_g, i > 0);
                tc::mma_commit_warp(&rb.empty[g % L::RB]);
                if (more) issue_s(i + 1, g + 1);
                ok = more ? warp_wait(abort_flag, ds, rb.landed(g + 1)) : warp_wait(abort_flag, ds);
                if (!ok) break;
                tc::tc_fence_after();
                mma_ab<kXRows, 64>(tmem + 384, tmem + 128, sbase + L::OFF_A + (g % L::RA) * L::TILE, id_g, i > 0);
                tc::mma_commit_warp(&ra.empty[g % L::RA]);
                if (more) issue_dp(i + 1, g + 1);
            }
            if (!ok) break;
            tc::mma_commit_warp(&bars[XB_ACC]);
            ++nonempty;
        }
        if (!ok && lane == 0) fail();
        // every MMA issued must be complete before TMEM is freed: one more phase of XB_ACC
        if (!ok) tc::mma_commit_warp(&bars[XB_ACC]);
        const int phases = nonempty + (ok ? 0 : 1);
        if (!__all_sync(0xffffffffu, tc::drain_armed(&bars[XB_ACC], phases, kXWaitNs)) && lane == 0) fail();
    }

    const int h = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                // key = TMEM lane
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float fv = kFp16 ? exp2f(-kShift) : 1.f;
    Work w{};
    float up = 0.f;                                      // exponent that dS is scaled by (windowed: of the thread's key)
    bool st_live = false;                                // the thread's key is there
    auto out = [&](int k) -> int64_t {                   // place of key row k in dK and dV; negative: none
        const int key = w.first + k;
        if (key >= (A.s2_pad ? A.s2_pad : w.seq.klen)) return -1;
        return (((int64_t)w.seq.k0 + key) * A.n2 + w.head) * D;
    };
    if (warp < 8) {
        bool ok = true;
        int g = 0, nonempty = 0;
        // what the next unit needs from memory is on its way while this one is stored
        float2 norms{};
        auto begin = [&](int k) {
            ok = units.read(k, abort_flag, lane, &w);
            if (!ok || w.n < 0) return;
            st_live = w.first + r < w.seq.klen && (!A.mask || A.mask[(int64_t)w.seq.k0 + w.first + r] != 0);
            if constexpr (kFp16 && kBand) norms.x = A.k_up[(int64_t)w.stat * kXRows + r];
            else if constexpr (kFp16) norms = ds_norms(A, w.b, w.head);
        };
        begin(0);
        for (int turn = 0; ok && w.n >= 0; ++turn) {
            const int n = w.n;
            if constexpr (kFp16) up = kBand ? norms.x : ds_exponent(norms.x, norms.y);
            const bool live = st_live;
            if (n > 0) {
                // ---------------------------------------------- softmax
                const float c = A.scale_log2;
                const float k = kFp16 ? exp2f(up - kShift) : 1.f;
                // columns of the first tile that the thread's key is seen by: from the first query's to the last one's
                const int col_p = w.first + r - (w.seq.klen - w.seq.qlen) - w.t0 * A.tpt;
                // One query tile; a copy of its own for key tiles with absent keys.
                auto tile = [&](auto masked, int i) -> bool {
                    constexpr bool kMasked = decltype(masked)::value;
                    KeyBits<2> seen;                     // windowed: which of the thread's 64 columns see the key
                    if constexpr (kMasked && kBand) {
                        const int at = col_p - i * A.tpt;
                        seen.set_first(live ? 64 : 0);
                        seen.clip(min(max(at - A.right, 0), A.tpt) * G - h * 64, min(max(at + A.left + 1, 0), A.tpt) * G - h * 64);
                    }
                    const float4 *st = reinterpret_cast<const float4 *>(smem + L::OFF_STAT + (g & 1) * 1024) + h * 16;
                    float p[64];
                    tmem_ld32(trow + h * 64, reinterpret_cast<uint32_t *>(p));
                    tmem_ld32(trow + h * 64 + 32, reinterpret_cast<uint32_t *>(p) + 32);
                    tc::tmem_wait_ld();
                    uint32_t q[32];
#pragma unroll
                    for (int j = 0; j < 64; j += 4) {
                        const float4 nl4 = st[j / 4];
                        const float2 c2 = make_float2(c, c), shift = make_float2(kShift, kShift);
                        float2 e = fma2(make_float2(p[j], p[j + 1]), c2, make_float2(nl4.x, nl4.y));
                        float2 o = fma2(make_float2(p[j + 2], p[j + 3]), c2, make_float2(nl4.z, nl4.w));
                        if (kFp16) {
                            e = add2(e, shift);
                            o = add2(o, shift);
                        }
                        p[j] = xex2(e.x);
                        p[j + 1] = xex2(e.y);
                        p[j + 2] = xex2(o.x);
                        p[j + 3] = xex2(o.y);
                        if constexpr (kMasked && kBand) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!((seen.w[(j + e) >> 5] >> ((j + e) & 31)) & 1u)) p[j + e] = 0.f;
                        }
                        q[j / 2] = xpack<kFp16>(p[j], p[j + 1]);
                        q[j / 2 + 1] = xpack<kFp16>(p[j + 2], p[j + 3]);
                        if (kMasked && !kBand && !live) q[j / 2] = q[j / 2 + 1] = 0u;
                    }
                    tmem_st32(trow + h * 64, q);
                    tmem_wait_st();
                    tc::tc_fence_before();
                    warp_arrive(&bars[XB_PF], lane);
                    if (!warp_wait(abort_flag, Phase{&bars[XB_DP], (uint32_t)g & 1u})) return false;
                    tc::tc_fence_after();
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        float y[32];
                        tmem_ld32(trow + 128 + h * 64 + f * 32, reinterpret_cast<uint32_t *>(y));
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 nd4 = st[32 + (f * 32 + j) / 4];
                            const float2 k2 = make_float2(k, k);
                            const float *pp = p + f * 32 + j;
                            float2 e = add2(make_float2(y[j], y[j + 1]), make_float2(nd4.x, nd4.y));
                            float2 o = add2(make_float2(y[j + 2], y[j + 3]), make_float2(nd4.z, nd4.w));
                            if (kFp16) {
                                e = mul2(e, k2);
                                o = mul2(o, k2);
                            }
                            e = mul2(e, make_float2(pp[0], pp[1]));
                            o = mul2(o, make_float2(pp[2], pp[3]));
                            q[(f * 32 + j) / 2] = xpack<kFp16>(e.x, e.y);
                            q[(f * 32 + j) / 2 + 1] = xpack<kFp16>(o.x, o.y);
                            if (kMasked && !live) q[(f * 32 + j) / 2] = q[(f * 32 + j) / 2 + 1] = 0u;
                        }
                    }
                    tmem_st32(trow + 128 + h * 64, q);
                    tmem_wait_st();
                    tc::tc_fence_before();
                    warp_arrive(&bars[XB_DS], lane);
                    if (lane == 0) tc::mbar_arrive(&rs.empty[g & 1]);
                    return true;
                };
                const bool all = __all_sync(0xffffffffu, live);
                for (int i = 0; i < n && ok; ++i, ++g) {
                    ok = warp_wait(abort_flag, rs.landed(g), Phase{&bars[XB_S], (uint32_t)g & 1u});
                    if (!ok) break;
                    tc::tc_fence_after();
                    ok = all && (!kBand || (i >= w.f0 && i < w.f1)) ? tile(std::false_type{}, i) : tile(std::true_type{}, i);
                }
            }
            // beside the last product: the places of this unit's rows, and the next unit
            const int piece = w.piece;
            RowStore<kFp16> rows;
            if (ns == 1 && ok) {
                // k_xpre has zeroed the rows of absent states, whose sums are not 0 where dY holds a NaN (P = 0 does not cancel
                // it).  Zeroing them here made one-tile loops 2 % longer (selects: 5 %) and masked ones 3 %.
                rows.rows(live ? out(r) : -1, lane);
                begin(turn + 1);
            }
            if (n > 0) {
                if (ok) ok = warp_wait(abort_flag, Phase{&bars[XB_ACC], (uint32_t)nonempty & 1u});
                ++nonempty;
                tc::tc_fence_after();
            }
            if (ns > 1 || !ok) break;                    // stored below
            // -------------------------------------------------- epilogue: warps 0-3 dV, warps 4-7 dK
            const float f = h ? A.scale * (kFp16 ? exp2f(-up) : 1.f) : fv;
            auto sums = [&](int j, float *y) {
                if (n > 0) {
                    tmem_ld32(trow + 256 + h * 128 + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = 0.f;
                }
            };
            auto store = [&](int j, float *y) {
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] *= f;
                rows.store(h ? A.dk : A.dv, y, j, lane);
            };
            if (piece < 0) {
#pragma unroll
                for (int j = 0; j < D; j += 32) {
                    float y[32];
                    sums(j, y);
                    store(j, y);
                }
            } else {
                const Pieces<D> part(A, piece, warp, lane);
#pragma unroll 1
                for (int j = 0; j < D; j += 32) {
                    float y[32];
                    sums(j, y);
                    part.put(j, y);
                }
                if (part.last(lane))
#pragma unroll 1
                    for (int j = 0; j < D; j += 32) {
                        float y[32];
                        part.sum(j, y);
                        store(j, y);
                    }
            }
            tc::tc_fence_before();                       // read before the next unit's products may follow
        }
        if (!ok && lane == 0) fail();
    }
    if (ns > 1) {
        // the CTA's only unit: partial sums into shared memory, then each rank joins its share of the rows
        float *xo = reinterpret_cast<float *>(smem);
        __syncthreads();                                 // loads and products on this memory are complete
        const float down = kFp16 && kBand && h ? exp2f(-up) : 1.f;   // of this key, undone before rows change threads
        if (warp < 8) {
#pragma unroll
            for (int j = 0; j < D; j += 32) {
                float y[32];
                if (w.n > 0) {
                    tmem_ld32(trow + 256 + h * 128 + j, reinterpret_cast<uint32_t *>(y));
                    tc::tmem_wait_ld();
                    if constexpr (kFp16 && kBand) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] *= down;
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(xo + (h * kXRows + r) * L::XROW + j + e) =
                        w.n > 0 && st_live ? make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        cluster_sync();
        if (warp < 8) {
            const float fk = A.scale * (kFp16 && !kBand ? exp2f(-up) : 1.f);
            join_rows<kFp16, D>(xo, A.dv, ns, rank, warp, lane, out, fv);
            join_rows<kFp16, D>(xo + kXRows * L::XROW, A.dk, ns, rank, warp, lane, out, fk);
        }
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

template <bool kFp16, int D, bool kBand>
cudaError_t launch(const XArgs &a, const sca_io &io, const sca_desc &d, bool dkv, bool after, cudaStream_t s) {
    BwdMaps m;
    if (!maps(&m, a, io, d)) return cudaErrorInvalidValue;
    return x_launch(dkv ? k_xdkv<kFp16, D, kBand> : k_xdq<kFp16, D, kBand>, a.ctas, kXThreads, a.nsplit, BwdSmem<D>::TOTAL, after, s, m.q, m.dy,
                    m.k, m.v, a);
}

template <bool kFp16, bool kBand>
cudaError_t launch(const XArgs &a, const sca_io &io, const sca_desc &d, bool dkv, bool after, cudaStream_t s) {
    return d.d == 128 ? launch<kFp16, 128, kBand>(a, io, d, dkv, after, s) : launch<kFp16, 64, kBand>(a, io, d, dkv, after, s);
}

template <bool kBand>
cudaError_t launch_bwd(const XArgs &a, const sca_io &io, const sca_desc &d, bool dkv, bool after, cudaStream_t s) {
    return d.dtype == SAG_FP16 ? launch<true, kBand>(a, io, d, dkv, after, s) : launch<false, kBand>(a, io, d, dkv, after, s);
}

}  // namespace
}  // namespace sag
