// Pieces shared by the cross-attention kernels: arguments, tile geometry, the
// TMEM and cluster instructions they add, and the masks of a key tile.
//
// A tile has 128 rows.  A query tile packs 128 / G tokens with the G heads that
// share a key/value head (row = token * G + head), so keys are read once for the
// whole group and the key gradients sum over it inside the matrix product.
#pragma once

#include "common.cuh"
#include "seqtab.cuh"
#include "tc.cuh"

namespace sag {

constexpr int kXRows = 128;             // rows of a query tile, keys of a key tile
constexpr int kMaxSplit = 8;            // CTAs of a cluster, pieces of a unit
constexpr int kMaxPieces = 304;         // pieces of a launch: each has its partial sums in the workspace
constexpr int kXThreads = 320;          // warps 0-7 softmax and epilogue, 8 TMA, 9 MMA
constexpr uint64_t kXWaitNs = 2000000000ull;
// A half keeps 11 bits down to 2^-14 only, and a probability of a long sequence lies below that.  Both passes shift
// fp16 probabilities up by a power of two that cannot overflow 65504, and undo it in fp32.
constexpr float kFwdShiftF16 = 7.f;     // forward: exp2(x - max) <= 2^8 (lazy maximum), so <= 2^15
constexpr float kGradShiftF16 = 15.f;   // gradient: P <= 1 (up to rounding), so <= 2^15

struct XArgs {
    SeqTab seq;
    int32_t n1, n2, group;
    int32_t tpt;                        // tokens per query tile
    int32_t s1_pad, s2_pad;             // BSND: padded lengths, else 0
    int32_t units;                      // query (k_xdkv: key) tiles times key/value heads
    int32_t nsplit;                     // CTAs (one cluster) that share a unit
    int32_t ctas;                       // of the launch: units * nsplit, or fewer that take unit after unit
    // gradient kernels: work items are `full` whole units, then pieces of the others, `pieces` each
    int32_t items, full, pieces;
    float *parts;                       // partial sums of the pieces
    unsigned *arrived;                  // pieces of a unit whose sums are there, for each softmax warp
    int32_t n_arrived;                  // such counters of the call
    unsigned *ticket;                   // next items of the two gradient kernels; zeroed by k_xpre, like the counters
    float scale, scale_log2;
    const uint8_t *mask;
    const uint16_t *o_in, *dy, *v_in;   // preprocess
    int64_t v_stride;
    uint16_t *o, *dq, *dk, *dv;
    float *lse;                         // forward: written, gradient: read
    float *stats;                       // [query tile][n2][256]: lse * log2(e), then Delta, of the tile's 128 rows
    unsigned *norms;                    // fp16: [batch][n2][2] largest squared row norms of dY and of V, as float bits
    float *row_norms;                   // fp16: [query tile][n2][128] squared norms of the rows of dY
    int32_t q_tiles, k_tiles;
    int32_t *count, *status;            // device status: number of words, one word for each CTA
    int32_t n_status;                   // value for *count
};

cudaError_t launch_xfwd(const XArgs &a, const sca_io &io, const sca_desc &d, bool long_loops, cudaStream_t s);
cudaError_t launch_xpre(const XArgs &a, bool fp16, int d, cudaStream_t s);
cudaError_t launch_xdq(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s);
cudaError_t launch_xdkv(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s);

namespace {

// ---------------------------------------------------------------- PTX
// Shared-memory descriptors (128-byte swizzle, 1024 bytes between groups of eight rows) as two words: the low one holds
// the address, so a step along K is one 32-bit addition, and the high one is a constant.  Descriptors built anew for each
// instruction were kept in registers by the compiler, and spilled: a thousand cycles a tile in the MMA warp.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// (the mask drops the CTA's rank, which addresses carry from bit 24 on in a cluster)
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}

// One elected lane of the (convergent) warp issues.  A and B from shared memory, or A from TMEM (K-major: lane = row, two
// elements a column).
__device__ __forceinline__ void xmma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void xmma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Waits of a whole (convergent) warp for one to three barriers: a test of a completed phase costs about 60 cycles, three
// independent ones little more, and one after the other three times that, which the MMA warps do not have.  Bounded like
// tc::mbar_wait; false when the limit ran out or *abort was set.  A barrier that has been seen complete stays so until
// this warp goes on, so testing it again with the others is safe.
struct Phase {
    uint64_t *bar;
    uint32_t parity;
};
template <class... P>
__device__ __forceinline__ bool warp_wait(volatile int *abort, const P &...p) {
    auto done = [&]() {
        bool all = true;
        ((all = tc::mbar_try_wait(p.bar, p.parity) && all), ...);
        return __all_sync(0xffffffffu, all) != 0;
    };
    if (done()) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (done()) return true;
        if ((i & 63) == 0 &&
            __any_sync(0xffffffffu, *abort != 0 || tc::globaltimer_ns() - t0 > kXWaitNs))
            return false;
    }
}

// One arrival for a warp whose lanes have all done what the barrier stands for.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
}

// global -> shared copy of `bytes` (a multiple of 16, both ends 16-byte aligned)
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     tc::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Kernels of one call: the next one's CTAs may be placed as this one's leave, and wait there for all its results.
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// address of the same shared-memory variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
// (no memory clobber: the reads of several ranks overlap; cluster_sync has one)
__device__ __forceinline__ float2 peer_ld2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ float xex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two fp32 operations an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

template <bool kFp16>
__device__ __forceinline__ uint32_t xpack(float a, float b) {
    if constexpr (kFp16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// ---------------------------------------------------------------- geometry
// Unit -> sequence, key/value head, tile within the sequence.  Units of a
// sequence are consecutive, and within it those of a head, so that CTAs that
// run at the same time read the same keys (or queries) from L2.
struct XUnit {
    SeqRow seq;
    int b, head, tile;
    int64_t tile_id;                    // (tiles of the sequences before + tile) * n2 + head
};
template <int32_t SeqRow::*field>
__device__ __forceinline__ XUnit x_decode(const XArgs &A, int unit) {
    XUnit x;
    x.b = seq_find<field>(A.seq, unit / A.n2);
    x.seq = seq_row(A.seq, x.b);
    const int first = x.seq.*field, nt = seq_get<field>(A.seq, x.b + 1) - first;
    const int local = unit - first * A.n2;
    x.head = local / nt;
    x.tile = local % nt;
    x.tile_id = (int64_t)(first + x.tile) * A.n2 + x.head;
    return x;
}

// A rank's share of `tiles`: first tile and number.
__device__ __forceinline__ void x_share(int tiles, int rank, int ranks, int *first, int *n) {
    *first = 0;
    *n = tiles;
    if (ranks > 1) {
        *first = tiles * rank / ranks;
        *n = tiles * (rank + 1) / ranks - *first;
    }
}

// Which of the kWords * 32 keys from key `first` of a sequence are there.
// Collective over a warp when there is a mask.
template <int kWords>
struct KeyBits {
    uint32_t w[kWords];
    __device__ __forceinline__ bool all() const {
        uint32_t x = w[0];
#pragma unroll
        for (int j = 1; j < kWords; ++j) x &= w[j];
        return x == 0xffffffffu;
    }
    // the first n
    __device__ __forceinline__ void set_first(int n) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            const int k = n - 32 * j;
            w[j] = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
        }
    }
};
// In two steps, so that a tile's mask bytes are on their way while the tile before is worked on.
template <int kWords>
struct KeyLoad {
    uint8_t byte[kWords];
    int left;
    bool masked;
    __device__ __forceinline__ void start(const uint8_t *mask, const SeqRow &seq, int first, int lane) {
        left = seq.klen - first;
        masked = mask != nullptr;
        if (!masked) return;
        const uint8_t *m = mask + (int64_t)seq.k0 + first;
#pragma unroll
        for (int j = 0; j < kWords; ++j) byte[j] = 32 * j + lane < left ? m[32 * j + lane] : (uint8_t)0;
    }
    __device__ __forceinline__ KeyBits<kWords> finish() const {
        KeyBits<kWords> k;
        if (!masked) {
            k.set_first(left);
            return k;
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) k.w[j] = __ballot_sync(0xffffffffu, byte[j] != 0);
        return k;
    }
};

// Zeros the rows of a [32 * kWords x 64 * kChunks] shared tile whose bit is not set, before a matrix product reads it: a
// probability of 0 does not cancel a NaN.  Shared by kThreads threads; each fences its writes for the products' proxy.
template <int kChunks, int kWords, int kThreads>
__device__ __forceinline__ void zero_rows(uint8_t *tile, const KeyBits<kWords> &k, int thread) {
    // consecutive threads take consecutive 16-byte pieces, so a pass of kPass rows has no bank conflicts (with a thread or
    // two a row this took 700 to 1000 cycles of a masked tile)
    constexpr int kRows = 32 * kWords, kPass = kThreads / (kChunks * 8);
    static_assert(kPass >= 1 && 32 % kPass == 0, "a pass lies within a word");
    const int c = thread % (kChunks * 8), r = thread / (kChunks * 8);
    uint8_t *at = tile + (c >> 3) * kRows * 128 + r * 128 + (c & 7) * 16;
#pragma unroll
    for (int j = 0; j < kRows; j += kPass)
        if (!((k.w[j >> 5] >> ((j & 31) + r)) & 1u)) *reinterpret_cast<uint4 *>(at + j * 128) = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async_smem();
}

// Products, each with K = 16 steps; a tile of R rows keeps its 64-column chunks 128 R bytes apart.
// A [128 x D] K-major, B [kN x D] K-major: columns 0..kN-1 of the accumulator.
template <int D, int kN>
__device__ __forceinline__ void mma_abt(uint32_t acc, uint32_t a, uint32_t b, uint32_t idesc) {
    const uint32_t al = desc_lo(a, 16), bl = desc_lo(b, 16);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        xmma_ss(acc, al + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), bl + (((kk >> 2) * kN * 128 + (kk & 3) * 32) >> 4),
                idesc, kk > 0);
}
// A [128 x kK] in TMEM (16-bit pairs; the second half of kK = 128 starts kGap columns after the first), B [kK x D] MN-major.
// Steps kFrom .. kTo - 1 of kK / 16.
template <int kK, int kGap, int kFrom = 0, int kTo = kK / 16>
__device__ __forceinline__ void mma_ab(uint32_t acc, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    const uint32_t bl = desc_lo(b, kK * 128);
#pragma unroll
    for (int kk = kFrom; kk < kTo; ++kk)
        xmma_ts(acc, a + (kk >> 2) * kGap + (kk & 3) * 8, bl + (kk * 2048 >> 4), idesc, accumulate || kk > 0);
}

// Stores of accumulator rows.  A lane holds 32 columns of its own row; written as they stand, each instruction of a warp
// would touch 32 lines for 16 bytes each.  Groups of four lanes swap their 16-byte pieces first (two steps of a 4 x 4
// transposition), so that an instruction writes 64 consecutive bytes of eight rows.  Collective over a warp.
template <bool kFp16>
struct RowStore {
    int64_t off[4];                     // elements from `base` to the rows of this lane's group; negative: not stored
    __device__ __forceinline__ void rows(int64_t mine, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = __shfl_sync(0xffffffffu, mine, (lane & ~3) + i);
    }
    // the lower lane of a pair gives b for the other's a
    __device__ __forceinline__ static void trade(uint32_t &a, uint32_t &b, bool upper, int with) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? a : b, with);
        a = upper ? got : a;
        b = upper ? b : got;
    }
    __device__ __forceinline__ static void trade(uint4 &a, uint4 &b, bool upper, int with) {
        trade(a.x, b.x, upper, with);
        trade(a.y, b.y, upper, with);
        trade(a.z, b.z, upper, with);
        trade(a.w, b.w, upper, with);
    }
    __device__ __forceinline__ void store(uint16_t *base, const float *y, int col, int lane) const {
        uint4 c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            c[k] = make_uint4(xpack<kFp16>(y[8 * k], y[8 * k + 1]), xpack<kFp16>(y[8 * k + 2], y[8 * k + 3]),
                              xpack<kFp16>(y[8 * k + 4], y[8 * k + 5]), xpack<kFp16>(y[8 * k + 6], y[8 * k + 7]));
        const bool odd = lane & 1, high = lane & 2;
#pragma unroll
        for (int k = 0; k < 4; k += 2) trade(c[k], c[k + 1], odd, 1);
#pragma unroll
        for (int k = 0; k < 2; ++k) trade(c[k], c[k + 2], high, 2);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (off[i] >= 0) *reinterpret_cast<uint4 *>(base + off[i] + col + 8 * (lane & 3)) = c[i];
    }
};

}  // namespace
}  // namespace sag
