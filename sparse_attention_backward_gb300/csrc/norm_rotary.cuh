// Norms of queries and keys for each head with the rotary positions in the same
// pass, and the gradient: what the two directions share.
//
// Mathematics.  A head x of d columns has r = 1 / sqrt(mean(x^2) + eps), its
// weight w and its row's rotation R (angles as in rotary.cu):
//     y = R (x r w)
//     gradient, with dn = R^T dy and g = dn w:
//     dx = r (g - x r^2 mean(g x)),   dw = sum over rows and heads of dn x r
// All in fp32, one rounding to the 16-bit type.
//
// A head belongs to a group of 4 to 32 neighbouring threads, each with vectors
// that turn together (halves: columns c and c + d_rot / 2), so that the rotation
// needs no exchange and the sums a few shuffles; groups take heads in the order
// of memory.  Sines are computed once a token for queries and keys, into shared
// memory, laid out so that neighbouring threads read neighbouring 16 bytes.
// Heads whose columns or strides are not multiples of the vectors take the same
// kernels element by element.
//
// These kernels issue about as many instructions as memory can feed: the
// arithmetic is in pairs (f32x2), the threads of a head are a constant, and few
// threads take a head, as many elements each as registers allow.
#pragma once

#include "f32x2.cuh"
#include "kernels.cuh"
#include "rotary.cuh"

namespace sag {

constexpr int kNormThreads = 256;
constexpr int kMaxNormTokens = 64, kMaxSines = 2048;     // of a block: tokens, pairs of all of them
constexpr int kGradBlocks = 304;                         // of a gradient launch: partial sums of the weights' gradients

struct NormArgs {
    SeqTab seq;
    uint64_t turns[kMaxRot / 2];
    float magnitude, eps, plus, inv_d;
    int32_t rows, d, d_rot, offset, s_max;
    int32_t heads[2];                   // of query, key
    int32_t half;                       // style
    int32_t units, rot_units;           // items of a head, the turning ones first
    int32_t weight_fp32;
    int32_t tokens;                     // of a tile
    int32_t chunk, parts;               // forward: heads of a block, blocks of a tile
    const int32_t *positions;
    const uint16_t *in[2], *dy[2];
    uint16_t *out[2];
    int64_t in_stride[2], out_stride[2], dy_stride[2];
    const void *weight[2];
    float *dw[2];
    float *part;                        // [kGradBlocks][query, key][d]
};

// Vectors of an item (two of 8, 4 or 1 elements that turn with each other, or one of 8 whose neighbours do), threads of a
// head, items of a thread.
struct NormShape {
    int vec, pair, group, slots;
};
cudaError_t launch_norm_fwd(const NormArgs &a, bool fp16, const NormShape &p, int blocks, int smem, cudaStream_t s);
cudaError_t launch_norm_grad(const NormArgs &a, bool fp16, const NormShape &p, int blocks, int smem, cudaStream_t s);

namespace {

__device__ __forceinline__ float norm_rsqrt(float x) {   // x is normal: eps is
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Where an item lies: the first column of its vectors, and which of them there are.  Columns that do not turn are paired up
// as they come.
template <bool kPair, int V>
struct Place {
    int a, b;
    bool has_a, has_b, turns;
    __device__ __forceinline__ Place() {}
    __device__ __forceinline__ Place(const NormArgs &A, int it) {
        has_a = it < A.units;
        turns = it < A.rot_units;
        has_b = false;
        b = 0;
        const int others = (A.d - A.d_rot) / V;
        auto other = [&](int i) { return i * V < A.offset ? i * V : i * V + A.d_rot; };
        if (turns) {
            const bool apart = kPair && (V > 1 || A.half);
            a = A.offset + (kPair && !apart ? 2 * it : it * V);
            if (kPair) {
                b = a + (apart ? A.d_rot / 2 : 1);
                has_b = true;
            }
        } else {
            const int i = it - A.rot_units;
            a = other(kPair ? 2 * i : i);
            if (kPair) {
                b = other(2 * i + 1);
                has_b = has_a && 2 * i + 1 < others;
            }
        }
    }
    // column of element k of the first and the second part
    __device__ __forceinline__ int col(int k, bool second) const {
        return kPair ? (second ? b : a) + k : a + 2 * k + second;
    }
    __device__ __forceinline__ bool has(bool second) const { return kPair && second ? has_b : has_a; }
};

// An item's elements: P of them, `a`, turn with P others, `b`.
template <bool kFp16, bool kPair, int V>
struct Item {
    static constexpr int P = kPair ? V : V / 2;
    static constexpr int W = (V + 1) / 2;
    uint32_t a[W], b[kPair ? W : 1];
    __device__ __forceinline__ static void take(uint32_t *w, const uint16_t *p) {
        if constexpr (V == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (V == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else {
            w[0] = *p;
        }
    }
    __device__ __forceinline__ static void give(uint16_t *p, const uint32_t *w) {
        if constexpr (V == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (V == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else *p = (uint16_t)w[0];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            a[i] = 0;
            if (kPair) b[i] = 0;
        }
    }
    __device__ __forceinline__ void load(const uint16_t *p, const Place<kPair, V> &at) {
        if (at.has_a) take(a, p + at.a);
        if (kPair && at.has_b) take(b, p + at.b);
    }
    __device__ __forceinline__ void get(float *fa, float *fb) const {
        if constexpr (V == 1) {
            fa[0] = u16_to_f<kFp16>((uint16_t)a[0]);
            fb[0] = u16_to_f<kFp16>((uint16_t)b[0]);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float2 x = unpack2<kFp16>(a[i]);
                if constexpr (kPair) {
                    const float2 y = unpack2<kFp16>(b[i]);
                    fa[2 * i] = x.x, fa[2 * i + 1] = x.y, fb[2 * i] = y.x, fb[2 * i + 1] = y.y;
                } else {
                    fa[i] = x.x, fb[i] = x.y;
                }
            }
        }
    }
    __device__ __forceinline__ static void store(uint16_t *p, const Place<kPair, V> &at, const float *fa, const float *fb) {
        uint32_t w[W];
        if (!at.has_a) return;
        if constexpr (V == 1) {
            p[at.a] = f_to_u16<kFp16>(fa[0]);
            if (at.has_b) p[at.b] = f_to_u16<kFp16>(fb[0]);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                w[i] = kPair ? round2<kFp16>(fa[(2 * i) % P], fa[(2 * i + 1) % P]) : round2<kFp16>(fa[i % P], fb[i % P]);
            give(p + at.a, w);
            if (kPair && at.has_b) {
#pragma unroll
                for (int i = 0; i < W; ++i) w[i] = round2<kFp16>(fb[(2 * i) % P], fb[(2 * i + 1) % P]);
                give(p + at.b, w);
            }
        }
    }
};

// P floats, in pairs where there are any.
template <int P, class F>
__device__ __forceinline__ void pairs(F &&f) {
    if constexpr (P > 1) {
#pragma unroll
        for (int k = 0; k < P; k += 2) f(k);
    } else {
        f(0);
    }
}
template <int P>
__device__ __forceinline__ float2 at2(const float *x, int k) {
    return P > 1 ? make_float2(x[k], x[k + (P > 1)]) : make_float2(x[0], 0.f);
}
template <int P>
__device__ __forceinline__ void put2(float *x, int k, float2 v) {
    x[k] = v.x;
    if (P > 1) x[k + (P > 1)] = v.y;
}
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// Turns an item's elements.
template <int P>
__device__ __forceinline__ void turn(float *fa, float *fb, const float *cs, const float *sn) {
    pairs<P>([&](int k) {
        const float2 x = at2<P>(fa, k), y = at2<P>(fb, k), c = at2<P>(cs, k), s = at2<P>(sn, k);
        put2<P>(fa, k, fma2(x, c, neg2(mul2(y, s))));
        put2<P>(fb, k, fma2(x, s, mul2(y, c)));
    });
}

// Runs of P floats for each of `items` items in shared memory, of which a thread reads four at a time: neighbouring items
// are 16 bytes apart.
template <int P>
__device__ __forceinline__ int run_at(int it, int k, int items) {
    constexpr int L = P >= 4 ? 4 : 1;
    return (k / L * items + it) * L + k % L;
}
template <int P>
__device__ __forceinline__ void run_read(const float *base, int it, int items, float *f) {
    if constexpr (P >= 4) {
#pragma unroll
        for (int k = 0; k < P; k += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(base + run_at<P>(it, k, items));
            f[k] = x.x, f[k + 1] = x.y, f[k + 2] = x.z, f[k + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < P; ++k) f[k] = base[run_at<P>(it, k, items)];
    }
}

// Sines of a block: [tokens][cos, sin][P of each turning item], in floats.
__host__ __device__ inline int norm_sines(int tokens, int d_rot) { return (tokens * d_rot + 3) & ~3; }

// A tile's rows: whether each is there, and its position.
struct TileRows {
    int32_t position[kMaxNormTokens];
    int8_t live[kMaxNormTokens];
    __device__ __forceinline__ void fill(const NormArgs &A, int row0, int n_tok) {
        if (threadIdx.x >= n_tok) return;
        const int row = row0 + threadIdx.x;
        int place;
        live[threadIdx.x] = locate_row(A.seq, A.s_max, A.positions, row, &place);
        position[threadIdx.x] = A.positions && live[threadIdx.x] ? __ldg(A.positions + row) : place;
    }
};

// The sines of a tile's tokens (of padding rows too: any position's).
template <int P>
__device__ __forceinline__ void fill_sines(const NormArgs &A, const uint64_t *turns, float *sines, const TileRows &rows, int n_tok) {
    const int half = A.d_rot / 2, by_tok = kNormThreads / half, by_pair = kNormThreads - by_tok * half;
    int tok = threadIdx.x / half, pair = threadIdx.x - tok * half;
    while (tok < n_tok) {
        const int32_t t = (int32_t)(((uint64_t)(int64_t)rows.position[tok] * turns[pair]) >> 32);
        float sn, cs;
        sincospif((float)t * 0x1p-31f, &sn, &cs);
        float *at = sines + tok * A.d_rot + run_at<P>(pair / P, pair % P, A.rot_units);
        at[0] = cs * A.magnitude;
        at[half] = sn * A.magnitude;
        tok += by_tok;
        pair += by_pair;
        if (pair >= half) {
            pair -= half;
            ++tok;
        }
    }
}

// A tensor's weights in shared memory: [first, second part][P of each item].
template <bool kFp16, bool kPair, int V>
__device__ __forceinline__ void fill_weights(const NormArgs &A, int w, float *to) {
    constexpr int P = Item<kFp16, kPair, V>::P;
    for (int i = threadIdx.x; i < A.units * P * 2; i += kNormThreads) {
        const bool second = i >= A.units * P;
        const int j = i - (second ? A.units * P : 0), it = j / P, k = j % P;
        const Place<kPair, V> at(A, it);
        float x = 0.f;
        if (at.has(second)) {
            x = 1.f;
            if (A.weight[w]) {
                const int c = at.col(k, second);
                if (A.weight_fp32) x = static_cast<const float *>(A.weight[w])[c];
                else x = u16_to_f<kFp16>(static_cast<const uint16_t *>(A.weight[w])[c]);
                x += A.plus;
            }
        }
        to[(second ? A.units * P : 0) + run_at<P>(it, k, A.units)] = x;
    }
}
template <int P>
__device__ __forceinline__ void read_weights(const float *from, int it, int units, float *wa, float *wb) {
    run_read<P>(from, it, units, wa);
    run_read<P>(from + units * P, it, units, wb);
}

template <int kGroup>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = kGroup >> 1; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The instantiation for a shape: f(pair, V, group, slots) as integral constants.
template <int N>
using Int = std::integral_constant<int, N>;
template <class F>
cudaError_t with_shape(const NormShape &p, F &&f) {
    auto sized = [&](auto pair, auto v, auto slots) {
        if (p.group == 4) return f(pair, v, Int<4>{}, slots);
        if (p.group == 8) return f(pair, v, Int<8>{}, slots);
        if (p.group == 16) return f(pair, v, Int<16>{}, slots);
        return f(pair, v, Int<32>{}, slots);
    };
    if (p.vec == 1) return f(Int<1>{}, Int<1>{}, Int<32>{}, Int<8>{});
    if (p.pair && p.vec == 8) return sized(Int<1>{}, Int<8>{}, Int<1>{});
    if (p.pair) return sized(Int<1>{}, Int<4>{}, Int<3>{});
    return p.slots == 2 ? sized(Int<0>{}, Int<8>{}, Int<2>{}) : sized(Int<0>{}, Int<8>{}, Int<3>{});
}

}  // namespace
}  // namespace sag
