// Norms of queries and keys for each head with the rotary positions in the same
// pass, and the gradient.
//
// Mathematics.  A head x of d columns has r = 1 / sqrt(mean(x^2) + eps), its
// weight w and its row's rotation R (angles as in rotary.cu):
//     y = R (x r w)
//     gradient, with dn = R^T dy and g = dn w:
//     dx = r (g - x r^2 mean(g x)),   dw = sum over rows and heads of dn x r
// The gradient's two sums over a head, of x^2 and of g x, are taken together; r
// is formed again from x, so the forward keeps nothing.  All in fp32, one
// rounding to the 16-bit type.
//
// Bound by memory: 4 bytes an element (gradient: 6).  A head belongs to a group
// of 4 to 32 neighbouring threads, each with the 16-byte vectors that turn
// together (halves: columns c and c + d_rot / 2), so that the rotation needs no
// exchange and the sums a few shuffles; groups take heads in the order of
// memory.  Sines are computed once a token and weights read once a block, into
// shared memory, laid out so that neighbouring threads read neighbouring 16
// bytes.  Heads whose columns or strides are not multiples of eight elements
// take the same kernels element by element.
//
// dw: every thread keeps the sums of its columns over all heads that its group
// takes; a block adds its groups up in their order, and k_norm_dw the blocks in
// theirs, so the result does not depend on timing.
#include <math.h>

#include "kernels.cuh"
#include "rotary.cuh"

namespace sag {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64, kMaxSines = 1024;         // of a block: tokens, pairs of all of them
constexpr int kGradBlocks = 608;                         // of a gradient launch: partial sums of the weights' gradients

struct NormArgs {
    SeqTab seq;
    uint64_t turns[kMaxRot / 2];
    float magnitude, eps, plus, inv_d;
    int32_t rows, n1, n2, d, d_rot, offset, s_max;
    int32_t half;                       // style
    int32_t group;                      // threads of a head
    int32_t units, rot_units;           // items of a head, the turning ones first
    int32_t tokens, chunk;              // of a block: tokens, and heads of them
    int32_t weight_fp32;
    int32_t q_blocks;                   // gradient: blocks that take queries
    const int32_t *positions;
    const uint16_t *in[2], *dy[2];
    uint16_t *out[2];
    int64_t in_stride[2], out_stride[2], dy_stride[2];
    const void *weight[2];
    float *dw[2];
    float *part;                        // [kGradBlocks][d]
};

// An item's vector of V elements.
template <bool kFp16, int V>
struct Elems;
template <bool kFp16>
struct Elems<kFp16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float *f) const {
        const uint32_t *w = &v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack2<kFp16>(w[i]);
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    }
    __device__ __forceinline__ static void store(uint16_t *p, const float *f) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(round2<kFp16>(f[0], f[1]), round2<kFp16>(f[2], f[3]),
                                                   round2<kFp16>(f[4], f[5]), round2<kFp16>(f[6], f[7]));
    }
};
template <bool kFp16>
struct Elems<kFp16, 1> {
    uint16_t v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *p; }
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void get(float *f) const { f[0] = u16_to_f<kFp16>(v); }
    __device__ __forceinline__ static void store(uint16_t *p, const float *f) { *p = f_to_u16<kFp16>(f[0]); }
};

// How items map to columns, and what a block keeps in shared memory.  kPair: an item that turns has two vectors, whose
// elements turn with each other (V = 1: a pair of columns in either style); otherwise its vector holds interleaved pairs.
template <bool kPair, int V>
struct Shape {
    static constexpr int P = kPair ? V : V / 2;          // pairs of an item
    static constexpr int L = V == 8 ? 4 : 1;             // floats that a thread reads at a time
    __device__ __forceinline__ static int col_a(const NormArgs &A, int it) {
        if (it < A.rot_units) return A.offset + (V == 1 && !A.half ? 2 * it : it * V);
        const int c = (it - A.rot_units) * V;
        return c < A.offset ? c : c + A.d_rot;
    }
    __device__ __forceinline__ static int gap(const NormArgs &A) { return V == 1 && !A.half ? 1 : A.d_rot / 2; }
    // float k of a run of N belonging to item `it`, of `items`: neighbouring items are 16 bytes apart
    template <int N>
    __device__ __forceinline__ static int at(int it, int k, int items) { return (k / L * items + it) * L + k % L; }
    template <int N>
    __device__ __forceinline__ static void read(const float *base, int it, int items, float *f) {
#pragma unroll
        for (int k = 0; k < N; k += L) {
            if constexpr (L == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(base + at<N>(it, k, items));
                f[k] = x.x;
                f[k + 1] = x.y;
                f[k + 2] = x.z;
                f[k + 3] = x.w;
            } else {
                f[k] = base[at<N>(it, k, items)];
            }
        }
    }
};

// Shared memory of a block, in floats: sines [tokens][cos, sin][P][rot_units], then weights [which][a, b][V][units].
__host__ __device__ inline int norm_sines(int tokens, int d_rot) { return (tokens * d_rot + 3) & ~3; }

template <bool kPair, int V>
__device__ __forceinline__ void fill_weights(const NormArgs &A, float *w, int which, bool fp16) {
    using H = Shape<kPair, V>;
    for (int i = threadIdx.x; i < A.units * V * 2; i += kThreads) {
        const int part = i / (A.units * V), k = i % (A.units * V) / A.units, it = i % A.units;
        if (part && !(kPair && it < A.rot_units)) continue;
        const int c = H::col_a(A, it) + k + (part ? H::gap(A) : 0);
        float x = 1.f;
        if (A.weight[which]) {
            if (A.weight_fp32) x = static_cast<const float *>(A.weight[which])[c];
            else if (fp16) x = u16_to_f<true>(static_cast<const uint16_t *>(A.weight[which])[c]);
            else x = u16_to_f<false>(static_cast<const uint16_t *>(A.weight[which])[c]);
            x += A.plus;
        }
        w[part * A.units * V + H::template at<V>(it, k, A.units)] = x;
    }
}

template <bool kPair, int V>
__device__ __forceinline__ void fill_sines(const NormArgs &A, const uint64_t *turns, float *sines, int row0, int n_tok) {
    using H = Shape<kPair, V>;
    const int pairs = A.d_rot / 2;
    for (int j = threadIdx.x; j < n_tok * pairs; j += kThreads) {
        const int tok = j / pairs, pair = j - tok * pairs, row = row0 + tok;
        int place;
        if (!locate_row(A.seq, A.s_max, A.positions, row, &place)) continue;
        const int64_t p = A.positions ? (int64_t)__ldg(A.positions + row) : (int64_t)place;
        const int32_t t = (int32_t)(((uint64_t)p * turns[pair]) >> 32);
        float sn, cs;
        sincospif((float)t * 0x1p-31f, &sn, &cs);
        float *at = sines + tok * A.d_rot;
        const int i = H::template at<H::P>(pair / H::P, pair % H::P, A.rot_units);
        at[i] = cs * A.magnitude;
        at[pairs + i] = sn * A.magnitude;
    }
}

// A thread's part of a head: items `lane`, `lane` + group, ...
template <bool kFp16, bool kPair, int V, int S>
struct Head {
    using H = Shape<kPair, V>;
    Elems<kFp16, V> a[S], b[kPair ? S : 1];
    __device__ __forceinline__ void load(const NormArgs &A, const uint16_t *p, int lane, bool live) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int it = lane + s * A.group;
            a[s].zero();
            if (kPair) b[s].zero();
            if (!live || it >= A.units) continue;
            const int c = H::col_a(A, it);
            a[s].load(p + c);
            if (kPair && it < A.rot_units) b[s].load(p + c + H::gap(A));
        }
    }
    __device__ __forceinline__ void get(int s, float *fa, float *fb) const {
        a[s].get(fa);
        if (kPair) b[s].get(fb);
    }
    __device__ __forceinline__ static void store(const NormArgs &A, uint16_t *p, int it, const float *fa, const float *fb) {
        const int c = H::col_a(A, it);
        Elems<kFp16, V>::store(p + c, fa);
        if (kPair && it < A.rot_units) Elems<kFp16, V>::store(p + c + H::gap(A), fb);
    }
    // Turns an item's elements by its token's angles.
    __device__ __forceinline__ static void turn(const NormArgs &A, const float *sines, int it, float *fa, float *fb) {
        if (it >= A.rot_units) return;
        float cs[H::P], sn[H::P];
        H::template read<H::P>(sines, it, A.rot_units, cs);
        H::template read<H::P>(sines + A.d_rot / 2, it, A.rot_units, sn);
#pragma unroll
        for (int k = 0; k < H::P; ++k) {
            float &x = kPair ? fa[k] : fa[2 * k], &y = kPair ? fb[k] : fa[2 * k + 1];
            const float u = x * cs[k] - y * sn[k], v = x * sn[k] + y * cs[k];
            x = u;
            y = v;
        }
    }
};

__device__ __forceinline__ float group_sum(float x, int group) {
    for (int o = group >> 1; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ------------------------------------------------------------------ forward
template <bool kFp16, bool kPair, int V, int S>
__global__ void __launch_bounds__(kThreads) k_norm_fwd(const __grid_constant__ NormArgs A) {
    using Hd = Head<kFp16, kPair, V, S>;
    using H = Shape<kPair, V>;
    constexpr int U = S == 1 ? 2 : 1;                    // heads of a thread in flight
    extern __shared__ __align__(16) float smem[];
    __shared__ uint64_t turns[kMaxRot / 2];
    __shared__ int8_t is_live[kMaxTokens];
    float *sines = smem, *weights = smem + norm_sines(A.tokens, A.d_rot);
    const int heads = A.n1 + A.n2, wsize = 2 * A.units * V;
    const int row0 = blockIdx.x * A.tokens, n_tok = min(A.tokens, A.rows - row0);
    const int lo = blockIdx.y * A.chunk, hi = min(lo + A.chunk, n_tok * heads);
    const int group = threadIdx.x / A.group, lane = threadIdx.x % A.group, groups = kThreads / A.group;
    for (int i = threadIdx.x; i < A.d_rot / 2; i += kThreads) turns[i] = A.turns[i];
    if (threadIdx.x < n_tok) {
        int place;
        is_live[threadIdx.x] = locate_row(A.seq, A.s_max, A.positions, row0 + threadIdx.x, &place);
    }
    __syncthreads();
    Hd x[U];
    auto where = [&](int i, int *tok, int *w, int *head) {
        *tok = i / heads;
        *head = i - *tok * heads;
        *w = *head >= A.n1;
        *head -= *w ? A.n1 : 0;
    };
    auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = base + k * groups + group;
            int tok, w, head;
            where(i < hi ? i : lo, &tok, &w, &head);
            x[k].load(A, A.in[w] + (int64_t)(row0 + tok) * A.in_stride[w] + head * A.d, lane, i < hi && is_live[tok]);
        }
    };
    load(lo);
    // while the first heads are on their way
    fill_weights<kPair, V>(A, weights, 0, kFp16);
    if (A.n2) fill_weights<kPair, V>(A, weights + wsize, 1, kFp16);
    fill_sines<kPair, V>(A, turns, sines, row0, n_tok);
    __syncthreads();
    for (int base = lo; base < hi; base += U * groups) {
        if (base > lo) load(base);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = base + k * groups + group;
            float sum = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float fa[V], fb[V];
                x[k].get(s, fa, fb);
#pragma unroll
                for (int e = 0; e < V; ++e) sum += fa[e] * fa[e] + (kPair ? fb[e] * fb[e] : 0.f);
            }
            const float r = rsqrtf(group_sum(sum, A.group) * A.inv_d + A.eps);
            if (i >= hi) continue;
            int tok, w, head;
            where(i, &tok, &w, &head);
            uint16_t *to = A.out[w] + (int64_t)(row0 + tok) * A.out_stride[w] + head * A.d;
            const bool live = is_live[tok];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int it = lane + s * A.group;
                if (it >= A.units) continue;
                float fa[V], fb[V], wa[V], wb[V];
                x[k].get(s, fa, fb);
                H::template read<V>(weights + w * wsize, it, A.units, wa);
#pragma unroll
                for (int e = 0; e < V; ++e) fa[e] *= r * wa[e];
                if (kPair && it < A.rot_units) {
                    H::template read<V>(weights + w * wsize + A.units * V, it, A.units, wb);
#pragma unroll
                    for (int e = 0; e < V; ++e) fb[e] *= r * wb[e];
                }
                if (live) {
                    Hd::turn(A, sines + tok * A.d_rot, it, fa, fb);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) fa[e] = fb[e] = 0.f;
                }
                Hd::store(A, to, it, fa, fb);
            }
        }
    }
}

// ----------------------------------------------------------------- gradient
template <bool kFp16, bool kPair, int V, int S>
__global__ void __launch_bounds__(kThreads) k_norm_grad(const __grid_constant__ NormArgs A) {
    using Hd = Head<kFp16, kPair, V, S>;
    using H = Shape<kPair, V>;
    extern __shared__ __align__(16) float smem[];
    __shared__ uint64_t turns[kMaxRot / 2];
    __shared__ int8_t is_live[kMaxTokens];
    float *sines = smem, *weights = smem + norm_sines(A.tokens, A.d_rot);
    const int w = (int)blockIdx.x >= A.q_blocks;
    const int block = blockIdx.x - (w ? A.q_blocks : 0), blocks = w ? gridDim.x - A.q_blocks : A.q_blocks;
    const int heads = w ? A.n2 : A.n1;
    const int group = threadIdx.x / A.group, lane = threadIdx.x % A.group, groups = kThreads / A.group;
    for (int i = threadIdx.x; i < A.d_rot / 2; i += kThreads) turns[i] = A.turns[i];
    fill_weights<kPair, V>(A, weights, w, kFp16);
    float da[S][V], db[kPair ? S : 1][V];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            da[s][e] = 0.f;
            if (kPair) db[s][e] = 0.f;
        }
    const int tiles = (A.rows + A.tokens - 1) / A.tokens;
    for (int tile = block; tile < tiles; tile += blocks) {
        const int row0 = tile * A.tokens, n_tok = min(A.tokens, A.rows - row0), hi = n_tok * heads;
        __syncthreads();                                 // the tile before is done with the sines
        if (threadIdx.x < n_tok) {
            int place;
            is_live[threadIdx.x] = locate_row(A.seq, A.s_max, A.positions, row0 + threadIdx.x, &place);
        }
        __syncthreads();
        Hd x, y;
        auto load = [&](int base) {
            const int i = min(base + group, hi - 1), tok = i / heads, head = i - tok * heads;
            const bool live = base + group < hi && is_live[tok];
            x.load(A, A.in[w] + (int64_t)(row0 + tok) * A.in_stride[w] + head * A.d, lane, live);
            y.load(A, A.dy[w] + (int64_t)(row0 + tok) * A.dy_stride[w] + head * A.d, lane, live);
        };
        load(0);
        fill_sines<kPair, V>(A, turns, sines, row0, n_tok);
        __syncthreads();
        for (int base = 0; base < hi; base += groups) {
            if (base) load(base);
            const int i = min(base + group, hi - 1), tok = i / heads, head = i - tok * heads;
            const bool live = is_live[tok];
            float sq = 0.f, dot = 0.f;
            float ga[S][V], gb[kPair ? S : 1][V];        // R^T dy
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int it = lane + s * A.group;
                float *pa = ga[s], *pb = gb[kPair ? s : 0];
                y.get(s, pa, pb);
                if (it >= A.units) continue;
                // (of padding rows the sines may be anything)
                if (live) Hd::turn(A, sines + tok * A.d_rot, it, pa, pb);
                float fa[V], fb[V], wa[V];
                x.get(s, fa, fb);
                H::template read<V>(weights, it, A.units, wa);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    sq += fa[e] * fa[e];
                    dot += fa[e] * (pa[e] * wa[e]);
                }
                if (kPair && it < A.rot_units) {
                    H::template read<V>(weights + A.units * V, it, A.units, wa);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        sq += fb[e] * fb[e];
                        dot += fb[e] * (pb[e] * wa[e]);
                    }
                }
            }
            sq = group_sum(sq, A.group);
            dot = group_sum(dot, A.group);
            if (base + group >= hi) continue;
            const float r = rsqrtf(sq * A.inv_d + A.eps), back = r * r * dot * A.inv_d;
            uint16_t *to = A.out[w] + (int64_t)(row0 + tok) * A.out_stride[w] + head * A.d;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int it = lane + s * A.group;
                if (it >= A.units) continue;
                float fa[V], fb[V], wa[V], oa[V], ob[V];
                x.get(s, fa, fb);
                H::template read<V>(weights, it, A.units, wa);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    oa[e] = r * (ga[s][e] * wa[e] - fa[e] * back);
                    da[s][e] += ga[s][e] * (fa[e] * r);
                }
                if (kPair && it < A.rot_units) {
                    H::template read<V>(weights + A.units * V, it, A.units, wa);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        ob[e] = r * (gb[s][e] * wa[e] - fb[e] * back);
                        db[s][e] += gb[s][e] * (fb[e] * r);
                    }
                }
                Hd::store(A, to, it, oa, ob);            // padding: all zeros
            }
        }
    }
    if (!A.dw[w]) return;
    // the block's sums: groups of a warp by shuffles, then the warps in their order
    const int warp = threadIdx.x >> 5, in_warp = threadIdx.x & 31;
    float *sums = smem;                                  // [warps][d]
    __syncthreads();
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int it = lane + s * A.group, c = it < A.units ? H::col_a(A, it) : 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float u = da[s][e], v = kPair ? db[s][e] : 0.f;
            for (int o = A.group; o < 32; o <<= 1) {
                u += __shfl_xor_sync(0xffffffffu, u, o);
                if (kPair) v += __shfl_xor_sync(0xffffffffu, v, o);
            }
            if (in_warp < A.group && it < A.units) {
                sums[warp * A.d + c + e] = u;
                if (kPair && it < A.rot_units) sums[warp * A.d + c + H::gap(A) + e] = v;
            }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < A.d; c += kThreads) {
        float u = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) u += sums[k * A.d + c];
        A.part[(int64_t)blockIdx.x * A.d + c] = u;
    }
}

// Adds the blocks' sums up: a block takes 32 columns of one tensor, its warps every eighth of the others' blocks.
__global__ void __launch_bounds__(kThreads) k_norm_dw(const float *part, int d, int q_blocks, int blocks, float *dwq, float *dwk) {
    __shared__ float sums[kThreads / 32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    float *dw = blockIdx.y ? dwk : dwq;
    const int first = blockIdx.y ? q_blocks : 0, last = blockIdx.y ? blocks : q_blocks;
    if (!dw) return;
    float u = 0.f;
    if (c < d) {
#pragma unroll 8
        for (int k = first + warp; k < last; k += kThreads / 32) u += part[(int64_t)k * d + c];
    }
    sums[warp][lane] = u;
    __syncthreads();
    if (warp == 0 && c < d) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) t += sums[k][lane];
        dw[c] = t;
    }
}

// ---------------------------------------------------------------- host side
sag_status check_norm(const snr_desc *d) {
    if (!d) return SAG_ERR_NULL;
    const sag_status st = check_rotary(&d->rotary);
    if (st != SAG_OK && st != SAG_ERR_UNSUPPORTED) return st;
    if (!(d->eps > 0.0) || !isfinite(d->eps) || (float)d->eps == 0.f || !isfinite((float)d->eps) || !isfinite(d->weight_offset) ||
        (d->weight_fp32 != 0 && d->weight_fp32 != 1) || d->reserved_ != 0)
        return SAG_ERR_SHAPE;
    const int64_t sy[] = {d->q_grad_stride, d->k_grad_stride};
    for (int i = 0; i < 2; ++i)
        if (sy[i] != 0 && (sy[i] < (int64_t)(i ? d->rotary.n2 : d->rotary.n1) * d->rotary.d || sy[i] > (1LL << 40)))
            return SAG_ERR_SHAPE;
    return st;
}

size_t norm_ws(const snr_desc *d, bool grad) {
    const size_t seq = (seq_ws_bytes(d->rotary.batch) + 255) / 256 * 256;
    return grad ? seq + sizeof(float) * kGradBlocks * d->rotary.d : seq_ws_bytes(d->rotary.batch);
}

template <bool kFp16, bool kPair, int V, int S>
cudaError_t launch(const NormArgs &a, bool grad, dim3 grid, int smem, cudaStream_t s) {
    if (grad) k_norm_grad<kFp16, kPair, V, S><<<grid, kThreads, smem, s>>>(a);
    else k_norm_fwd<kFp16, kPair, V, S><<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <bool kFp16>
cudaError_t launch(const NormArgs &a, int vec, bool pair, int slots, bool grad, dim3 grid, int smem, cudaStream_t s) {
    if (vec == 1) return launch<kFp16, true, 1, 16>(a, grad, grid, smem, s);
    if (pair) {
        if (slots == 1) return launch<kFp16, true, 8, 1>(a, grad, grid, smem, s);
        if (slots == 2) return launch<kFp16, true, 8, 2>(a, grad, grid, smem, s);
        return launch<kFp16, true, 8, 3>(a, grad, grid, smem, s);
    }
    if (slots == 1) return launch<kFp16, false, 8, 1>(a, grad, grid, smem, s);
    if (slots == 2) return launch<kFp16, false, 8, 2>(a, grad, grid, smem, s);
    return launch<kFp16, false, 8, 3>(a, grad, grid, smem, s);
}

sag_status run_norm(const snr_desc *desc, const snr_io *io, void *workspace, size_t workspace_bytes, void *stream, bool grad) {
    sag_status st = check_norm(desc);
    if (st != SAG_OK) return st;
    const srt_desc *d = &desc->rotary;
    const bool bsnd = d->layout == SAG_LAYOUT_BSND;
    const int32_t rows = bsnd ? d->batch * d->s_max : d->cu_seqlens[d->batch];
    const size_t need = norm_ws(desc, grad);
    if (!io) return SAG_ERR_NULL;
    if (need && (!workspace || workspace_bytes < need)) return SAG_ERR_WORKSPACE;
    auto off = [](const void *p, int mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
    if (need && off(workspace, 15)) return SAG_ERR_ALIGN;
    float *const dws[] = {io->query_weight ? io->query_weight_grad : nullptr,
                          io->key_weight && d->n2 ? io->key_weight_grad : nullptr};
    const void *ins[] = {io->query, io->key}, *dys[] = {io->query_out_grad, io->key_out_grad};
    void *outs[] = {grad ? io->query_grad : io->query_out, grad ? io->key_grad : io->key_out};
    const void *weights[] = {io->query_weight, io->key_weight};
    const int sides = d->n2 ? 2 : 1;
    for (int i = 0; i < sides; ++i) {
        if (rows && (!ins[i] || !outs[i] || (grad && !dys[i]))) return SAG_ERR_NULL;
        if (rows && (off(ins[i], 15) || off(outs[i], 15) || (grad && off(dys[i], 15)))) return SAG_ERR_ALIGN;
        if (off(weights[i], 15) || (grad && off(dws[i], 15))) return SAG_ERR_ALIGN;
    }
    if (off(io->positions, 3)) return SAG_ERR_ALIGN;
    NormArgs a{};
    const int64_t dense[] = {(int64_t)d->n1 * d->d, (int64_t)d->n2 * d->d};
    const int64_t si[] = {d->q_stride, d->k_stride}, so[] = {d->q_out_stride, d->k_out_stride},
                  sy[] = {desc->q_grad_stride, desc->k_grad_stride};
    for (int i = 0; i < 2; ++i) {
        a.in_stride[i] = si[i] ? si[i] : dense[i];
        a.out_stride[i] = so[i] ? so[i] : dense[i];
        a.dy_stride[i] = sy[i] ? sy[i] : dense[i];
        a.in[i] = static_cast<const uint16_t *>(ins[i]);
        a.dy[i] = static_cast<const uint16_t *>(dys[i]);
        a.out[i] = static_cast<uint16_t *>(outs[i]);
        a.weight[i] = weights[i];
        a.dw[i] = dws[i];
    }
    // an output over an input (a group has read its head whole before it writes) has to have its rows where that has them
    for (int i = 0; rows && i < sides; ++i)
        if ((outs[i] == ins[i] && a.in_stride[i] != a.out_stride[i]) ||
            (grad && outs[i] == dys[i] && a.dy_stride[i] != a.out_stride[i]))
            return SAG_ERR_SHAPE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard wg, dg;
    if (need && !wg.bind_memory(workspace)) return SAG_ERR_CUDA;         // a kernel writes there: host memory is refused
    if (rows == 0) {                                                     // sums of nothing
        for (int i = 0; grad && i < sides; ++i)
            if (dws[i] && cudaMemsetAsync(dws[i], 0, sizeof(float) * d->d, s) != cudaSuccess) return SAG_ERR_CUDA;
        return SAG_OK;
    }
    if (!dg.bind_memory(outs[0])) return SAG_ERR_CUDA;
    rotary_turns(d, grad, a.turns);
    a.magnitude = (float)d->magnitude;
    a.eps = (float)desc->eps;
    a.plus = (float)desc->weight_offset;
    a.inv_d = 1.f / d->d;
    a.rows = rows;
    a.n1 = d->n1;
    a.n2 = d->n2;
    a.d = d->d;
    a.d_rot = d->d_rot;
    a.offset = d->offset;
    a.s_max = bsnd ? d->s_max : 0;
    a.half = d->style == SRT_HALF;
    a.weight_fp32 = desc->weight_fp32;
    a.positions = io->positions;
    // vectors of eight where every address, stride and part boundary allows them
    int64_t all = (int64_t)d->d | d->offset | (a.half ? d->d_rot / 2 : d->d_rot);
    for (int i = 0; i < sides; ++i) all |= a.in_stride[i] | a.out_stride[i] | (grad ? a.dy_stride[i] : 0);
    const int vec = all % 8 == 0 ? 8 : 1;
    const bool pair = a.half || vec == 1;
    a.rot_units = pair ? d->d_rot / 2 / vec : d->d_rot / vec;
    a.units = a.rot_units + (d->d - d->d_rot) / vec;
    // threads of a head and items of a thread: the fewest places that hold the items, then the fewest items
    int slots = 16;
    a.group = 32;
    if (vec == 8) {
        int best = 1 << 30;
        for (int t = 1; t <= 3; ++t)
            for (int g = 4; g <= 32; g *= 2)
                if (g * t >= a.units && g * t < best) {
                    best = g * t;
                    a.group = g;
                    slots = t;
                }
    }
    const int groups = kThreads / a.group;
    if (fill_seq_tab(&a.seq, d->batch, static_cast<SeqRow *>(workspace), s, [&](int b) {
            SeqRow r{};
            r.q0 = bsnd ? b * d->s_max : d->cu_seqlens[b];
            r.qlen = b < d->batch ? d->cu_seqlens[b + 1] - d->cu_seqlens[b] : 0;
            return r;
        }) != cudaSuccess)
        return SAG_ERR_CUDA;
    dim3 grid;
    const int heads = d->n1 + d->n2;
    const int sms = current_device_sms();
    auto tokens_of = [&](int64_t target, int per) {
        int64_t t = target / per;
        if (t > kMaxTokens) t = kMaxTokens;
        if (t > kMaxSines / (d->d_rot / 2)) t = kMaxSines / (d->d_rot / 2);
        return t < 1 ? 1 : (int)t;
    };
    if (!grad) {
        // several rounds of heads a block where there is work for all SMs; else one, of a part of a token if need be
        const int64_t total = (int64_t)rows * heads, want = total / ((int64_t)sms * 8);
        const int round = groups * (slots == 1 ? 2 : 1);
        const int64_t target = want >= 8 * round ? 8 * round : want >= round ? round : groups;
        a.tokens = tokens_of(target, heads);
        a.chunk = a.tokens > 1 || heads <= target ? a.tokens * heads : (int)target;
        grid = dim3((unsigned)((rows + a.tokens - 1) / a.tokens), (unsigned)((a.tokens * heads + a.chunk - 1) / a.chunk));
    } else {
        // blocks shared between queries and keys by their heads; each walks over tokens
        a.tokens = tokens_of(8 * groups, d->n1);
        const int64_t tiles = ((int64_t)rows + a.tokens - 1) / a.tokens;
        int64_t k_blocks = d->n2 ? (int64_t)kGradBlocks * d->n2 / heads : 0;
        if (d->n2 && k_blocks < 1) k_blocks = 1;
        int64_t q_blocks = kGradBlocks - k_blocks;
        if (q_blocks > tiles) q_blocks = tiles;
        if (k_blocks > tiles) k_blocks = tiles;
        a.q_blocks = (int)q_blocks;
        a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + (need - sizeof(float) * kGradBlocks * d->d));
        grid = dim3((unsigned)(q_blocks + k_blocks));
    }
    int smem = (norm_sines(a.tokens, d->d_rot) + 2 * a.units * vec * (grad ? 1 : 2)) * (int)sizeof(float);
    if (grad && smem < kThreads / 32 * d->d * (int)sizeof(float)) smem = kThreads / 32 * d->d * (int)sizeof(float);
    const cudaError_t e = d->dtype == SAG_FP16 ? launch<true>(a, vec, pair, slots, grad, grid, smem, s)
                                               : launch<false>(a, vec, pair, slots, grad, grid, smem, s);
    if (e != cudaSuccess) return SAG_ERR_CUDA;
    if (grad && (dws[0] || dws[1])) {
        k_norm_dw<<<dim3((unsigned)(d->d + 31) / 32, sides), kThreads, 0, s>>>(a.part, d->d, a.q_blocks, (int)grid.x, dws[0], dws[1]);
        if (cudaGetLastError() != cudaSuccess) return SAG_ERR_CUDA;
    }
    return SAG_OK;
}

sag_status norm_size(const snr_desc *desc, size_t *bytes, bool grad) {
    if (!bytes) return SAG_ERR_NULL;
    const sag_status st = check_norm(desc);
    if (st == SAG_OK) *bytes = norm_ws(desc, grad);
    return st;
}

}  // namespace
}  // namespace sag

using namespace sag;

extern "C" sag_status norm_rotary_fwd_workspace_size(const snr_desc *desc, size_t *workspace_bytes) {
    return norm_size(desc, workspace_bytes, false);
}

extern "C" sag_status norm_rotary_grad_workspace_size(const snr_desc *desc, size_t *workspace_bytes) {
    return norm_size(desc, workspace_bytes, true);
}

extern "C" sag_status norm_rotary_fwd(const snr_desc *desc, const snr_io *io, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    return run_norm(desc, io, workspace, workspace_bytes, stream, false);
}

extern "C" sag_status norm_rotary_grad(const snr_desc *desc, const snr_io *io, void *workspace, size_t workspace_bytes,
                                       void *stream) {
    return run_norm(desc, io, workspace, workspace_bytes, stream, true);
}
