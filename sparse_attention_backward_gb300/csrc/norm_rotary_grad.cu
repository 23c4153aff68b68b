// Norms with rotation, gradient (norm_rotary.cuh).
//
// 6 bytes an element: x and dy read, dx written; r is formed again from x, so
// the forward keeps nothing, and the two sums over a head, of x^2 and of g x,
// are taken together.
//
// Blocks walk over tiles of tokens, first a tile's queries, then its keys, which
// share the sines; a tile's sines are computed while the one before is worked
// on, and a head's loads are on their way while the one before it is.  dw: a
// thread keeps the sums of its columns over all heads that its group takes (the
// other side's in shared memory meanwhile); a block adds its groups up in their
// order, and k_norm_dw the blocks in theirs, so the result does not depend on
// timing.  4 x 4095 padded tokens of 32 heads of 192, 64 of them turning: 103
// us, 5.4 TB/s; 32768 tokens of 40 heads of 128: 182 us.  (Blocks of queries
// and of keys apart, each with sines of its own: 120 and 226 us.)
#include <type_traits>

#include "norm_rotary.cuh"

namespace sag {

namespace {

template <bool kFp16, bool kPair, int V, int kGroup, int S>
__global__ void __launch_bounds__(kNormThreads, V == 1 ? 1 : 2) k_norm_grad(const __grid_constant__ NormArgs A) {
    using I = Item<kFp16, kPair, V>;
    constexpr int P = I::P, kGroups = kNormThreads / kGroup, kSums = 2 * S * P;
    constexpr bool kHeld = kSums <= 16 && V > 1;         // weights in registers
    extern __shared__ __align__(16) float smem[];        // two tiles' sines, weights, the other side's sums of each thread
    __shared__ uint64_t turns[kMaxRot / 2];
    __shared__ TileRows rows[4];                         // of this block's tiles, by their number, two ahead
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tokens = A.tokens, half = A.d_rot / 2, sines_size = norm_sines(tokens, A.d_rot), wsize = 2 * A.units * P;
    const int sides = A.heads[1] ? 2 : 1;
    float *weights = smem + 2 * sines_size, *others = weights + sides * wsize + threadIdx.x;
    const int group = threadIdx.x / kGroup, lane = threadIdx.x % kGroup;
    const bool padded = A.s_max != 0;
    for (int i = threadIdx.x; i < half; i += kNormThreads) turns[i] = A.turns[i];
    for (int w = 0; w < sides; ++w) fill_weights<kFp16, kPair, V>(A, w, weights + w * wsize);
    float sums[kSums];                                   // of the columns of this side's items: `a` parts, then `b`
    Place<kPair, V> at[S];
    I nx[S], ny[S];                                      // of the next head; what is never loaded stays zero
#pragma unroll
    for (int s = 0; s < S; ++s) {
        at[s] = Place<kPair, V>(A, lane + s * kGroup);
        nx[s].zero();
        ny[s].zero();
    }
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        sums[i] = 0.f;
        others[i * kNormThreads] = 0.f;
    }
    const int tiles = (A.rows + tokens - 1) / tokens;
    auto tile_tokens = [&](int tile) { return min(tokens, A.rows - tile * tokens); };
    auto place_rows = [&](int number) {
        const int tile = blockIdx.x + number * gridDim.x;
        if (tile < tiles) rows[number & 3].fill(A, tile * tokens, tile_tokens(tile));
    };
    auto angles = [&](int number) {
        const int tile = blockIdx.x + number * gridDim.x;
        if (tile < tiles)
            fill_sines<P>(A, turns, smem + (number & 1) * sines_size, rows[number & 3], tile_tokens(tile));
    };
    // a group's heads of a tile and side, one every kGroups
    struct Steps {
        int heads, by_tok, by_head, tok, head;
        __device__ __forceinline__ void start(int n, int group) {
            heads = n;
            by_tok = kGroups / n;
            by_head = kGroups - by_tok * n;
            tok = group / n;
            head = group - tok * n;
        }
        __device__ __forceinline__ void next() {
            tok += by_tok;
            head += by_head;
            if (head >= heads) {
                head -= heads;
                ++tok;
            }
        }
    };
    // of the next loads
    Steps l;
    int l_tile = blockIdx.x, l_number = 0, l_side = 0, l_left;
    auto begin = [&]() {
        l.start(A.heads[l_side], group);
        l_left = l_tile < tiles ? tile_tokens(l_tile) * l.heads : 0;
    };
    auto load = [&]() {
        if (l_left > group && (!padded || rows[l_number & 3].live[l.tok])) {
            const int64_t row = (int64_t)l_tile * tokens + l.tok;
            const uint16_t *px = A.in[l_side] + (row * A.in_stride[l_side] + l.head * A.d);
            const uint16_t *py = A.dy[l_side] + (row * A.dy_stride[l_side] + l.head * A.d);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                nx[s].load(px, at[s]);
                ny[s].load(py, at[s]);
            }
        }
        l.next();
        l_left -= kGroups;
        if (l_left <= 0) {                               // the same for the block: the other side, or the next tile
            if (++l_side >= sides) {
                l_side = 0;
                l_tile += gridDim.x;
                ++l_number;
            }
            begin();
        }
    };
    place_rows(0);
    place_rows(1);
    __syncthreads();                                     // frequencies, rows, weights
    begin();
    load();
    angles(0);
    float ha[kHeld ? S : 1][P], hb[kHeld ? S : 1][P];
    int number = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++number) {
        __syncthreads();                                 // this tile's sines are there, and the other buffer is free
        angles(number + 1);
        place_rows(number + 2);
        const float *sines = smem + (number & 1) * sines_size;
        for (int w = 0; w < sides; ++w) {
            Steps c;
            c.start(A.heads[w], group);
            const float *from = weights + w * wsize;
            if constexpr (kHeld) {
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (at[s].has_a) read_weights<P>(from, lane + s * kGroup, A.units, ha[s], hb[s]);
            }
            auto weight = [&](int s, float *wa, float *wb) {
                if constexpr (kHeld) {
#pragma unroll
                    for (int k = 0; k < P; ++k) wa[k] = ha[s][k], wb[k] = hb[s][k];
                } else {
                    read_weights<P>(from, lane + s * kGroup, A.units, wa, wb);
                }
            };
            for (int left = tile_tokens(tile) * c.heads; left > 0; left -= kGroups, c.next()) {
                const bool mine = left > group, live = mine && (!padded || rows[number & 3].live[c.tok]);
                float2 sq = make_float2(0.f, 0.f), dot = sq;
                float ga[S][P], gb[S][P];
                I x[S];
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    x[s] = nx[s];
                    ny[s].get(ga[s], gb[s]);
                }
                load();                                  // the next head
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    if (!at[s].has_a || !live) continue;
                    if (at[s].turns) {
                        float cs[P], sn[P];
                        run_read<P>(sines + c.tok * A.d_rot, lane + s * kGroup, A.rot_units, cs);
                        run_read<P>(sines + c.tok * A.d_rot + half, lane + s * kGroup, A.rot_units, sn);
                        turn<P>(ga[s], gb[s], cs, sn);   // R^T dy
                    }
                    float fa[P], fb[P], wa[P], wb[P];
                    weight(s, wa, wb);
                    x[s].get(fa, fb);
                    pairs<P>([&](int k) {
                        const float2 u = at2<P>(fa, k), v = at2<P>(fb, k);
                        sq = fma2(v, v, fma2(u, u, sq));
                        dot = fma2(v, mul2(at2<P>(gb[s], k), at2<P>(wb, k)), fma2(u, mul2(at2<P>(ga[s], k), at2<P>(wa, k)), dot));
                    });
                }
                const float sum = group_sum<kGroup>(sq.x + sq.y), gx = group_sum<kGroup>(dot.x + dot.y);
                if (mine) {
                    const float r = norm_rsqrt(sum * A.inv_d + A.eps), back = -r * r * gx * A.inv_d * r;
                    const float2 r2 = make_float2(r, r), b2 = make_float2(back, back);
                    uint16_t *to = A.out[w] + (((int64_t)tile * tokens + c.tok) * A.out_stride[w] + c.head * A.d);
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        if (!at[s].has_a) continue;
                        float oa[P], ob[P];
                        if (live) {
                            float wa[P], wb[P], fa[P], fb[P];
                            weight(s, wa, wb);
                            x[s].get(fa, fb);
                            // g r - x r^3 mean(g x); dw gets dn x r
                            pairs<P>([&](int k) {
                                const float2 u = at2<P>(fa, k), v = at2<P>(fb, k);
                                const float2 m = mul2(at2<P>(ga[s], k), r2), n = mul2(at2<P>(gb[s], k), r2);
                                put2<P>(oa, k, fma2(m, at2<P>(wa, k), mul2(u, b2)));
                                put2<P>(ob, k, fma2(n, at2<P>(wb, k), mul2(v, b2)));
                                put2<P>(sums + s * P, k, fma2(m, u, at2<P>(sums + s * P, k)));
                                put2<P>(sums + (S + s) * P, k, fma2(n, v, at2<P>(sums + (S + s) * P, k)));
                            });
                        } else {                         // padding
#pragma unroll
                            for (int e = 0; e < P; ++e) oa[e] = ob[e] = 0.f;
                        }
                        I::store(to, at[s], oa, ob);
                    }
                }
            }
            if (sides > 1) {                             // the other side's sums
#pragma unroll
                for (int i = 0; i < kSums; ++i) {
                    const float x = others[i * kNormThreads];
                    others[i * kNormThreads] = sums[i];
                    sums[i] = x;
                }
            }
        }
    }
    // the block's sums: groups of a warp by shuffles, then the warps in their order (after whole tiles they are the query's)
    const int warp = threadIdx.x >> 5, in_warp = threadIdx.x & 31;
    float more[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) more[i] = others[i * kNormThreads];
    for (int w = 0; w < sides; ++w) {
        if (w) {
#pragma unroll
            for (int i = 0; i < kSums; ++i) sums[i] = more[i];
        }
        if (!A.dw[w]) continue;
        float *to = smem;                                // [warps][d]
        __syncthreads();
#pragma unroll
        for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                float u = sums[s * P + e], v = sums[(S + s) * P + e];
#pragma unroll
                for (int o = kGroup; o < 32; o <<= 1) {
                    u += __shfl_xor_sync(0xffffffffu, u, o);
                    v += __shfl_xor_sync(0xffffffffu, v, o);
                }
                if (in_warp < kGroup) {
                    if (at[s].has(false)) to[warp * A.d + at[s].col(e, false)] = u;
                    if (at[s].has(true)) to[warp * A.d + at[s].col(e, true)] = v;
                }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < A.d; c += kNormThreads) {
            float u = 0.f;
#pragma unroll
            for (int k = 0; k < kNormThreads / 32; ++k) u += to[k * A.d + c];
            A.part[((int64_t)blockIdx.x * 2 + w) * A.d + c] = u;
        }
    }
}

// Adds the blocks' sums up: a block takes 32 columns of one tensor, its warps every 32nd of the blocks.  It is placed while
// k_norm_grad runs.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) k_norm_dw(const float *part, int d, int blocks, float *dwq, float *dwk) {
    __shared__ float sums[kSumWarps][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    float *dw = blockIdx.y ? dwk : dwq;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!dw) return;
    float u = 0.f;
    if (c < d) {
#pragma unroll
        for (int i = 0; i < (kGradBlocks + kSumWarps - 1) / kSumWarps; ++i) {
            const int k = warp + i * kSumWarps;
            if (k < blocks) u += part[((int64_t)k * 2 + blockIdx.y) * d + c];
        }
    }
    sums[warp][lane] = u;
    __syncthreads();
    // warp w adds the sums of column w of the 32 up, in the warps' order
    float t = sums[lane][warp];
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0 && blockIdx.x * 32 + warp < d) dw[blockIdx.x * 32 + warp] = t;
}

}  // namespace

cudaError_t launch_norm_grad(const NormArgs &a, bool fp16, const NormShape &p, int blocks, int smem, cudaStream_t s) {
    const cudaError_t e = with_shape(p, [&](auto pair, auto v, auto group, auto slots) {
        auto *kernel = fp16 ? k_norm_grad<true, pair.value, v.value, group.value, slots.value>
                            : k_norm_grad<false, pair.value, v.value, group.value, slots.value>;
        if (smem > 48 * 1024) {
            const cudaError_t wide =
                cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (wide != cudaSuccess) return wide;
        }
        kernel<<<blocks, kNormThreads, smem, s>>>(a);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || !(a.dw[0] || a.dw[1])) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.d + 31) / 32, a.heads[1] ? 2 : 1);
    cfg.blockDim = dim3(kSumWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const float *part = a.part;
    return cudaLaunchKernelEx(&cfg, k_norm_dw, part, (int)a.d, blocks, a.dw[0], a.dw[1]);
}

}  // namespace sag
