// Norms with rotation: forward, C ABI (norm_rotary.cuh).
//
// 4 bytes an element.  A block takes a tile of tokens, queries and keys, or a
// part of one token's heads; two heads' loads are on their way beyond a group's
// current one.  32768 tokens of 68 heads of 128: 180 us, 6.3 TB/s (blocks that
// walked over tiles, with the next one's loads ahead, had more instructions and
// a third of the registers less for loads: 208 us).  16 tokens: 3.6 us, a launch.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "norm_rotary.cuh"

namespace sag {

namespace {

template <bool kFp16, bool kPair, int V, int kGroup, int S>
__global__ void __launch_bounds__(kNormThreads, V == 1 ? 1 : S == 3 ? 2 : 4) k_norm_fwd(const __grid_constant__ NormArgs A) {
    using I = Item<kFp16, kPair, V>;
    constexpr int P = I::P, kGroups = kNormThreads / kGroup;
    extern __shared__ __align__(16) float smem[];        // sines, [query, key] weights
    __shared__ uint64_t turns[kMaxRot / 2];
    __shared__ TileRows rows;
    const int n1 = A.heads[0], heads = n1 + A.heads[1], half = A.d_rot / 2;
    const int tile = blockIdx.x / A.parts, row0 = tile * A.tokens, n_tok = min(A.tokens, A.rows - row0);
    const int lo = (blockIdx.x - tile * A.parts) * A.chunk, hi = min(lo + A.chunk, n_tok * heads);
    const int group = threadIdx.x / kGroup, lane = threadIdx.x % kGroup, wsize = 2 * A.units * P;
    const bool padded = A.s_max != 0;
    rows.fill(A, row0, n_tok);
    if (padded) __syncthreads();                         // only padded batches have rows that are not loaded
    Place<kPair, V> at[S];
#pragma unroll
    for (int s = 0; s < S; ++s) at[s] = Place<kPair, V>(A, lane + s * kGroup);
    // a group's heads, one every kGroups
    const int by_tok = kGroups / heads, by_head = kGroups % heads;
    int tok = (lo + group) / heads, head = lo + group - tok * heads, left = hi - lo - group;
    struct Ahead {
        I x[S];
        int tok, head;
    };
    auto load = [&](Ahead &a) {
        a.tok = tok;
        a.head = head;
        if (left > 0 && (!padded || rows.live[tok])) {
            const int w = head >= n1;
            const uint16_t *p = A.in[w] + ((int64_t)(row0 + tok) * A.in_stride[w] + (head - (w ? n1 : 0)) * A.d);
#pragma unroll
            for (int s = 0; s < S; ++s) a.x[s].load(p, at[s]);
        }
        tok += by_tok;
        head += by_head;
        if (head >= heads) {
            head -= heads;
            ++tok;
        }
        left -= kGroups;
    };
    Ahead first, second;                                 // what is never loaded stays zero
#pragma unroll
    for (int s = 0; s < S; ++s) first.x[s].zero(), second.x[s].zero();
    load(first);
    load(second);
    for (int i = threadIdx.x; i < half; i += kNormThreads) turns[i] = A.turns[i];
    float *weights = smem + norm_sines(A.tokens, A.d_rot);
    fill_weights<kFp16, kPair, V>(A, 0, weights);
    if (A.heads[1]) fill_weights<kFp16, kPair, V>(A, 1, weights + wsize);
    __syncthreads();
    fill_sines<P>(A, turns, smem, rows, n_tok);
    __syncthreads();
    int todo = hi - lo;
    auto work = [&](Ahead &a) {
        float2 sq = make_float2(0.f, 0.f);
        float fa[S][P], fb[S][P];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            a.x[s].get(fa[s], fb[s]);
            pairs<P>([&](int k) {
                const float2 u = at2<P>(fa[s], k), v = at2<P>(fb[s], k);
                sq = fma2(v, v, fma2(u, u, sq));
            });
        }
        const int t = a.tok, h = a.head;
        const bool mine = todo > group, live = !padded || (mine && rows.live[t]);
        load(a);                                         // two rounds on
        const float r = norm_rsqrt(group_sum<kGroup>(sq.x + sq.y) * A.inv_d + A.eps);
        todo -= kGroups;
        if (!mine) return;
        const int w = h >= n1;
        uint16_t *to = A.out[w] + ((int64_t)(row0 + t) * A.out_stride[w] + (h - (w ? n1 : 0)) * A.d);
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int it = lane + s * kGroup;
            if (!at[s].has_a) continue;
            if (live) {
                float wa[P], wb[P];
                read_weights<P>(weights + w * wsize, it, A.units, wa, wb);
                pairs<P>([&](int k) {
                    put2<P>(fa[s], k, mul2(at2<P>(fa[s], k), mul2(at2<P>(wa, k), r2)));
                    put2<P>(fb[s], k, mul2(at2<P>(fb[s], k), mul2(at2<P>(wb, k), r2)));
                });
                if (at[s].turns) {
                    float cs[P], sn[P];
                    run_read<P>(smem + t * A.d_rot, it, A.rot_units, cs);
                    run_read<P>(smem + t * A.d_rot + half, it, A.rot_units, sn);
                    turn<P>(fa[s], fb[s], cs, sn);
                }
            } else {                                     // padding
#pragma unroll
                for (int e = 0; e < P; ++e) fa[s][e] = fb[s][e] = 0.f;
            }
            I::store(to, at[s], fa[s], fb[s]);
        }
    };
    while (todo > 0) {                                   // the same for the block
        work(first);
        if (todo > 0) work(second);
    }
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs &a, bool fp16, const NormShape &p, int blocks, int smem, cudaStream_t s) {
    return with_shape(p, [&](auto pair, auto v, auto group, auto slots) {
        if (fp16) k_norm_fwd<true, pair.value, v.value, group.value, slots.value><<<blocks, kNormThreads, smem, s>>>(a);
        else k_norm_fwd<false, pair.value, v.value, group.value, slots.value><<<blocks, kNormThreads, smem, s>>>(a);
        return cudaGetLastError();
    });
}

namespace {

// ---------------------------------------------------------------- host side
sag_status check_norm(const snr_desc *d) {
    if (!d) return SAG_ERR_NULL;
    const sag_status st = check_rotary(&d->rotary);
    if (st != SAG_OK && st != SAG_ERR_UNSUPPORTED) return st;
    if (!(d->eps > 0.0) || !isfinite(d->eps) || !((float)d->eps >= FLT_MIN) || !isfinite((float)d->eps) || !isfinite(d->weight_offset) ||
        (d->weight_fp32 != 0 && d->weight_fp32 != 1) || d->reserved_ != 0)
        return SAG_ERR_SHAPE;
    const int64_t sy[] = {d->q_grad_stride, d->k_grad_stride};
    for (int i = 0; i < 2; ++i)
        if (sy[i] != 0 && (sy[i] < (int64_t)(i ? d->rotary.n2 : d->rotary.n1) * d->rotary.d || sy[i] > (1LL << 40)))
            return SAG_ERR_SHAPE;
    return st;
}

size_t seq_part(int batch) { return (seq_ws_bytes(batch) + 255) / 256 * 256; }
size_t norm_ws(const snr_desc *d, bool grad) {
    if (!grad) return seq_ws_bytes(d->rotary.batch);
    return seq_part(d->rotary.batch) + sizeof(float) * 2 * kGradBlocks * d->rotary.d;
}

int norm_units(const srt_desc &d, const NormShape &p) {
    const int others = (d.d - d.d_rot) / p.vec;
    return p.pair ? d.d_rot / 2 / p.vec + (others + 1) / 2 : d.d_rot / p.vec + others;
}

// Threads of a head are a power of two, so heads of 192 or 80 columns would leave a quarter to a third of them without work
// with one item each; three smaller items a thread fit better.  Of shapes that leave as many idle, the one with more
// elements a thread.  32768 tokens of 40 heads of 192 columns in halves, one item against three: 214 and 190 us forward.
NormShape norm_shape(const srt_desc &d, int vec) {
    const bool half = d.style == SRT_HALF;
    if (vec == 1 || (!half && vec < 8)) return {1, 1, 32, 8};
    NormShape best{0, 0, 0, 0};
    int places = 0;
    auto consider = [&](int v, int pair, int slots) {
        NormShape p{v, pair, 4, slots};
        const int units = norm_units(d, p);
        while (p.group * slots < units) p.group *= 2;
        if (p.group > 32) return;
        const int n = p.group * slots * v * (pair ? 2 : 1);             // elements there would be room for
        if (places && n >= places) return;
        places = n;
        best = p;
    };
    if (half) {
        if (vec == 8) consider(8, 1, 1);
        consider(4, 1, 3);
    } else {
        consider(8, 0, 2);
        consider(8, 0, 3);
    }
    return best.vec ? best : NormShape{1, 1, 32, 8};
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
        if (off(weights[i], desc->weight_fp32 ? 3 : 1) || (grad && off(dws[i], 3))) return SAG_ERR_ALIGN;
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
    a.heads[0] = d->n1;
    a.heads[1] = d->n2;
    a.d = d->d;
    a.d_rot = d->d_rot;
    a.offset = d->offset;
    a.s_max = bsnd ? d->s_max : 0;
    a.half = d->style == SRT_HALF;
    a.weight_fp32 = desc->weight_fp32;
    a.positions = io->positions;
    // vectors as wide as every address, stride and part boundary allows
    int64_t all = (int64_t)d->d | d->offset | (a.half ? d->d_rot / 2 : d->d_rot);
    for (int i = 0; i < sides; ++i) all |= a.in_stride[i] | a.out_stride[i] | (grad ? a.dy_stride[i] : 0);
    const NormShape shape = norm_shape(*d, all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 1);
    a.rot_units = shape.pair ? d->d_rot / 2 / shape.vec : d->d_rot / shape.vec;
    a.units = norm_units(*d, shape);
    const int groups = kNormThreads / shape.group;
    if (fill_seq_tab(&a.seq, d->batch, static_cast<SeqRow *>(workspace), s, [&](int b) {
            SeqRow r{};
            r.q0 = bsnd ? b * d->s_max : d->cu_seqlens[b];
            r.qlen = b < d->batch ? d->cu_seqlens[b + 1] - d->cu_seqlens[b] : 0;
            return r;
        }) != cudaSuccess)
        return SAG_ERR_CUDA;
    const int heads = d->n1 + d->n2;
    // Tokens of a tile: about `target` heads, so many that they fill the groups' last round.
    auto tokens_of = [&](int64_t target, int per) {
        int most = kMaxSines / (d->d_rot / 2);
        if (most > kMaxNormTokens) most = kMaxNormTokens;
        int64_t t = target / per;
        if (t > most) t = most;
        if (t < 1) t = 1;
        int best = (int)t;
        auto waste = [&](int64_t x) { return (double)((x * per + groups - 1) / groups * groups) / (double)(x * per); };
        for (int x = best; x <= 2 * t && x <= most; ++x)
            if (waste(x) < waste(best) - 0.01) best = x;
        return best;
    };
    const int P = shape.pair ? shape.vec : shape.vec / 2;
    const int held = 2 * a.units * P;                    // floats of a tensor's weights
    int64_t blocks;
    int smem;
    if (!grad) {
        // several rounds of heads a block where there is work for all SMs; else one, of a part of a token if need be
        const int64_t want = (int64_t)rows * heads / ((int64_t)current_device_sms() * 8);
        const int64_t target = want >= 16 * groups ? 16 * groups : want >= groups ? want / groups * groups : groups;
        a.tokens = target >= heads ? tokens_of(target, heads) : 1;
        a.chunk = a.tokens > 1 || heads <= target ? a.tokens * heads : (int)target;
        a.parts = (a.tokens * heads + a.chunk - 1) / a.chunk;
        blocks = (int64_t)((rows + a.tokens - 1) / a.tokens) * a.parts;
        smem = (norm_sines(a.tokens, d->d_rot) + sides * held) * (int)sizeof(float);
    } else {
        // each block walks over tiles, four or more if there are as many
        const int64_t share = (int64_t)rows * heads / kGradBlocks / 4;
        a.tokens = tokens_of(share < 8 * groups ? share : 8 * groups, heads);
        const int64_t tiles = ((int64_t)rows + a.tokens - 1) / a.tokens;
        blocks = tiles < kGradBlocks ? tiles : kGradBlocks;
        a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + seq_part(d->batch));
        smem = (2 * norm_sines(a.tokens, d->d_rot) + sides * held + 2 * shape.slots * P * kNormThreads) * (int)sizeof(float);
        if (smem < kNormThreads / 32 * d->d * (int)sizeof(float)) smem = kNormThreads / 32 * d->d * (int)sizeof(float);
    }
    const bool fp16 = d->dtype == SAG_FP16;
    const cudaError_t e = grad ? launch_norm_grad(a, fp16, shape, (int)blocks, smem, s)
                               : launch_norm_fwd(a, fp16, shape, (int)blocks, smem, s);
    return e == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
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
