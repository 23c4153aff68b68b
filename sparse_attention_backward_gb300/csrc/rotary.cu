// Rotary positions of queries and keys, and their gradient (the same map with
// the angle negated).
//
// Mathematics.  A row of position p turns each of its d_rot / 2 pairs of
// columns by the angle p * f_i.  The angle is wanted modulo one turn, so f_i /
// 2 pi is held as a 64-bit fixed-point fraction of a turn and multiplied by
// the integer position modulo 2^64: the whole turns fall off the top exactly,
// whatever the position.  The top 32 bits, as a signed fraction of half a turn,
// go to sincospif.  Each 16-bit output is rounded once, from fp32.
//
// Bound by memory: 4 bytes per element (read once, written once).  A block
// takes a few tokens, or a part of one, and walks over their vectors in the
// order of memory, four loads of a thread in flight, like a copy; the sines of
// its tokens are computed once, into shared memory, while the first loads are on
// their way.  A thread that kept its columns and walked over heads instead had
// its sines in registers, but spread each access over several tokens' rows:
// 106 us against 90 for 32768 tokens of 68 heads of 64 (85 at the measured copy
// rate; 6.3 TB/s).  64 tokens: 3 us, a launch.
#include <math.h>

#include <type_traits>

#include "kernels.cuh"
#include "rotary.cuh"

namespace sag {

sag_status check_rotary(const srt_desc *d) {
    if (!d || !d->cu_seqlens || !d->inv_freq) return SAG_ERR_NULL;
    if (d->dtype != SAG_BF16 && d->dtype != SAG_FP16) return SAG_ERR_DTYPE;
    if (d->style != SRT_HALF && d->style != SRT_INTERLEAVED) return SAG_ERR_SHAPE;
    if (d->n1 < 1 || d->n1 > 128 || d->n2 < 0 || d->n2 > 128 || d->d < 1 || d->d > 512) return SAG_ERR_SHAPE;
    if (d->d_rot < 2 || d->d_rot > kMaxRot || d->d_rot % 2 || d->offset < 0 || d->offset + d->d_rot > d->d)
        return SAG_ERR_SHAPE;
    if (!isfinite(d->magnitude)) return SAG_ERR_SHAPE;
    for (int i = 0; i < d->d_rot / 2; ++i)
        if (!isfinite(d->inv_freq[i])) return SAG_ERR_SHAPE;
    const int64_t st[] = {d->q_stride, d->q_out_stride, d->k_stride, d->k_out_stride};
    for (int i = 0; i < 4; ++i)
        if (st[i] != 0 && (st[i] < (int64_t)(i < 2 ? d->n1 : d->n2) * d->d || st[i] > (1LL << 40))) return SAG_ERR_SHAPE;
    return check_seqs(d->batch, d->layout, d->cu_seqlens, d->s_max);
}

void rotary_turns(const srt_desc *d, bool grad, uint64_t *turns) {
    for (int i = 0; i < d->d_rot / 2; ++i) {
        // fraction of a turn per position, then 64 bits of it
        double t = d->inv_freq[i] / (2.0 * M_PI);
        t -= floor(t);
        uint64_t q = t >= 1.0 ? 0 : (uint64_t)ldexp(t, 64);
        turns[i] = grad ? (uint64_t)0 - q : q;
    }
}

namespace {

constexpr int kRotThreads = 256;
constexpr int kInFlight = 4;
constexpr int kMaxTokens = 256, kMaxSines = 2048;   // of a block

struct RotArgs {
    SeqTab seq;
    uint64_t turns[kMaxRot / 2];        // inv_freq / 2 pi in 2^-64 turns, negated for the gradient
    float magnitude;
    int32_t rows;                       // rows that the call covers
    int32_t n1, d, d_rot, offset, s_max;
    int32_t units, rot_units;           // vectors of a head, the rotating ones first
    int32_t items;                      // vectors of a token: (n1 + n2) * units
    uint32_t by_units, by_items;        // ceil(2^32 / units), ceil(2^32 / items): divisions as multiplications
    int32_t tokens, chunk;              // of a block: tokens, and vectors of them (one token may be split over blockIdx.y)
    const int32_t *positions;
    const uint16_t *in[2];              // query, key
    uint16_t *out[2];
    int64_t in_stride[2], out_stride[2];
};

template <int V> struct Vec;
template <> struct Vec<8> { using T = uint4; };
template <> struct Vec<4> { using T = uint2; };
template <> struct Vec<2> { using T = uint32_t; };
template <> struct Vec<1> { using T = uint16_t; };

// V elements as words of two (V = 1: one element in the low half of a word)
template <int V>
union Pack {
    typename Vec<V>::T v;
    uint32_t w[(V + 1) / 2];
};

// kHalf: the vector at column c and its partner at c + d_rot / 2; otherwise V / 2 interleaved pairs in one vector.
template <bool kFp16, bool kHalf, int V>
__global__ void __launch_bounds__(kRotThreads, 4) k_rotary(const __grid_constant__ RotArgs A) {
    constexpr int kWords = (V + 1) / 2;
    constexpr int kPairs = kHalf ? V : V / 2;            // of a rotating vector
    // Sines of a word: (cos, cos, sin, sin) of its two pairs (half style), (cos, sin) of its one (interleaved), at
    // [token][word][rotating vector], so that neighbouring threads read neighbours.
    using Sines = typename std::conditional<kHalf, float4, float2>::type;
    using T = typename Vec<V>::T;
    __shared__ uint64_t turns[kMaxRot / 2];
    __shared__ Sines table[kHalf && V > 1 ? kMaxSines / 2 : kMaxSines];
    __shared__ int8_t is_live[kMaxTokens];
    const int row0 = blockIdx.x * A.tokens, n_tok = min(A.tokens, A.rows - row0);
    const int lo = blockIdx.y * A.chunk, hi = min(lo + A.chunk, n_tok * A.items);
    const int words = kWords * A.rot_units;              // of a token in the table

    auto locate = [&](int row, int *place) { return locate_row(A.seq, A.s_max, A.positions, row, place); };
    for (int i = threadIdx.x; i < A.d_rot / 2; i += kRotThreads) turns[i] = A.turns[i];
    if (threadIdx.x < n_tok) {
        int place;
        is_live[threadIdx.x] = locate(row0 + threadIdx.x, &place);
    }
    __syncthreads();

    Pack<V> a[kInFlight], b[kInFlight];
    uint16_t *to[kInFlight];
    int sines[kInFlight];               // place in the table; -1: of a padding row, -2: passes unchanged
    // loads vectors i, i + kRotThreads, ...
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int i = i0 + k * kRotThreads;
            if (i >= hi) break;
            const int tok = A.tokens == 1 ? 0 : A.items > 1 ? (int)__umulhi((uint32_t)i, A.by_items) : i;
            const int at = i - tok * A.items;
            int head = A.units > 1 ? (int)__umulhi((uint32_t)at, A.by_units) : at;
            const int u = at - head * A.units;
            const int w = head >= A.n1;
            head -= w ? A.n1 : 0;
            const bool turning = u < A.rot_units, live = is_live[tok];
            int col = turning ? A.offset + u * V : (u - A.rot_units) * V;
            if (!turning && col >= A.offset) col += A.d_rot;
            const int64_t row = row0 + tok;
            const uint16_t *p = A.in[w] + row * A.in_stride[w] + (head * A.d + col);
            to[k] = A.out[w] + row * A.out_stride[w] + (head * A.d + col);
            sines[k] = turning ? (live ? tok * words + u : -1) : -2;
            a[k].v = b[k].v = T{};
            if (live) {
                a[k].v = *reinterpret_cast<const T *>(p);
                if (kHalf && turning) b[k].v = *reinterpret_cast<const T *>(p + A.d_rot / 2);
            }
        }
    };
    int i = lo + threadIdx.x;
    load(i);
    // sines, while the first vectors are on their way
    const int pairs = A.d_rot / 2;
    float *flat = reinterpret_cast<float *>(table);
    for (int j = threadIdx.x; j < n_tok * pairs; j += kRotThreads) {
        const int tok = j / pairs, pair = j - tok * pairs, row = row0 + tok;
        int place;
        if (!locate(row, &place)) continue;
        const int64_t p = A.positions ? (int64_t)__ldg(A.positions + row) : (int64_t)place;
        const int32_t t = (int32_t)(((uint64_t)p * turns[pair]) >> 32);
        float sn, cs;
        sincospif((float)t * 0x1p-31f, &sn, &cs);
        const int in_vec = pair % kPairs, per_word = kHalf && V > 1 ? 2 : 1;
        float *at = flat + (tok * words + in_vec / per_word * A.rot_units + pair / kPairs) * (kHalf ? 4 : 2);
        at[in_vec % per_word] = cs * A.magnitude;
        at[(kHalf ? 2 : 1) + in_vec % per_word] = sn * A.magnitude;
    }
    __syncthreads();
    for (; i < hi; i += kInFlight * kRotThreads) {
        if (i >= lo + kInFlight * kRotThreads) load(i);
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            if (i + k * kRotThreads >= hi) break;
            if (sines[k] >= 0) {
#pragma unroll
                for (int j = 0; j < kWords; ++j) {
                    const Sines t = table[sines[k] + j * A.rot_units];
                    if constexpr (kHalf && V == 1) {
                        const float x = u16_to_f<kFp16>((uint16_t)a[k].w[0]), y = u16_to_f<kFp16>((uint16_t)b[k].w[0]);
                        a[k].w[0] = f_to_u16<kFp16>(x * t.x - y * t.z);
                        b[k].w[0] = f_to_u16<kFp16>(x * t.z + y * t.x);
                    } else if constexpr (kHalf) {
                        const float2 x = unpack2<kFp16>(a[k].w[j]), y = unpack2<kFp16>(b[k].w[j]);
                        a[k].w[j] = round2<kFp16>(x.x * t.x - y.x * t.z, x.y * t.y - y.y * t.w);
                        b[k].w[j] = round2<kFp16>(x.x * t.z + y.x * t.x, x.y * t.w + y.y * t.y);
                    } else {
                        const float2 x = unpack2<kFp16>(a[k].w[j]);
                        a[k].w[j] = round2<kFp16>(x.x * t.x - x.y * t.y, x.x * t.y + x.y * t.x);
                    }
                }
            }
            *reinterpret_cast<T *>(to[k]) = a[k].v;
            if (kHalf && sines[k] >= -1) *reinterpret_cast<T *>(to[k] + A.d_rot / 2) = b[k].v;
        }
    }
}

template <bool kFp16, bool kHalf>
cudaError_t launch_vec(const RotArgs &a, int vec, dim3 grid, cudaStream_t s) {
    switch (vec) {
    case 8: k_rotary<kFp16, kHalf, 8><<<grid, kRotThreads, 0, s>>>(a); break;
    case 4: k_rotary<kFp16, kHalf, 4><<<grid, kRotThreads, 0, s>>>(a); break;
    case 2: k_rotary<kFp16, kHalf, 2><<<grid, kRotThreads, 0, s>>>(a); break;
    default:
        if constexpr (kHalf) k_rotary<kFp16, true, 1><<<grid, kRotThreads, 0, s>>>(a);
        break;
    }
    return cudaGetLastError();
}

sag_status run_rotary(const srt_desc *d, const srt_io *io, void *workspace, size_t workspace_bytes, void *stream,
                      bool grad) {
    sag_status st = check_rotary(d);
    if (st != SAG_OK) return st;
    const bool bsnd = d->layout == SAG_LAYOUT_BSND;
    const int32_t rows = bsnd ? d->batch * d->s_max : d->cu_seqlens[d->batch];
    const size_t need = seq_ws_bytes(d->batch);
    if (!io) return SAG_ERR_NULL;
    if (need && (!workspace || workspace_bytes < need)) return SAG_ERR_WORKSPACE;
    auto off16 = [](const void *p, int mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
    if (need && off16(workspace, 15)) return SAG_ERR_ALIGN;
    if (rows == 0) return SAG_OK;
    if (!io->query || !io->query_out || (d->n2 && (!io->key || !io->key_out))) return SAG_ERR_NULL;
    if (off16(io->query, 15) || off16(io->query_out, 15) || off16(io->positions, 3) ||
        (d->n2 && (off16(io->key, 15) || off16(io->key_out, 15))))
        return SAG_ERR_ALIGN;
    RotArgs a;
    a.in_stride[0] = d->q_stride ? d->q_stride : (int64_t)d->n1 * d->d;
    a.in_stride[1] = d->k_stride ? d->k_stride : (int64_t)d->n2 * d->d;
    a.out_stride[0] = d->q_out_stride ? d->q_out_stride : (int64_t)d->n1 * d->d;
    a.out_stride[1] = d->k_out_stride ? d->k_out_stride : (int64_t)d->n2 * d->d;
    // an output over its own input has to have its rows where the input has them
    if ((io->query == io->query_out && a.in_stride[0] != a.out_stride[0]) ||
        (d->n2 && io->key == io->key_out && a.in_stride[1] != a.out_stride[1]))
        return SAG_ERR_SHAPE;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard wg, dg;
    if (need && !wg.bind_memory(workspace)) return SAG_ERR_CUDA;         // a kernel writes there: host memory is refused
    if (!dg.bind_memory(io->query_out)) return SAG_ERR_CUDA;
    a.n1 = d->n1;
    a.d = d->d;
    a.d_rot = d->d_rot;
    a.offset = d->offset;
    a.s_max = bsnd ? d->s_max : 0;
    a.rows = rows;
    a.magnitude = (float)d->magnitude;
    a.positions = io->positions;
    a.in[0] = static_cast<const uint16_t *>(io->query);
    a.in[1] = static_cast<const uint16_t *>(io->key);
    a.out[0] = static_cast<uint16_t *>(io->query_out);
    a.out[1] = static_cast<uint16_t *>(io->key_out);
    rotary_turns(d, grad, a.turns);
    // widest vector that every address, stride and part boundary allows
    const bool half = d->style == SRT_HALF;
    int64_t all = (int64_t)d->d | d->offset | (half ? d->d_rot / 2 : d->d_rot) | a.in_stride[0] | a.out_stride[0];
    if (d->n2) all |= a.in_stride[1] | a.out_stride[1];
    int vec = 8;
    while (vec > 1 && (all % vec)) vec >>= 1;
    // an odd column count leaves interleaved pairs at odd addresses: single elements, handled as vectors of two, would
    // be misaligned, so such heads are refused
    if (!half && vec == 1) return SAG_ERR_UNSUPPORTED;
    a.rot_units = half ? d->d_rot / 2 / vec : d->d_rot / vec;
    // in place, the columns that pass unchanged are where they belong -- except padding rows, which get zeros
    const bool inplace = io->query == io->query_out && a.in_stride[0] == a.out_stride[0] &&
                         (!d->n2 || (io->key == io->key_out && a.in_stride[1] == a.out_stride[1]));
    a.units = a.rot_units + (inplace && !bsnd ? 0 : (d->d - d->d_rot) / vec);
    if (fill_seq_tab(&a.seq, d->batch, static_cast<SeqRow *>(workspace), s, [&](int b) {
            SeqRow r{};
            r.q0 = bsnd ? b * d->s_max : d->cu_seqlens[b];
            r.qlen = b < d->batch ? d->cu_seqlens[b + 1] - d->cu_seqlens[b] : 0;
            return r;
        }) != cudaSuccess)
        return SAG_ERR_CUDA;
    a.items = (d->n1 + d->n2) * a.units;
    a.by_units = (uint32_t)(((1ull << 32) + a.units - 1) / a.units);     // exact below 2^16 * 2^16
    a.by_items = (uint32_t)(((1ull << 32) + a.items - 1) / a.items);
    // several rounds of loads a block where there is work for all SMs; else one round, of a part of a token if need be
    const int64_t total = (int64_t)rows * a.items;
    const int round = kRotThreads * kInFlight;
    const int64_t want = total / ((int64_t)current_device_sms() * 8);
    const int target = want >= 2 * round ? 2 * round : want >= round ? round : kRotThreads;
    int tokens = target / a.items;
    if (tokens > kMaxTokens) tokens = kMaxTokens;
    if (tokens > kMaxSines / (d->d_rot / 2)) tokens = kMaxSines / (d->d_rot / 2);
    a.tokens = tokens < 1 ? 1 : tokens;
    a.chunk = a.tokens > 1 || a.items <= target ? a.tokens * a.items : target;
    const dim3 grid((unsigned)((rows + a.tokens - 1) / a.tokens),
                    (unsigned)((a.tokens * a.items + a.chunk - 1) / a.chunk));
    const bool fp16 = d->dtype == SAG_FP16;
    const cudaError_t e = fp16 ? (half ? launch_vec<true, true>(a, vec, grid, s) : launch_vec<true, false>(a, vec, grid, s))
                               : (half ? launch_vec<false, true>(a, vec, grid, s) : launch_vec<false, false>(a, vec, grid, s));
    return e == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
}

}  // namespace
}  // namespace sag

using namespace sag;

extern "C" sag_status rotary_frequencies(int32_t d_rot, double base, int32_t scaling, double factor,
                                         double original_length, double beta_fast, double beta_slow, double low,
                                         double high, double *inv_freq, double *magnitude) {
    if (!inv_freq || !magnitude) return SAG_ERR_NULL;
    if (d_rot < 2 || d_rot > kMaxRot || d_rot % 2 || !(base > 1.0) || !isfinite(base)) return SAG_ERR_SHAPE;
    if (scaling < SRT_SCALE_NONE || scaling > SRT_SCALE_BANDS) return SAG_ERR_SHAPE;
    if (scaling != SRT_SCALE_NONE && (!(factor >= 1.0) || !isfinite(factor))) return SAG_ERR_SHAPE;
    if (scaling == SRT_SCALE_BASE && d_rot < 4) return SAG_ERR_SHAPE;
    if (scaling >= SRT_SCALE_RAMP && (!(original_length >= 1.0) || !isfinite(original_length))) return SAG_ERR_SHAPE;
    if (scaling == SRT_SCALE_RAMP && (!(beta_slow > 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast)))
        return SAG_ERR_SHAPE;
    if (scaling == SRT_SCALE_BANDS && (!(low >= 0.0) || !(high > low) || !isfinite(high))) return SAG_ERR_SHAPE;
    if (scaling == SRT_SCALE_BASE) base *= pow(factor, (double)d_rot / (d_rot - 2));
    // pair index at which a pair makes `beta` turns over the original length
    auto edge = [&](double beta) { return d_rot * log(original_length / (2.0 * M_PI * beta)) / (2.0 * log(base)); };
    double lo = 0, hi = 1;
    if (scaling == SRT_SCALE_RAMP) {
        lo = fmax(floor(edge(beta_fast)), 0.0);
        hi = fmin(ceil(edge(beta_slow)), d_rot - 1.0);
    }
    for (int i = 0; i < d_rot / 2; ++i) {
        double f = pow(base, -2.0 * i / d_rot);
        double keep = 1.0;      // share that is not divided by the factor
        if (scaling == SRT_SCALE_LINEAR) keep = 0.0;
        if (scaling == SRT_SCALE_RAMP) keep = 1.0 - fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
        if (scaling == SRT_SCALE_BANDS)
            keep = fmin(fmax((original_length * f / (2.0 * M_PI) - low) / (high - low), 0.0), 1.0);
        inv_freq[i] = keep == 1.0 ? f : f * keep + f / factor * (1.0 - keep);
    }
    *magnitude = scaling == SRT_SCALE_RAMP ? 0.1 * log(factor) + 1.0 : 1.0;
    return SAG_OK;
}

extern "C" sag_status rotary_workspace_size(const srt_desc *desc, size_t *workspace_bytes) {
    if (!workspace_bytes) return SAG_ERR_NULL;
    const sag_status st = check_rotary(desc);
    if (st != SAG_OK) return st;
    *workspace_bytes = seq_ws_bytes(desc->batch);
    return SAG_OK;
}

extern "C" sag_status rotary_fwd(const srt_desc *desc, const srt_io *io, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    return run_rotary(desc, io, workspace, workspace_bytes, stream, false);
}

extern "C" sag_status rotary_grad(const srt_desc *desc, const srt_io *io, void *workspace, size_t workspace_bytes,
                                  void *stream) {
    return run_rotary(desc, io, workspace, workspace_bytes, stream, true);
}
