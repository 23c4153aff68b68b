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
// Bound by memory: 4 bytes per element (read once, written once).  A thread
// owns one vector of columns of one token (a pair of vectors for the half
// style), computes that vector's sines once and walks over heads, four loads
// in flight, so sines cost 1 / heads of an element and neighbouring threads
// touch neighbouring columns.
#include <math.h>

#include "kernels.cuh"
#include "seqtab.cuh"

namespace sag {

namespace {

constexpr int kRotThreads = 256;
constexpr int kMaxRot = 256;
constexpr int kHeadsInFlight = 4;

struct RotArgs {
    SeqTab seq;
    uint64_t turns[kMaxRot / 2];        // inv_freq / 2 pi in 2^-64 turns, negated for the gradient
    float magnitude;
    int32_t rows;                       // rows that the call covers
    int32_t n1, n2, d, d_rot, offset, s_max;
    int32_t units, rot_units;           // vectors a head and token, the rotating ones first
    int32_t tokens_per_block, heads_per_block;
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

template <int V>
union Pack {
    typename Vec<V>::T v;
    uint16_t e[V];
};

// kHalf: the vector at column c and its partner at c + d_rot / 2; otherwise V / 2 interleaved pairs in one vector.
template <bool kFp16, bool kHalf, int V>
__global__ void __launch_bounds__(kRotThreads) k_rotary(const __grid_constant__ RotArgs A) {
    constexpr int kPairs = kHalf ? V : V / 2;
    __shared__ uint64_t turns[kMaxRot / 2];
    for (int i = threadIdx.x; i < A.d_rot / 2; i += kRotThreads) turns[i] = A.turns[i];
    __syncthreads();
    const int tok = threadIdx.x / A.units, u = threadIdx.x % A.units;
    const int64_t row64 = (int64_t)blockIdx.x * A.tokens_per_block + tok;
    if (tok >= A.tokens_per_block || row64 >= A.rows) return;
    const int row = (int)row64;

    // the row's sequence, and whether it is padding
    int place = 0;
    bool live = true;
    if (A.s_max) {
        const int b = row / A.s_max;
        place = row - b * A.s_max;
        live = place < seq_get<&SeqRow::qlen>(A.seq, b);
    } else if (!A.positions) {
        place = row - seq_get<&SeqRow::q0>(A.seq, seq_find<&SeqRow::q0>(A.seq, row));
    }
    const bool rot = u < A.rot_units;
    int col;                            // first column of the vector
    float cs[kPairs], sn[kPairs];
    if (rot) {
        col = A.offset + u * V;
        const int64_t p = A.positions && live ? (int64_t)__ldg(A.positions + row) : (int64_t)place;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const int32_t t = (int32_t)(((uint64_t)p * turns[u * kPairs + j]) >> 32);
            sincospif((float)t * 0x1p-31f, &sn[j], &cs[j]);
            sn[j] *= A.magnitude;
            cs[j] *= A.magnitude;
        }
    } else {
        // columns outside [offset, offset + d_rot)
        col = (u - A.rot_units) * V;
        if (col >= A.offset) col += A.d_rot;
    }
    const int half = kHalf && rot ? A.d_rot / 2 : 0;
    const int h_lo = blockIdx.y * A.heads_per_block;
    const int h_hi = min(h_lo + A.heads_per_block, A.n1 + A.n2);
    using T = typename Vec<V>::T;
    auto src = [&](int h) {
        const int w = h >= A.n1;
        return A.in[w] + (int64_t)row * A.in_stride[w] + (int64_t)(h - (w ? A.n1 : 0)) * A.d + col;
    };
    auto dst = [&](int h) {
        const int w = h >= A.n1;
        return A.out[w] + (int64_t)row * A.out_stride[w] + (int64_t)(h - (w ? A.n1 : 0)) * A.d + col;
    };
    for (int h0 = h_lo; h0 < h_hi; h0 += kHeadsInFlight) {
        Pack<V> a[kHeadsInFlight], b[kHeadsInFlight];
#pragma unroll
        for (int i = 0; i < kHeadsInFlight; ++i)
            if (h0 + i < h_hi) {
                if (live) {
                    const uint16_t *p = src(h0 + i);
                    a[i].v = *reinterpret_cast<const T *>(p);
                    if (kHalf) b[i].v = *reinterpret_cast<const T *>(p + half);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) a[i].e[j] = b[i].e[j] = 0;
                }
            }
#pragma unroll
        for (int i = 0; i < kHeadsInFlight; ++i) {
            if (h0 + i >= h_hi) break;
            if (rot && live) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    uint16_t &xa = kHalf ? a[i].e[j] : a[i].e[(2 * j) % V];
                    uint16_t &xb = kHalf ? b[i].e[j] : a[i].e[(2 * j + 1) % V];
                    const float x = u16_to_f<kFp16>(xa), y = u16_to_f<kFp16>(xb);
                    xa = f_to_u16<kFp16>(x * cs[j] - y * sn[j]);
                    xb = f_to_u16<kFp16>(x * sn[j] + y * cs[j]);
                }
            }
            uint16_t *p = dst(h0 + i);
            *reinterpret_cast<T *>(p) = a[i].v;
            if (kHalf && rot) *reinterpret_cast<T *>(p + half) = b[i].v;
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

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard dg;
    if (!dg.bind_memory(io->query_out)) return SAG_ERR_CUDA;
    RotArgs a;
    a.n1 = d->n1;
    a.n2 = d->n2;
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
    a.in_stride[0] = d->q_stride ? d->q_stride : (int64_t)d->n1 * d->d;
    a.in_stride[1] = d->k_stride ? d->k_stride : (int64_t)d->n2 * d->d;
    a.out_stride[0] = d->q_out_stride ? d->q_out_stride : (int64_t)d->n1 * d->d;
    a.out_stride[1] = d->k_out_stride ? d->k_out_stride : (int64_t)d->n2 * d->d;
    for (int i = 0; i < d->d_rot / 2; ++i) {
        // fraction of a turn per position, then 64 bits of it
        double t = d->inv_freq[i] / (2.0 * M_PI);
        t -= floor(t);
        uint64_t q = t >= 1.0 ? 0 : (uint64_t)ldexp(t, 64);
        a.turns[i] = grad ? (uint64_t)0 - q : q;
    }
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
    if (a.units > kRotThreads) return SAG_ERR_UNSUPPORTED;
    if (fill_seq_tab(&a.seq, d->batch, static_cast<SeqRow *>(workspace), s, [&](int b) {
            SeqRow r{};
            r.q0 = bsnd ? b * d->s_max : d->cu_seqlens[b];
            r.qlen = b < d->batch ? d->cu_seqlens[b + 1] - d->cu_seqlens[b] : 0;
            return r;
        }) != cudaSuccess)
        return SAG_ERR_CUDA;
    a.tokens_per_block = kRotThreads / a.units;
    const int heads = d->n1 + d->n2;
    // heads stay together (sines once a token) unless that leaves SMs without blocks: then groups of kHeadsInFlight
    const int64_t blocks = (rows + a.tokens_per_block - 1) / a.tokens_per_block;
    const int64_t want = 8LL * current_device_sms();
    int64_t groups = blocks >= want ? 1 : (want + blocks - 1) / blocks;
    const int64_t most = (heads + kHeadsInFlight - 1) / kHeadsInFlight;
    if (groups > most) groups = most;
    a.heads_per_block = (int)(((heads + groups - 1) / groups + kHeadsInFlight - 1) / kHeadsInFlight * kHeadsInFlight);
    const dim3 grid((unsigned)blocks, (unsigned)((heads + a.heads_per_block - 1) / a.heads_per_block));
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
