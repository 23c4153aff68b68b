// What the rotary positions and the norms with rotation share: checks of a
// descriptor, angles, and two elements of a word.
#pragma once

#include "common.cuh"
#include "seqtab.cuh"

namespace sag {

constexpr int kMaxRot = 256;

sag_status check_rotary(const srt_desc *d);
// inv_freq / 2 pi in 2^-64 turns, negated for the gradient
void rotary_turns(const srt_desc *d, bool grad, uint64_t *turns);

template <bool kFp16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (kFp16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <bool kFp16>
__device__ __forceinline__ uint32_t round2(float a, float b) {
    if constexpr (kFp16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// The row's sequence and place in it; false for padding.
__device__ __forceinline__ bool locate_row(const SeqTab &seq, int s_max, const int32_t *positions, int row, int *place) {
    *place = 0;
    if (s_max) {
        const int b = row / s_max;
        *place = row - b * s_max;
        return *place < seq_get<&SeqRow::qlen>(seq, b);
    }
    if (!positions) *place = row - seq_get<&SeqRow::q0>(seq, seq_find<&SeqRow::q0>(seq, row));
    return true;
}

}  // namespace sag
