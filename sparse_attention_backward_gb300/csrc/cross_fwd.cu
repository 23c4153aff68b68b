// Cross attention, forward: launches of k_xfwd (xfwd.cuh) over all keys of a sequence.
#include "xfwd.cuh"

namespace sag {

namespace {

template <bool kFp16, int D, int kKeys>
cudaError_t launch(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!x_map_q(&mq, io.query, d, a, d.q_stride) || !x_map_k(&mk, io.key, io.query, d, d.k_stride, kKeys) ||
        !x_map_k(&mv, io.value, io.query, d, d.v_stride, kKeys))
        return cudaErrorInvalidValue;
    return x_launch(k_xfwd<kFp16, D, kKeys, kAll>, a.ctas, kFwdThreads, a.nsplit, FwdShape<D, kKeys>::TOTAL, false, s, mq,
                    mk, mv, a);
}

}  // namespace

// Tiles of 128 keys take 64 cycles a step for their scores where two of 64 take 96 (M = 128 rows re-read per instruction),
// but leave one score tile in flight instead of two.  They are taken for 128-wide heads where products dominate: full
// query tiles and long loops.  Measured, 64 against 128: 8192 x 4096 tokens 825 / 742 us, 130 x 131072 233 / 205;
// 1024 x 1024 33 / 35, 2048 x 512 70 / 74, one token x 4096 69 / 74 us; 64-wide heads 582 / 596 us.  (Sharing a row of 128
// keys between two threads, for a shorter softmax, was slower: 792 us for the first, and 235 for the second.)
cudaError_t launch_xfwd(const XArgs &a, const sca_io &io, const sca_desc &d, bool long_loops, cudaStream_t s) {
    const bool fp16 = d.dtype == SAG_FP16;
    if (d.d == 128 && long_loops)
        return fp16 ? launch<true, 128, 128>(a, io, d, s) : launch<false, 128, 128>(a, io, d, s);
    if (d.d == 128) return fp16 ? launch<true, 128, 64>(a, io, d, s) : launch<false, 128, 64>(a, io, d, s);
    return fp16 ? launch<true, 64, 64>(a, io, d, s) : launch<false, 64, 64>(a, io, d, s);
}

}  // namespace sag
