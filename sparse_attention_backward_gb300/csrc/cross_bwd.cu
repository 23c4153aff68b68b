// Cross attention, gradient: launches of k_xpre, k_xdq and k_xdkv (xbwd.cuh) over all keys of a sequence.
#include "xbwd.cuh"

namespace sag {

cudaError_t launch_xpre(const XArgs &a, bool fp16, int d, cudaStream_t s) {
    const int64_t ctas = (int64_t)a.q_tiles * a.n2 + (fp16 || a.mask || a.s2_pad ? (int64_t)a.k_tiles * a.n2 : 0);
    if (ctas == 0) return cudaSuccess;
    if (d == 128) {
        if (fp16 && a.key_norms) k_xpre<true, 128, true><<<(unsigned)ctas, 256, 0, s>>>(a);
        else if (fp16) k_xpre<true, 128, false><<<(unsigned)ctas, 256, 0, s>>>(a);
        else k_xpre<false, 128, false><<<(unsigned)ctas, 256, 0, s>>>(a);
    } else {
        if (fp16 && a.key_norms) k_xpre<true, 64, true><<<(unsigned)ctas, 256, 0, s>>>(a);
        else if (fp16) k_xpre<true, 64, false><<<(unsigned)ctas, 256, 0, s>>>(a);
        else k_xpre<false, 64, false><<<(unsigned)ctas, 256, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_xdq(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s) {
    return launch_bwd<false>(a, io, d, false, true, s);
}

cudaError_t launch_xdkv(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s) {
    // without query rows there is no kernel of this call before it
    const bool after = a.q_tiles > 0;
    return launch_bwd<false>(a, io, d, true, after, s);
}

}  // namespace sag
