// Windowed attention, gradient: launches of k_xdq and k_xdkv (xbwd.cuh) over the tiles that a window reaches.
#include "xbwd.cuh"

namespace sag {

cudaError_t launch_wdq(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s) {
    return launch_bwd<true>(a, io, d, false, true, s);
}

cudaError_t launch_wdkv(const XArgs &a, const sca_io &io, const sca_desc &d, cudaStream_t s) {
    // without query rows there is no kernel of this call before it
    return launch_bwd<true>(a, io, d, true, a.q_tiles > 0, s);
}

}  // namespace sag
