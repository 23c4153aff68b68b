// Windowed attention, gradient: launches of k_xdkv and k_xdq (xbwd.cuh) over the tiles that a window reaches.
//
// k_xdkv goes first, since its units are longer, and k_xdq does not wait for it:
// both need only k_xpre, which is complete once k_xdkv lets the next kernel's
// CTAs in.  They start as k_xdkv's leave, and take units by ticket, so the one's
// last, unfilled round is filled by the other.
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
