// Upload of large sequence tables and the descriptor checks around them.
#include "kernels.cuh"
#include "seqtab.cuh"

namespace sag {

namespace {
constexpr int64_t kMaxRows = 2LL * 1024 * 1024;   // rows in all, as for the selected attention

__global__ void k_seq_upload(const __grid_constant__ SeqUpload u, SeqRow *dst, int n) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = u.row[i];
}
}  // namespace

cudaError_t launch_seq_upload(const SeqUpload &u, SeqRow *dst, int n, cudaStream_t s) {
    k_seq_upload<<<1, 256, 0, s>>>(u, dst, n);
    return cudaGetLastError();
}

sag_status check_seqs(int batch, int layout, const int32_t *cu, int32_t s_max) {
    if (!cu) return SAG_ERR_NULL;
    if (layout != SAG_LAYOUT_TND && layout != SAG_LAYOUT_BSND) return SAG_ERR_SHAPE;
    if (batch < 1 || batch > kMaxRows) return SAG_ERR_SHAPE;
    const bool bsnd = layout == SAG_LAYOUT_BSND;
    if (bsnd ? (s_max < 0 || (int64_t)batch * s_max > kMaxRows) : s_max != 0) return SAG_ERR_SHAPE;
    if (cu[0] != 0) return SAG_ERR_SHAPE;
    for (int b = 0; b < batch; ++b) {
        const int64_t n = (int64_t)cu[b + 1] - cu[b];
        if (n < 0 || n > (bsnd ? (int64_t)s_max : kMaxRows)) return SAG_ERR_SHAPE;
    }
    if (cu[batch] > kMaxRows) return SAG_ERR_SHAPE;
    return batch > kMaxSeqs ? SAG_ERR_UNSUPPORTED : SAG_OK;
}

int current_device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        return 148;
    return sms;
}

}  // namespace sag
