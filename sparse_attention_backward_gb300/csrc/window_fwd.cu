// Windowed attention, forward, over rows and over pages: launches of k_xfwd and k_xjoin (xfwd.cuh).
#include "xfwd.cuh"

namespace sag {

namespace {

// The cache as the kernel reads it: boxes of `box` rows of a page, 64 columns of one head.
bool cache_map(CUtensorMap *m, const void *base, const spa_desc &d, int64_t row, int64_t page, int box_rows) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d.d, (cuuint64_t)d.n2, (cuuint64_t)d.page_size, (cuuint64_t)d.pages};
    cuuint64_t strides[3] = {(cuuint64_t)d.d * 2, (cuuint64_t)row * 2, (cuuint64_t)page * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, d.dtype == SAG_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFp16, int D, int kKeys, int kMode>
cudaError_t launch(const XArgs &a_in, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t s) {
    // CTAs that run at once take unit after unit
    const int room = 152 * FwdShape<D, kKeys>::CTAS;
    XArgs a = a_in;
    if (x_walks(kMode, D, kKeys) && a.nsplit * a.pieces == 1 && a.ctas > room) a.ctas = a.n_status = room;
    cudaError_t e = x_launch(k_xfwd<kFp16, D, kKeys, kMode>, a.ctas, kFwdThreads, a.nsplit, FwdShape<D, kKeys>::TOTAL, false, s,
                             mq, mk, mv, a);
    if (e != cudaSuccess || a.pieces == 1) return e;
    return x_launch(k_xjoin<kFp16, D>, a.units * a.join_rows, kJoinWarps * 32, 1, 0, true, s, a);
}

template <int kMode>
cudaError_t launch(const XArgs &a, bool fp16, int d, int keys, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                   cudaStream_t s) {
    if (d == 128 && keys == 128)
        return fp16 ? launch<true, 128, 128, kMode>(a, q, k, v, s) : launch<false, 128, 128, kMode>(a, q, k, v, s);
    if (d == 128) return fp16 ? launch<true, 128, 64, kMode>(a, q, k, v, s) : launch<false, 128, 64, kMode>(a, q, k, v, s);
    return fp16 ? launch<true, 64, 64, kMode>(a, q, k, v, s) : launch<false, 64, 64, kMode>(a, q, k, v, s);
}

}  // namespace

cudaError_t launch_wfwd(const XArgs &a, const sca_io &io, const sca_desc &d, bool long_loops, cudaStream_t s) {
    const int keys = d.d == 128 && long_loops ? 128 : 64;
    CUtensorMap mq, mk, mv;
    if (!x_map_q(&mq, io.query, d, a, d.q_stride) || !x_map_k(&mk, io.key, io.query, d, d.k_stride, keys) ||
        !x_map_k(&mv, io.value, io.query, d, d.v_stride, keys))
        return cudaErrorInvalidValue;
    return launch<kBand>(a, d.dtype == SAG_FP16, d.d, keys, mq, mk, mv, s);
}

cudaError_t launch_pfwd(const XArgs &a_in, const spa_io &io, const spa_desc &d, bool long_loops, cudaStream_t s) {
    const int keys = d.d == 128 && long_loops ? 128 : 64;
    XArgs a = a_in;
    a.box = 16;
    while (a.box < keys && d.page_size % (2 * a.box) == 0) a.box *= 2;
    const int64_t rows = d.layout == SAG_LAYOUT_BSND ? (int64_t)d.batch * d.s1_max : d.cu_seqlens_q[d.batch];
    const int64_t row = (int64_t)d.n2 * d.d;
    const int64_t k_row = d.k_row ? d.k_row : row, v_row = d.v_row ? d.v_row : row;
    CUtensorMap mq, mk, mv;
    if (!x_map(&mq, io.query, d.dtype == SAG_FP16, d.d, d.n1, rows, d.q_stride ? d.q_stride : (int64_t)d.n1 * d.d, a.group, a.tpt) ||
        !cache_map(&mk, io.key_cache, d, k_row, d.k_page ? d.k_page : k_row * d.page_size, a.box) ||
        !cache_map(&mv, io.value_cache, d, v_row, d.v_page ? d.v_page : v_row * d.page_size, a.box))
        return cudaErrorInvalidValue;
    return launch<kPaged>(a, d.dtype == SAG_FP16, d.d, keys, mq, mk, mv, s);
}

}  // namespace sag
