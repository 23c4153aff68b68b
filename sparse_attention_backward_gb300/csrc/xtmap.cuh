// Host side of the cross-attention launches: tensor maps and cluster launch.
#pragma once

#include "cross.cuh"
#include "tmap.cuh"

namespace sag {

// [rows, heads, d] 16-bit tensor with its own row stride (elements), box {64 columns, box_heads, box_rows}, 128-byte
// swizzle, out-of-range elements read as zero.
inline bool x_map(CUtensorMap *m, const void *base, bool fp16, int d, int heads, int64_t rows, int64_t stride,
                  int box_heads, int box_rows) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int64_t x_rows_q(const sca_desc &d) {
    return d.layout == SAG_LAYOUT_BSND ? (int64_t)d.batch * d.s1_max : d.cu_seqlens_q[d.batch];
}
inline int64_t x_rows_k(const sca_desc &d) {
    return d.layout == SAG_LAYOUT_BSND ? (int64_t)d.batch * d.s2_max : d.cu_seqlens_kv[d.batch];
}
// A side without rows has no tile that would be loaded; its map is encoded over one row of the other side's tensor.
inline bool x_map_q(CUtensorMap *m, const void *base, const sca_desc &d, const XArgs &a, int64_t stride,
                    const void *other = nullptr) {
    const int64_t rows = x_rows_q(d);
    return x_map(m, rows ? base : other, d.dtype == SAG_FP16, d.d, rows ? d.n1 : d.n2, rows ? rows : 1,
                 rows && stride ? stride : (int64_t)(rows ? d.n1 : d.n2) * d.d, rows ? a.group : 1, a.tpt);
}
inline bool x_map_k(CUtensorMap *m, const void *base, const void *other, const sca_desc &d, int64_t stride,
                    int box_rows) {
    const int64_t rows = x_rows_k(d);
    return x_map(m, rows ? base : other, d.dtype == SAG_FP16, d.d, rows ? d.n2 : d.n1, rows ? rows : 1,
                 rows && stride ? stride : (int64_t)(rows ? d.n2 : d.n1) * d.d, 1, box_rows);
}

// `after`: a kernel of this call that starts while the one before it ends (its CTAs set up, then wait for that one's
// results with grid_wait).
template <class... P, class... Args>
cudaError_t x_launch(void (*kernel)(P...), int ctas, int threads, int cluster, int smem, bool after, cudaStream_t s,
                     const Args &...args) {
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (after) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace sag
