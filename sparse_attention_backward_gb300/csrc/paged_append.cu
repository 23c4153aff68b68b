// New tokens' keys and values into their places of a paged cache.
//
// Bound by memory: 2 bytes read and 2 written an element, or, for a step of few
// tokens, by a launch and two dependent reads (length, page).  A warp takes a
// token; its first loads are on their way before it looks the page up.
#include "kernels.cuh"
#include "xplan.cuh"

namespace sag {

namespace {

constexpr int kThreads = 256, kInFlight = 4;
constexpr int kMaxBlocks = 152 * 8;

struct AppendArgs {
    SeqTab seq;
    int32_t rows, s_max;
    int32_t vecs;                       // 16-byte vectors of a token's keys (and of its values)
    int32_t page, pages, width;
    const int32_t *table, *klens;
    const uint16_t *in[2];              // key, value
    uint16_t *cache[2];
    int64_t in_stride[2], row[2], page_stride[2];
    int32_t *count, *status;
};

__global__ void __launch_bounds__(kThreads) k_append(const __grid_constant__ AppendArgs A) {
    __shared__ int bad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    const int total = 2 * A.vecs;
    for (int row = blockIdx.x * (kThreads / 32) + warp; row < A.rows; row += gridDim.x * (kThreads / 32)) {
        int b, place;
        if (A.s_max) {
            b = row / A.s_max;
            place = row - b * A.s_max;
        } else {
            b = seq_find<&SeqRow::q0>(A.seq, row);
            place = row - seq_get<&SeqRow::q0>(A.seq, b);
        }
        const int qlen = seq_get<&SeqRow::qlen>(A.seq, b);
        if (place >= qlen) continue;                     // padding
        uint4 x[kInFlight];
        auto load = [&](int i0) {
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                const int i = i0 + k * 32, w = i >= A.vecs;
                if (i < total) x[k] = *reinterpret_cast<const uint4 *>(A.in[w] + row * A.in_stride[w] + (i - w * A.vecs) * 8);
            }
        };
        load(lane);
        const int given = __ldg(A.klens + b), klen = min(max(given, 0), A.width * A.page);
        const int at = klen - qlen + place;
        if (given != klen) bad = 1;
        if (at < 0) continue;
        const int id = __ldg(A.table + (int64_t)b * A.width + at / A.page);
        if ((unsigned)id >= (unsigned)A.pages) {
            bad = 1;
            continue;
        }
        const int in_page = at % A.page;
        uint16_t *to[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) to[w] = A.cache[w] + id * A.page_stride[w] + in_page * A.row[w];
        for (int i0 = lane; i0 < total; i0 += 32 * kInFlight) {
            if (i0 != lane) load(i0);
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                const int i = i0 + k * 32, w = i >= A.vecs;
                if (i < total) *reinterpret_cast<uint4 *>((w ? to[1] : to[0]) + (i - w * A.vecs) * 8) = x[k];
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        A.status[blockIdx.x] = bad ? SAG_ERR_INDEX : SAG_OK;
        if (blockIdx.x == 0) *A.count = gridDim.x;
    }
}

size_t append_ws(const spa_desc *d, size_t *o_seq) {
    *o_seq = up256(kStatusAt + sizeof(int32_t) * kMaxBlocks);
    return up256(*o_seq + seq_ws_bytes(d->batch));
}

}  // namespace
}  // namespace sag

using namespace sag;

extern "C" sag_status paged_append_workspace_size(const spa_desc *desc, size_t *workspace_bytes) {
    if (!workspace_bytes) return SAG_ERR_NULL;
    const sag_status st = check_paged(desc);
    size_t o_seq;
    if (st == SAG_OK) *workspace_bytes = append_ws(desc, &o_seq);
    return st;
}

extern "C" sag_status paged_append(const spa_desc *d, const spa_io *io, void *workspace, size_t workspace_bytes, void *stream) {
    const sag_status st = check_paged(d);
    if (st != SAG_OK) return st;
    if (!io) return SAG_ERR_NULL;
    const bool bsnd = d->layout == SAG_LAYOUT_BSND;
    const int32_t rows = bsnd ? d->batch * d->s1_max : d->cu_seqlens_q[d->batch];
    const void *need[] = {io->key, io->value, io->key_cache, io->value_cache};
    if (rows) {
        for (const void *x : need)
            if (!x) return SAG_ERR_NULL;
        if (!io->page_table || !io->kv_lens) return SAG_ERR_NULL;
    }
    size_t o_seq;
    if (!workspace || workspace_bytes < append_ws(d, &o_seq)) return SAG_ERR_WORKSPACE;
    auto off = [](const void *x, int mask) { return (reinterpret_cast<uintptr_t>(x) & mask) != 0; };
    if (rows) {
        for (const void *x : need)
            if (off(x, 15)) return SAG_ERR_ALIGN;
        if (off(io->page_table, 3) || off(io->kv_lens, 3)) return SAG_ERR_ALIGN;
    }
    if (off(workspace, 15)) return SAG_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard dg;
    if (!dg.bind_memory(workspace)) return SAG_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    if (rows == 0) return cudaMemsetAsync(ws, 0, sizeof(int32_t), s) == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
    AppendArgs a{};
    const int64_t dense = (int64_t)d->n2 * d->d;
    const int64_t in[] = {d->k_stride, d->v_stride}, row[] = {d->k_row, d->v_row}, page[] = {d->k_page, d->v_page};
    for (int i = 0; i < 2; ++i) {
        a.in_stride[i] = in[i] ? in[i] : dense;
        a.row[i] = row[i] ? row[i] : dense;
        a.page_stride[i] = page[i] ? page[i] : a.row[i] * d->page_size;
    }
    a.in[0] = static_cast<const uint16_t *>(io->key);
    a.in[1] = static_cast<const uint16_t *>(io->value);
    a.cache[0] = static_cast<uint16_t *>(io->key_cache);
    a.cache[1] = static_cast<uint16_t *>(io->value_cache);
    a.rows = rows;
    a.s_max = bsnd ? d->s1_max : 0;
    a.vecs = (int32_t)(dense / 8);
    a.page = d->page_size;
    a.pages = d->pages;
    a.width = d->width;
    a.table = io->page_table;
    a.klens = io->kv_lens;
    a.count = reinterpret_cast<int32_t *>(ws);
    a.status = reinterpret_cast<int32_t *>(ws + kStatusAt);
    if (fill_seq_tab(&a.seq, d->batch, reinterpret_cast<SeqRow *>(ws + o_seq), s, [&](int b) {
            SeqRow r{};
            r.q0 = bsnd ? b * d->s1_max : d->cu_seqlens_q[b];
            r.qlen = b < d->batch ? d->cu_seqlens_q[b + 1] - d->cu_seqlens_q[b] : 0;
            return r;
        }) != cudaSuccess)
        return SAG_ERR_CUDA;
    const int blocks = (rows + kThreads / 32 - 1) / (kThreads / 32);
    k_append<<<blocks < kMaxBlocks ? blocks : kMaxBlocks, kThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
}
