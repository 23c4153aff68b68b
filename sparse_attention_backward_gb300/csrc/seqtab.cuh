// Sequence tables of the operators that take free sequence lengths (rotary
// positions, cross attention).  A problem of up to kInlineSeqs sequences
// carries its table in the kernel parameters: no copy, no extra launch, and a
// captured call keeps its own.  A larger one puts it into the workspace by
// k_seq_upload launches whose payload is a kernel parameter too (a copy from
// pageable host memory could not be captured).
#pragma once

#include "common.cuh"

namespace sag {

constexpr int kInlineSeqs = 64;
constexpr int kMaxSeqs = 65536;

// One sequence; entry [batch] holds the totals of the tile counts.
struct SeqRow {
    int32_t q0, qlen;       // first query row, valid query rows
    int32_t k0, klen;       // first key row, valid key rows
    int32_t qtile0, ktile0; // query / key tiles of the sequences before it
};

struct SeqTab {
    int32_t batch;
    const SeqRow *ext;                  // in the workspace, or nullptr: row[]
    SeqRow row[kInlineSeqs + 1];
};

// Row b of the table.  Two plain accesses, not one pointer: row[] is then read
// through the constant bank (about 40 cycles), which a generic pointer into the
// parameters is not (it cost over a thousand cycles at the start of each block).
__device__ __forceinline__ SeqRow seq_row(const SeqTab &t, int b) {
    if (t.ext) return t.ext[b];
    return t.row[b];
}
template <int32_t SeqRow::*field>
__device__ __forceinline__ int seq_get(const SeqTab &t, int b) {
    if (t.ext) return t.ext[b].*field;
    return t.row[b].*field;
}

// Last sequence whose `field` is <= x (empty sequences share their successor's
// value, so the last one is the one that holds x).
template <int32_t SeqRow::*field>
__device__ __forceinline__ int seq_find(const SeqTab &t, int x) {
    int lo = 0, hi = t.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq_get<field>(t, mid) <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Fills a table: `make(b)` gives row b, 0 <= b <= batch, and is called in
// order, once each.  ext_ws: where the workspace keeps the rows of a large
// batch.  Enqueues the uploads on `s`.
constexpr int kUploadRows = 1024;       // 24 KB of kernel parameters a launch
struct SeqUpload {
    SeqRow row[kUploadRows];
};
cudaError_t launch_seq_upload(const SeqUpload &u, SeqRow *dst, int n, cudaStream_t s);

inline size_t seq_ws_bytes(int batch) { return batch > kInlineSeqs ? sizeof(SeqRow) * ((size_t)batch + 1) : 0; }

template <class Make>
cudaError_t fill_seq_tab(SeqTab *tab, int batch, SeqRow *ext_ws, cudaStream_t s, Make &&make) {
    tab->batch = batch;
    tab->ext = nullptr;
    if (batch <= kInlineSeqs) {
        for (int b = 0; b <= batch; ++b) tab->row[b] = make(b);
        return cudaSuccess;
    }
    tab->ext = ext_ws;
    SeqUpload u;
    for (int b0 = 0; b0 <= batch; b0 += kUploadRows) {
        const int n = batch + 1 - b0 < kUploadRows ? batch + 1 - b0 : kUploadRows;
        for (int i = 0; i < n; ++i) u.row[i] = make(b0 + i);
        const cudaError_t e = launch_seq_upload(u, ext_ws + b0, n, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Checks shared by the two operators' descriptors: batch, layout, prefix sums.
sag_status check_seqs(int batch, int layout, const int32_t *cu, int32_t s_max);

int current_device_sms();

}  // namespace sag
