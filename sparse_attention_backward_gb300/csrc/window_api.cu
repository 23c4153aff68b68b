// C ABI of windowed and paged attention: validation and workspace sizes (phase 1),
// sequence tables and launches (phase 2).
#include "xplan.cuh"

namespace sag {

namespace {

int32_t limit_of(int32_t keys) { return keys < 0 || keys >= kMaxPos ? kNoLimit : keys; }

// Keys that the `rows` tokens of a query tile may see, of `most`; queries that see the 128 keys of a key tile.
int64_t reach(int32_t left, int32_t right, int64_t rows, int64_t most) {
    const int64_t all = (int64_t)limit_of(left) + limit_of(right) + rows;
    return all < most ? all : most;
}

// Workspace behind a plan's own: O, maximum and sum of the pieces of units.
struct Parts {
    XSplit split;
    size_t o_parts, o_ml, total;
};
Parts parts_of(int64_t units, int64_t keys, int d, size_t at) {
    Parts p{};
    p.split = fwd_split(units, (int)((keys + 63) / 64), d == 64 ? 4 : 2);
    const size_t rows = p.split.pieces > 1 ? (size_t)units * p.split.pieces * kXRows : 0;
    p.o_parts = at;
    p.o_ml = up256(p.o_parts + rows * d * sizeof(float));
    p.total = up256(p.o_ml + rows * sizeof(float2));
    return p;
}

sag_status w_plan(const swa_desc *d, bool grad, XPlan *p, Parts *parts) {
    const sag_status st = x_plan(d ? &d->attn : nullptr, grad, p);
    if (st != SAG_OK || grad) return st;
    int64_t most = 0;
    for (int b = 0; b < d->attn.batch; ++b) {
        const int64_t k = d->attn.cu_seqlens_kv[b + 1] - d->attn.cu_seqlens_kv[b];
        most = k > most ? k : most;
    }
    *parts = parts_of(p->q_tiles * d->attn.n2, reach(d->left, d->right, p->tpt, most), d->attn.d, p->total);
    p->total = parts->total;
    return SAG_OK;
}

struct PPlan {
    bool bsnd;
    int tpt, max_q;
    int64_t q_tiles, rows, keys;
    Parts parts;
    size_t o_seq, total;
};

}  // namespace

sag_status check_paged(const spa_desc *d) {
    if (!d || !d->cu_seqlens_q) return SAG_ERR_NULL;
    if (d->dtype != SAG_BF16 && d->dtype != SAG_FP16) return SAG_ERR_DTYPE;
    if (d->n1 < 1 || d->n1 > 128 || d->n2 < 1 || d->n2 > 128 || d->n1 % d->n2 != 0 || d->n1 / d->n2 > 32) return SAG_ERR_SHAPE;
    if (d->d < 1 || d->d > 512 || !(d->scale > 0.0) || d->scale > 1e30 || d->reserved_ != 0) return SAG_ERR_SHAPE;
    if (d->page_size < 1 || d->page_size > 65536 || d->pages < 1 || d->width < 1 || d->kv_expected < 0 ||
        (int64_t)d->width * d->page_size > kMaxPos)
        return SAG_ERR_SHAPE;
    const sag_status st = check_seqs(d->batch, d->layout, d->cu_seqlens_q, d->s1_max);
    if (st != SAG_OK) return st;
    const int64_t row = (int64_t)d->n2 * d->d;
    const int64_t news[] = {d->q_stride, d->k_stride, d->v_stride};
    for (int i = 0; i < 3; ++i)
        if (news[i] != 0 && (news[i] % 8 != 0 || news[i] < (int64_t)(i ? d->n2 : d->n1) * d->d || news[i] > (1LL << 36)))
            return SAG_ERR_SHAPE;
    const int64_t rows[] = {d->k_row, d->v_row}, pages[] = {d->k_page, d->v_page};
    for (int i = 0; i < 2; ++i) {
        if (rows[i] != 0 && (rows[i] % 8 != 0 || rows[i] < row || rows[i] > (1LL << 36))) return SAG_ERR_SHAPE;
        const int64_t r = rows[i] ? rows[i] : row;
        // pages may be interleaved with others (keys and values in one tensor), but not overlap
        if (pages[i] != 0 && (pages[i] % 8 != 0 || pages[i] < r * (d->page_size - 1) + row || pages[i] > (1LL << 36)))
            return SAG_ERR_SHAPE;
    }
    if (d->d % 8 != 0 || d->page_size % 16 != 0) return SAG_ERR_UNSUPPORTED;
    return SAG_OK;
}

namespace {

sag_status p_plan(const spa_desc *d, PPlan *p) {
    const sag_status st = check_paged(d);
    if (st != SAG_OK) return st;
    if (d->d != 64 && d->d != 128) return SAG_ERR_UNSUPPORTED;
    p->bsnd = d->layout == SAG_LAYOUT_BSND;
    p->tpt = kXRows / (d->n1 / d->n2);
    p->q_tiles = 0;
    p->max_q = 0;
    for (int b = 0; b < d->batch; ++b) {
        const int ql = d->cu_seqlens_q[b + 1] - d->cu_seqlens_q[b];
        p->q_tiles += ((p->bsnd ? d->s1_max : ql) + p->tpt - 1) / p->tpt;
        const int qw = (ql + p->tpt - 1) / p->tpt;
        if (qw > p->max_q) p->max_q = qw;
    }
    p->rows = p->bsnd ? (int64_t)d->batch * d->s1_max : d->cu_seqlens_q[d->batch];
    int64_t most = (int64_t)d->width * d->page_size;
    if (d->kv_expected && d->kv_expected < most) most = d->kv_expected;
    p->keys = reach(d->left, d->right, p->tpt, most);
    p->o_seq = up256(kStatusAt + sizeof(int32_t) * (size_t)(p->q_tiles * d->n2 + kSplitCtas));
    p->parts = parts_of(p->q_tiles * d->n2, p->keys, d->d, up256(p->o_seq + seq_ws_bytes(d->batch)));
    p->total = p->parts.total;
    return SAG_OK;
}

// longest: most rows of a sequence that the outputs have (padding included)
void use_parts(XArgs *a, const Parts &p, char *ws, int longest) {
    a->join_rows = (longest < a->tpt ? longest : a->tpt) * a->group;
    a->nsplit = p.split.nsplit;
    a->pieces = p.split.pieces;
    a->parts = reinterpret_cast<float *>(ws + p.o_parts);
    a->part_ml = reinterpret_cast<float2 *>(ws + p.o_ml);
    a->n_status = a->ctas = a->units * a->nsplit * a->pieces;
}

template <class Desc>
int longest_of(const Desc &d) {
    if (d.layout == SAG_LAYOUT_BSND) return d.s1_max;
    int most = 0;
    for (int b = 0; b < d.batch; ++b) {
        const int n = d.cu_seqlens_q[b + 1] - d.cu_seqlens_q[b];
        most = n > most ? n : most;
    }
    return most;
}

// 128-key tiles: full query tiles, and at least 2048 keys a CTA (xfwd.cuh has the times)
bool long_loops(int max_q, int64_t keys, const XArgs &a) { return max_q > 1 && keys >= 2048LL * a.nsplit * a.pieces; }

bool off16(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15) != 0; }

}  // namespace
}  // namespace sag

using namespace sag;

extern "C" sag_status window_attn_fwd_workspace_size(const swa_desc *desc, size_t *workspace_bytes) {
    if (!workspace_bytes) return SAG_ERR_NULL;
    XPlan p;
    Parts parts;
    const sag_status st = w_plan(desc, false, &p, &parts);
    if (st == SAG_OK) *workspace_bytes = p.total;
    return st;
}

extern "C" sag_status window_attn_grad_workspace_size(const swa_desc *desc, size_t *workspace_bytes) {
    if (!workspace_bytes) return SAG_ERR_NULL;
    XPlan p;
    const sag_status st = w_plan(desc, true, &p, nullptr);
    if (st == SAG_OK) *workspace_bytes = p.total;
    return st;
}

extern "C" sag_status window_attn_fwd(const swa_desc *desc, const sca_io *io, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    XPlan p;
    Parts parts;
    sag_status st = w_plan(desc, false, &p, &parts);
    if (st != SAG_OK) return st;
    const sca_desc *d = &desc->attn;
    st = x_check(d, io, p, false, workspace, workspace_bytes);
    if (st != SAG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard dg;
    if (!dg.bind_memory(workspace)) return SAG_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    if (p.q_tiles == 0)                     // no query rows: nothing to write, no device status
        return cudaMemsetAsync(ws, 0, sizeof(int32_t), s) == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
    XArgs a = x_args(d, io, p, ws);
    a.left = limit_of(desc->left);
    a.right = limit_of(desc->right);
    if (x_table(&a, d, p, ws, s) != cudaSuccess) return SAG_ERR_CUDA;
    a.units = (int)(p.q_tiles * d->n2);
    use_parts(&a, parts, ws, longest_of(*d));
    const int64_t keys = reach(desc->left, desc->right, p.tpt, (int64_t)p.max_k * kXRows);
    return launch_wfwd(a, *io, *d, long_loops(p.max_q, keys, a), s) == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
}

extern "C" sag_status window_attn_grad(const swa_desc *desc, const sca_io *io, void *workspace, size_t workspace_bytes,
                                       void *stream) {
    XPlan p;
    sag_status st = w_plan(desc, true, &p, nullptr);
    if (st != SAG_OK) return st;
    const sca_desc *d = &desc->attn;
    st = x_check(d, io, p, true, workspace, workspace_bytes);
    if (st != SAG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard dg;
    if (!dg.bind_memory(workspace)) return SAG_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    const int q_units = (int)(p.q_tiles * d->n2), k_units = (int)(p.k_tiles * d->n2);
    if (k_units == 0 && cudaMemsetAsync(ws, 0, sizeof(int32_t), s) != cudaSuccess) return SAG_ERR_CUDA;
    XArgs a = x_args(d, io, p, ws);
    a.left = limit_of(desc->left);
    a.right = limit_of(desc->right);
    if (x_table(&a, d, p, ws, s) != cudaSuccess) return SAG_ERR_CUDA;
    const int sms = current_device_sms();
    if (p.fp16 && cudaMemsetAsync(a.norms, 0, sizeof(unsigned) * 2 * (size_t)d->batch * d->n2, s) != cudaSuccess)
        return SAG_ERR_CUDA;
    // one CTA an SM: CTAs that take unit after unit, or a cluster for each unit where loops are long enough for its join to pay
    // (8 heads of 128, 1000 x 1000 tokens, 8 tiles: 24 us, split 35; 1 x 4000 tokens, 32 tiles: 49 us, split 27)
    auto use = [&](int units, int64_t tiles) {
        a.units = a.full = a.items = units;
        a.pieces = 1;
        a.nsplit = tiles < 12 ? 1 : split_of(units, (int)tiles / 2, 1, 152);
        a.ctas = a.nsplit > 1 ? units * a.nsplit : units < sms ? units : sms;
    };
    if (launch_xpre(a, p.fp16, d->d, s) != cudaSuccess) return SAG_ERR_CUDA;
    // k_xpre zeroes the tickets; without query rows there is none
    if (!q_units && cudaMemsetAsync(a.ticket, 0, 2 * sizeof(unsigned), s) != cudaSuccess) return SAG_ERR_CUDA;
    // k_xdkv first; k_xdq starts as its CTAs leave (window_bwd.cu).  Status words: k_xdq's, then k_xdkv's
    XArgs q = a;
    if (q_units) {
        use(q_units, (reach(desc->left, desc->right, p.tpt, (int64_t)p.max_k * kXRows) + kXRows - 1) / kXRows);
        q = a;
        q.late = k_units > 0;
    }
    if (k_units) {
        const int before = q_units ? q.ctas : 0;
        a.status += before;
        a.ticket += 1;
        use(k_units, (reach(desc->left, desc->right, kXRows, (int64_t)p.max_q * p.tpt) + p.tpt - 1) / p.tpt);
        a.n_status = before + a.ctas;
        if (launch_wdkv(a, *io, *d, s) != cudaSuccess) return SAG_ERR_CUDA;
    }
    if (q_units && launch_wdq(q, *io, *d, s) != cudaSuccess) return SAG_ERR_CUDA;
    return SAG_OK;
}

extern "C" sag_status window_attn_query_error(const void *workspace, void *stream) {
    return cross_attn_query_error(workspace, stream);
}

extern "C" sag_status paged_attn_fwd_workspace_size(const spa_desc *desc, size_t *workspace_bytes) {
    if (!workspace_bytes) return SAG_ERR_NULL;
    PPlan p;
    const sag_status st = p_plan(desc, &p);
    if (st == SAG_OK) *workspace_bytes = p.total;
    return st;
}

extern "C" sag_status paged_attn_fwd(const spa_desc *desc, const spa_io *io, void *workspace, size_t workspace_bytes,
                                     void *stream) {
    PPlan p;
    const sag_status st = p_plan(desc, &p);
    if (st != SAG_OK) return st;
    if (!io) return SAG_ERR_NULL;
    const void *need[] = {io->query, io->key_cache, io->value_cache, io->attention_out, io->softmax_lse};
    if (p.q_tiles) {
        for (const void *x : need)
            if (!x) return SAG_ERR_NULL;
        if (!io->page_table || !io->kv_lens) return SAG_ERR_NULL;
    }
    if (!workspace || workspace_bytes < p.total) return SAG_ERR_WORKSPACE;
    if (p.q_tiles) {
        for (const void *x : need)
            if (off16(x)) return SAG_ERR_ALIGN;
        if ((reinterpret_cast<uintptr_t>(io->page_table) | reinterpret_cast<uintptr_t>(io->kv_lens)) & 3) return SAG_ERR_ALIGN;
    }
    if (off16(workspace)) return SAG_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard dg;
    if (!dg.bind_memory(workspace)) return SAG_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    if (p.q_tiles == 0)                     // no new tokens: nothing to write, no device status
        return cudaMemsetAsync(ws, 0, sizeof(int32_t), s) == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
    XArgs a{};
    a.n1 = desc->n1;
    a.n2 = desc->n2;
    a.group = desc->n1 / desc->n2;
    a.tpt = p.tpt;
    a.s1_pad = p.bsnd ? desc->s1_max : 0;
    a.scale = (float)desc->scale;
    a.scale_log2 = (float)(desc->scale * 1.4426950408889634);
    a.left = limit_of(desc->left);
    a.right = limit_of(desc->right);
    a.table = io->page_table;
    a.klens = io->kv_lens;
    a.width = desc->width;
    a.page = desc->page_size;
    a.pages = desc->pages;
    a.o = static_cast<uint16_t *>(io->attention_out);
    a.lse = io->softmax_lse;
    a.count = reinterpret_cast<int32_t *>(ws);
    a.status = reinterpret_cast<int32_t *>(ws + kStatusAt);
    a.q_tiles = (int)p.q_tiles;
    int qt = 0;
    if (fill_seq_tab(&a.seq, desc->batch, reinterpret_cast<SeqRow *>(ws + p.o_seq), s, [&](int b) {
            SeqRow r{};
            r.qtile0 = qt;
            r.q0 = p.bsnd ? b * desc->s1_max : desc->cu_seqlens_q[b];
            if (b < desc->batch) {
                r.qlen = desc->cu_seqlens_q[b + 1] - desc->cu_seqlens_q[b];
                qt += ((p.bsnd ? desc->s1_max : r.qlen) + p.tpt - 1) / p.tpt;
            }
            return r;
        }) != cudaSuccess)
        return SAG_ERR_CUDA;
    a.units = (int)(p.q_tiles * desc->n2);
    use_parts(&a, p.parts, ws, longest_of(*desc));
    return launch_pfwd(a, *io, *desc, long_loops(p.max_q, p.keys, a), s) == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
}

extern "C" sag_status paged_query_error(const void *workspace, void *stream) {
    return cross_attn_query_error(workspace, stream);
}
