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

// How a gradient kernel's units are shared: a cluster for each; or CTAs (one an SM) that take units, or `pieces` of each, as they
// come to them, from the longest on.
struct Share {
    int units, nsplit, pieces;
    int64_t items() const { return (int64_t)units * pieces; }
    size_t part_bytes(int cols) const { return pieces > 1 ? (size_t)items() * 256 * cols * sizeof(float) : 0; }
};
// One way to share them: the longest item and all of them together, in tiles of the loop.  A piece takes about fourteen tiles
// more (its start, its sums' way through the workspace) and one for each piece added up, a cluster's join four.
struct Way {
    Share share;
    int64_t one, all;
};
int ways_of(int64_t units, int64_t longest, int64_t total, Way *to) {
    int n = 0;
    to[n++] = {{(int)units, 1, 1}, longest, total};
    if (units == 0 || units > kMaxPieces || longest < 12) return n;
    const int ns = split_of(units, (int)(longest / 2), 1, 152);
    if (ns > 1) {
        const int64_t one = (longest + ns - 1) / ns + 4;
        to[n++] = {{(int)units, ns, 1}, one, one * units * ns};
    }
    for (int s = 2; s <= kMaxSplit && s * 2 <= longest && units * s <= kMaxPieces; ++s)
        to[n++] = {{(int)units, 1, s}, (longest + s - 1) / s + 14 + s, total + 14 * units * s};
    return n;
}
// Both kernels run side by side on 152 SMs; a tile of k_xdkv takes five units of time, one of k_xdq four.  Causal units differ: 64
// key tiles of 2 heads have loops of 4 to 256 query tiles of 32 tokens, and the longest would hold up the rest (8192 tokens, 8 / 2
// heads of 128: 381 us, the units of k_xdkv in two pieces each 286).  From the descriptor alone, so that a call's sums have the
// same order on every GB300.
void share_both(int64_t q_units, int64_t q_most, int64_t q_all, int64_t k_units, int64_t k_most, int64_t k_all, Share *q, Share *k) {
    Way qs[kMaxSplit + 2], ks[kMaxSplit + 2];
    const int nq = ways_of(q_units, q_most, q_all, qs), nk = ways_of(k_units, k_most, k_all, ks);
    int64_t best = INT64_MAX;
    for (int i = 0; i < nq; ++i)
        for (int j = 0; j < nk; ++j) {
            int64_t t = (4 * qs[i].all + 5 * ks[j].all) / 152;
            t = 4 * qs[i].one > t ? 4 * qs[i].one : t;
            t = 5 * ks[j].one > t ? 5 * ks[j].one : t;
            if (t >= best) continue;
            best = t;
            *q = qs[i].share;
            *k = ks[j].share;
        }
}

struct GradPlan {
    Share q, k;
    size_t o_parts_q, o_parts_k, o_arrived, o_key_norms, o_tops, o_up, total;
};
GradPlan grad_plan(const swa_desc *desc, const XPlan &p) {
    const sca_desc *d = &desc->attn;
    GradPlan g{};
    const int64_t left = limit_of(desc->left), right = limit_of(desc->right);
    const int64_t q_units = p.q_tiles * d->n2, k_units = p.k_tiles * d->n2;
    int64_t q_most = 0, q_all = 0, k_most = 0, k_all = 0;
    for (int b = 0; b < d->batch && (q_units <= kMaxPieces || k_units <= kMaxPieces); ++b) {
        const int64_t ql = d->cu_seqlens_q[b + 1] - d->cu_seqlens_q[b], kl = d->cu_seqlens_kv[b + 1] - d->cu_seqlens_kv[b];
        const int64_t off = kl - ql;
        auto count = [](int64_t lo, int64_t hi, int64_t step) { return hi > lo ? (hi - lo + step - 1) / step : 0; };
        if (q_units <= kMaxPieces)
            for (int64_t t = 0; t < ql; t += p.tpt) {
                const int64_t last = (t + p.tpt < ql ? t + p.tpt : ql) - 1, lo = t + off - left, hi = last + off + right + 1;
                const int64_t n = count(lo > 0 ? lo : 0, hi < kl ? hi : kl, kXRows);
                q_most = n > q_most ? n : q_most;
                q_all += n * d->n2;
            }
        if (k_units <= kMaxPieces)
            for (int64_t k = 0; k < kl; k += kXRows) {
                const int64_t last = (k + kXRows < kl ? k + kXRows : kl) - 1, lo = k - off - right, hi = last - off + left + 1;
                const int64_t from = lo > 0 ? lo / p.tpt * p.tpt : 0, n = count(from, hi < ql ? hi : ql, p.tpt);
                k_most = n > k_most ? n : k_most;
                k_all += n * d->n2;
            }
    }
    // pairs of tiles are about as many on either side
    if (q_units > kMaxPieces) q_all = k_all;
    if (k_units > kMaxPieces) k_all = q_all;
    share_both(q_units, q_most, q_all, k_units, k_most, k_all, &g.q, &g.k);
    g.o_parts_q = p.o_parts;                // (x_plan's own are the last)
    g.o_parts_k = up256(g.o_parts_q + g.q.part_bytes(d->d / 2));
    g.o_arrived = up256(g.o_parts_k + g.k.part_bytes(d->d));
    g.o_key_norms =
        up256(g.o_arrived + sizeof(unsigned) * 8 * (size_t)((g.q.pieces > 1 ? g.q.units : 0) + (g.k.pieces > 1 ? g.k.units : 0)));
    // fp16: of each key, and of query and key tiles, and of query rows and keys (k_wscale)
    const size_t scaled = p.fp16 ? (size_t)(q_units + k_units) : 0;
    g.o_tops = up256(g.o_key_norms + (p.fp16 ? sizeof(float) * kXRows * (size_t)k_units : 0));
    g.o_up = up256(g.o_tops + sizeof(float2) * scaled);
    g.total = up256(g.o_up + sizeof(float) * kXRows * scaled);
    return g;
}

sag_status w_plan(const swa_desc *d, bool grad, XPlan *p, Parts *parts, GradPlan *g) {
    const sag_status st = x_plan(d ? &d->attn : nullptr, grad, p);
    if (st != SAG_OK) return st;
    if (grad) {
        *g = grad_plan(d, *p);
        p->total = g->total;
        return SAG_OK;
    }
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
    const sag_status st = w_plan(desc, false, &p, &parts, nullptr);
    if (st == SAG_OK) *workspace_bytes = p.total;
    return st;
}

extern "C" sag_status window_attn_grad_workspace_size(const swa_desc *desc, size_t *workspace_bytes) {
    if (!workspace_bytes) return SAG_ERR_NULL;
    XPlan p;
    GradPlan g;
    const sag_status st = w_plan(desc, true, &p, nullptr, &g);
    if (st == SAG_OK) *workspace_bytes = p.total;
    return st;
}

extern "C" sag_status window_attn_fwd(const swa_desc *desc, const sca_io *io, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    XPlan p;
    Parts parts;
    sag_status st = w_plan(desc, false, &p, &parts, nullptr);
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
    GradPlan g;
    sag_status st = w_plan(desc, true, &p, nullptr, &g);
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
    if (p.fp16) {
        a.key_norms = reinterpret_cast<float *>(ws + g.o_key_norms);
        a.q_tops = reinterpret_cast<float2 *>(ws + g.o_tops);
        a.k_tops = a.q_tops + q_units;
        a.q_up = reinterpret_cast<float *>(ws + g.o_up);
        a.k_up = a.q_up + (size_t)q_units * kXRows;
    }
    auto use = [&](XArgs *x, const Share &h, size_t parts) {
        x->units = h.units;
        x->full = h.pieces > 1 ? 0 : h.units;
        x->pieces = h.pieces;
        x->nsplit = h.nsplit;
        x->items = (int)h.items();
        x->ctas = h.nsplit > 1 ? h.units * h.nsplit : x->items < sms ? x->items : sms;
        x->parts = reinterpret_cast<float *>(ws + parts);
    };
    unsigned *arrived = reinterpret_cast<unsigned *>(ws + g.o_arrived);
    const int q_counts = g.q.pieces > 1 ? 8 * g.q.units : 0;
    a.arrived = arrived;
    a.n_arrived = q_counts + (g.k.pieces > 1 ? 8 * g.k.units : 0);
    if (launch_xpre(a, p.fp16, d->d, s) != cudaSuccess) return SAG_ERR_CUDA;
    if (p.fp16 && launch_wscale(a, s) != cudaSuccess) return SAG_ERR_CUDA;
    // k_xpre zeroes the tickets and counters; without query rows there may be none (and no pieces)
    if (!q_units && cudaMemsetAsync(a.ticket, 0, 2 * sizeof(unsigned), s) != cudaSuccess) return SAG_ERR_CUDA;
    // k_xdkv first; k_xdq starts as its CTAs leave (window_bwd.cu).  Status words: k_xdq's, then k_xdkv's
    XArgs q = a;
    if (q_units) {
        use(&q, g.q, g.o_parts_q);
        q.late = k_units > 0;
    }
    if (k_units) {
        const int before = q_units ? q.ctas : 0;
        a.status += before;
        a.ticket += 1;
        a.arrived = arrived + q_counts;
        use(&a, g.k, g.o_parts_k);
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
