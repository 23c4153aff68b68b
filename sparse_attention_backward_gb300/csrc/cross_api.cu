// C ABI of the cross attention: validation and workspace sizes (phase 1),
// sequence tables and launches (phase 2).
#include <math.h>

#include "cross.cuh"
#include "kernels.cuh"

namespace sag {

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kTicketAt = 16;            // two ticket counters
constexpr size_t kStatusAt = 256;           // status words, behind the workspace's header
size_t up256(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
// most CTAs of a launch whose units are split, for the status words
constexpr int64_t kSplitCtas = 1024;

struct XPlan {
    bool fp16, bsnd;
    int tpt;
    int64_t q_tiles, k_tiles;               // query and key tiles of all sequences, padding included
    int max_q, max_k;                       // most query / key tiles of one sequence that have work
    int min_q, min_k;                       // fewest
    bool padding;                           // some tiles are padding
    size_t o_seq, o_stats, o_norms, o_row_norms, o_parts, o_arrived, total;
};

// Whether units with loops of `least` to `longest` tiles may be cut (tail_of): below 14 a piece never pays, and short units
// fill the last round as it is (a ragged padded batch: 155 -> 165 us with pieces).  The shortest loop then has 13 tiles, one
// at least for each of up to 8 pieces, which the kernels rely on.
bool may_cut(const XPlan &p, int longest, int least) { return !p.padding && longest >= 14 && least * 8 >= longest * 7; }

sag_status x_plan(const sca_desc *d, bool grad, XPlan *p) {
    if (!d || !d->cu_seqlens_q || !d->cu_seqlens_kv) return SAG_ERR_NULL;
    if (d->dtype != SAG_BF16 && d->dtype != SAG_FP16) return SAG_ERR_DTYPE;
    if (d->n1 < 1 || d->n1 > 128 || d->n2 < 1 || d->n2 > 128 || d->n1 % d->n2 != 0 || d->n1 / d->n2 > 32)
        return SAG_ERR_SHAPE;
    if (d->d < 1 || !(d->scale > 0.0) || d->scale > 1e30) return SAG_ERR_SHAPE;
    sag_status st = check_seqs(d->batch, d->layout, d->cu_seqlens_q, d->s1_max);
    const sag_status st2 = check_seqs(d->batch, d->layout, d->cu_seqlens_kv, d->s2_max);
    if (st == SAG_OK || (st == SAG_ERR_UNSUPPORTED && st2 != SAG_OK)) st = st2;
    if (st != SAG_OK) return st;
    const int64_t strides[] = {d->q_stride, d->k_stride, d->v_stride};
    for (int i = 0; i < 3; ++i)
        if (strides[i] != 0 && (strides[i] % 8 != 0 || strides[i] < (int64_t)(i ? d->n2 : d->n1) * d->d ||
                                strides[i] > (1LL << 36)))
            return SAG_ERR_SHAPE;
    if (d->d != 64 && d->d != 128) return SAG_ERR_UNSUPPORTED;
    p->fp16 = d->dtype == SAG_FP16;
    p->bsnd = d->layout == SAG_LAYOUT_BSND;
    p->tpt = kXRows / (d->n1 / d->n2);
    p->q_tiles = p->k_tiles = 0;
    p->max_q = p->max_k = 0;
    p->min_q = p->min_k = 1 << 30;
    p->padding = false;
    for (int b = 0; b < d->batch; ++b) {
        const int ql = d->cu_seqlens_q[b + 1] - d->cu_seqlens_q[b], kl = d->cu_seqlens_kv[b + 1] - d->cu_seqlens_kv[b];
        const int qt = ((p->bsnd ? d->s1_max : ql) + p->tpt - 1) / p->tpt;
        const int kt = ((p->bsnd ? d->s2_max : kl) + kXRows - 1) / kXRows;
        p->q_tiles += qt;
        p->k_tiles += kt;
        const int qw = (ql + p->tpt - 1) / p->tpt, kw = (kl + kXRows - 1) / kXRows;
        if (qw > p->max_q) p->max_q = qw;
        if (kw > p->max_k) p->max_k = kw;
        if (qw < p->min_q) p->min_q = qw;
        if (kw < p->min_k) p->min_k = kw;
        if (qw < qt || kw < kt) p->padding = true;
    }
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o = up256(o + bytes); return at; };
    take(kStatusAt);                        // header: number of status words
    const int64_t ctas = grad ? (p->q_tiles + p->k_tiles) * d->n2 + 2 * kSplitCtas : p->q_tiles * d->n2 + kSplitCtas;
    take(sizeof(int32_t) * ctas);           // status words, one a CTA
    p->o_seq = take(seq_ws_bytes(d->batch));
    p->o_stats = take(grad ? sizeof(float) * 256 * p->q_tiles * d->n2 : 0);
    p->o_norms = take(grad && p->fp16 ? sizeof(unsigned) * 2 * (size_t)d->batch * d->n2 : 0);
    p->o_row_norms = take(grad && p->fp16 ? sizeof(float) * kXRows * p->q_tiles * d->n2 : 0);
    const int64_t most = (p->q_tiles > p->k_tiles ? p->q_tiles : p->k_tiles) * d->n2;
    const int64_t pieces = most < kMaxPieces / kMaxSplit ? most * kMaxSplit : kMaxPieces;
    const bool cut = grad && (may_cut(*p, p->max_k, p->min_k) || may_cut(*p, p->max_q, p->min_q));
    p->o_parts = take(cut ? sizeof(float) * 2 * kXRows * d->d * pieces : 0);
    p->o_arrived = take(cut ? sizeof(unsigned) * 2 * 8 * kMaxPieces : 0);
    p->total = o;
    return SAG_OK;
}

// CTAs that share a unit: as many as run at once, up to a cluster's 8, as long as each has a tile of the loop.  A cluster
// lies within one of the GPU's parts (GPCs), so not every size fills all SMs, and with fewer CTAs an SM fewer sizes do.
// Most clusters that run at once on 152 SMs: with one and two CTAs an SM what cudaOccupancyMaxActiveClusters gives for
// that shared memory (asked for the kernels themselves it counts one CTA an SM), with four up to where the next smaller size
// is faster.  The limits show in the times of one query tile against 4096 states, us at them and one cluster beyond:
//   gradient, 128 wide (one an SM)   15 of 8: 36.4 | 47.9   23 of 6: 51.4 | 65.7   28 of 5: 58.9 | 75.3   36 of 4: 69.7 | 85.7
//   forward, 128 wide (two)          36 of 8: 18.6 | 29.1   46 of 6: 22.1 | 34.9   58 of 5: 30.0 | 44.5   74 of 4: 38.4 | 54.9
//   forward, 64 wide (four)          64 of 8: 22.2, 66: 25.3, 69: 33.7, where 7 take 27.1
// They are fixed, not asked for, so that a call's sums have the same order on every GB300.
int split_of(int64_t units, int tiles, int per_sm, int sms) {
    static const int fits[3][kMaxSplit + 1] = {
        {0, 152, 76, 46, 36, 28, 23, 15, 15}, {0, 304, 152, 97, 74, 58, 46, 38, 36}, {0, 608, 304, 194, 146, 114, 94, 77, 66}};
    const int *row = fits[per_sm >> 1];
    for (int ns = kMaxSplit; ns > 1; --ns)
        if (ns <= tiles && units * ns <= kSplitCtas && units * 152 <= (int64_t)row[ns] * sms) return ns;
    return 1;
}

// Units of a gradient kernel beyond full rounds of the SMs are cut into pieces of their loops if those fill the last round
// better: `full` whole units, then `pieces` of each other one.  Times in tiles of the loop: a piece costs about six more
// for its start, its sums' way to the workspace and the last one's adding up, which takes one for each piece.  160 units of
// 64 tiles: 260 -> 207 us, 512 units of 256 tiles: 2320 -> 2150 us, 320 units of 24 tiles: 190 -> 179 us.
void tail_of(int units, int tiles, int sms, int *full, int *pieces) {
    *full = units;
    *pieces = 1;
    const int rest = units % sms;
    int best = tiles + 1;
    for (int s = 2; s <= kMaxSplit && s <= tiles && rest * s <= kMaxPieces; ++s) {
        const int t = (rest * s + sms - 1) / sms * ((tiles + s - 1) / s + 6) + s;
        if (rest == 0 || t >= best) continue;
        best = t;
        *full = units - rest;
        *pieces = s;
    }
}

XArgs x_args(const sca_desc *d, const sca_io *io, const XPlan &p, char *ws) {
    XArgs a{};
    a.n1 = d->n1;
    a.n2 = d->n2;
    a.group = d->n1 / d->n2;
    a.tpt = p.tpt;
    a.s1_pad = p.bsnd ? d->s1_max : 0;
    a.s2_pad = p.bsnd ? d->s2_max : 0;
    a.nsplit = 1;
    a.scale = (float)d->scale;
    a.scale_log2 = (float)(d->scale * 1.4426950408889634);
    a.mask = io->key_mask;
    a.o_in = static_cast<const uint16_t *>(io->attention_out);
    a.dy = static_cast<const uint16_t *>(io->attention_out_grad);
    a.v_in = static_cast<const uint16_t *>(io->value);
    a.v_stride = d->v_stride ? d->v_stride : (int64_t)d->n2 * d->d;
    a.o = static_cast<uint16_t *>(io->attention_out);
    a.dq = static_cast<uint16_t *>(io->dq);
    a.dk = static_cast<uint16_t *>(io->dk);
    a.dv = static_cast<uint16_t *>(io->dv);
    a.lse = io->softmax_lse;
    a.stats = reinterpret_cast<float *>(ws + p.o_stats);
    a.norms = reinterpret_cast<unsigned *>(ws + p.o_norms);
    a.row_norms = reinterpret_cast<float *>(ws + p.o_row_norms);
    a.parts = reinterpret_cast<float *>(ws + p.o_parts);
    a.arrived = reinterpret_cast<unsigned *>(ws + p.o_arrived);
    a.q_tiles = (int)p.q_tiles;
    a.k_tiles = (int)p.k_tiles;
    a.count = reinterpret_cast<int32_t *>(ws);
    a.ticket = reinterpret_cast<unsigned *>(ws + kTicketAt);
    a.status = reinterpret_cast<int32_t *>(ws + kStatusAt);
    return a;
}

cudaError_t x_table(XArgs *a, const sca_desc *d, const XPlan &p, char *ws, cudaStream_t s) {
    int qt = 0, kt = 0;
    return fill_seq_tab(&a->seq, d->batch, reinterpret_cast<SeqRow *>(ws + p.o_seq), s, [&](int b) {
        SeqRow r{};
        r.qtile0 = qt;
        r.ktile0 = kt;
        r.q0 = p.bsnd ? b * d->s1_max : d->cu_seqlens_q[b];
        r.k0 = p.bsnd ? b * d->s2_max : d->cu_seqlens_kv[b];
        if (b < d->batch) {
            r.qlen = d->cu_seqlens_q[b + 1] - d->cu_seqlens_q[b];
            r.klen = d->cu_seqlens_kv[b + 1] - d->cu_seqlens_kv[b];
            qt += ((p.bsnd ? d->s1_max : r.qlen) + p.tpt - 1) / p.tpt;
            kt += ((p.bsnd ? d->s2_max : r.klen) + kXRows - 1) / kXRows;
        }
        return r;
    });
}

// required pointers and alignment; those of a side without rows may be NULL
sag_status x_check(const sca_desc *d, const sca_io *io, const XPlan &p, bool grad, const void *ws, size_t ws_bytes) {
    if (!io) return SAG_ERR_NULL;
    const bool has_q = p.q_tiles > 0, has_k = p.k_tiles > 0;
    const void *qs[] = {io->query, io->attention_out, io->softmax_lse, grad ? io->attention_out_grad : io->query,
                        grad ? io->dq : io->query};
    const void *ks[] = {io->key, io->value, grad ? io->dk : io->key, grad ? io->dv : io->key};
    for (const void *x : qs)
        if (has_q && !x) return SAG_ERR_NULL;
    for (const void *x : ks)
        if (has_k && !x) return SAG_ERR_NULL;
    if (!ws || ws_bytes < p.total) return SAG_ERR_WORKSPACE;
    auto off = [](const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15) != 0; };
    for (const void *x : qs)
        if (has_q && off(x)) return SAG_ERR_ALIGN;
    for (const void *x : ks)
        if (has_k && off(x)) return SAG_ERR_ALIGN;
    if (off(ws)) return SAG_ERR_ALIGN;
    return SAG_OK;
}

}  // namespace
}  // namespace sag

using namespace sag;

extern "C" sag_status cross_attn_fwd_workspace_size(const sca_desc *desc, size_t *workspace_bytes) {
    if (!workspace_bytes) return SAG_ERR_NULL;
    XPlan p;
    const sag_status st = x_plan(desc, false, &p);
    if (st == SAG_OK) *workspace_bytes = p.total;
    return st;
}

extern "C" sag_status cross_attn_grad_workspace_size(const sca_desc *desc, size_t *workspace_bytes) {
    if (!workspace_bytes) return SAG_ERR_NULL;
    XPlan p;
    const sag_status st = x_plan(desc, true, &p);
    if (st == SAG_OK) *workspace_bytes = p.total;
    return st;
}

extern "C" sag_status cross_attn_fwd(const sca_desc *desc, const sca_io *io, void *workspace, size_t workspace_bytes,
                                     void *stream) {
    XPlan p;
    sag_status st = x_plan(desc, false, &p);
    if (st != SAG_OK) return st;
    st = x_check(desc, io, p, false, workspace, workspace_bytes);
    if (st != SAG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard dg;
    if (!dg.bind_memory(workspace)) return SAG_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    if (p.q_tiles == 0)                     // no query rows: nothing to write, no device status
        return cudaMemsetAsync(ws, 0, sizeof(int32_t), s) == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
    XArgs a = x_args(desc, io, p, ws);
    if (x_table(&a, desc, p, ws, s) != cudaSuccess) return SAG_ERR_CUDA;
    a.units = (int)(p.q_tiles * desc->n2);
    a.nsplit = split_of(a.units, 2 * p.max_k, desc->d == 64 ? 4 : 2, current_device_sms());   // tiles of 64 keys; CTAs an SM
    a.n_status = a.ctas = a.units * a.nsplit;
    // full query tiles, and at least 2048 keys a CTA
    const bool long_loops = p.max_q > 1 && p.max_k >= 16 * a.nsplit;
    return launch_xfwd(a, *io, *desc, long_loops, s) == cudaSuccess ? SAG_OK : SAG_ERR_CUDA;
}

extern "C" sag_status cross_attn_grad(const sca_desc *desc, const sca_io *io, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    XPlan p;
    sag_status st = x_plan(desc, true, &p);
    if (st != SAG_OK) return st;
    st = x_check(desc, io, p, true, workspace, workspace_bytes);
    if (st != SAG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard dg;
    if (!dg.bind_memory(workspace)) return SAG_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    const int q_units = (int)(p.q_tiles * desc->n2), k_units = (int)(p.k_tiles * desc->n2);
    if (k_units == 0 && cudaMemsetAsync(ws, 0, sizeof(int32_t), s) != cudaSuccess) return SAG_ERR_CUDA;
    XArgs a = x_args(desc, io, p, ws);
    if (x_table(&a, desc, p, ws, s) != cudaSuccess) return SAG_ERR_CUDA;
    const int sms = current_device_sms();
    if (p.fp16 && cudaMemsetAsync(a.norms, 0, sizeof(unsigned) * 2 * (size_t)desc->batch * desc->n2, s) != cudaSuccess)
        return SAG_ERR_CUDA;
    // one CTA an SM: a cluster for each unit, or CTAs that take item after item
    struct Share {
        int units, nsplit, full, pieces, items, ctas;
    };
    auto share = [&](int units, int tiles, int least) {
        Share x;
        x.units = x.full = units;
        x.nsplit = split_of(units, tiles, 1, sms);
        x.pieces = 1;
        if (x.nsplit == 1 && may_cut(p, tiles, least)) tail_of(units, tiles, sms, &x.full, &x.pieces);
        x.items = x.full + (units - x.full) * x.pieces;
        x.ctas = x.nsplit > 1 ? units * x.nsplit : x.items < sms ? x.items : sms;
        return x;
    };
    auto use = [&](const Share &x) {
        a.units = x.units;
        a.nsplit = x.nsplit;
        a.full = x.full;
        a.pieces = x.pieces;
        a.items = x.items;
        a.ctas = x.ctas;
    };
    const Share sq = share(q_units, p.max_k, p.min_k), sk = share(k_units, p.max_q, p.min_q);
    const int counts = (sq.units - sq.full) * 8;
    a.n_arrived = counts + (sk.units - sk.full) * 8;
    if (launch_xpre(a, p.fp16, desc->d, s) != cudaSuccess) return SAG_ERR_CUDA;
    int before = 0;
    // k_xpre zeroes the tickets; without query rows there is none
    if (!q_units && cudaMemsetAsync(a.ticket, 0, 2 * sizeof(unsigned), s) != cudaSuccess) return SAG_ERR_CUDA;
    if (q_units) {
        use(sq);
        if (launch_xdq(a, *io, *desc, s) != cudaSuccess) return SAG_ERR_CUDA;
        before = a.ctas;
    }
    if (k_units) {
        a.status += before;
        a.ticket += 1;
        use(sk);
        a.arrived += counts;
        a.n_status = before + a.ctas;
        if (launch_xdkv(a, *io, *desc, s) != cudaSuccess) return SAG_ERR_CUDA;
    }
    return SAG_OK;
}

extern "C" sag_status cross_attn_query_error(const void *workspace, void *stream) {
    if (!workspace) return SAG_ERR_NULL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceGuard dg;
    if (!dg.bind_memory(workspace)) return SAG_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return SAG_ERR_CUDA;
    const char *ws = static_cast<const char *>(workspace);
    int32_t count = 0, words[1024];
    if (cudaMemcpy(&count, ws, sizeof(count), cudaMemcpyDeviceToHost) != cudaSuccess) return SAG_ERR_CUDA;
    for (int32_t at = 0; at < count; at += 1024) {
        const int n = count - at < 1024 ? count - at : 1024;
        if (cudaMemcpy(words, ws + kStatusAt + sizeof(int32_t) * (size_t)at, sizeof(int32_t) * n, cudaMemcpyDeviceToHost) !=
            cudaSuccess)
            return SAG_ERR_CUDA;
        for (int i = 0; i < n; ++i)
            if (words[i] != SAG_OK) return static_cast<sag_status>(words[i]);
    }
    return SAG_OK;
}
