// C ABI of the cross attention: validation and workspace sizes (phase 1),
// sequence tables and launches (phase 2).
#include "xplan.cuh"

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
