"""GB300 (sm_103a) selected-attention backward: thin Python binding.

Every step of the backward runs in the CUDA kernels of ``libselattn.so``; this
module only marshals arguments into its C ABI (``include/selattn.h``) with
ctypes.  PyTorch is used for device memory and streams.  There is no CPU path:
if the library is missing, importing the binding's entry points raises.

    import sparse_attention_backward_gb300 as sab
    dq, dk, dv = sab.backward(q, k, v, o, dy, softmax_max, softmax_sum, topk,
                              cu_seqlens_q, cu_seqlens_kv, scale,
                              block_size, block_count, deterministic=False)

Tensors are TND ([T, N, D]) or, given as 4-D tensors, BSND ([B, S, N, D] with
every batch padded to S rows; cu_seqlens then give the valid lengths).  With
``q_rope`` / ``k_rope`` the head dim is split (Q = [q, q_rope] along D) and
the gradients come back as (dq, dk, dv, dq_rope, dk_rope).

Next to it, in the same layouts: ``forward`` and ``indexer_backward``; rotary
positions (``Rotary``, ``rotary_forward`` / ``rotary_backward``, or ``rotary=``
of forward and backward); cross attention to an encoder's states
(``cross_forward`` / ``cross_backward``); norms of queries and keys with the
rotation in the same pass (``norm_rotary_forward`` / ``norm_rotary_backward``);
causal and windowed attention (``window_forward`` / ``window_backward``); and,
for new tokens over a paged cache, ``paged_append`` and ``paged_forward``.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libselattn.so")

SAG_OK, SAG_ERR_NULL, SAG_ERR_SHAPE, SAG_ERR_DTYPE, SAG_ERR_UNSUPPORTED = 0, 1, 2, 3, 4
SAG_ERR_WORKSPACE, SAG_ERR_ALIGN, SAG_ERR_CUDA, SAG_ERR_INDEX, SAG_ERR_TIMEOUT = 5, 6, 7, 8, 9
SAG_BF16, SAG_FP16 = 0, 1
SAG_LAYOUT_TND, SAG_LAYOUT_BSND = 0, 1

EXPORTED = ("sel_attn_grad_workspace_size", "sel_attn_grad", "sel_attn_grad_timed", "sel_attn_grad_ex",
            "sel_attn_grad_plan_info", "sel_attn_grad_query_error", "sel_attn_grad_status_string",
            "sel_attn_fwd_workspace_size", "sel_attn_fwd", "sel_attn_fwd_timed", "sel_attn_fwd_ex",
            "lightning_indexer_grad_workspace_size", "lightning_indexer_grad", "sel_attn_selftest_wait_timeout")


class SagDesc(ctypes.Structure):
    """Mirror of ``sag_desc`` in include/selattn.h."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("n1", ctypes.c_int32), ("n2", ctypes.c_int32),
        ("d_qk", ctypes.c_int32), ("d_v", ctypes.c_int32),
        ("block_size", ctypes.c_int32), ("block_count", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("deterministic", ctypes.c_int32), ("layout", ctypes.c_int32),
        ("scale", ctypes.c_double),
        ("cu_seqlens_q", ctypes.POINTER(ctypes.c_int32)),
        ("cu_seqlens_kv", ctypes.POINTER(ctypes.c_int32)),
        ("s1_max", ctypes.c_int32), ("s2_max", ctypes.c_int32), ("d_rope", ctypes.c_int32),
        ("reserved_", ctypes.c_int32),
    ]


class SagIo(ctypes.Structure):
    """Mirror of ``sag_io`` in include/selattn.h (device pointers as ints)."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "query", "key", "value", "attention_out", "attention_out_grad", "softmax_max", "softmax_sum",
        "topk_indices", "query_rope", "key_rope", "dq", "dk", "dv", "dq_rope", "dk_rope")]


class SagPlanInfo(ctypes.Structure):
    """Mirror of ``sag_plan_info`` in include/selattn.h."""
    _fields_ = [("workspace_bytes", ctypes.c_uint64), ("launches", ctypes.c_int32),
                ("token_chunks", ctypes.c_int32), ("items", ctypes.c_int64),
                ("main_kernel", ctypes.c_int32), ("dq_path", ctypes.c_int32)]


class SagError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({status_string(status)})")
        self.status = status


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libselattn.so (built by ``build.py``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} not found: build it with "
                           "`python -m sparse_attention_backward_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    D = ctypes.POINTER(SagDesc)
    lib.sel_attn_grad_workspace_size.argtypes = [D, ctypes.POINTER(sz)]
    lib.sel_attn_grad_workspace_size.restype = ctypes.c_int
    lib.sel_attn_grad.argtypes = [D] + [vp] * 11 + [vp, sz, vp]
    lib.sel_attn_grad.restype = ctypes.c_int
    lib.sel_attn_grad_timed.argtypes = [D] + [vp] * 11 + [vp, sz, vp, vp, vp]
    lib.sel_attn_grad_timed.restype = ctypes.c_int
    IO = ctypes.POINTER(SagIo)
    lib.sel_attn_grad_ex.argtypes = [D, IO, vp, sz, vp, vp, vp]
    lib.sel_attn_grad_ex.restype = ctypes.c_int
    lib.sel_attn_fwd_ex.argtypes = [D, IO, vp, sz, vp, vp, vp]
    lib.sel_attn_fwd_ex.restype = ctypes.c_int
    lib.sel_attn_grad_plan_info.argtypes = [D, ctypes.POINTER(SagPlanInfo)]
    lib.sel_attn_grad_plan_info.restype = ctypes.c_int
    lib.sel_attn_grad_query_error.argtypes = [vp, vp]
    lib.sel_attn_grad_query_error.restype = ctypes.c_int
    lib.sel_attn_fwd_workspace_size.argtypes = [D, ctypes.POINTER(sz)]
    lib.sel_attn_fwd_workspace_size.restype = ctypes.c_int
    lib.sel_attn_fwd.argtypes = [D] + [vp] * 7 + [vp, sz, vp]
    lib.sel_attn_fwd.restype = ctypes.c_int
    lib.sel_attn_fwd_timed.argtypes = [D] + [vp] * 7 + [vp, sz, vp, vp, vp]
    lib.sel_attn_fwd_timed.restype = ctypes.c_int
    lib.sel_attn_grad_status_string.argtypes = [ctypes.c_int]
    lib.sel_attn_grad_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().sel_attn_grad_status_string(int(status)).decode()


def make_desc(cu_seqlens_q, cu_seqlens_kv, n1, n2, d_qk, d_v, block_size, block_count, scale,
              dtype=SAG_BF16, deterministic=False, layout=SAG_LAYOUT_TND, s1_max=0, s2_max=0, d_rope=0):
    """Build a descriptor; keeps the host cu_seqlens arrays alive on the object.

    ``d_qk`` is the head dim of the query / key tensors (without the rope
    part when ``d_rope`` is set); BSND takes the padded lengths s1_max, s2_max.
    """
    cq = (ctypes.c_int32 * len(cu_seqlens_q))(*[int(x) for x in cu_seqlens_q])
    ck = (ctypes.c_int32 * len(cu_seqlens_kv))(*[int(x) for x in cu_seqlens_kv])
    d = SagDesc(batch=len(cu_seqlens_q) - 1, n1=n1, n2=n2, d_qk=d_qk, d_v=d_v,
                block_size=block_size, block_count=block_count, dtype=dtype,
                deterministic=1 if deterministic else 0, layout=int(layout), scale=float(scale),
                cu_seqlens_q=ctypes.cast(cq, ctypes.POINTER(ctypes.c_int32)),
                cu_seqlens_kv=ctypes.cast(ck, ctypes.POINTER(ctypes.c_int32)),
                s1_max=int(s1_max), s2_max=int(s2_max), d_rope=int(d_rope), reserved_=0)
    d._keep = (cq, ck)
    return d


def make_io(**ptrs) -> SagIo:
    """sag_io from device pointers (ints); names as in the C struct, others NULL."""
    io = SagIo()
    for k, v in ptrs.items():
        setattr(io, k, v)
    return io


def sel_attn_grad_ex(desc: SagDesc, io: SagIo, workspace, workspace_bytes: int, stream, main_start=None,
                     main_stop=None) -> None:
    """Phase 2 with every tensor in one sag_io; raises on a non-OK status."""
    st = load().sel_attn_grad_ex(ctypes.byref(desc), ctypes.byref(io), workspace, workspace_bytes, stream,
                                 main_start, main_stop)
    if st != SAG_OK:
        raise SagError(st, "sel_attn_grad_ex")


def sel_attn_fwd_ex(desc: SagDesc, io: SagIo, workspace, workspace_bytes: int, stream, passes_start=None,
                    passes_stop=None) -> None:
    """Forward phase 2 with every tensor in one sag_io; raises on a non-OK status."""
    st = load().sel_attn_fwd_ex(ctypes.byref(desc), ctypes.byref(io), workspace, workspace_bytes, stream,
                                passes_start, passes_stop)
    if st != SAG_OK:
        raise SagError(st, "sel_attn_fwd_ex")


def _layout_of(q, k, q_rope):
    """(layout, s1_max, s2_max, n1, d_qk, n2, d_rope) from the tensors' shapes."""
    if q.dim() == 4:
        if k.dim() != 4:
            raise ValueError("BSND needs 4-D query and key tensors")
        layout, s1_max, s2_max = SAG_LAYOUT_BSND, q.shape[1], k.shape[1]
    else:
        layout, s1_max, s2_max = SAG_LAYOUT_TND, 0, 0
    return layout, s1_max, s2_max, q.shape[-2], q.shape[-1], k.shape[-2], (q_rope.shape[-1] if q_rope is not None else 0)


def workspace_size(desc: SagDesc) -> int:
    """Phase 1: validate and return the workspace size in bytes."""
    n = ctypes.c_size_t(0)
    st = load().sel_attn_grad_workspace_size(ctypes.byref(desc), ctypes.byref(n))
    if st != SAG_OK:
        raise SagError(st, "sel_attn_grad_workspace_size")
    return n.value


def plan_info(desc: SagDesc) -> SagPlanInfo:
    """Launch plan of a problem (host only)."""
    info = SagPlanInfo()
    st = load().sel_attn_grad_plan_info(ctypes.byref(desc), ctypes.byref(info))
    if st != SAG_OK:
        raise SagError(st, "sel_attn_grad_plan_info")
    return info


def sel_attn_grad(desc: SagDesc, query, key, value, attention_out, attention_out_grad,
                  softmax_max, softmax_sum, topk_indices, dq, dk, dv, workspace,
                  workspace_bytes: int, stream, main_start=None, main_stop=None) -> None:
    """Phase 2 on raw device pointers (ints); raises on a non-OK status.

    ``main_start`` / ``main_stop`` are optional raw cudaEvent_t handles recorded
    around the main backward kernel (``sel_attn_grad_timed``).
    """
    lib = load()
    if main_start is None and main_stop is None:
        st = lib.sel_attn_grad(ctypes.byref(desc), query, key, value, attention_out,
                               attention_out_grad, softmax_max, softmax_sum, topk_indices,
                               dq, dk, dv, workspace, workspace_bytes, stream)
    else:
        st = lib.sel_attn_grad_timed(ctypes.byref(desc), query, key, value, attention_out,
                                     attention_out_grad, softmax_max, softmax_sum, topk_indices,
                                     dq, dk, dv, workspace, workspace_bytes, stream, main_start,
                                     main_stop)
    if st != SAG_OK:
        raise SagError(st, "sel_attn_grad")


def selftest_wait_timeout(workspace, limit_ns: int, stream) -> None:
    """Enqueue the bounded-wait self-test (see include/selattn.h); read its
    status with ``query_error``."""
    lib = load()
    f = lib.sel_attn_selftest_wait_timeout
    f.argtypes = [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]
    f.restype = ctypes.c_int
    st = f(workspace, int(limit_ns), stream)
    if st != SAG_OK:
        raise SagError(st, "sel_attn_selftest_wait_timeout")


def query_error(workspace, stream) -> int:
    """Wait for the stream; return the status the device recorded."""
    return load().sel_attn_grad_query_error(workspace, stream)


def backward(q, k, v, o, dy, softmax_max, softmax_sum, topk, cu_seqlens_q, cu_seqlens_kv, scale,
             block_size, block_count, deterministic=False, out=None, workspace=None, stream=None,
             check=False, q_rope=None, k_rope=None, rotary=None, q_positions=None, k_positions=None):
    """torch-tensor convenience over the C ABI (allocation and marshalling only).

    All tensors must be contiguous CUDA tensors, TND ([T, N, D]) or BSND
    ([B, S, N, D], 4-D); returns (dq, dk, dv), or (dq, dk, dv, dq_rope,
    dk_rope) with the rope split.  With ``check`` the device status is read
    back (this synchronizes the stream).  With ``rotary`` (see ``forward``) q
    and k, and their gradients, are those before the rotation.
    """
    import torch
    if not q.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    if rotary is not None:
        q, k, q_rope, k_rope = _rotated(q, k, q_rope, k_rope, rotary, cu_seqlens_q, cu_seqlens_kv, q_positions,
                                        k_positions, stream)
    dtype = SAG_FP16 if q.dtype == torch.float16 else SAG_BF16
    layout, s1_max, s2_max, n1, d_qk, n2, d_rope = _layout_of(q, k, q_rope)
    d_v = v.shape[-1]
    desc = make_desc(cu_seqlens_q, cu_seqlens_kv, n1, n2, d_qk, d_v, block_size, block_count, scale,
                     dtype, deterministic, layout, s1_max, s2_max, d_rope)
    need = workspace_size(desc)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
        if d_rope:
            out = out + (torch.empty_like(q_rope), torch.empty_like(k_rope))
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    named = dict(query=q, key=k, value=v, attention_out=o, attention_out_grad=dy, softmax_max=softmax_max,
                 softmax_sum=softmax_sum, topk_indices=topk, dq=out[0], dk=out[1], dv=out[2])
    if d_rope:
        named.update(query_rope=q_rope, key_rope=k_rope, dq_rope=out[3], dk_rope=out[4])
    for t in named.values():
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    io = make_io(**{k_: t.data_ptr() for k_, t in named.items()})
    sel_attn_grad_ex(desc, io, workspace.data_ptr(), need, stream.cuda_stream)
    if rotary is not None:      # the gradients of the tensors that were rotated, in place
        dq, dk = (out[3], out[4]) if d_rope else (out[0], out[1])
        rotary_backward(dq, None, rotary, cu_seqlens_q, q_positions, out=dq, stream=stream)
        rotary_backward(dk, None, rotary, cu_seqlens_kv, k_positions, out=dk, stream=stream)
    if check:
        st = query_error(workspace.data_ptr(), stream.cuda_stream)
        if st != SAG_OK:
            raise SagError(st, "device")
    return out


def _rotated(q, k, q_rope, k_rope, rotary, cu_seqlens_q, cu_seqlens_kv, q_positions, k_positions, stream):
    """(q, k, q_rope, k_rope) with the rotation applied to the rope tensors, or
    to q and k where there are none."""
    turn = lambda x, cu, pos: rotary_forward(x, None, rotary, cu, pos, stream=stream)  # noqa: E731
    if q_rope is not None:
        return q, k, turn(q_rope, cu_seqlens_q, q_positions), turn(k_rope, cu_seqlens_kv, k_positions)
    return turn(q, cu_seqlens_q, q_positions), turn(k, cu_seqlens_kv, k_positions), None, None


def fwd_workspace_size(desc: SagDesc) -> int:
    """Forward phase 1: validate and return the forward's workspace size."""
    n = ctypes.c_size_t(0)
    st = load().sel_attn_fwd_workspace_size(ctypes.byref(desc), ctypes.byref(n))
    if st != SAG_OK:
        raise SagError(st, "sel_attn_fwd_workspace_size")
    return n.value


def sel_attn_fwd(desc: SagDesc, query, key, value, topk_indices, attention_out, softmax_max,
                 softmax_sum, workspace, workspace_bytes: int, stream, passes_start=None,
                 passes_stop=None) -> None:
    """Forward phase 2 on raw device pointers (ints); raises on a non-OK status."""
    lib = load()
    if passes_start is None and passes_stop is None:
        st = lib.sel_attn_fwd(ctypes.byref(desc), query, key, value, topk_indices, attention_out,
                              softmax_max, softmax_sum, workspace, workspace_bytes, stream)
    else:
        st = lib.sel_attn_fwd_timed(ctypes.byref(desc), query, key, value, topk_indices,
                                    attention_out, softmax_max, softmax_sum, workspace,
                                    workspace_bytes, stream, passes_start, passes_stop)
    if st != SAG_OK:
        raise SagError(st, "sel_attn_fwd")


def forward(q, k, v, topk, cu_seqlens_q, cu_seqlens_kv, scale, block_size, block_count,
            out=None, workspace=None, stream=None, check=False, q_rope=None, k_rope=None, rotary=None,
            q_positions=None, k_positions=None):
    """torch-tensor convenience over the forward's C ABI: returns
    (attention_out [.., n1, d_v], softmax_max [.., n1, 8], softmax_sum [.., n1, 8])
    in the layout of q (TND or 4-D BSND).

    ``rotary`` (a ``Rotary``) rotates q_rope and k_rope, or q and k where there
    is no rope split, before the attention; ``q_positions`` / ``k_positions``
    as in ``rotary_forward``."""
    import torch
    if not q.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    if rotary is not None:
        q, k, q_rope, k_rope = _rotated(q, k, q_rope, k_rope, rotary, cu_seqlens_q, cu_seqlens_kv, q_positions,
                                        k_positions, stream)
    dtype = SAG_FP16 if q.dtype == torch.float16 else SAG_BF16
    layout, s1_max, s2_max, n1, d_qk, n2, d_rope = _layout_of(q, k, q_rope)
    d_v = v.shape[-1]
    desc = make_desc(cu_seqlens_q, cu_seqlens_kv, n1, n2, d_qk, d_v, block_size, block_count, scale,
                     dtype, False, layout, s1_max, s2_max, d_rope)
    need = fwd_workspace_size(desc)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    lead = tuple(q.shape[:-1])
    if out is None:
        out = (torch.empty(lead + (d_v,), dtype=q.dtype, device=q.device),
               torch.empty(lead + (8,), dtype=torch.float32, device=q.device),
               torch.empty(lead + (8,), dtype=torch.float32, device=q.device))
    o, smax, ssum = out
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    named = dict(query=q, key=k, value=v, topk_indices=topk, attention_out=o, softmax_max=smax, softmax_sum=ssum)
    if d_rope:
        named.update(query_rope=q_rope, key_rope=k_rope)
    for t in named.values():
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    io = make_io(**{k_: t.data_ptr() for k_, t in named.items()})
    sel_attn_fwd_ex(desc, io, workspace.data_ptr(), need, stream.cuda_stream)
    if check:
        st = query_error(workspace.data_ptr(), stream.cuda_stream)
        if st != SAG_OK:
            raise SagError(st, "device")
    return o, smax, ssum


# ------------------------------------------------------------ lightning indexer
class SliDesc(ctypes.Structure):
    """Mirror of ``sli_desc`` in include/selattn.h."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("n1", ctypes.c_int32), ("n2", ctypes.c_int32), ("d", ctypes.c_int32),
        ("topk", ctypes.c_int32), ("dtype", ctypes.c_int32), ("deterministic", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("cu_seqlens_q", ctypes.POINTER(ctypes.c_int32)), ("cu_seqlens_kv", ctypes.POINTER(ctypes.c_int32)),
        ("s1_max", ctypes.c_int32), ("s2_max", ctypes.c_int32),
    ]


class SliIo(ctypes.Structure):
    """Mirror of ``sli_io`` in include/selattn.h (device pointers as ints)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("query", "key", "weights", "dy", "indices", "dq", "dk", "dweights")]


def _lib_indexer():
    lib = load()
    if not getattr(lib, "_sli_ready", False):
        D, IO, vp, sz = ctypes.POINTER(SliDesc), ctypes.POINTER(SliIo), ctypes.c_void_p, ctypes.c_size_t
        lib.lightning_indexer_grad_workspace_size.argtypes = [D, ctypes.POINTER(sz)]
        lib.lightning_indexer_grad_workspace_size.restype = ctypes.c_int
        lib.lightning_indexer_grad.argtypes = [D, IO, vp, sz, vp]
        lib.lightning_indexer_grad.restype = ctypes.c_int
        lib._sli_ready = True
    return lib


def make_indexer_desc(cu_seqlens_q, cu_seqlens_kv, n1, n2, d, topk, dtype=SAG_BF16, deterministic=False,
                      layout=SAG_LAYOUT_TND, s1_max=0, s2_max=0) -> SliDesc:
    cq = (ctypes.c_int32 * len(cu_seqlens_q))(*[int(x) for x in cu_seqlens_q])
    ck = (ctypes.c_int32 * len(cu_seqlens_kv))(*[int(x) for x in cu_seqlens_kv])
    desc = SliDesc(batch=len(cu_seqlens_q) - 1, n1=n1, n2=n2, d=d, topk=topk, dtype=dtype,
                   deterministic=1 if deterministic else 0, layout=int(layout),
                   cu_seqlens_q=ctypes.cast(cq, ctypes.POINTER(ctypes.c_int32)),
                   cu_seqlens_kv=ctypes.cast(ck, ctypes.POINTER(ctypes.c_int32)), s1_max=int(s1_max),
                   s2_max=int(s2_max))
    desc._keep = (cq, ck)
    return desc


def indexer_workspace_size(desc: SliDesc) -> int:
    n = ctypes.c_size_t(0)
    st = _lib_indexer().lightning_indexer_grad_workspace_size(ctypes.byref(desc), ctypes.byref(n))
    if st != SAG_OK:
        raise SagError(st, "lightning_indexer_grad_workspace_size")
    return n.value


def lightning_indexer_grad(desc: SliDesc, io: SliIo, workspace, workspace_bytes: int, stream) -> None:
    """Phase 2 on raw device pointers (ints); raises on a non-OK status."""
    st = _lib_indexer().lightning_indexer_grad(ctypes.byref(desc), ctypes.byref(io), workspace, workspace_bytes,
                                               stream)
    if st != SAG_OK:
        raise SagError(st, "lightning_indexer_grad")


def indexer_backward(q, k, weights, dy, indices, cu_seqlens_q, cu_seqlens_kv, deterministic=False, out=None,
                     workspace=None, stream=None, check=False):
    """torch-tensor convenience for the lightning-indexer backward: returns
    (dq, dk, dweights).  TND tensors ([T, N, D]) or BSND (4-D, padded)."""
    import torch
    if not q.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    dtype = SAG_FP16 if q.dtype == torch.float16 else SAG_BF16
    bsnd = q.dim() == 4
    layout = SAG_LAYOUT_BSND if bsnd else SAG_LAYOUT_TND
    desc = make_indexer_desc(cu_seqlens_q, cu_seqlens_kv, q.shape[-2], k.shape[-2], q.shape[-1], indices.shape[-1],
                             dtype, deterministic, layout, q.shape[1] if bsnd else 0, k.shape[1] if bsnd else 0)
    need = indexer_workspace_size(desc)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(weights))
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    named = dict(query=q, key=k, weights=weights, dy=dy, indices=indices, dq=out[0], dk=out[1], dweights=out[2])
    for t in named.values():
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    io = SliIo(**{k_: t.data_ptr() for k_, t in named.items()})
    lightning_indexer_grad(desc, io, workspace.data_ptr(), need, stream.cuda_stream)
    if check:
        st = query_error(workspace.data_ptr(), stream.cuda_stream)
        if st != SAG_OK:
            raise SagError(st, "device")
    return out


# ------------------------------------------- rotary positions, cross attention
EXPORTED_NEIGHBOURS = ("rotary_frequencies", "rotary_workspace_size", "rotary_fwd", "rotary_grad",
                       "cross_attn_fwd_workspace_size", "cross_attn_fwd", "cross_attn_grad_workspace_size",
                       "cross_attn_grad", "cross_attn_query_error")
EXPORTED_LAYER = ("norm_rotary_fwd_workspace_size", "norm_rotary_grad_workspace_size", "norm_rotary_fwd", "norm_rotary_grad",
                  "window_attn_fwd_workspace_size", "window_attn_grad_workspace_size", "window_attn_fwd",
                  "window_attn_grad", "window_attn_query_error", "paged_attn_fwd_workspace_size",
                  "paged_append_workspace_size", "paged_attn_fwd", "paged_append", "paged_query_error")
SRT_HALF, SRT_INTERLEAVED = 0, 1
_ROTARY_STYLES = {"half": SRT_HALF, "interleaved": SRT_INTERLEAVED}
_ROTARY_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3, "bands": 4}


class SrtDesc(ctypes.Structure):
    """Mirror of ``srt_desc`` in include/selattn.h."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("n1", ctypes.c_int32), ("n2", ctypes.c_int32), ("d", ctypes.c_int32),
        ("d_rot", ctypes.c_int32), ("offset", ctypes.c_int32), ("style", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("layout", ctypes.c_int32), ("s_max", ctypes.c_int32),
        ("cu_seqlens", ctypes.POINTER(ctypes.c_int32)), ("inv_freq", ctypes.POINTER(ctypes.c_double)),
        ("magnitude", ctypes.c_double),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
        ("k_out_stride", ctypes.c_int64),
    ]


class SrtIo(ctypes.Structure):
    """Mirror of ``srt_io`` in include/selattn.h (device pointers as ints)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("query", "key", "positions", "query_out", "key_out")]


class ScaDesc(ctypes.Structure):
    """Mirror of ``sca_desc`` in include/selattn.h."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("n1", ctypes.c_int32), ("n2", ctypes.c_int32), ("d", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32), ("scale", ctypes.c_double),
        ("cu_seqlens_q", ctypes.POINTER(ctypes.c_int32)), ("cu_seqlens_kv", ctypes.POINTER(ctypes.c_int32)),
        ("s1_max", ctypes.c_int32), ("s2_max", ctypes.c_int32),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
    ]


class SwaDesc(ctypes.Structure):
    """Mirror of ``swa_desc`` in include/selattn.h (the cross attention's fields by their own names)."""
    _anonymous_ = ("attn",)
    _fields_ = [("attn", ScaDesc), ("left", ctypes.c_int32), ("right", ctypes.c_int32)]


class SnrDesc(ctypes.Structure):
    """Mirror of ``snr_desc`` in include/selattn.h (the rotary positions' fields by their own names)."""
    _anonymous_ = ("rotary",)
    _fields_ = [("rotary", SrtDesc), ("eps", ctypes.c_double), ("weight_offset", ctypes.c_double),
                ("weight_fp32", ctypes.c_int32), ("reserved_", ctypes.c_int32),
                ("q_grad_stride", ctypes.c_int64), ("k_grad_stride", ctypes.c_int64)]


class SnrIo(ctypes.Structure):
    """Mirror of ``snr_io`` in include/selattn.h (device pointers as ints)."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "query", "key", "query_weight", "key_weight", "positions", "query_out", "key_out", "query_out_grad", "key_out_grad",
        "query_grad", "key_grad", "query_weight_grad", "key_weight_grad")]


class SpaDesc(ctypes.Structure):
    """Mirror of ``spa_desc`` in include/selattn.h."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("n1", ctypes.c_int32), ("n2", ctypes.c_int32), ("d", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32), ("scale", ctypes.c_double),
        ("cu_seqlens_q", ctypes.POINTER(ctypes.c_int32)), ("s1_max", ctypes.c_int32),
        ("left", ctypes.c_int32), ("right", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("pages", ctypes.c_int32), ("width", ctypes.c_int32),
        ("kv_expected", ctypes.c_int32), ("reserved_", ctypes.c_int32),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
        ("k_row", ctypes.c_int64), ("k_page", ctypes.c_int64), ("v_row", ctypes.c_int64), ("v_page", ctypes.c_int64),
    ]


class SpaIo(ctypes.Structure):
    """Mirror of ``spa_io`` in include/selattn.h (device pointers as ints)."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "query", "key", "value", "key_cache", "value_cache", "page_table", "kv_lens", "attention_out", "softmax_lse")]


class ScaIo(ctypes.Structure):
    """Mirror of ``sca_io`` in include/selattn.h (device pointers as ints)."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "query", "key", "value", "attention_out", "attention_out_grad", "softmax_lse", "key_mask", "dq", "dk", "dv")]


_neighbours = None
_torch = None       # the module, for calls that take microseconds: an import statement costs a quarter of one


def _lib_neighbours():
    global _neighbours, _torch
    if _neighbours is not None:
        return _neighbours
    import torch
    _torch = torch
    lib = load()
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    dbl, psz = ctypes.c_double, ctypes.POINTER(ctypes.c_size_t)
    lib.rotary_frequencies.argtypes = [ctypes.c_int32, dbl, ctypes.c_int32] + [dbl] * 6 + [ctypes.POINTER(dbl)] * 2
    lib.cross_attn_query_error.argtypes = [vp, vp]
    for prefix, desc, io, names in (("rotary", SrtDesc, SrtIo, ("fwd", "grad")),
                                    ("cross_attn", ScaDesc, ScaIo, ("fwd", "grad")),
                                    ("window_attn", SwaDesc, ScaIo, ("fwd", "grad")),
                                    ("norm_rotary", SnrDesc, SnrIo, ("fwd", "grad")),
                                    ("paged", SpaDesc, SpaIo, ("attn_fwd", "append"))):
        for n in names:
            getattr(lib, f"{prefix}_{n}").argtypes = [ctypes.POINTER(desc), ctypes.POINTER(io), vp, sz, vp]
            if prefix not in ("rotary", "cross_attn"):
                getattr(lib, f"{prefix}_{n}_workspace_size").argtypes = [ctypes.POINTER(desc), psz]
    lib.window_attn_query_error.argtypes = lib.paged_query_error.argtypes = [vp, vp]
    lib.rotary_workspace_size.argtypes = [ctypes.POINTER(SrtDesc), psz]
    lib.cross_attn_fwd_workspace_size.argtypes = [ctypes.POINTER(ScaDesc), psz]
    lib.cross_attn_grad_workspace_size.argtypes = [ctypes.POINTER(ScaDesc), psz]
    for n in EXPORTED_NEIGHBOURS + EXPORTED_LAYER:
        getattr(lib, n).restype = ctypes.c_int
    _neighbours = lib
    return lib


def _phase1(name: str, desc) -> int:
    n = ctypes.c_size_t(0)
    st = getattr(_lib_neighbours(), name)(ctypes.byref(desc), ctypes.byref(n))
    if st != SAG_OK:
        raise SagError(st, name)
    return n.value


def _i32(xs):
    return (ctypes.c_int32 * len(xs))(*[int(x) for x in xs])


def _sag_dtype(t):
    import torch
    if t.dtype == torch.bfloat16:
        return SAG_BF16
    if t.dtype == torch.float16:
        return SAG_FP16
    raise SagError(SAG_ERR_DTYPE, f"tensor of {t.dtype}")


def _torch_dtype(desc):
    import torch
    return torch.float16 if desc.dtype == SAG_FP16 else torch.bfloat16


def _row_stride(name, t, heads, d):
    """Elements from one row (token) to the next of a TND or BSND tensor whose
    rows are dense; 0 for a dense tensor."""
    if t.is_contiguous():
        return 0
    if (d > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != d):
        raise ValueError(f"{name}: the heads and columns of a row must be dense")
    if t.dim() == 3:
        step = t.stride(0) if t.shape[0] > 1 else heads * d
    else:
        b, s = t.shape[0], t.shape[1]
        step = t.stride(1) if s > 1 else (t.stride(0) if b > 1 else heads * d)
        if b > 1 and t.stride(0) != s * step:
            raise ValueError(f"{name}: the batches of a padded tensor must follow one another in memory")
    if step < heads * d:
        raise ValueError(f"{name}: rows overlap")
    return step


def _check_rows(name, t, shape, dtype):
    """A tensor of the descriptor's rows and type: a padded batch of just its
    shape, or packed rows, possibly with more behind them."""
    if t.dtype is not dtype:
        raise SagError(SAG_ERR_DTYPE, f"{name}: tensor of {t.dtype}, expected {dtype}")
    if t.shape == shape:
        return
    if len(shape) == 4 or t.dim() != 3 or tuple(t.shape[1:]) != shape[1:] or t.shape[0] < shape[0]:
        raise ValueError(f"{name}: shape {tuple(t.shape)} does not hold the descriptor's {shape}")


def _check(name, t, device, shape, dtype):
    if t.dtype is not dtype:
        raise SagError(SAG_ERR_DTYPE, f"{name}: tensor of {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, not on device {device}")


def _dense(name, t, device, shape, dtype):
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    _check(name, t, device, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _new(like):
    """A dense tensor of the same shape, type and device."""
    if like.is_contiguous():
        return _torch.empty_like(like)
    return _torch.empty_like(like, memory_format=_torch.contiguous_format)


_PREFIXES = ("cu_seqlens", "cu_seqlens_q", "cu_seqlens_kv")


def _rows_of(desc, cu, s_max):
    if desc.layout == SAG_LAYOUT_BSND:
        return (desc.batch, s_max)
    return (cu[desc.batch] if desc.batch >= 0 else 0,)


def _derive(desc, dense=False):
    """What calls with the descriptor go by: the tensors' shapes and type.  Strides come from the tensors, so the
    descriptor serves dense tensors as it is only while its own are 0."""
    if isinstance(desc, (SrtDesc, SnrDesc)):
        lead = _rows_of(desc, desc.cu_seqlens, desc.s_max)
        desc._shapes = (lead + (desc.n1, desc.d), lead + (desc.n2, desc.d))
    elif isinstance(desc, SpaDesc):
        lead = _rows_of(desc, desc.cu_seqlens_q, desc.s1_max)
        desc._shapes = (lead + (desc.n1, desc.d), lead + (desc.n2, desc.d),
                        (desc.pages, desc.page_size, desc.n2, desc.d), (desc.batch, desc.width))
    else:
        desc._shapes = (_rows_of(desc, desc.cu_seqlens_q, desc.s1_max) + (desc.n1, desc.d),
                        _rows_of(desc, desc.cu_seqlens_kv, desc.s2_max) + (desc.n2, desc.d))
    for size in _SIZES:
        desc.__dict__.pop(size, None)
    desc._dtype = _torch_dtype(desc)
    desc._dense = dense
    desc._bytes = bytes(desc)
    # the prefix sums, which the descriptor has by address only (of batches that the library takes)
    views = [(ctypes.c_char * (4 * (desc.batch + 1))).from_address(ctypes.addressof(p.contents))
             for p in (getattr(desc, name, None) for name in _PREFIXES) if p and 0 <= desc.batch <= 65536]
    desc._lengths = [(v, v.raw) for v in views]
    return desc


def _unchanged(desc):
    """Whether a kept descriptor, and the lengths that it points to, are what _derive saw."""
    if bytes(desc) != desc._bytes:
        return False
    for view, seen in desc._lengths:
        if view.raw != seen:
            return False
    return True


def _size_of(desc, size):
    """Phase 1 of a kept descriptor, once."""
    need = desc.__dict__.get(size)
    if need is None:
        need = desc.__dict__[size] = size(desc)
    return need


def _scratch(workspace, need, device):
    """The caller's workspace where it is large enough, or a new one."""
    if workspace is None or workspace.numel() < need:
        return _torch.empty(need, dtype=_torch.uint8, device=device)
    if not workspace.is_contiguous():       # an expanded tensor has more elements than memory
        raise ValueError("workspace must be contiguous")
    return workspace


def _given(desc):
    """A kept descriptor, brought up to date if fields or lengths were set since."""
    return desc if _unchanged(desc) else _derive(desc)


def _with(desc, **fields):
    """The descriptor, or a copy where a field differs (a kept one is never changed)."""
    if all(getattr(desc, k) == v for k, v in fields.items()):
        return desc
    new = type(desc).from_buffer_copy(desc)
    new.__dict__.update(desc.__dict__, _dense=False)
    for k, v in fields.items():
        setattr(new, k, v)
    return new


def _launch(device, stream, call):
    """call(raw stream) with the tensors' device current; what the call
    allocates comes from the pool of the stream that it runs on."""
    if stream is not None:
        with _torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    if _torch._C._cuda_getDevice() != device:
        with _torch.cuda.device(device):
            return call(_torch.cuda.current_stream().cuda_stream)
    return call(_torch._C._cuda_getCurrentRawStream(device))   # a stream object costs several microseconds


class Rotary:
    """Frequencies, column range and style of rotary positions (see
    ``rotary_frequencies`` and ``srt_desc`` in include/selattn.h).

    ``d_rot`` columns from ``offset`` on are rotated; ``style`` is "half" or
    "interleaved", ``scaling`` "none", "linear", "base", "ramp" or "bands".
    ``inv_freq`` (radians per position, d_rot / 2 floats) and ``magnitude``
    replace the computed ones.
    """

    def __init__(self, d_rot, base=10000.0, style="half", offset=0, scaling="none", factor=1.0, original_length=0,
                 beta_fast=32.0, beta_slow=1.0, low=1.0, high=4.0, inv_freq=None, magnitude=None):
        if style not in _ROTARY_STYLES:
            raise ValueError(f"style {style!r} is none of {sorted(_ROTARY_STYLES)}")
        if scaling not in _ROTARY_SCALINGS:
            raise ValueError(f"scaling {scaling!r} is none of {sorted(_ROTARY_SCALINGS)}")
        self.d_rot, self.offset, self.style = int(d_rot), int(offset), _ROTARY_STYLES[style]
        self._freq = (ctypes.c_double * max(1, self.d_rot // 2))()
        mag = ctypes.c_double(1.0)
        if inv_freq is None:
            st = _lib_neighbours().rotary_frequencies(self.d_rot, base, _ROTARY_SCALINGS[scaling], factor,
                                                      original_length, beta_fast, beta_slow, low, high, self._freq,
                                                      ctypes.byref(mag))
            if st != SAG_OK:
                raise SagError(st, "rotary_frequencies")
        else:
            if len(inv_freq) != self.d_rot // 2:
                raise ValueError(f"{len(inv_freq)} frequencies for {self.d_rot} columns")
            self._freq[:] = [float(f) for f in inv_freq]
        self.magnitude = mag.value if magnitude is None else float(magnitude)

    @property
    def inv_freq(self):
        return list(self._freq)


def make_rotary_desc(rotary: Rotary, cu_seqlens, n1, n2, d, dtype=SAG_BF16, layout=SAG_LAYOUT_TND, s_max=0) -> SrtDesc:
    """Descriptor of a rotation (n2 = 0: no key); keeps the host arrays alive.
    The tensor calls take strides from the tensors, whatever the fields say."""
    cu = _i32(cu_seqlens)
    desc = SrtDesc(batch=len(cu) - 1, n1=n1, n2=n2, d=d, d_rot=rotary.d_rot, offset=rotary.offset, style=rotary.style,
                   dtype=dtype, layout=int(layout), s_max=int(s_max),
                   cu_seqlens=ctypes.cast(cu, ctypes.POINTER(ctypes.c_int32)),
                   inv_freq=ctypes.cast(rotary._freq, ctypes.POINTER(ctypes.c_double)), magnitude=rotary.magnitude)
    desc._keep = (cu, rotary._freq)
    return _derive(desc, dense=True)


def rotary_workspace_size(desc: SrtDesc) -> int:
    """Phase 1: validate and return the workspace size in bytes (0 for small batches)."""
    return _phase1("rotary_workspace_size", desc)


def _rotary(entry, q, k, rotary, cu_seqlens, positions, out, workspace, stream, desc):
    if not q.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    shape = q.shape
    n1, d = shape[-2:]
    n2 = k.shape[-2] if k is not None else 0
    if desc is None:
        bsnd = q.dim() == 4
        desc = make_rotary_desc(rotary, cu_seqlens, n1, n2, d, _sag_dtype(q), SAG_LAYOUT_BSND if bsnd else SAG_LAYOUT_TND,
                                shape[1] if bsnd else 0)
    else:
        desc = _given(desc)
    qs, ks = desc._shapes
    dtype, device = desc._dtype, q.get_device()
    if q.dtype is not dtype or shape != qs:
        _check_rows("q", q, qs, dtype)
    lead = shape[:-2]
    if k is not None:
        _check("k", k, device, lead + ks[-2:], dtype)
    elif ks[-2]:
        raise ValueError("the descriptor has a key")
    pos = _dense("positions", positions, device, lead, _torch.int32) if positions is not None else None

    def call(handle):
        use = desc
        if out is None:
            qo = _new(q)
            ko = _new(k) if k is not None else None
            plain = desc._dense and q.is_contiguous() and (k is None or k.is_contiguous())
        else:
            qo, ko = (out, None) if k is None and not isinstance(out, (tuple, list)) else out
            _check("out", qo, device, q.shape, dtype)
            if k is not None:
                _check("out", ko, device, k.shape, dtype)
            plain = False
        if not plain:
            use = _with(desc, q_stride=_row_stride("q", q, n1, d), q_out_stride=_row_stride("out", qo, n1, d),
                        k_stride=_row_stride("k", k, n2, d) if n2 else 0,
                        k_out_stride=_row_stride("out", ko, n2, d) if n2 else 0)
        io = SrtIo(q.data_ptr(), k.data_ptr() if n2 else None, pos, qo.data_ptr(), ko.data_ptr() if n2 else None)
        ws, need = None, 0
        if use.batch > 64:          # smaller tables travel with the launch
            need = rotary_workspace_size(use)
            ws = _scratch(workspace, need, q.device)
        st = entry(use, io, ws.data_ptr() if need else None, need, handle)
        if st != SAG_OK:
            raise SagError(st, entry.__name__)
        return (qo, ko) if k is not None else qo

    return _launch(device, stream, call)


def rotary_forward(q, k, rotary, cu_seqlens=None, positions=None, out=None, workspace=None, stream=None, desc=None):
    """Rotary positions of q [.., n1, d] and k [.., n2, d] (or None), TND or 4-D
    BSND tensors of the same rows: returns (q, k) rotated, or q alone.

    A row's position is its place in its sequence (``cu_seqlens``), or
    ``positions[row]`` (int32, the shape of q without heads and columns).
    ``out=(q, k)`` rotates in place; rows may be strided (slices of a fused
    projection).  ``desc`` (make_rotary_desc) replaces rotary and cu_seqlens.
    """
    return _rotary(_lib_neighbours().rotary_fwd, q, k, rotary, cu_seqlens, positions, out, workspace, stream, desc)


def rotary_backward(dq, dk, rotary, cu_seqlens=None, positions=None, out=None, workspace=None, stream=None, desc=None):
    """Gradient of ``rotary_forward``: the gradients of its outputs to those of
    its inputs; arguments alike."""
    return _rotary(_lib_neighbours().rotary_grad, dq, dk, rotary, cu_seqlens, positions, out, workspace, stream, desc)


def make_cross_desc(cu_seqlens_q, cu_seqlens_kv, n1, n2, d, scale, dtype=SAG_BF16, layout=SAG_LAYOUT_TND, s1_max=0,
                    s2_max=0) -> ScaDesc:
    """Descriptor of a cross attention; keeps the host arrays alive.  The tensor
    calls take strides from the tensors, whatever the fields say."""
    cq, ck = _i32(cu_seqlens_q), _i32(cu_seqlens_kv)
    if len(cq) != len(ck):
        raise ValueError("cu_seqlens_q and cu_seqlens_kv are of different batches")
    desc = ScaDesc(batch=len(cq) - 1, n1=n1, n2=n2, d=d, dtype=dtype, layout=int(layout), scale=float(scale),
                   cu_seqlens_q=ctypes.cast(cq, ctypes.POINTER(ctypes.c_int32)),
                   cu_seqlens_kv=ctypes.cast(ck, ctypes.POINTER(ctypes.c_int32)), s1_max=int(s1_max), s2_max=int(s2_max))
    desc._keep = (cq, ck)
    return _derive(desc, dense=True)


def cross_fwd_workspace_size(desc: ScaDesc) -> int:
    """Phase 1 of the forward: validate and return the workspace size in bytes."""
    return _phase1("cross_attn_fwd_workspace_size", desc)


def cross_grad_workspace_size(desc: ScaDesc) -> int:
    """Phase 1 of the gradient: validate and return the workspace size in bytes."""
    return _phase1("cross_attn_grad_workspace_size", desc)


def cross_query_error(workspace, stream) -> int:
    """Wait for the stream; return the status the device recorded."""
    return _lib_neighbours().cross_attn_query_error(workspace, stream)


def _cross(entry, size, q, k, v, cu_seqlens_q, cu_seqlens_kv, scale, key_mask, workspace, stream, check, desc, tensors,
           make=None):
    """Shared by the two directions of cross and windowed attention:
    ``tensors(io, device, dtype)`` fills in the remaining sca_io pointers and
    gives the outputs; ``make`` is what builds the descriptor."""
    if not q.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    q_shape, k_shape = q.shape, k.shape
    n1, d = q_shape[-2:]
    n2 = k_shape[-2]
    if desc is None:
        bsnd = q.dim() == 4
        if bsnd and k.dim() != 4:
            raise ValueError("BSND needs 4-D query and key tensors")
        desc = (make or make_cross_desc)(cu_seqlens_q, cu_seqlens_kv, n1, n2, d, scale, dtype=_sag_dtype(q),
                                         layout=SAG_LAYOUT_BSND if bsnd else SAG_LAYOUT_TND,
                                         s1_max=q_shape[1] if bsnd else 0, s2_max=k_shape[1] if bsnd else 0)
    else:
        desc = _given(desc)
    dtype, device = desc._dtype, q.get_device()
    qs, ks = desc._shapes
    if q.dtype is not dtype or q_shape != qs:
        _check_rows("q", q, qs, dtype)
    if k.dtype is not dtype or k_shape != ks:
        _check_rows("k", k, ks, dtype)
    if v.dtype is not dtype or v.shape != k_shape or v.get_device() != device:
        _check("v", v, device, k_shape, dtype)
    if k.get_device() != device:
        raise ValueError(f"k: on {k.device}, not on {q.device}")
    use = desc
    if not (desc._dense and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        use = _with(desc, q_stride=_row_stride("q", q, n1, d), k_stride=_row_stride("k", k, n2, d),
                    v_stride=_row_stride("v", v, n2, d))
    io = ScaIo(q.data_ptr(), k.data_ptr(), v.data_ptr())
    if key_mask is not None:
        if key_mask.dtype not in (_torch.bool, _torch.uint8):
            raise ValueError("key_mask must be a bool or uint8 tensor")
        io.key_mask = _dense("key_mask", key_mask, device, k_shape[:-2], key_mask.dtype)

    def call(handle):
        outs = tensors(io, device, dtype)
        need = _size_of(desc, size)
        ws = _scratch(workspace, need, q.device)
        st = entry(use, io, ws.data_ptr(), need, handle)
        if st == SAG_OK and check:
            st = cross_query_error(ws.data_ptr(), handle)
        if st != SAG_OK:
            raise SagError(st, entry.__name__)
        return outs

    return _launch(device, stream, call)


def _usual_forward(entry, size, q, k, v, key_mask, workspace, desc):
    """The forward of a kept descriptor with dense tensors of just its shapes on the current device, which is what calls of a
    few microseconds are: the checks of ``_cross`` in one condition.  None: not such a call."""
    if not desc._dense or not _unchanged(desc):
        return None
    qs, ks = desc._shapes
    dtype, device = desc._dtype, q.get_device()
    if not (q.dtype is dtype and k.dtype is dtype and v.dtype is dtype and q.shape == qs and k.shape == ks and v.shape == ks
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and device >= 0 and k.get_device() == device
            and v.get_device() == device and _torch._C._cuda_getDevice() == device):
        return None
    mask = None
    if key_mask is not None:
        if key_mask.dtype is not _torch.bool or key_mask.shape != ks[:-2] or not key_mask.is_contiguous() \
                or key_mask.get_device() != device:
            return None
        mask = key_mask.data_ptr()
    where = q.device
    o, lse = _torch.empty_like(q), _torch.empty(qs[:-1], dtype=_torch.float32, device=where)
    need = _size_of(desc, size)
    ws = _scratch(workspace, need, where)
    io = ScaIo(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), None, lse.data_ptr(), mask)
    st = entry(desc, io, ws.data_ptr(), need, _torch._C._cuda_getCurrentRawStream(device))
    if st != SAG_OK:
        raise SagError(st, entry.__name__)
    return o, lse


def _attention_out(q, out):
    """The forward's outputs as _cross wants them."""
    def tensors(io, device, dtype):
        if out is None:
            o, lse = _new(q), _torch.empty(q.shape[:-1], dtype=_torch.float32, device=q.device)
            io.attention_out, io.softmax_lse = o.data_ptr(), lse.data_ptr()
        else:
            o, lse = out
            io.attention_out = _dense("attention_out", o, device, q.shape, dtype)
            io.softmax_lse = _dense("softmax_lse", lse, device, q.shape[:-1], _torch.float32)
        return o, lse
    return tensors


def _attention_grads(q, k, v, o, dy, lse, out):
    """The gradient's remaining inputs and its outputs as _cross wants them."""
    def tensors(io, device, dtype):
        io.attention_out = _dense("o", o, device, q.shape, dtype)
        io.attention_out_grad = _dense("dy", dy, device, q.shape, dtype)
        io.softmax_lse = _dense("lse", lse, device, q.shape[:-1], _torch.float32)
        if out is None:
            outs = dq, dk, dv = _new(q), _new(k), _new(v)
            io.dq, io.dk, io.dv = dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
        else:
            outs = dq, dk, dv = out
            io.dq = _dense("dq", dq, device, q.shape, dtype)
            io.dk = _dense("dk", dk, device, k.shape, dtype)
            io.dv = _dense("dv", dv, device, k.shape, dtype)
        return outs
    return tensors


def cross_forward(q, k, v, cu_seqlens_q=None, cu_seqlens_kv=None, scale=None, key_mask=None, out=None, workspace=None,
                  stream=None, check=False, desc=None):
    """Cross attention of q [.., n1, d] to the encoder states k, v [.., n2, d] of
    the same sequences, TND or 4-D BSND: returns (attention_out [.., n1, d],
    softmax_lse [.., n1] in fp32).

    ``key_mask`` (bool or uint8, the shape of k without heads and columns):
    states where it is 0 are not there.  q, k and v may be strided by rows.
    ``desc`` (make_cross_desc) replaces cu_seqlens_* and scale; ``check`` reads
    the device status back (this synchronizes the stream).
    """
    entry = _lib_neighbours().cross_attn_fwd
    if desc is not None and out is None and stream is None and not check:
        done = _usual_forward(entry, cross_fwd_workspace_size, q, k, v, key_mask, workspace, desc)
        if done is not None:
            return done
    return _cross(entry, cross_fwd_workspace_size, q, k, v, cu_seqlens_q, cu_seqlens_kv, scale, key_mask,
                  workspace, stream, check, desc, _attention_out(q, out))


def cross_backward(q, k, v, o, dy, lse, cu_seqlens_q=None, cu_seqlens_kv=None, scale=None, key_mask=None, out=None,
                   workspace=None, stream=None, check=False, desc=None):
    """Gradient of ``cross_forward``: returns (dq, dk, dv), from the forward's o
    and lse and the gradient dy of o; the other arguments as there."""
    return _cross(_lib_neighbours().cross_attn_grad, cross_grad_workspace_size, q, k, v, cu_seqlens_q, cu_seqlens_kv, scale, key_mask,
                  workspace, stream, check, desc, _attention_grads(q, k, v, o, dy, lse, out))


# ------------------------------------------------------- windowed attention
def _reach(keys):
    """A window's side as the descriptors hold it: beyond 32 bits it has no limit that shows."""
    return max(-1, min(int(keys), 2 ** 31 - 1))


def make_window_desc(cu_seqlens_q, cu_seqlens_kv, n1, n2, d, scale, left=-1, right=0, dtype=SAG_BF16, layout=SAG_LAYOUT_TND,
                     s1_max=0, s2_max=0) -> SwaDesc:
    """Descriptor of a windowed attention; ``left`` and ``right`` are the keys
    before and behind a query's position that it attends to (-1: all of them).
    Keeps the host arrays alive; the tensor calls take strides from the tensors."""
    base = make_cross_desc(cu_seqlens_q, cu_seqlens_kv, n1, n2, d, scale, dtype, layout, s1_max, s2_max)
    desc = SwaDesc(attn=base, left=_reach(left), right=_reach(right))
    desc._keep = base._keep
    return _derive(desc, dense=True)


def window_fwd_workspace_size(desc: SwaDesc) -> int:
    """Phase 1 of the forward: validate and return the workspace size in bytes."""
    return _phase1("window_attn_fwd_workspace_size", desc)


def window_grad_workspace_size(desc: SwaDesc) -> int:
    """Phase 1 of the gradient: validate and return the workspace size in bytes."""
    return _phase1("window_attn_grad_workspace_size", desc)


def window_query_error(workspace, stream) -> int:
    """Wait for the stream; return the status the device recorded."""
    return _lib_neighbours().window_attn_query_error(workspace, stream)


def _make_window(left, right):
    return lambda *args, **kw: make_window_desc(*args, left=left, right=right, **kw)


def window_forward(q, k, v, cu_seqlens_q=None, cu_seqlens_kv=None, scale=None, left=-1, right=0, key_mask=None, out=None,
                   workspace=None, stream=None, check=False, desc=None):
    """Attention of q [.., n1, d] to the keys k, v [.., n2, d] of the same
    sequences from ``left`` before to ``right`` behind each query's position
    (-1: all; the last query stands at the last key), TND or 4-D BSND: returns
    (attention_out [.., n1, d], softmax_lse [.., n1] in fp32).

    Causal by default; the other arguments as in ``cross_forward``, with
    ``desc`` from make_window_desc (it replaces left and right too)."""
    entry = _lib_neighbours().window_attn_fwd
    if desc is not None and out is None and stream is None and not check:
        done = _usual_forward(entry, window_fwd_workspace_size, q, k, v, key_mask, workspace, desc)
        if done is not None:
            return done
    return _cross(entry, window_fwd_workspace_size, q, k, v, cu_seqlens_q, cu_seqlens_kv, scale,
                  key_mask, workspace, stream, check, desc, _attention_out(q, out), _make_window(left, right))


def window_backward(q, k, v, o, dy, lse, cu_seqlens_q=None, cu_seqlens_kv=None, scale=None, left=-1, right=0, key_mask=None,
                    out=None, workspace=None, stream=None, check=False, desc=None):
    """Gradient of ``window_forward``: returns (dq, dk, dv), from the forward's
    o and lse and the gradient dy of o; the probabilities are formed again."""
    return _cross(_lib_neighbours().window_attn_grad, window_grad_workspace_size, q, k, v, cu_seqlens_q, cu_seqlens_kv, scale,
                  key_mask, workspace, stream, check, desc, _attention_grads(q, k, v, o, dy, lse, out),
                  _make_window(left, right))


# ------------------------------------------------------------- paged cache
def make_paged_desc(cu_seqlens_q, n1, n2, d, scale, pages, page_size, width, left=-1, right=0, dtype=SAG_BF16,
                    layout=SAG_LAYOUT_TND, s1_max=0, kv_expected=0) -> SpaDesc:
    """Descriptor of new tokens over a paged cache of ``pages`` pages of
    ``page_size`` rows, ``width`` of them a sequence at most; serves
    ``paged_append`` and ``paged_forward``.  Keeps the host array alive; the
    tensor calls take strides from the tensors."""
    cq = _i32(cu_seqlens_q)
    desc = SpaDesc(batch=len(cq) - 1, n1=n1, n2=n2, d=d, dtype=dtype, layout=int(layout), scale=float(scale),
                   cu_seqlens_q=ctypes.cast(cq, ctypes.POINTER(ctypes.c_int32)), s1_max=int(s1_max), left=_reach(left),
                   right=_reach(right), page_size=int(page_size), pages=int(pages), width=int(width),
                   kv_expected=int(kv_expected), reserved_=0)
    desc._keep = (cq,)
    return _derive(desc, dense=True)


def paged_fwd_workspace_size(desc: SpaDesc) -> int:
    """Phase 1 of the attention: validate and return the workspace size in bytes."""
    return _phase1("paged_attn_fwd_workspace_size", desc)


def paged_append_workspace_size(desc: SpaDesc) -> int:
    """Phase 1 of the append: validate and return the workspace size in bytes."""
    return _phase1("paged_append_workspace_size", desc)


def paged_query_error(workspace, stream) -> int:
    """Wait for the stream; return the status the device recorded."""
    return _lib_neighbours().paged_query_error(workspace, stream)


def _cache_strides(name, t, shape, dtype, device):
    """(row, page) strides of a cache tensor; 0 for a dense one."""
    _check(name, t, device, shape, dtype)
    if t.is_contiguous():
        return 0, 0
    pages, page, heads, d = shape
    if (d > 1 and t.stride(3) != 1) or (heads > 1 and t.stride(2) != d):
        raise ValueError(f"{name}: the heads and columns of a row must be dense")
    row = t.stride(1) if page > 1 else heads * d
    between = t.stride(0) if pages > 1 else row * page
    if row < heads * d or between < row * (page - 1) + heads * d:
        raise ValueError(f"{name}: rows and pages must not overlap or interleave")
    return row, between


def _paged(entry, size, x, desc, k_cache, v_cache, page_table, kv_lens, workspace, stream, check, fill):
    """Shared by the append and the attention: ``x`` is a tensor of new tokens,
    ``fill(io, device, dtype)`` sets the other pointers and gives the outputs
    and the strides that differ from 0."""
    desc = _given(desc)
    dtype, device = desc._dtype, x.get_device()
    cache, table = desc._shapes[2:]
    io = SpaIo()
    io.key_cache, io.value_cache = k_cache.data_ptr(), v_cache.data_ptr()
    k_row, k_page = _cache_strides("k_cache", k_cache, cache, dtype, device)
    v_row, v_page = _cache_strides("v_cache", v_cache, cache, dtype, device)
    io.page_table = _dense("page_table", page_table, device, table, _torch.int32)
    io.kv_lens = _dense("kv_lens", kv_lens, device, table[:1], _torch.int32)

    def call(handle):
        outs, strides = fill(io, device, dtype)
        use = desc
        if not desc._dense or strides or k_row or v_row or k_page or v_page:
            use = _with(desc, **dict(dict(q_stride=0, k_stride=0, v_stride=0), **strides), k_row=k_row, k_page=k_page, v_row=v_row,
                        v_page=v_page)
        need = _size_of(desc, size)
        ws = _scratch(workspace, need, x.device)
        st = entry(use, io, ws.data_ptr(), need, handle)
        if st == SAG_OK and check:
            st = paged_query_error(ws.data_ptr(), handle)
        if st != SAG_OK:
            raise SagError(st, entry.__name__)
        return outs

    return _launch(device, stream, call)


def _usual_paged(entry, q, k_cache, v_cache, page_table, kv_lens, workspace, desc):
    """As ``_usual_forward``, over pages."""
    if not desc._dense or not _unchanged(desc):
        return None
    qs, _, cache, table = desc._shapes
    dtype, device, i32 = desc._dtype, q.get_device(), _torch.int32
    if not (q.dtype is dtype and k_cache.dtype is dtype and v_cache.dtype is dtype and page_table.dtype is i32
            and kv_lens.dtype is i32 and q.shape == qs and k_cache.shape == cache and v_cache.shape == cache
            and page_table.shape == table and kv_lens.shape == table[:1] and q.is_contiguous() and k_cache.is_contiguous()
            and v_cache.is_contiguous() and page_table.is_contiguous() and kv_lens.is_contiguous() and device >= 0
            and k_cache.get_device() == device and v_cache.get_device() == device and page_table.get_device() == device
            and kv_lens.get_device() == device and _torch._C._cuda_getDevice() == device):
        return None
    where = q.device
    o, lse = _torch.empty_like(q), _torch.empty(qs[:-1], dtype=_torch.float32, device=where)
    need = _size_of(desc, paged_fwd_workspace_size)
    ws = _scratch(workspace, need, where)
    io = SpaIo(q.data_ptr(), None, None, k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(),
               o.data_ptr(), lse.data_ptr())
    st = entry(desc, io, ws.data_ptr(), need, _torch._C._cuda_getCurrentRawStream(device))
    if st != SAG_OK:
        raise SagError(st, entry.__name__)
    return o, lse


def _paged_layout(x):
    bsnd = x.dim() == 4
    return dict(dtype=_sag_dtype(x), layout=SAG_LAYOUT_BSND if bsnd else SAG_LAYOUT_TND, s1_max=x.shape[1] if bsnd else 0)


def paged_append(k, v, k_cache, v_cache, page_table, kv_lens, cu_seqlens_q=None, workspace=None, stream=None, check=False,
                 desc=None):
    """Writes the new tokens' k, v [.., n2, d] (TND or 4-D BSND) into the caches
    [pages, page_size, n2, d]: token i of a sequence with q new ones goes to
    position kv_lens - q + i, in page page_table[sequence, position //
    page_size].  page_table [batch, width] and kv_lens [batch] are int32 tensors
    on the device (the lengths include the new tokens).  Returns the caches.  No
    two tokens may go to the same place: it would hold parts of both.

    ``desc`` (make_paged_desc) replaces cu_seqlens_q; ``check`` reads the device
    status back (a page or length out of range)."""
    lib = _lib_neighbours()
    if not k.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    if desc is None:
        desc = make_paged_desc(cu_seqlens_q, k.shape[-2], k.shape[-2], k.shape[-1], 1.0, k_cache.shape[0], k_cache.shape[1],
                               page_table.shape[1], **_paged_layout(k))

    def fill(io, device, dtype):
        shape = desc._shapes[1]
        _check_rows("k", k, shape, dtype)
        _check("v", v, device, k.shape, dtype)
        io.key, io.value = k.data_ptr(), v.data_ptr()
        strides = {}
        if not (k.is_contiguous() and v.is_contiguous()):
            strides = dict(k_stride=_row_stride("k", k, *shape[-2:]), v_stride=_row_stride("v", v, *shape[-2:]))
        return (k_cache, v_cache), strides

    return _paged(lib.paged_append, paged_append_workspace_size, k, desc, k_cache, v_cache, page_table, kv_lens, workspace, stream,
                  check, fill)


def paged_forward(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens_q=None, scale=None, left=-1, right=0, out=None,
                  workspace=None, stream=None, check=False, desc=None):
    """Attention of the new tokens' q [.., n1, d] (TND or 4-D BSND) to a paged
    cache (see ``paged_append``), which holds their own keys and values already:
    returns (attention_out [.., n1, d], softmax_lse [.., n1] in fp32).

    Causal by default, or within a window as in ``window_forward``; ``desc``
    (make_paged_desc) replaces cu_seqlens_q, scale, left and right.  The page
    table and the lengths are read on the device, so a captured call may be
    replayed as sequences grow.  How few tokens' loops are split is planned for
    the whole width of the table, or for a descriptor's ``kv_expected``, where
    tables are much wider than sequences are long."""
    lib = _lib_neighbours()
    if desc is not None and out is None and stream is None and not check:
        done = _usual_paged(lib.paged_attn_fwd, q, k_cache, v_cache, page_table, kv_lens, workspace, desc)
        if done is not None:
            return done
    if not q.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    if desc is None:
        desc = make_paged_desc(cu_seqlens_q, q.shape[-2], k_cache.shape[-2], q.shape[-1], scale, k_cache.shape[0],
                               k_cache.shape[1], page_table.shape[1], left, right, **_paged_layout(q))

    def fill(io, device, dtype):
        shape = desc._shapes[0]
        if q.dtype is not dtype or q.shape != shape:
            _check_rows("q", q, shape, dtype)
        io.query = q.data_ptr()
        outs = _attention_out(q, out)(io, device, dtype)
        return outs, {} if q.is_contiguous() else dict(q_stride=_row_stride("q", q, *shape[-2:]))

    return _paged(lib.paged_attn_fwd, paged_fwd_workspace_size, q, desc, k_cache, v_cache, page_table, kv_lens, workspace, stream,
                  check, fill)


# ---------------------------------------- norms of queries and keys, rotated
def make_norm_rotary_desc(rotary: Rotary, cu_seqlens, n1, n2, d, eps=1e-6, weight_offset=0.0, dtype=SAG_BF16,
                          layout=SAG_LAYOUT_TND, s_max=0) -> SnrDesc:
    """Descriptor of norms with rotation (n2 = 0: no key); keeps the host arrays
    alive.  The tensor calls take strides and the weights' type from the tensors."""
    base = make_rotary_desc(rotary, cu_seqlens, n1, n2, d, dtype, layout, s_max)
    desc = SnrDesc(rotary=base, eps=float(eps), weight_offset=float(weight_offset), weight_fp32=0, reserved_=0)
    desc._keep = base._keep
    return _derive(desc, dense=True)


def norm_rotary_fwd_workspace_size(desc: SnrDesc) -> int:
    """Phase 1 of the forward: validate and return the workspace size in bytes (0 for small batches)."""
    return _phase1("norm_rotary_fwd_workspace_size", desc)


def norm_rotary_grad_workspace_size(desc: SnrDesc) -> int:
    """Phase 1 of the gradient: validate and return the workspace size in bytes."""
    return _phase1("norm_rotary_grad_workspace_size", desc)


def _norm_rotary(entry, size, q, k, dq, dk, rotary, q_weight, k_weight, eps, weight_offset, cu_seqlens, positions, out, workspace,
                 stream, desc):
    """Both directions: with dq (and dk) the gradient."""
    if not q.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    shape = q.shape
    n1, d = shape[-2:]
    n2 = k.shape[-2] if k is not None else 0
    if desc is None:
        bsnd = q.dim() == 4
        desc = make_norm_rotary_desc(rotary, cu_seqlens, n1, n2, d, eps, weight_offset, _sag_dtype(q),
                                     SAG_LAYOUT_BSND if bsnd else SAG_LAYOUT_TND, shape[1] if bsnd else 0)
    else:
        desc = _given(desc)
    qs, ks = desc._shapes
    dtype, device, grad = desc._dtype, q.get_device(), dq is not None
    if q.dtype is not dtype or shape != qs:
        _check_rows("q", q, qs, dtype)
        lead = shape[:-2]
        ks = lead + ks[-2:]
    else:
        lead = qs[:-2]
    dense = desc._dense and q.is_contiguous()
    if k is not None:
        if k.dtype is not dtype or k.shape != ks or k.get_device() != device:
            _check("k", k, device, ks, dtype)
        dense = dense and k.is_contiguous()
    elif ks[-2]:
        raise ValueError("the descriptor has a key")
    if not n2:
        k_weight = None
    w = q_weight if q_weight is not None else k_weight
    wtype, fp32 = dtype, 0
    if w is not None and w.dtype is _torch.float32:
        wtype, fp32 = w.dtype, 1
    wq = wk = pos = None
    if q_weight is not None:
        wq = _dense("q_weight", q_weight, device, (d,), wtype)
    if k_weight is not None:
        wk = _dense("k_weight", k_weight, device, (d,), wtype)
    if positions is not None:
        pos = _dense("positions", positions, device, lead, _torch.int32)
    if grad:
        _check("dq", dq, device, shape, dtype)
        dense = dense and dq.is_contiguous()
        if n2:
            _check("dk", dk, device, ks, dtype)
            dense = dense and dk.is_contiguous()

    def call(handle):
        gq = gk = None
        if out is None:
            qo, ko = _new(q), _new(k) if k is not None else None
            if grad:
                gq = _torch.empty(d, dtype=_torch.float32, device=q.device) if wq else None
                gk = _torch.empty(d, dtype=_torch.float32, device=q.device) if wk else None
        else:
            given = tuple(out) if isinstance(out, (tuple, list)) else (out,)
            if grad and k is None:
                given = given[:1] + (None,) + given[1:]
            given += (None,) * ((4 if grad else 2) - len(given))
            qo, ko = given[:2]
            _check("out", qo, device, shape, dtype)
            if k is not None:
                _check("out", ko, device, ks, dtype)
            if grad:
                gq, gk = given[2:]
        use = desc
        if not dense or out is not None:
            use = _with(desc, weight_fp32=fp32, q_stride=_row_stride("q", q, n1, d), q_out_stride=_row_stride("out", qo, n1, d),
                        k_stride=_row_stride("k", k, n2, d) if n2 else 0,
                        k_out_stride=_row_stride("out", ko, n2, d) if n2 else 0,
                        q_grad_stride=_row_stride("dq", dq, n1, d) if grad else 0,
                        k_grad_stride=_row_stride("dk", dk, n2, d) if grad and n2 else 0)
        elif fp32 != desc.weight_fp32:
            use = _with(desc, weight_fp32=fp32)
        kp, kop = (k.data_ptr(), ko.data_ptr()) if n2 else (None, None)
        if grad:
            io = SnrIo(q.data_ptr(), kp, wq, wk, pos, None, None, dq.data_ptr(), dk.data_ptr() if n2 else None, qo.data_ptr(), kop,
                       _dense("dq_weight", gq, device, (d,), _torch.float32) if gq is not None else None,
                       _dense("dk_weight", gk, device, (d,), _torch.float32) if gk is not None else None)
        else:
            io = SnrIo(q.data_ptr(), kp, wq, wk, pos, qo.data_ptr(), kop)
        ws, need = None, 0
        if grad or desc.batch > 64:
            need = _size_of(desc, size)
            ws = _scratch(workspace, need, q.device)
        st = entry(use, io, ws.data_ptr() if need else None, need, handle)
        if st != SAG_OK:
            raise SagError(st, entry.__name__)
        if grad:
            return (qo, ko, gq, gk) if k is not None else (qo, gq)
        return (qo, ko) if k is not None else qo

    return _launch(device, stream, call)


def _usual_norm(entry, q, k, q_weight, k_weight, positions, desc):
    """As ``_usual_forward``: queries and keys, each with a weight of its type, and few sequences."""
    if not desc._dense or desc.batch > 64 or desc.weight_fp32 or not _unchanged(desc):
        return None
    qs, ks = desc._shapes
    dtype, device, d = desc._dtype, q.get_device(), ks[-1:]
    if not (q.dtype is dtype and k.dtype is dtype and q_weight.dtype is dtype and k_weight.dtype is dtype and q.shape == qs
            and k.shape == ks and q_weight.shape == d and k_weight.shape == d and q.is_contiguous() and k.is_contiguous()
            and q_weight.is_contiguous() and k_weight.is_contiguous() and device >= 0 and k.get_device() == device
            and q_weight.get_device() == device and k_weight.get_device() == device
            and _torch._C._cuda_getDevice() == device):
        return None
    pos = None
    if positions is not None:
        if positions.dtype is not _torch.int32 or positions.shape != qs[:-2] or not positions.is_contiguous() \
                or positions.get_device() != device:
            return None
        pos = positions.data_ptr()
    qo, ko = _torch.empty_like(q), _torch.empty_like(k)
    io = SnrIo(q.data_ptr(), k.data_ptr(), q_weight.data_ptr(), k_weight.data_ptr(), pos, qo.data_ptr(), ko.data_ptr())
    st = entry(desc, io, None, 0, _torch._C._cuda_getCurrentRawStream(device))
    if st != SAG_OK:
        raise SagError(st, entry.__name__)
    return qo, ko


def norm_rotary_forward(q, k, rotary, q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, cu_seqlens=None, positions=None,
                        out=None, workspace=None, stream=None, desc=None):
    """Each head of q [.., n1, d] and k [.., n2, d] (or None) over its root mean
    square, times ``q_weight`` / ``k_weight`` [d] (fp32 or the tensors' type, plus
    ``weight_offset``; None: no weight), then rotated: returns (q, k), or q alone.

    The other arguments as in ``rotary_forward``; ``desc``
    (make_norm_rotary_desc) replaces rotary, cu_seqlens, eps and weight_offset."""
    entry = _lib_neighbours().norm_rotary_fwd
    if desc is not None and out is None and stream is None and k is not None and q_weight is not None and k_weight is not None:
        done = _usual_norm(entry, q, k, q_weight, k_weight, positions, desc)
        if done is not None:
            return done
    return _norm_rotary(entry, norm_rotary_fwd_workspace_size, q, k, None, None, rotary, q_weight,
                        k_weight, eps, weight_offset, cu_seqlens, positions, out, workspace, stream, desc)


def norm_rotary_backward(q, k, dq, dk, rotary, q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, cu_seqlens=None,
                         positions=None, out=None, workspace=None, stream=None, desc=None):
    """Gradient of ``norm_rotary_forward`` from its inputs q, k and the gradients
    dq, dk of its outputs: returns (q's, k's, q_weight's, k_weight's), the
    weights' in fp32 (None without a weight); without k (q's, q_weight's).
    ``out`` takes the same tuple; a weight's gradient left out of it is not computed."""
    if dq is None or (dk is None) != (k is None):
        raise ValueError("dq and, with k, dk are needed")
    return _norm_rotary(_lib_neighbours().norm_rotary_grad, norm_rotary_grad_workspace_size, q, k, dq, dk, rotary, q_weight, k_weight,
                        eps, weight_offset, cu_seqlens, positions, out, workspace, stream, desc)


# phase 1 of calls that keep its result with their descriptor
_SIZES = (cross_fwd_workspace_size, cross_grad_workspace_size, window_fwd_workspace_size, window_grad_workspace_size,
          paged_fwd_workspace_size, paged_append_workspace_size, norm_rotary_fwd_workspace_size, norm_rotary_grad_workspace_size)
