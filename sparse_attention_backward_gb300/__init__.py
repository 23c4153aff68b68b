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
(``cross_forward`` / ``cross_backward``).
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
                                    ("cross_attn", ScaDesc, ScaIo, ("fwd", "grad"))):
        for n in names:
            getattr(lib, f"{prefix}_{n}").argtypes = [ctypes.POINTER(desc), ctypes.POINTER(io), vp, sz, vp]
    lib.rotary_workspace_size.argtypes = [ctypes.POINTER(SrtDesc), psz]
    lib.cross_attn_fwd_workspace_size.argtypes = [ctypes.POINTER(ScaDesc), psz]
    lib.cross_attn_grad_workspace_size.argtypes = [ctypes.POINTER(ScaDesc), psz]
    for n in EXPORTED_NEIGHBOURS:
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
    _check(name, t, device, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _new(like):
    """A dense tensor of the same shape, type and device."""
    return _torch.empty_like(like, memory_format=_torch.contiguous_format)


def _rows_of(desc, cu, s_max):
    if desc.layout == SAG_LAYOUT_BSND:
        return (desc.batch, s_max)
    return (cu[desc.batch] if desc.batch >= 0 else 0,)


def _derive(desc, dense=False):
    """What calls with the descriptor go by: the tensors' shapes and type.  Strides come from the tensors, so the
    descriptor serves dense tensors as it is only while its own are 0."""
    if isinstance(desc, SrtDesc):
        lead = _rows_of(desc, desc.cu_seqlens, desc.s_max)
        desc._shapes = (lead + (desc.n1, desc.d), lead + (desc.n2, desc.d))
    else:
        desc._shapes = (_rows_of(desc, desc.cu_seqlens_q, desc.s1_max) + (desc.n1, desc.d),
                        _rows_of(desc, desc.cu_seqlens_kv, desc.s2_max) + (desc.n2, desc.d))
        for size in (cross_fwd_workspace_size, cross_grad_workspace_size):
            desc.__dict__.pop(size, None)
    desc._dtype = _torch_dtype(desc)
    desc._dense = dense
    desc._bytes = bytes(desc)
    return desc


def _given(desc):
    """A kept descriptor, brought up to date if fields were set since."""
    return desc if bytes(desc) == desc._bytes else _derive(desc)


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
        ws, need = workspace, 0
        if use.batch > 64:          # smaller tables travel with the launch
            need = rotary_workspace_size(use)
            if ws is None or ws.numel() < need:
                ws = _torch.empty(need, dtype=_torch.uint8, device=q.device)
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


def _cross(entry, size, q, k, v, cu_seqlens_q, cu_seqlens_kv, scale, key_mask, workspace, stream, check, desc, tensors):
    """Shared by the two directions: ``tensors(io, device, dtype)`` fills in
    the remaining sca_io pointers and gives the outputs."""
    if not q.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    q_shape, k_shape = q.shape, k.shape
    n1, d = q_shape[-2:]
    n2 = k_shape[-2]
    if desc is None:
        bsnd = q.dim() == 4
        if bsnd and k.dim() != 4:
            raise ValueError("BSND needs 4-D query and key tensors")
        desc = make_cross_desc(cu_seqlens_q, cu_seqlens_kv, n1, n2, d, scale, _sag_dtype(q),
                               SAG_LAYOUT_BSND if bsnd else SAG_LAYOUT_TND, q_shape[1] if bsnd else 0,
                               k_shape[1] if bsnd else 0)
    else:
        desc = _given(desc)
    dtype, device = desc._dtype, q.get_device()
    qs, ks = desc._shapes
    if q.dtype is not dtype or q_shape != qs:
        _check_rows("q", q, qs, dtype)
    if k.dtype is not dtype or k_shape != ks:
        _check_rows("k", k, ks, dtype)
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
        need = desc.__dict__.get(size)
        if need is None:
            need = desc.__dict__[size] = size(desc)
        ws = workspace
        if ws is None or ws.numel() < need:
            ws = _torch.empty(need, dtype=_torch.uint8, device=q.device)
        st = entry(use, io, ws.data_ptr(), need, handle)
        if st == SAG_OK and check:
            st = cross_query_error(ws.data_ptr(), handle)
        if st != SAG_OK:
            raise SagError(st, entry.__name__)
        return outs

    return _launch(device, stream, call)


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
    def tensors(io, device, dtype):
        if out is None:
            o, lse = _new(q), _torch.empty(q.shape[:-1], dtype=_torch.float32, device=q.device)
            io.attention_out, io.softmax_lse = o.data_ptr(), lse.data_ptr()
        else:
            o, lse = out
            io.attention_out = _dense("attention_out", o, device, q.shape, dtype)
            io.softmax_lse = _dense("softmax_lse", lse, device, q.shape[:-1], _torch.float32)
        return o, lse

    return _cross(_lib_neighbours().cross_attn_fwd, cross_fwd_workspace_size, q, k, v, cu_seqlens_q, cu_seqlens_kv, scale, key_mask,
                  workspace, stream, check, desc, tensors)


def cross_backward(q, k, v, o, dy, lse, cu_seqlens_q=None, cu_seqlens_kv=None, scale=None, key_mask=None, out=None,
                   workspace=None, stream=None, check=False, desc=None):
    """Gradient of ``cross_forward``: returns (dq, dk, dv), from the forward's o
    and lse and the gradient dy of o; the other arguments as there."""
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

    return _cross(_lib_neighbours().cross_attn_grad, cross_grad_workspace_size, q, k, v, cu_seqlens_q, cu_seqlens_kv, scale, key_mask,
                  workspace, stream, check, desc, tensors)
