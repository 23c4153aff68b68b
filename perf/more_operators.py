"""Cases that measure four operators that a decoder layer runs around the selected attention, in training and in serving:

* norms of queries and keys with the rotation in the same pass (``norm_rotary_forward`` / ``norm_rotary_backward``), for each
  head x of d columns with its learned weight w (plus an offset), r = 1 / sqrt(mean x^2 + eps) and the rotation R of its position:
      y = R (x r w),    g = w R^T dy,  dx = r (g - x r^2 mean(g x)),  dw = sum of (R^T dy) x r over tokens and heads;
* attention within a window (``window_forward`` / ``window_backward``): query i of a sequence stands at key position
  p = i + (keys - queries) and attends to the keys p - left .. p + right (-1: no limit) that are there,
      S = scale Q K^T,  lse = ln sum exp S,  O = exp(S - lse) V,
      dP = dY V^T,  dS = P (dP - rowsum(dY O)),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dY;
  a row with nothing to attend to has O = 0 and lse = -inf and gives no gradient;
* the same forward for a chunk of new tokens over keys and values in pages (``paged_forward``), with the page table and the
  lengths in device memory;
* the new tokens' keys and values into their places of such a cache (``paged_append``).

``run`` computes them with elementary torch operations in 32 bits, or, with ``own`` set, by the calls that a user makes of the
framework.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token for each of 16 running sequences at far positions: latency
        dict(name="norm_token", op="norm", dtype="bf16", batch=16, s=1, ragged=False, padded=False, n1=64, n2=4, d=128, rot=128,
             offset=0, style="half", far=True, weight="own", plus=0.0, grad=False),
        # the long training context (32768 tokens, 64 and 4 heads)
        dict(name="norm_long_context", op="norm", dtype="bf16", batch=1, s=32768, ragged=False, padded=False, n1=64, n2=4, d=128,
             rot=128, offset=0, style="half", far=False, weight="own", plus=0.0, grad=False),
        # gradients of a padded batch of 192-wide heads, the last 64 columns rotated in neighbouring pairs, 32-bit weights around 1
        dict(name="norm_grad_padded_f16", op="norm", dtype="f16", batch=4, s=4095, ragged=True, padded=True, n1=24, n2=8, d=192, rot=64,
             offset=128, style="interleaved", far=False, weight="f32", plus=1.0, grad=True),
        # an ordinary packed batch of short sequences, 64-wide heads, each token seeing 64 before it
        dict(name="window_packed_f16", op="window", dtype="f16", batch=5, s1=421, s2=421, ragged=True, padded=False, n1=16, n2=16, d=64,
             left=63, right=0, holes=False, grad=False),
        # the local branch at the long training context: a window of 512
        dict(name="window_long_context", op="window", dtype="bf16", batch=1, s1=32768, s2=32768, ragged=False, padded=False, n1=64, n2=4,
             d=128, left=511, right=0, holes=False, grad=False),
        # gradients of a padded batch with holes in its keys and a window to both sides, groups of three heads
        dict(name="window_grad_padded_f16", op="window", dtype="f16", batch=4, s1=1500, s2=1500, ragged=True, padded=True, n1=24, n2=8,
             d=128, left=200, right=55, holes=True, grad=True),
        # the largest gradient: causal attention of long sequences
        dict(name="causal_grad_large", op="window", dtype="bf16", batch=2, s1=8192, s2=8192, ragged=False, padded=False, n1=32, n2=8,
             d=128, left=-1, right=0, holes=False, grad=True),
        # decoding: one token for each of 64 sequences over ragged caches
        dict(name="paged_decode", op="paged", dtype="bf16", batch=64, s1=1, s2=4096, ragged=True, padded=False, n1=64, n2=4, d=128,
             left=-1, right=0, page=64),
        # one token of one sequence at the end of a very long cache of small pages
        dict(name="paged_token_long_f16", op="paged", dtype="f16", batch=1, s1=1, s2=131072, ragged=False, padded=False, n1=32, n2=4,
             d=128, left=-1, right=0, page=16),
        # chunks of new tokens behind long caches
        dict(name="paged_chunk", op="paged", dtype="bf16", batch=4, s1=2048, s2=16384, ragged=True, padded=False, n1=32, n2=8, d=128,
             left=-1, right=0, page=32),
        # the tokens of one decoding step
        dict(name="append_decode", op="append", dtype="bf16", batch=64, s1=1, s2=4096, ragged=True, padded=False, n1=64, n2=4, d=128,
             page=64),
        # chunks of new tokens, padded to one length
        dict(name="append_chunk_padded_f16", op="append", dtype="f16", batch=8, s1=4095, s2=8190, ragged=True, padded=True, n1=32, n2=8,
             d=128, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    padded, ragged = rng.random() < 0.4, rng.random() < 0.7
    dtype = rng.choice(["bf16", "f16"])
    op = rng.choice(["norm", "window", "window", "paged", "append"])
    if op == "norm":
        d = rng.choice([64, 80, 128, 192, 256])
        rot = rng.choice([r for r in (16, 32, 64, 80, 128, 192, 256) if r <= d])
        n2 = rng.choice([1, 2, 4, 8])
        n1 = n2 * rng.choice([1, 2, 3, 5, 8])
        batch, grad = _log(rng, 1, 64), rng.random() < 0.5
        # no more elements than the long context has; a gradient moves half as much again for each
        s = max(1, min(_log(rng, 1, 32768), 32768 * 68 * 128 * 2 // (batch * (n1 + n2) * d * (3 if grad else 2))))
        return dict(op=op, dtype=dtype, batch=batch, s=s, ragged=ragged, padded=padded, n1=n1, n2=n2, d=d, rot=rot,
                    offset=rng.choice([0, d - rot]), style=rng.choice(["half", "interleaved"]), far=rng.random() < 0.3,
                    weight=rng.choice(["own", "f32"]), plus=rng.choice([0.0, 1.0]), grad=grad)
    d = rng.choice([64, 128])
    n2 = rng.choice([1, 2, 4, 8, 16])
    n1 = n2 * rng.choice([1, 1, 2, 3, 4, 5, 8])
    if op == "window":
        grad, batch = rng.random() < 0.5, _log(rng, 1, 16)
        s1 = max(1, min(_log(rng, 1, 8192), 2 * 8192 * 32 * 128 // (batch * n1 * d)))
        # a sequence attends to itself, or its last tokens to all of it (or to less than its own length)
        s2 = s1 if rng.random() < 0.6 else max(1, min(_log(rng, 1, 16384), 2 * 8192 * 8192 * 32 * 128 // (2 * batch * s1 * n1 * d)))
        left = -1 if rng.random() < 0.4 else _log(rng, 1, 2048) - 1
        right = rng.choice([0, 0, 0, -1, _log(rng, 1, 512)])
        if right == -1 and left == -1:
            left = 255
        return dict(op=op, dtype=dtype, batch=batch, s1=s1, s2=s2, ragged=ragged, padded=padded, n1=n1, n2=n2, d=d, left=left,
                    right=right, holes=rng.random() < 0.3, grad=grad)
    page, batch = rng.choice([16, 32, 48, 64, 128, 256]), _log(rng, 1, 64)
    s1 = 1 if rng.random() < 0.4 else _log(rng, 1, 4096)
    s2 = max(s1, _log(rng, 1, 65536))
    # no more cache than the decoding step's, no more pairs than the chunks'
    s2 = max(1, min(s2, 64 * 4096 * 4 * 128 // (batch * n2 * d)))
    s1 = max(1, min(s1, s2, 4 * 2048 * 16384 * 32 * 128 // (batch * s2 * n1 * d)))
    case = dict(op=op, dtype=dtype, batch=batch, s1=s1, s2=s2, ragged=ragged, padded=padded, n1=n1, n2=n2, d=d, page=page)
    if op == "paged":
        case.update(left=-1 if rng.random() < 0.6 else _log(rng, 1, 4096) - 1, right=0)
    return case


# ------------------------------------------------------------- what is in hand
def _lengths(batch, s, ragged, step):
    """Lengths of the sequences, the longest of them s."""
    return [s - (b * step) % (s // 2 + 1) if ragged else s for b in range(batch)]


def _prefix(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _both(case):
    """Lengths of the queries (new tokens) and of the keys of each sequence."""
    l1 = _lengths(case["batch"], case["s1"], case["ragged"], 97)
    if case["op"] == "window":
        return l1, l1 if case["s1"] == case["s2"] else _lengths(case["batch"], case["s2"], case["ragged"], 389)
    return l1, [max(a, b) for a, b in zip(l1, _lengths(case["batch"], case["s2"], case["ragged"], 389))]


def _rows(lengths, s, padded):
    """(row of each valid token in the tensor, its place in a [batch, s] grid, rows of the tensor)."""
    row, place, at = [], [], 0
    for b, n in enumerate(lengths):
        first = b * s if padded else at
        row.append(torch.arange(first, first + n))
        place.append(torch.arange(b * s, b * s + n))
        at += n
    return torch.cat(row).cuda(), torch.cat(place).cuda(), len(lengths) * s if padded else at


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        return _prepare_norm(case, gen, dtype)
    l1, l2 = _both(case)
    row1, place1, r1 = _rows(l1, case["s1"], case["padded"])
    lead1 = (case["batch"], case["s1"]) if case["padded"] else (r1,)
    state = dict(case=case, cu1=_prefix(l1), row1=row1, place1=place1, lead1=lead1, scale=case["d"] ** -0.5,
                 l1=torch.tensor(l1, device="cuda", dtype=torch.int32), l2=torch.tensor(l2, device="cuda", dtype=torch.int32))
    n1, n2, d = case["n1"], case["n2"], case["d"]
    if case["op"] == "window":
        row2, place2, r2 = _rows(l2, case["s2"], case["padded"])
        lead2 = (case["batch"], case["s2"]) if case["padded"] else (r2,)
        state.update(cu2=_prefix(l2), row2=row2, place2=place2, lead2=lead2, q=_normal(gen, lead1 + (n1, d), dtype),
                     k=_normal(gen, lead2 + (n2, d), dtype), v=_normal(gen, lead2 + (n2, d), dtype), mask=None)
        if case["holes"]:  # an eighth of the keys are masked out
            state["mask"] = torch.rand(lead2, generator=gen, device="cuda") >= 0.125
        if case["grad"]:
            state["dy"] = _normal(gen, lead1 + (n1, d), dtype)
            state["o"], state["lse"] = _attention_plain(state)
    else:
        # pages in the order in which a server that has run for a while hands them out, some of them free
        width = -(-max(l2) // case["page"])
        used = case["batch"] * width
        pages = used + used // 8 + 1
        table = torch.randperm(pages, generator=gen, device="cuda")[:used].reshape(case["batch"], width).to(torch.int32)
        cache = (pages, case["page"], n2, d)
        state.update(table=table, k_cache=_normal(gen, cache, dtype), v_cache=_normal(gen, cache, dtype), mask=None)
        if case["op"] == "paged":
            state["q"] = _normal(gen, lead1 + (n1, d), dtype)
        else:
            state["k"], state["v"] = _normal(gen, lead1 + (n2, d), dtype), _normal(gen, lead1 + (n2, d), dtype)
    if own:
        state["kept"] = _keep(case, state)
    return state


def _prepare_norm(case, gen, dtype):
    lengths = _lengths(case["batch"], case["s"], case["ragged"], 211)
    row, place, rows = _rows(lengths, case["s"], case["padded"])
    lead = (case["batch"], case["s"]) if case["padded"] else (rows,)
    n1, n2, d = case["n1"], case["n2"], case["d"]
    state = dict(case=case, cu=_prefix(lengths), row=row, place=place, q=_normal(gen, lead + (n1, d), dtype),
                 k=_normal(gen, lead + (n2, d), dtype), positions=None)
    state["wq"], state["wk"] = (((1.0 - case["plus"]) + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(
        dtype if case["weight"] == "own" else torch.float32) for _ in range(2))
    if case["far"]:  # each row's own position in a long context
        state["positions"] = torch.randint(0, 131072, lead, generator=gen, device="cuda", dtype=torch.int32)
    state["frequencies"] = torch.tensor([500000.0 ** (-2 * i / case["rot"]) for i in range(case["rot"] // 2)], dtype=torch.float64,
                                        device="cuda")
    if case["grad"]:
        state["dq"], state["dk"] = _normal(gen, lead + (n1, d), dtype), _normal(gen, lead + (n2, d), dtype)
    if own:
        state["kept"] = _keep_norm(case, state)
    return state


# --------------------------------------------------------- the framework's calls
def _sag_type(case):
    import sparse_attention_backward_gb300 as sab
    return sab.SAG_FP16 if case["dtype"] == "f16" else sab.SAG_BF16


def _layout(case):
    import sparse_attention_backward_gb300 as sab
    return sab.SAG_LAYOUT_BSND if case["padded"] else sab.SAG_LAYOUT_TND


def _bytes(n):
    return torch.empty(max(1, n), dtype=torch.uint8, device="cuda")


def _keep_norm(case, state):
    """The frequencies, the descriptor and the workspace of the problem."""
    import sparse_attention_backward_gb300 as sab
    rotary = sab.Rotary(case["rot"], base=500000.0, style=case["style"], offset=case["offset"])
    desc = sab.make_norm_rotary_desc(rotary, state["cu"], case["n1"], case["n2"], case["d"], eps=EPS, weight_offset=case["plus"],
                                     dtype=_sag_type(case), layout=_layout(case), s_max=case["s"] if case["padded"] else 0)
    need = sab.norm_rotary_grad_workspace_size(desc) if case["grad"] else sab.norm_rotary_fwd_workspace_size(desc)
    return dict(desc=desc, workspace=_bytes(need))


def _keep(case, state):
    """The descriptor and the workspace of the problem."""
    import sparse_attention_backward_gb300 as sab
    s1 = case["s1"] if case["padded"] else 0
    if case["op"] == "window":
        desc = sab.make_window_desc(state["cu1"], state["cu2"], case["n1"], case["n2"], case["d"], state["scale"], left=case["left"],
                                    right=case["right"], dtype=_sag_type(case), layout=_layout(case), s1_max=s1,
                                    s2_max=case["s2"] if case["padded"] else 0)
        need = sab.window_grad_workspace_size(desc) if case["grad"] else sab.window_fwd_workspace_size(desc)
        return dict(desc=desc, workspace=_bytes(need))
    desc = sab.make_paged_desc(state["cu1"], case["n1"], case["n2"], case["d"], state["scale"], state["k_cache"].shape[0], case["page"],
                               state["table"].shape[1], left=case.get("left", -1), right=case.get("right", 0), dtype=_sag_type(case),
                               layout=_layout(case), s1_max=s1)
    need = sab.paged_fwd_workspace_size(desc) if case["op"] == "paged" else sab.paged_append_workspace_size(desc)
    return dict(desc=desc, workspace=_bytes(need))


def _own(state):
    import sparse_attention_backward_gb300 as sab
    case, s, kept = state["case"], state, state["kept"]
    if case["op"] == "norm":
        if case["grad"]:
            return sab.norm_rotary_backward(s["q"], s["k"], s["dq"], s["dk"], None, s["wq"], s["wk"], positions=s["positions"],
                                            workspace=kept["workspace"], desc=kept["desc"])
        return sab.norm_rotary_forward(s["q"], s["k"], None, s["wq"], s["wk"], positions=s["positions"], workspace=kept["workspace"],
                                       desc=kept["desc"])
    if case["op"] == "paged":
        return sab.paged_forward(s["q"], s["k_cache"], s["v_cache"], s["table"], s["l2"], workspace=kept["workspace"], desc=kept["desc"])
    if case["op"] == "append":
        return sab.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["l2"], workspace=kept["workspace"],
                                desc=kept["desc"])
    if case["grad"]:
        return sab.window_backward(s["q"], s["k"], s["v"], s["o"], s["dy"], s["lse"], key_mask=s["mask"], workspace=kept["workspace"],
                                   desc=kept["desc"])
    return sab.window_forward(s["q"], s["k"], s["v"], key_mask=s["mask"], workspace=kept["workspace"], desc=kept["desc"])


# ------------------------------------------------------------- the plain forms
def _sines(state):
    case = state["case"]
    pos = state["place"] % case["s"] if state["positions"] is None else state["positions"].reshape(-1)[state["row"]]
    angle = pos.double()[:, None] * state["frequencies"]  # 64 bits: far positions make many turns
    return angle.sin().float()[:, None], angle.cos().float()[:, None]


def _turn(case, x, sin, cos):
    r, off = case["rot"], case["offset"]
    z = x[..., off:off + r]
    a, b = (z[..., :r // 2], z[..., r // 2:]) if case["style"] == "half" else (z[..., 0::2], z[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    z = torch.cat((a, b), -1) if case["style"] == "half" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((x[..., :off], z, x[..., off + r:]), -1)


def _spread(state, y, like):
    """Rows of the valid tokens as a tensor like `like`, zeros in its padding."""
    return torch.zeros_like(like).reshape(-1, *like.shape[-2:]).index_copy(0, state["row"], y.to(like.dtype)).reshape(like.shape)


def _norm_plain(state):
    case = state["case"]
    sin, cos = _sines(state)
    answers, weights = [], []
    for x, w, dy in ((state["q"], state["wq"], state.get("dq")), (state["k"], state["wk"], state.get("dk"))):
        z = x.reshape(-1, *x.shape[-2:])[state["row"]].float()
        r = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
        w = w.float() + case["plus"]
        if not case["grad"]:
            answers.append(_spread(state, _turn(case, z * r * w, sin, cos), x))
            continue
        dn = _turn(case, dy.reshape(-1, *x.shape[-2:])[state["row"]].float(), -sin, cos)
        g = dn * w
        answers.append(_spread(state, r * (g - z * (r * r * (g * z).mean(-1, keepdim=True))), x))
        weights.append((dn * z * r).sum((0, 1), dtype=torch.float64).float())  # 64 bits: a long sum
    return tuple(answers + weights)


def _grid(state, x, which):
    """Valid rows of x as [batch, heads, s, d] in 32 bits, zeros elsewhere."""
    case = state["case"]
    s, tail = case["s%d" % which], x.shape[-2:]
    out = torch.zeros((case["batch"] * s,) + tuple(tail), dtype=torch.float32, device=x.device)
    out[state["place%d" % which]] = x.reshape((-1,) + tuple(tail))[state["row%d" % which]].float()
    return out.reshape((case["batch"], s) + tuple(tail)).transpose(1, 2)


def _back(state, x, which, like):
    """[batch, heads, s, ...] as rows of the tensors' layout, zeros in its padding."""
    lead = state["lead%d" % which]
    x = x.transpose(1, 2)
    tail = x.shape[2:]
    out = torch.zeros((math.prod(lead),) + tail, dtype=like, device=x.device)
    out[state["row%d" % which]] = x.reshape((-1,) + tail)[state["place%d" % which]].to(like)
    return out.reshape(tuple(lead) + tail)


def _slots(state, width):
    """Row in the cache of each of `width` key positions of each sequence (any row where the sequence has none)."""
    page, table = state["case"]["page"], state["table"]
    at = torch.arange(width, device="cuda")
    return table[:, (at // page).clamp(max=table.shape[1] - 1)].long() * page + at % page


def _keys(state):
    """Keys and values [batch, n2, s2, d] in 32 bits, zeros where there are none, and which are there [batch, s2]."""
    case = state["case"]
    b, s2 = case["batch"], case["s2"]
    if case["op"] == "paged":
        s2 = state["table"].shape[1] * case["page"]
        there = torch.arange(s2, device="cuda") < state["l2"][:, None]
        slots = _slots(state, s2)
        k, v = (c.reshape(-1, *c.shape[-2:])[slots].float().transpose(1, 2) for c in (state["k_cache"], state["v_cache"]))
    else:
        there = torch.zeros(b * s2, dtype=torch.bool, device="cuda")
        there[state["place2"]] = True if state["mask"] is None else state["mask"].reshape(-1)[state["row2"]]
        there = there.reshape(b, s2)
        k, v = _grid(state, state["k"], 2), _grid(state, state["v"], 2)
    keep = there[:, None, :, None]
    return torch.where(keep, k, 0.0), torch.where(keep, v, 0.0), there


def _pieces(state, s2):
    """Query rows in pieces whose scores fit, each with the keys that any of its rows may see: (i0, i1, j0, j1)."""
    case = state["case"]
    l1, l2 = _both(case)
    shift = [b - a for a, b in zip(l1, l2)]
    left, right = case["left"], case["right"]
    i0 = 0
    while i0 < case["s1"]:
        # rows at a time: as many as the window is wide, within 2^28 scores
        rows = max(1, min(case["s1"] - i0, max(512, left if right >= 0 else 0), (1 << 28) // (case["batch"] * case["n1"] * s2)))
        i1 = i0 + rows
        j0 = 0 if left < 0 else min(max(0, min(shift) + i0 - left), s2)
        j1 = s2 if right < 0 else max(j0, min(s2, max(shift) + i1 + right))
        yield i0, i1, j0, j1
        i0 = i1


def _scores(state, q, k, there, piece):
    """Masked scores [batch, n2, G, rows, keys] of a piece, -inf where there is nothing to attend to."""
    case = state["case"]
    i0, i1, j0, j1 = piece
    b, n2, g, d = case["batch"], case["n2"], case["n1"] // case["n2"], case["d"]
    p = torch.arange(i0, i1, device="cuda") + (state["l2"] - state["l1"])[:, None]
    j = torch.arange(j0, j1, device="cuda")
    seen = there[:, None, j0:j1].expand(b, i1 - i0, j1 - j0)
    if case["left"] >= 0:
        seen = seen & (j >= p[..., None] - case["left"])
    if case["right"] >= 0:
        seen = seen & (j <= p[..., None] + case["right"])
    s = torch.matmul(q[:, :, i0:i1].reshape(b, n2, g * (i1 - i0), d), k[:, :, j0:j1].transpose(2, 3)).mul_(state["scale"])
    return s.reshape(b, n2, g, i1 - i0, j1 - j0).masked_fill_(~seen[:, None, None], -math.inf).reshape(b, n2, g * (i1 - i0), j1 - j0)


def _attention_plain(state):
    case = state["case"]
    b, n1, s1, d = case["batch"], case["n1"], case["s1"], case["d"]
    q = _grid(state, state["q"], 1)
    k, v, there = _keys(state)
    o, lse = torch.empty_like(q), torch.full((b, n1, s1), -math.inf, device="cuda")
    for piece in _pieces(state, k.shape[2]):
        i0, i1, j0, j1 = piece
        if j0 == j1:
            o[:, :, i0:i1] = 0.0
            continue
        s = _scores(state, q, k, there, piece)
        top = s.amax(-1, keepdim=True)
        p = s.sub_(torch.where(top.isinf(), 0.0, top)).exp_()
        total = p.sum(-1, keepdim=True)
        o[:, :, i0:i1] = (torch.matmul(p, v[:, :, j0:j1]) / torch.where(total > 0, total, 1.0)).reshape(b, n1, i1 - i0, d)
        lse[:, :, i0:i1] = (total.log() + top).reshape(b, n1, i1 - i0)
    return _back(state, o, 1, state["q"].dtype), _back(state, lse, 1, torch.float32)


def _attention_grad_plain(state):
    case = state["case"]
    b, n1, n2, d = case["batch"], case["n1"], case["n2"], case["d"]
    q, o, dy = (_grid(state, state[x], 1) for x in ("q", "o", "dy"))
    lse = _grid(state, state["lse"][..., None], 1)
    delta = (o * dy).sum(-1, keepdim=True)
    k, v, there = _keys(state)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for piece in _pieces(state, k.shape[2]):
        i0, i1, j0, j1 = piece
        if j0 == j1:
            continue
        part = lambda x: x[:, :, i0:i1].reshape(b, n2, -1, x.shape[-1])  # noqa: E731
        row = part(lse)
        p = _scores(state, q, k, there, piece).sub_(torch.where(row.isinf(), 0.0, row)).exp_()
        dv[:, :, j0:j1] += torch.matmul(p.transpose(2, 3), part(dy))
        ds = torch.matmul(part(dy), v[:, :, j0:j1].transpose(2, 3)).sub_(part(delta)).mul_(p).mul_(state["scale"])
        dq[:, :, i0:i1] = torch.matmul(ds, k[:, :, j0:j1]).reshape(b, n1, i1 - i0, d)
        dk[:, :, j0:j1] += torch.matmul(ds.transpose(2, 3), part(q))
    t = state["q"].dtype
    return _back(state, dq, 1, t), _back(state, dk, 2, t), _back(state, dv, 2, t)


def _append_plain(state):
    case = state["case"]
    b, s1 = torch.div(state["place1"], case["s1"], rounding_mode="floor"), state["place1"] % case["s1"]
    position = s1 + (state["l2"] - state["l1"])[b]
    slot = state["table"][b, position // case["page"]].long() * case["page"] + position % case["page"]
    for cache, new in ((state["k_cache"], state["k"]), (state["v_cache"], state["v"])):
        tail = new.shape[-2:]
        cache.view((-1,) + tuple(tail))[slot] = new.reshape((-1,) + tuple(tail))[state["row1"]]
    return state["k_cache"], state["v_cache"]


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "norm":
        return _norm_plain(state)
    if case["op"] == "append":
        return _append_plain(state)
    return _attention_grad_plain(state) if case.get("grad") else _attention_plain(state)


# --------------------------------------------------------------- the floor
def _pairs(case):
    """Pairs of a query and a key that it attends to, and keys that any query attends to."""
    pairs = keys = 0
    for a, b in zip(*_both(case)):
        p = torch.arange(a) + (b - a)
        lo = (p - case["left"]).clamp(min=0) if case["left"] >= 0 else torch.zeros_like(p)
        hi = (p + case["right"] + 1).clamp(max=b) if case["right"] >= 0 else torch.full_like(p, b)
        pairs += int((hi - lo).clamp(min=0).sum())
        keys += max(0, int(hi[-1]) - int(lo[0]))
    return pairs, keys


def work(case):
    n1, n2, d = case["n1"], case["n2"], case["d"]
    if case["op"] == "norm":
        tokens = sum(_lengths(case["batch"], case["s"], case["ragged"], 211))
        size = tokens * (n1 + n2)
        weights = 2 * d * (2 if case["weight"] == "own" else 4) + (8 * d if case["grad"] else 0)
        # an element: square, sum, two products (a gradient: two sums, four products more); a rotated pair: six
        return {"bytes": size * d * (6 if case["grad"] else 4) + (4 * tokens if case["far"] else 0) + weights,
                "flops": size * (d * (12 if case["grad"] else 4) + case["rot"] * 3)}
    l1, l2 = _both(case)
    t1 = sum(l1)
    if case["op"] == "append":
        return {"bytes": t1 * n2 * d * 8 + 4 * sum(-(-a // case["page"]) for a in l1) + 4 * case["batch"], "flops": 0}
    pairs, keys = _pairs(case)
    q, stat = t1 * n1 * d * 2, t1 * n1 * 4
    if case["op"] == "paged":
        return {"bytes": 2 * q + 2 * keys * n2 * d * 2 + stat + 4 * (-(-keys // case["page"]) + case["batch"]), "flops": 4 * pairs * n1 * d}
    pairs *= 0.875 if case["holes"] else 1.0
    kv, mask = sum(l2) * n2 * d * 2, sum(l2) if case["holes"] else 0
    if case["grad"]:  # q, o, dy, dq; k, v, dk, dv
        return {"bytes": int(4 * q + 4 * kv + stat + mask), "flops": int(10 * pairs * n1 * d)}
    return {"bytes": int(2 * q + 2 * kv + stat + mask), "flops": int(4 * pairs * n1 * d)}


# --------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, state)
    if case["op"] == "append":
        return _exact_append(case, state)
    if _pairs(case)[0] * case["n1"] * case["d"] * (10 if case.get("grad") else 4) > 6e12:
        return None
    return _exact_attention(case, state)


def _exact_norm(case, state):
    """Head by head as unit vectors times the weight, pairs of columns as complex numbers."""
    half, sign = case["rot"] // 2, -1.0 if case["grad"] else 1.0
    cols = torch.arange(case["rot"], device="cuda") + case["offset"]
    first, second = (cols[:half], cols[half:]) if case["style"] == "half" else (cols[0::2], cols[1::2])
    answers, weights = [], []
    for x, w, dy in ((state["q"], state["wq"], state.get("dq")), (state["k"], state["wk"], state.get("dk"))):
        out, dw = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), torch.zeros(case["d"], dtype=torch.float64, device="cuda")
        w = w.double() + case["plus"]
        for b, n in enumerate(_lengths(case["batch"], case["s"], case["ragged"], 211)):
            rows = (b, slice(0, n)) if case["padded"] else slice(state["cu"][b], state["cu"][b] + n)
            p = torch.arange(n, device="cuda") if state["positions"] is None else state["positions"][rows]
            phase = torch.polar(torch.ones((n, 1, half), dtype=torch.float64, device="cuda"),
                                sign * p.double().reshape(n, 1, 1) * state["frequencies"])
            z = x[rows].double()
            size = (z.square().sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
            unit = z / size
            y = dy[rows].double() if case["grad"] else unit * w
            turned = torch.complex(y[..., first], y[..., second]) * phase
            y[..., first], y[..., second] = turned.real, turned.imag
            if case["grad"]:
                dw += (y * unit).sum((0, 1))
                y = y * w
                y = (y - unit * (unit * y).sum(-1, keepdim=True) / case["d"]) / size
            out[rows] = y
        answers.append(out)
        weights.append(dw)
    return tuple(answers + (weights if case["grad"] else []))


def _exact_append(case, state):
    """Token by token of each sequence, page by page."""
    page, caches = case["page"], []
    for cache, new in ((state["k_cache"], state["k"]), (state["v_cache"], state["v"])):
        cache = cache.double()
        for b, (a, n) in enumerate(zip(*_both(case))):
            first, done = n - a, 0
            source = new[b, :a] if case["padded"] else new[state["cu1"][b]:state["cu1"][b] + a]
            while done < a:
                at = (first + done) % page
                take = min(a - done, page - at)
                cache[int(state["table"][b, (first + done) // page]), at:at + take] = source[done:done + take].double()
                done += take
        caches.append(cache)
    return tuple(caches)


def _exact_attention(case, state):
    """Sequence by sequence, head by head, a block of queries at a time, over the keys that are there."""
    n1, n2, d, scale, grad = case["n1"], case["n2"], case["d"], state["scale"], case.get("grad")
    new = lambda lead, *tail: torch.zeros(tuple(lead) + tail, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse, dq = new(state["lead1"], n1, d), new(state["lead1"], n1), new(state["lead1"], n1, d)
    if grad:
        dk, dv = new(state["lead2"], n2, d), new(state["lead2"], n2, d)
    for b, (a, n) in enumerate(zip(*_both(case))):
        rows = state["q"][b, :a] if case["padded"] else state["q"][state["cu1"][b]:state["cu1"][b] + a]
        if case["op"] == "paged":
            pages = state["table"][b].long()
            keys, values = (c[pages].reshape(-1, n2, d)[:n] for c in (state["k_cache"], state["v_cache"]))
            at = torch.arange(n, device="cuda")
        else:
            first = b * case["s2"] if case["padded"] else state["cu2"][b]
            at = torch.arange(first, first + n, device="cuda")
            keys, values = (state[x].reshape(-1, n2, d)[at] for x in ("k", "v"))
        own_key = torch.ones(n, dtype=torch.bool, device="cuda") if state["mask"] is None else state["mask"].reshape(-1)[at]
        head_rows = (lambda i, j: (b, slice(i, j))) if case["padded"] else (lambda i, j: (slice(state["cu1"][b] + i, state["cu1"][b] + j),))
        for i in range(0, a, 1024):
            j = min(a, i + 1024)
            p = torch.arange(i, j, device="cuda") + (n - a)
            lo = max(0, int(p[0]) - case["left"]) if case["left"] >= 0 else 0
            hi = max(lo, min(n, int(p[-1]) + case["right"] + 1)) if case["right"] >= 0 else n
            if lo >= hi:
                lse[head_rows(i, j)] = -math.inf
                continue
            c = torch.arange(lo, hi, device="cuda")
            seen = own_key[lo:hi].expand(j - i, hi - lo).clone()
            if case["left"] >= 0:
                seen &= c >= p[:, None] - case["left"]
            if case["right"] >= 0:
                seen &= c <= p[:, None] + case["right"]
            some = seen.any(1, keepdim=True)
            for h in range(n1):
                kv = h // (n1 // n2)
                q, k, v = rows[i:j, h].double(), keys[lo:hi, kv].double(), values[lo:hi, kv].double()
                k, v = torch.where(own_key[lo:hi, None], k, 0.0), torch.where(own_key[lo:hi, None], v, 0.0)
                s = (q @ k.T * scale).masked_fill(~seen, -math.inf)
                place = head_rows(i, j) + (h,)
                if not grad:
                    lse[place] = torch.logsumexp(s, 1)
                    o[place] = torch.where(some, torch.softmax(s, 1), 0.0) @ v
                    continue
                y, was = state["dy"][place].double(), state["o"][place].double()
                prob = torch.where(seen, (s - torch.where(some, state["lse"][place].double()[:, None], 0.0)).exp(), 0.0)
                ds = prob * (y @ v.T - (y * was).sum(1, keepdim=True)) * scale
                dq[place] = ds @ k
                dk.reshape(-1, n2, d)[at[lo:hi], kv] += ds.T @ q
                dv.reshape(-1, n2, d)[at[lo:hi], kv] += prob.T @ y
    return (dq, dk, dv) if grad else (o, lse)
