"""Cases that measure two operators next to the selected attention, in training and in serving:

* rotary positions of queries and keys (``rotary_forward`` / ``rotary_backward``):
      y = m * R(p f) x  on the rotated columns, the other columns unchanged; the gradient is m * R(-p f) dy,
  with p the row's position, f the frequency of its pair of columns and m a magnitude;
* cross attention of a batch's tokens to an encoder's states of another length
  (``cross_forward`` / ``cross_backward``), G query heads sharing a key/value head:
      S = scale Q K^T over the states that are there,  lse = ln sum exp S,  O = exp(S - lse) V,
      dP = dY V^T,  dS = P (dP - rowsum(dY O)),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dY;
  a row with no state to attend to has O = 0 and lse = -inf and gives no gradient.

``run`` computes them with elementary torch operations in 32 bits, or, with ``own`` set, by the calls that a user
makes of the framework.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token for each of 64 running sequences at far positions; the last 64 columns of 192-wide heads are rotated
        dict(name="rotary_decode", op="rotary", dtype="bf16", batch=64, s=1, ragged=False, padded=False, n1=64, n2=4, d=192,
             rot=64, offset=128, style="half", scaling="bands", far=True, grad=False),
        # the long training context (32768 tokens, 64 and 4 heads): the rope tensors of the split heads, pairs interleaved
        dict(name="rotary_long_context", op="rotary", dtype="bf16", batch=1, s=32768, ragged=False, padded=False, n1=64, n2=4, d=64,
             rot=64, offset=0, style="interleaved", scaling="none", far=False, grad=False),
        # packed sequences of other lengths, 128-wide heads rotated as halves, frequencies stretched for a longer context
        dict(name="rotary_packed_f16", op="rotary", dtype="f16", batch=5, s=8191, ragged=True, padded=False, n1=8, n2=8, d=128,
             rot=128, offset=0, style="half", scaling="ramp", far=False, grad=False),
        # gradients of a padded batch, 96 of 192 columns rotated
        dict(name="rotary_grad_padded", op="rotary", dtype="bf16", batch=4, s=4095, ragged=True, padded=True, n1=16, n2=1, d=192,
             rot=96, offset=0, style="half", scaling="linear", far=False, grad=True),
        # one token of one sequence against a short encoder output: latency
        dict(name="cross_token", op="cross", dtype="bf16", batch=1, s1=1, s2=577, ragged=False, padded=False, n1=16, n2=16, d=128,
             holes=False, empty=False, grad=False),
        # decoding: one token for each of 64 sequences against ragged encoder states
        dict(name="cross_decode", op="cross", dtype="bf16", batch=64, s1=1, s2=4096, ragged=True, padded=False, n1=64, n2=4, d=128,
             holes=False, empty=False, grad=False),
        # an ordinary packed batch, 64-wide heads, one sequence without encoder states
        dict(name="cross_packed_f16", op="cross", dtype="f16", batch=6, s1=1021, s2=1531, ragged=True, padded=False, n1=16, n2=16, d=64,
             holes=False, empty=True, grad=False),
        # a few query tokens against one very long memory
        dict(name="cross_long_memory", op="cross", dtype="bf16", batch=1, s1=130, s2=131072, ragged=False, padded=False, n1=32, n2=4,
             d=128, holes=False, empty=False, grad=False),
        # the largest forward: long sequences on both sides
        dict(name="cross_large", op="cross", dtype="bf16", batch=2, s1=8192, s2=4096, ragged=False, padded=False, n1=32, n2=8, d=128,
             holes=False, empty=False, grad=False),
        # gradients of a padded batch with holes in its states and groups of three heads
        dict(name="cross_grad_padded_f16", op="cross", dtype="f16", batch=4, s1=1000, s2=1290, ragged=True, padded=True, n1=24, n2=8,
             d=128, holes=True, empty=True, grad=True),
        # gradients of long sequences against short encoder states
        dict(name="cross_grad_short_states", op="cross", dtype="bf16", batch=3, s1=8192, s2=77, ragged=True, padded=False, n1=8, n2=8,
             d=64, holes=False, empty=False, grad=True),
        # the largest gradient
        dict(name="cross_grad_large", op="cross", dtype="bf16", batch=2, s1=8192, s2=4096, ragged=False, padded=False, n1=32, n2=8,
             d=128, holes=False, empty=False, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    padded, ragged = rng.random() < 0.4, rng.random() < 0.7
    dtype = rng.choice(["bf16", "f16"])
    if rng.random() < 0.4:
        d = rng.choice([64, 128, 192])
        rot = rng.choice([r for r in (16, 32, 64, 96, 128, 192) if r <= d])
        n2 = rng.choice([1, 2, 4, 8])
        n1 = n2 * rng.choice([1, 2, 3, 5, 8])
        batch = _log(rng, 1, 64)
        s = max(1, min(_log(rng, 1, 32768), 32768 * 68 * 64 // (batch * (n1 + n2) * d)))
        return dict(op="rotary", dtype=dtype, batch=batch, s=s, ragged=ragged, padded=padded, n1=n1, n2=n2, d=d, rot=rot,
                    offset=rng.choice([0, d - rot]), style=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "ramp", "bands"]), far=rng.random() < 0.3, grad=rng.random() < 0.5)
    d = rng.choice([64, 128])
    n2 = rng.choice([1, 2, 4, 8, 16])
    n1 = n2 * rng.choice([1, 1, 2, 3, 4, 5, 8])
    grad = rng.random() < 0.5
    batch = _log(rng, 1, 32)
    # no more queries and scores than the largest listed case has, no more states than the long memory
    s1 = 1 if rng.random() < 0.2 else min(_log(rng, 1, 8192), 2 * 8192 * 32 * 128 // (batch * n1 * d))
    s2 = _log(rng, 1, 65536)
    s2 = max(1, min(s2, 2 * 8192 * 4096 * 32 // (batch * s1 * n1), 131072 * 4 * 128 // (batch * n2 * d)))
    return dict(op="cross", dtype=dtype, batch=batch, s1=s1, s2=s2, ragged=ragged, padded=padded, n1=n1, n2=n2, d=d,
                holes=rng.random() < 0.3, empty=batch > 1 and rng.random() < 0.3, grad=grad)


# ------------------------------------------------------------- what is in hand
def _lengths(batch, s, ragged, step):
    """Lengths of the sequences, the longest of them s."""
    return [s - (b * step) % (s // 2 + 1) if ragged else s for b in range(batch)]


def _prefix(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _states_lengths(case):
    l2 = _lengths(case["batch"], case["s2"], case["ragged"], 389)
    if case["empty"]:
        l2[case["batch"] // 2] = 0
    if not any(l2):
        l2[0] = case["s2"]
    return l2


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


ROTARY = dict(base=10000.0, factor=4.0, original_length=8192, beta_fast=32.0, beta_slow=1.0, low=1.0, high=4.0)


def _frequencies(case):
    """Frequencies (radians a position) of the pairs of columns, and the magnitude m, in Python floats."""
    r, base, factor, length = case["rot"], ROTARY["base"], ROTARY["factor"], ROTARY["original_length"]
    kind = case["scaling"]
    if kind == "base":
        base *= factor ** (r / (r - 2))
    f = [base ** (-2 * i / r) for i in range(r // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    elif kind == "ramp":
        edge = [r * math.log(length / (2 * math.pi * beta)) / (2 * math.log(base)) for beta in (ROTARY["beta_fast"], ROTARY["beta_slow"])]
        lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), r - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(r // 2)]
        f = [x * (1 - g) + x / factor * g for x, g in zip(f, ramp)]
    elif kind == "bands":
        turns = [length * x / (2 * math.pi) for x in f]
        share = [min(max((t - ROTARY["low"]) / (ROTARY["high"] - ROTARY["low"]), 0.0), 1.0) for t in turns]
        f = [x / factor * (1 - g) + x * g for x, g in zip(f, share)]
    return f, (0.1 * math.log(factor) + 1.0 if kind == "ramp" else 1.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "rotary":
        lengths = _lengths(case["batch"], case["s"], case["ragged"], 211)
        row, place, rows = _rows(lengths, case["s"], case["padded"])
        lead = (case["batch"], case["s"]) if case["padded"] else (rows,)
        state = dict(case=case, cu=_prefix(lengths), row=row, place=place, q=_normal(gen, lead + (case["n1"], case["d"]), dtype),
                     k=_normal(gen, lead + (case["n2"], case["d"]), dtype), positions=None)
        if case["far"]:  # each row's own position in a long context
            state["positions"] = torch.randint(0, 131072, lead, generator=gen, device="cuda", dtype=torch.int32)
        f, state["magnitude"] = _frequencies(case)
        state["frequencies"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        if own:
            state["kept"] = _keep_rotary(case, state)
        return state
    l1, l2 = _lengths(case["batch"], case["s1"], case["ragged"], 97), _states_lengths(case)
    row1, place1, r1 = _rows(l1, case["s1"], case["padded"])
    row2, place2, r2 = _rows(l2, case["s2"], case["padded"])
    lead1 = (case["batch"], case["s1"]) if case["padded"] else (r1,)
    lead2 = (case["batch"], case["s2"]) if case["padded"] else (r2,)
    state = dict(case=case, cu1=_prefix(l1), cu2=_prefix(l2), row1=row1, place1=place1, row2=row2, place2=place2, lead1=lead1,
                 lead2=lead2, scale=case["d"] ** -0.5, q=_normal(gen, lead1 + (case["n1"], case["d"]), dtype),
                 k=_normal(gen, lead2 + (case["n2"], case["d"]), dtype), v=_normal(gen, lead2 + (case["n2"], case["d"]), dtype),
                 mask=None)
    if case["holes"]:  # an eighth of the states are masked out
        state["mask"] = torch.rand(lead2, generator=gen, device="cuda") >= 0.125
    if case["grad"]:
        state["dy"] = _normal(gen, lead1 + (case["n1"], case["d"]), dtype)
        state["o"], state["lse"] = _cross_plain(state)
    if own:
        state["kept"] = _keep_cross(case, state)
    return state


# --------------------------------------------------------- the framework's calls
def _sag_type(case):
    import sparse_attention_backward_gb300 as sab
    return sab.SAG_FP16 if case["dtype"] == "f16" else sab.SAG_BF16


def _layout(case):
    import sparse_attention_backward_gb300 as sab
    return sab.SAG_LAYOUT_BSND if case["padded"] else sab.SAG_LAYOUT_TND


def _keep_rotary(case, state):
    """The frequencies, the descriptor and the workspace of the problem."""
    import sparse_attention_backward_gb300 as sab
    rotary = sab.Rotary(case["rot"], base=ROTARY["base"], style=case["style"], offset=case["offset"], scaling=case["scaling"],
                        factor=ROTARY["factor"], original_length=ROTARY["original_length"], beta_fast=ROTARY["beta_fast"],
                        beta_slow=ROTARY["beta_slow"], low=ROTARY["low"], high=ROTARY["high"])
    desc = sab.make_rotary_desc(rotary, state["cu"], case["n1"], case["n2"], case["d"], dtype=_sag_type(case), layout=_layout(case),
                                s_max=case["s"] if case["padded"] else 0)
    work = torch.empty(max(1, sab.rotary_workspace_size(desc)), dtype=torch.uint8, device="cuda")
    return dict(rotary=rotary, desc=desc, workspace=work)


def _keep_cross(case, state):
    """The descriptor and the workspace of the problem."""
    import sparse_attention_backward_gb300 as sab
    desc = sab.make_cross_desc(state["cu1"], state["cu2"], case["n1"], case["n2"], case["d"], state["scale"], dtype=_sag_type(case),
                               layout=_layout(case), s1_max=case["s1"] if case["padded"] else 0,
                               s2_max=case["s2"] if case["padded"] else 0)
    need = sab.cross_grad_workspace_size(desc) if case["grad"] else sab.cross_fwd_workspace_size(desc)
    return dict(desc=desc, workspace=torch.empty(max(1, need), dtype=torch.uint8, device="cuda"))


def _own(state):
    import sparse_attention_backward_gb300 as sab
    case, kept = state["case"], state["kept"]
    if case["op"] == "rotary":
        call = sab.rotary_backward if case["grad"] else sab.rotary_forward
        return call(state["q"], state["k"], kept["rotary"], positions=state["positions"], workspace=kept["workspace"], desc=kept["desc"])
    if case["grad"]:
        return sab.cross_backward(state["q"], state["k"], state["v"], state["o"], state["dy"], state["lse"], key_mask=state["mask"],
                                  workspace=kept["workspace"], desc=kept["desc"])
    return sab.cross_forward(state["q"], state["k"], state["v"], key_mask=state["mask"], workspace=kept["workspace"], desc=kept["desc"])


# ------------------------------------------------------------- the plain forms
def _rotary_plain(state):
    case = state["case"]
    r, off, s = case["rot"], case["offset"], case["s"]
    if state["positions"] is not None:
        pos = state["positions"].reshape(-1)[state["row"]]
    else:
        pos = state["place"] % s
    angle = pos.double()[:, None] * state["frequencies"]  # 64 bits: far positions make many turns
    sin, cos = angle.sin() * (-1.0 if case["grad"] else 1.0), angle.cos()
    sin, cos = (sin * state["magnitude"]).float()[:, None], (cos * state["magnitude"]).float()[:, None]

    def turn(x):
        flat = x.reshape(-1, x.shape[-2], x.shape[-1])
        y = flat[state["row"]].float()
        z = y[..., off:off + r]
        a, b = (z[..., :r // 2], z[..., r // 2:]) if case["style"] == "half" else (z[..., 0::2], z[..., 1::2])
        a, b = a * cos - b * sin, a * sin + b * cos
        z = torch.cat((a, b), -1) if case["style"] == "half" else torch.stack((a, b), -1).flatten(-2)
        y = torch.cat((y[..., :off], z, y[..., off + r:]), -1)
        return torch.zeros_like(flat).index_copy(0, state["row"], y.to(x.dtype)).reshape(x.shape)

    return turn(state["q"]), turn(state["k"])


def _grid(state, x, which):
    """Valid rows of x as [batch, heads, s, ...] in 32 bits, zeros elsewhere."""
    case = state["case"]
    s = case["s1"] if which == 1 else case["s2"]
    tail = x.shape[2 if case["padded"] else 1:]
    flat = x.reshape((-1,) + tail)[state["row%d" % which]].float()
    out = torch.zeros((case["batch"] * s,) + tail, dtype=torch.float32, device=x.device)
    out[state["place%d" % which]] = flat
    return out.reshape((case["batch"], s) + tail).transpose(1, 2) if len(tail) else out.reshape(case["batch"], s)


def _back(state, x, which, like):
    """[batch, heads, s, ...] as rows of a tensor like `like`, zeros in its padding."""
    lead = state["lead%d" % which]
    x = x.transpose(1, 2)
    tail = x.shape[2:]
    x = x.reshape((-1,) + tail)[state["place%d" % which]]
    out = torch.zeros((math.prod(lead),) + tail, dtype=like, device=x.device)
    out[state["row%d" % which]] = x.to(like)
    return out.reshape(tuple(lead) + tail)


def _scores(state):
    """Masked scores [batch, n2, G, s1, s2], -inf where there is nothing to attend to."""
    case = state["case"]
    b, n2, g, s1, s2, d = case["batch"], case["n2"], case["n1"] // case["n2"], case["s1"], case["s2"], case["d"]
    there = torch.zeros(b * s2, dtype=torch.bool, device="cuda")
    there[state["place2"]] = True if state["mask"] is None else state["mask"].reshape(-1)[state["row2"]]
    q, k, v = _grid(state, state["q"], 1), _grid(state, state["k"], 2), _grid(state, state["v"], 2)
    keep = there.reshape(b, 1, s2, 1)
    q, k, v = q.reshape(b, n2, g * s1, d), torch.where(keep, k, 0.0), torch.where(keep, v, 0.0)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(state["scale"]).masked_fill_(~there.reshape(b, 1, 1, s2), -math.inf)
    return q, k, v, s


def _cross_plain(state):
    case = state["case"]
    b, n1, s1, d = case["batch"], case["n1"], case["s1"], case["d"]
    q, k, v, s = _scores(state)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top.isinf(), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = total.log() + top
    return _back(state, o.reshape(b, n1, s1, d), 1, state["q"].dtype), _back(state, lse.reshape(b, n1, s1), 1, torch.float32)


def _cross_grad_plain(state):
    case = state["case"]
    b, n1, n2, s1, d = case["batch"], case["n1"], case["n2"], case["s1"], case["d"]
    q, k, v, s = _scores(state)
    lse = _grid(state, state["lse"][..., None], 1).reshape(b, n2, -1, 1)
    dy = _grid(state, state["dy"], 1).reshape(b, n2, -1, d)
    delta = (_grid(state, state["o"], 1).reshape(b, n2, -1, d) * dy).sum(-1, keepdim=True)
    p = s.sub_(torch.where(lse.isinf(), 0.0, lse)).exp_()
    dv = torch.matmul(p.transpose(2, 3), dy)
    ds = torch.matmul(dy, v.transpose(2, 3)).sub_(delta).mul_(p).mul_(state["scale"])
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(2, 3), q)
    t = state["q"].dtype
    return _back(state, dq.reshape(b, n1, s1, d), 1, t), _back(state, dk, 2, t), _back(state, dv, 2, t)


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"] == "rotary":
        return _rotary_plain(state)
    return _cross_grad_plain(state) if state["case"]["grad"] else _cross_plain(state)


# --------------------------------------------------------------- the floor
def work(case):
    if case["op"] == "rotary":
        tokens = sum(_lengths(case["batch"], case["s"], case["ragged"], 211))
        # 8 operations for each pair of columns: two products and a sum, twice, and the scaling of sine and cosine
        return {"bytes": tokens * ((case["n1"] + case["n2"]) * case["d"] * 4 + (4 if case["far"] else 0)),
                "flops": tokens * (case["n1"] + case["n2"]) * case["rot"] // 2 * 8}
    l1, l2 = _lengths(case["batch"], case["s1"], case["ragged"], 97), _states_lengths(case)
    t1, t2, keep = sum(l1), sum(l2), 0.875 if case["holes"] else 1.0
    pairs = sum(a * b for a, b in zip(l1, l2)) * keep
    d, n1, n2 = case["d"], case["n1"], case["n2"]
    q, kv, stat, mask = t1 * n1 * d * 2, t2 * n2 * d * 2, t1 * n1 * 4, t2 if case["holes"] else 0
    if case["grad"]:  # q, o, dy, dq; k, v, dk, dv
        return {"bytes": int(4 * q + 4 * kv + stat + mask), "flops": int(10 * pairs * n1 * d)}
    return {"bytes": int(2 * q + 2 * kv + stat + mask), "flops": int(4 * pairs * n1 * d)}


# --------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, state)
    l1, l2 = _lengths(case["batch"], case["s1"], case["ragged"], 97), _states_lengths(case)
    if sum(a * b for a, b in zip(l1, l2)) * case["n1"] * case["d"] * (10 if case["grad"] else 4) > 6e12:
        return None
    return _exact_cross(case, state, l1, l2)


def _exact_rotary(case, state):
    """Pairs of columns as complex numbers, turned sequence by sequence."""
    freq, half = state["frequencies"], case["rot"] // 2
    sign = -1.0 if case["grad"] else 1.0
    cols = torch.arange(case["rot"], device="cuda") + case["offset"]
    first, second = (cols[:half], cols[half:]) if case["style"] == "half" else (cols[0::2], cols[1::2])
    answers = []
    for x in (state["q"], state["k"]):
        y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(case["batch"], case["s"], case["ragged"], 211)):
            part = (b, slice(0, n)) if case["padded"] else slice(state["cu"][b], state["cu"][b] + n)
            p = torch.arange(n, device="cuda") if state["positions"] is None else state["positions"][part]
            z = x[part].double()
            turned = torch.complex(z[..., first], z[..., second]) * torch.polar(
                torch.full((n, 1, half), state["magnitude"], dtype=torch.float64, device="cuda"),
                sign * p.double().reshape(n, 1, 1) * freq)
            z[..., first], z[..., second] = turned.real, turned.imag
            y[part] = z
        answers.append(y)
    return tuple(answers)


def _exact_cross(case, state, l1, l2):
    """Batch by batch and head by head, over the states that are there."""
    g, d, scale = case["n1"] // case["n2"], case["d"], state["scale"]
    new = lambda lead, *tail: torch.zeros(tuple(lead) + tail, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = new(state["lead1"], case["n1"], d), new(state["lead1"], case["n1"])
    dq, dk, dv = new(state["lead1"], case["n1"], d), new(state["lead2"], case["n2"], d), new(state["lead2"], case["n2"], d)
    for b in range(case["batch"]):
        rows = (b, slice(0, l1[b])) if case["padded"] else (slice(state["cu1"][b], state["cu1"][b] + l1[b]),)
        first = b * case["s2"] if case["padded"] else state["cu2"][b]
        at = torch.arange(first, first + l2[b], device="cuda")
        if state["mask"] is not None:
            at = at[state["mask"].reshape(-1)[at]]
        for h in range(case["n1"]):
            n = h // g
            q = state["q"][rows][:, h].double()
            k, v = state["k"].reshape(-1, case["n2"], d)[at, n].double(), state["v"].reshape(-1, case["n2"], d)[at, n].double()
            s = q @ k.T * scale
            if not case["grad"]:
                lse[rows + (h,)] = s.logsumexp(1)
                o[rows + (h,)] = s.softmax(1) @ v
                continue
            if not len(at):
                continue
            y, a = state["dy"][rows][:, h].double(), state["o"][rows][:, h].double()
            p = (s - state["lse"][rows][:, h].double()[:, None]).exp()
            ds = p * (y @ v.T - (y * a).sum(1, keepdim=True)) * scale
            dq[rows + (h,)] = ds @ k
            dk.reshape(-1, case["n2"], d)[at, n] += ds.T @ q
            dv.reshape(-1, case["n2"], d)[at, n] += p.T @ y
    return (dq, dk, dv) if case["grad"] else (o, lse)
