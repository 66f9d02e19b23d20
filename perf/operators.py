"""What is measured of the operators beside the attention kernels: the per-head norm of
queries and keys with the position rotation in the same pass (forward, backward), and
linear attention with a decay per head (prompts, backward, single tokens).

qk_norm_rope, per valid row and head, x the head's d values, w the weight, eps > 0:
    y = rotate(x / sqrt(mean(x^2) + eps) * w),    rotate: pair p of the first rot_dim values
    turned by the angle position[axis(p)] * inv_freq(p), inv_freq(p) = base^(-2p / rot_dim)
linear attention, per sequence and head h, lambda = exp(log_decay[h]):
    S_t = lambda S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t
Pad rows (at or past a sequence's length) give 0 in every output.

``own`` False runs plain torch operations in 32 bits (angles in 64); ``own`` True makes the
library's calls.
"""
import math
import random

import torch

own = False

CHUNK = 64


# --------------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of each of 64 sequences before a decoding step's attention
        {"name": "qk_tokens", "op": "qk_fwd", "layout": "padded", "B": 64, "N": 1, "lengths": "full", "seed": 1,
         "Hq": 8, "Hk": 8, "d": 64, "rot": 64, "axes": 1, "interleaved": False, "base": 10000.0, "far": 200000},
        # the single-cell batch: genes carry no position, so the norm alone
        {"name": "qk_single_cell", "op": "qk_fwd", "layout": "padded", "B": 32, "N": 2048, "lengths": "log", "seed": 1002,
         "Hq": 8, "Hk": 8, "d": 64, "rot": 0, "axes": 0, "interleaved": False, "base": 10000.0, "far": 0},
        # patches of images or video: time, height and width, fewer key heads than query heads, odd rows
        {"name": "qk_images", "op": "qk_fwd", "layout": "padded", "B": 2, "N": 8191, "lengths": "uniform", "seed": 3,
         "Hq": 16, "Hk": 4, "d": 128, "rot": 96, "axes": 3, "interleaved": False, "base": 10000.0, "far": 0},
        # training, a small odd batch, pairs side by side, part of the head rotated
        {"name": "qk_grad_odd", "op": "qk_bwd", "layout": "padded", "B": 3, "N": 1021, "lengths": "uniform", "seed": 4,
         "Hq": 6, "Hk": 2, "d": 64, "rot": 32, "axes": 2, "interleaved": True, "base": 1000.0, "far": 0},
        # training on packed documents, the largest ordinary batch
        {"name": "qk_grad_documents", "op": "qk_bwd", "layout": "packed", "B": 64, "N": 32768, "lengths": "documents", "seed": 1004,
         "Hq": 16, "Hk": 16, "d": 128, "rot": 128, "axes": 1, "interleaved": False, "base": 500000.0, "far": 0},
        # the smallest prompts: four short sequences, latency counts
        {"name": "linear_tiny", "op": "lin_fwd", "layout": "padded", "B": 4, "N": 128, "lengths": "tiny", "seed": 1001,
         "H": 2, "d": 64, "state": False},
        # the long ragged batch
        {"name": "linear_long", "op": "lin_fwd", "layout": "padded", "B": 8, "N": 16384, "lengths": "uniform4", "seed": 1003,
         "H": 16, "d": 128, "state": False},
        # one prompt of odd length that leaves its state for generation: few rows to share out
        {"name": "linear_prompt", "op": "lin_fwd", "layout": "packed", "B": 1, "N": 10007, "lengths": "full", "seed": 8,
         "H": 16, "d": 128, "state": True},
        # training on the single-cell batch, with gradients into and out of the state
        {"name": "linear_grad_single_cell", "op": "lin_bwd", "layout": "padded", "B": 32, "N": 2048, "lengths": "log", "seed": 1002,
         "H": 8, "d": 64, "state": True},
        # training on packed documents, causal within each
        {"name": "linear_grad_documents", "op": "lin_bwd", "layout": "packed", "B": 64, "N": 32768, "lengths": "documents", "seed": 1004,
         "H": 16, "d": 128, "state": False},
        # one sequence generates
        {"name": "linear_step_one", "op": "lin_step", "B": 1, "H": 16, "d": 128, "seed": 11},
        # a large batch generates
        {"name": "linear_step_batch", "op": "lin_step", "B": 256, "H": 16, "d": 128, "seed": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "lin_fwd", "lin_bwd", "lin_step"])
    d = rng.choice([64, 128])
    case = {"op": op, "d": d, "seed": rng.randrange(1 << 30)}
    if op == "lin_step":
        case.update(B=_log_int(rng, 1, 256), H=rng.choice([1, 2, 3, 8, 12, 16]))
        return case
    case["layout"] = rng.choice(["padded", "packed"])
    rows = _log_int(rng, 64, 32768)
    if case["layout"] == "padded":
        case["B"] = _log_int(rng, 1, min(rows, 32))
        case["N"] = max(1, rows // case["B"])
        case["lengths"] = rng.choice(["full", "uniform", "log"])
    else:
        case["B"] = _log_int(rng, 1, min(rows, 64))
        case["N"] = rows
        case["lengths"] = "full" if case["B"] == 1 else "documents"
    if op in ("qk_fwd", "qk_bwd"):
        case["Hq"] = rng.choice([1, 3, 6, 8, 16])
        case["Hk"] = rng.choice([h for h in (1, 2, 3, 6, 8, 16) if h <= case["Hq"] and case["Hq"] % h == 0])
        case["axes"] = rng.choice([0, 1, 1, 2, 3])
        case["rot"] = 0 if case["axes"] == 0 else rng.choice([r for r in (32, 48, 64, 96, 128) if r <= d])
        case["interleaved"] = rng.random() < 0.5
        case["base"] = rng.choice([1000.0, 10000.0, 500000.0])
        case["far"] = rng.choice([0, 0, 1000000]) if case["axes"] == 1 else 0
    else:
        case["H"] = rng.choice([1, 2, 5, 8, 16])
        case["state"] = rng.random() < 0.5
    return case


def _lengths(case):
    """The sequences' lengths (host list): a function of the case alone."""
    rng = random.Random(case["seed"] * 7 + 1)
    B, N, kind = case["B"], case["N"], case["lengths"]
    if kind == "tiny":
        return [37, 64, 100, 128]
    if kind == "full":
        return [N] * B
    if kind == "uniform":
        return [rng.randint(max(1, N // 3), N) for _ in range(B - 1)] + [N]
    if kind == "uniform4":
        return [rng.randint(N // 4, N) for _ in range(B - 1)] + [N]
    if kind == "log":
        lo = max(1, N // 10)
        return [min(N, int(math.exp(rng.uniform(math.log(lo), math.log(N + 1))))) for _ in range(B - 1)] + [N]
    # documents: N rows cut at B - 1 random places (lengths of zero may occur)
    cuts = sorted(rng.randint(0, N) for _ in range(B - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [N])]


def _sections(case):
    pairs, axes = case["rot"] // 2, case["axes"]
    base = [pairs // axes] * axes
    base[0] += pairs - sum(base)
    return base


# --------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(1000003 * seed + case["seed"] % 1000003)
    normal = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    bf = lambda *s: normal(*s).to(torch.bfloat16)  # noqa: E731
    st = {"case": case}
    d = case["d"]
    if case["op"] == "lin_step":
        B, H = case["B"], case["H"]
        st.update(q=bf(B, H, d), k=bf(B, H, d), v=bf(B, H, d), state=3.0 * normal(B, H, d, d), log_decay=_decay(H, dev))
        st["new_state"] = torch.empty_like(st["state"])
        return st
    ln = _lengths(case)
    B, N = case["B"], case["N"]
    st["lengths"] = torch.tensor(ln, dtype=torch.int32, device=dev)
    rows = (B, N) if case["layout"] == "padded" else (sum(ln),)
    if case["layout"] == "packed":
        st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(st["lengths"], 0)]).to(torch.int32)
        st["longest"] = max(ln)
    if case["op"] in ("qk_fwd", "qk_bwd"):
        # projections of one layer: heads of unequal size
        st["q"] = (normal(*rows, case["Hq"], d) * (0.5 + 2.0 * torch.rand(case["Hq"], 1, generator=gen, device=dev))).to(torch.bfloat16)
        st["k"] = (normal(*rows, case["Hk"], d) * (0.5 + 2.0 * torch.rand(case["Hk"], 1, generator=gen, device=dev))).to(torch.bfloat16)
        st["wq"] = 1.0 + 0.2 * normal(d)
        st["wk"] = 1.0 + 0.2 * normal(d)
        st["rope"] = {}
        if case["axes"]:
            p = torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64)
            st["rope"] = {"positions": _positions(case, st, gen, dev), "inv_freq": case["base"] ** (-2.0 * p / case["rot"]),
                          "sections": _sections(case), "interleaved": case["interleaved"]}
        if case["op"] == "qk_bwd":
            st["dyq"] = bf(*rows, case["Hq"], d)
            st["dyk"] = bf(*rows, case["Hk"], d)
        return st
    H = case["H"]
    st.update(q=bf(*rows, H, d), k=bf(*rows, H, d), v=bf(*rows, H, d), log_decay=_decay(H, dev))
    st["state"] = 3.0 * normal(B, H, d, d) if case["state"] else None
    if case["op"] == "lin_bwd":
        st["do"] = bf(*rows, H, d)
        st["dstate"] = normal(B, H, d, d) if case["state"] else None
    return st


def _decay(H, dev):
    """Slopes from 1/2 down to 1/256 over the heads: short and long memories."""
    return -torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H)


def _positions(case, st, gen, dev):
    """int32 [axes, rows...]: rows counted from the sequence's start (plus an offset per
    sequence where the cache already holds tokens), or time, height and width of patches."""
    B, N = case["B"], case["N"]
    if case["layout"] == "padded":
        row = torch.arange(N, device=dev)[None].expand(B, N)
        seq = torch.arange(B, device=dev)[:, None].expand(B, N)
    else:
        row, seq = _rows_of(st["cu"], st["q"].shape[0])
    if case["far"]:
        off = torch.randint(0, case["far"], (B,), generator=gen, device=dev)
        row = row + off[seq]
    if case["axes"] == 1:
        pos = row[None]
    else:
        side = 37  # patches of one image row
        axes = [row // (side * side), (row // side) % side, row % side]
        pos = torch.stack(axes[3 - case["axes"]:])
    return pos.to(torch.int32).contiguous()


def _rows_of(cu, T):
    """Of each packed row: its place in its sequence, and the sequence."""
    t = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), t, right=True)
    return t - cu.long()[seq], seq


# --------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    return {"qk_fwd": _run_qk_fwd, "qk_bwd": _run_qk_bwd, "lin_fwd": _run_lin_fwd, "lin_bwd": _run_lin_bwd,
            "lin_step": _run_lin_step}[case["op"]](st, case)


def _run_qk_fwd(st, case):
    lengths = st["lengths"] if case["layout"] == "padded" else None
    if own:
        from padded_variable_length_b200 import binding as Bd
        return Bd.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], eps=1e-6, lengths=lengths, **st["rope"])
    cs = _cos_sin(case, st["rope"])
    return tuple(_keep(_rotate(_norm(st[x].float())[0] * st["w" + x], cs, case, 1.0), lengths).to(torch.bfloat16) for x in ("q", "k"))


def _run_qk_bwd(st, case):
    lengths = st["lengths"] if case["layout"] == "padded" else None
    if own:
        from padded_variable_length_b200 import binding as Bd
        dq, dk, dwq, dwk = Bd.qk_norm_rope_bwd(st["q"], st["k"], st["dyq"], st["dyk"], st["wq"], st["wk"], eps=1e-6, lengths=lengths, **st["rope"])
        return dq, dwq, dk, dwk
    cs = _cos_sin(case, st["rope"])
    return _qk_grad(st, "q", cs, case, lengths) + _qk_grad(st, "k", cs, case, lengths)


def _qk_grad(st, x, cs, case, lengths):
    """(dx, dw) of one of the two tensors."""
    g = _rotate(_keep(st["dy" + x].float(), lengths), cs, case, -1.0)  # the rotation's transpose
    u, r = _norm(st[x].float())
    dw = _keep(g * u, lengths).reshape(-1, case["d"]).sum(0)
    h = g * st["w" + x]
    dx = r * (h - u * (h * u).mean(-1, keepdim=True))
    return _keep(dx, lengths).to(torch.bfloat16), dw


def _run_lin_fwd(st, case):
    scale = 1.0 / math.sqrt(case["d"])
    if own:
        from padded_variable_length_b200 import binding as Bd
        o, new = Bd.linear_fwd(st["q"], st["k"], st["v"], st["log_decay"], scale=scale, state=st["state"], return_state=case["state"], **_ragged(st, case))
        return (o, new) if case["state"] else o
    g, n = st["log_decay"], st["lengths"]
    q, k, v = (_spread(st[x], st, case) for x in ("q", "k", "v"))
    o = scale * _causal(q, k, v, g)
    if not case["state"]:
        return _gather(o, st, case)
    t = torch.arange(q.shape[1], device=q.device, dtype=torch.float32)
    o = o + scale * torch.exp(g * (t[:, None] + 1.0))[None, :, :, None] * _heads(q, st["state"])
    left = n[:, None].float() - 1.0 - t  # tokens after this one
    w = torch.exp(g * left.clamp(min=0)[:, :, None])[..., None]
    new = torch.einsum("bnhi,bnhj->bhij", k * w, v) + torch.exp(g * n[:, None])[:, :, None, None] * st["state"]
    return _gather(o, st, case), new


def _run_lin_bwd(st, case):
    scale = 1.0 / math.sqrt(case["d"])
    if own:
        from padded_variable_length_b200 import binding as Bd
        dq, dk, dv, ds = Bd.linear_bwd(st["q"], st["k"], st["v"], st["do"], st["log_decay"], scale=scale, state=st["state"], dstate=st["dstate"],
                                       **_ragged(st, case))
        return (dq, dk, dv, ds) if case["state"] else (dq, dk, dv)
    g, n = st["log_decay"], st["lengths"]
    q, k, v, do = (_spread(st[x], st, case) for x in ("q", "k", "v", "do"))
    back = lambda *x: _causal(*(y.flip(1) for y in x), g).flip(1)  # noqa: E731
    dq = scale * _causal(do, v, k, g)
    dk = scale * back(v, do, q)
    dv = scale * back(k, q, do)
    if not case["state"]:
        return tuple(_gather(x, st, case) for x in (dq, dk, dv))
    t = torch.arange(q.shape[1], device=q.device, dtype=torch.float32)
    since = torch.exp(g * (t[:, None] + 1.0))[None, :, :, None]
    left = torch.exp(g * (n[:, None].float() - 1.0 - t).clamp(min=0)[:, :, None])[..., None]
    dq = dq + scale * since * _heads(do, st["state"].transpose(2, 3))
    dk = dk + left * _heads(v, st["dstate"].transpose(2, 3))
    dv = dv + left * _heads(k, st["dstate"])
    ds = scale * torch.einsum("bnhi,bnhj->bhij", q * since, do) + torch.exp(g * n[:, None])[:, :, None, None] * st["dstate"]
    return tuple(_gather(x, st, case) for x in (dq, dk, dv)) + (ds,)


def _run_lin_step(st, case):
    scale = 1.0 / math.sqrt(case["d"])
    if own:
        from padded_variable_length_b200 import binding as Bd
        o = Bd.linear_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], state_out=st["new_state"], scale=scale)
        return o, st["new_state"]
    q, k, v = (st[x].float() for x in ("q", "k", "v"))
    new = torch.exp(st["log_decay"])[:, None, None] * st["state"] + k[..., :, None] * v[..., None, :]
    return (scale * (q[..., :, None] * new).sum(-2)).to(torch.bfloat16), new


def _ragged(st, case):
    if case["layout"] == "padded":
        return {"lengths": st["lengths"]}
    return {"cu_seqlens": st["cu"], "max_seqlen": st["longest"]}


# --------------------------------------------------------------------------- plain parts
def _norm(x):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return x * r, r


def _cos_sin(case, rope):
    """cos and sin [rows..., 1, pairs] in 32 bits, from angles in 64 (far positions)."""
    if not rope:
        return None
    axis = [a for a, pairs in enumerate(rope["sections"]) for _ in range(pairs)]
    angle = rope["positions"].double()[axis].movedim(0, -1) * rope["inv_freq"]
    return torch.cos(angle).float()[..., None, :], torch.sin(angle).float()[..., None, :]


def _rotate(x, cs, case, way):
    if cs is None:
        return x
    cos, sin = cs
    rot, rest = x[..., :case["rot"]], x[..., case["rot"]:]
    if case["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
    else:
        a, b = rot[..., :case["rot"] // 2], rot[..., case["rot"] // 2:]
    a, b = a * cos - way * b * sin, way * a * sin + b * cos
    rot = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([rot, rest], -1)


def _keep(x, lengths):
    """Pad rows become 0."""
    if lengths is None:
        return x
    t = torch.arange(x.shape[1], device=x.device)
    return torch.where((t < lengths[:, None])[:, :, None, None], x, x.new_zeros(()))


def _spread(x, st, case):
    """32-bit [B, N, H, d], zero behind each sequence, from the padded or packed tensor."""
    n = st["lengths"]
    if case["layout"] == "padded":
        return _keep(x.float(), n)
    t = torch.arange(max(1, st["longest"]), device=x.device)
    at = (st["cu"][:-1, None].long() + t).clamp(max=max(0, x.shape[0] - 1))
    return _keep(x.float()[at], n)


def _gather(x, st, case):
    """The tensor's own layout, rounded once."""
    if case["layout"] == "padded":
        return _keep(x, st["lengths"]).to(torch.bfloat16)
    row, seq = _rows_of(st["cu"], st["q"].shape[0])
    return x[seq, row].to(torch.bfloat16)


def _heads(x, s):
    """x [B, N, H, i] times s [B, H, i, j] for each head."""
    return torch.einsum("bnhi,bhij->bnhj", x, s)


def _causal(q, k, v, g):
    """sum_{j <= i} exp(g (i - j)) (q_i . k_j) v_j, [B, N, H, d] in 32 bits, in chunks: the
    tokens of a chunk against each other, and against the states that earlier chunks leave."""
    B, N, H, d = q.shape
    C = (N + CHUNK - 1) // CHUNK
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, C * CHUNK - N)).reshape(B, C, CHUNK, H, d).permute(0, 3, 1, 2, 4) for x in (q, k, v))
    i = torch.arange(CHUNK, device=g.device, dtype=torch.float32)
    gap = i[:, None] - i
    w = torch.where(gap >= 0, torch.exp(g[:, None, None] * gap.clamp(min=0)), 0.0)[:, None]
    near = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * w, v)
    left = torch.matmul((k * torch.exp(g[:, None] * (CHUNK - 1.0 - i))[:, None, :, None]).transpose(-1, -2), v)  # [B, H, C, d, d]
    c = torch.arange(C, device=g.device, dtype=torch.float32)
    gap = c[:, None] - 1.0 - c
    w = torch.where(gap >= 0, torch.exp(g[:, None, None] * CHUNK * gap.clamp(min=0)), 0.0)
    start = torch.matmul(w, left.reshape(B, H, C, d * d)).reshape(B, H, C, d, d)
    far = torch.matmul(q * torch.exp(g[:, None] * (i + 1.0))[:, None, :, None], start)
    return (near + far).permute(0, 2, 3, 1, 4).reshape(B, C * CHUNK, H, d)[:, :N]


# --------------------------------------------------------------------------- the work
def work(case):
    d = case["d"]
    if case["op"] == "lin_step":
        n = case["B"] * case["H"]
        return {"bytes": n * (2 * 4 * d * d + 4 * 2 * d), "flops": 5 * n * d * d}
    ln = _lengths(case)
    valid = sum(ln)
    rows = case["B"] * case["N"] if case["layout"] == "padded" else valid
    if case["op"] in ("qk_fwd", "qk_bwd"):
        el = (case["Hq"] + case["Hk"]) * d
        reads = 1 if case["op"] == "qk_fwd" else 2
        return {"bytes": 2 * el * (reads * valid + rows) + 4 * case["axes"] * valid, "flops": (8 if reads == 1 else 16) * el * valid}
    H = case["H"]
    states = case["B"] * H * d * d * 4 if case["state"] else 0
    # the recurrence's products, or those of all pairs where a sequence is shorter
    one = H * d * sum(2 * n * min(d, (n + 1) / 2) for n in ln)
    if case["op"] == "lin_fwd":
        return {"bytes": 2 * H * d * (3 * valid + rows) + 2 * states, "flops": 2 * one}
    return {"bytes": 2 * H * d * (4 * valid + 3 * rows) + 3 * states, "flops": 5 * one}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence, all pairs of tokens for linear attention."""
    st = prepare(case, seed)
    f = lambda x: None if x is None else x.double()  # noqa: E731
    if case["op"] == "lin_step":
        q, k, v, s, g = (f(st[x]) for x in ("q", "k", "v", "state", "log_decay"))
        s = torch.einsum("h,bhij->bhij", g.exp(), s) + torch.einsum("bhi,bhj->bhij", k, v)
        return torch.einsum("bhi,bhij->bhj", q, s) / math.sqrt(case["d"]), s
    ln = _lengths(case)
    if case["layout"] == "padded":
        places = [(b, slice(0, n)) for b, n in enumerate(ln)]
    else:
        ends = [sum(ln[:b + 1]) for b in range(len(ln))]
        places = [(slice(e - n, e),) for e, n in zip(ends, ln)]
    if case["op"] in ("qk_fwd", "qk_bwd"):
        return _exact_qk(case, st, places)
    return _exact_lin(case, st, places, ln)


def _exact_qk(case, st, places):
    d, rot = case["d"], case["rot"]
    outs = []
    for x in ("q", "k"):
        full = torch.zeros(st[x].shape, dtype=torch.float64, device=st[x].device)
        dw = torch.zeros(d, dtype=torch.float64, device=full.device)
        for at in places:
            v = st[x][at].double()
            root = (v.square().sum(-1, keepdim=True) / d + 1e-6).sqrt()
            w = st["w" + x].double()
            turn = None
            if rot:
                sec = [a for a, c in enumerate(_sections(case)) for _ in range(c)]
                ang = torch.stack([st["rope"]["positions"][a][at].double() / case["base"] ** (2.0 * p / rot) for p, a in enumerate(sec)], -1)
                turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]
            if case["op"] == "qk_fwd":
                full[at] = _exact_turn(v / root * w, turn, rot, case["interleaved"])
                continue
            g = _exact_turn(st["dy" + x][at].double(), None if turn is None else turn.conj(), rot, case["interleaved"])
            dw += (g * v / root).sum((0, 1))
            g = g * w
            full[at] = g / root - v * (g * v).sum(-1, keepdim=True) / (d * root ** 3)
        outs += [full] if case["op"] == "qk_fwd" else [full, dw]
    return tuple(outs)


def _exact_turn(x, turn, rot, interleaved):
    if turn is None:
        return x
    out = x.clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., one].contiguous(), x[..., two].contiguous()) * turn
    out[..., one], out[..., two] = z.real, z.imag
    return out


def _exact_lin(case, st, places, ln):
    grad = case["op"] == "lin_bwd"
    c = 1.0 / math.sqrt(case["d"])
    lam = st["log_decay"].double()[:, None, None]
    outs = [torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda") for _ in range(3 if grad else 1)]
    states = []
    for b, at in enumerate(places):
        n = ln[b]
        q, k, v, do = (st[x][at].double().transpose(0, 1) if x in st else None for x in ("q", "k", "v", "do"))  # [H, n, d]
        acc = [torch.zeros_like(q) for _ in outs]
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            gap = torch.arange(i0, i1, device="cuda")[:, None] - torch.arange(i1, device="cuda")
            w = c * torch.exp(lam * gap.clamp(min=0)) * (gap >= 0)
            if not grad:
                acc[0][:, i0:i1] = (q[:, i0:i1] @ k[:, :i1].mT * w) @ v[:, :i1]
                continue
            p = do[:, i0:i1] @ v[:, :i1].mT * w
            acc[0][:, i0:i1] = p @ k[:, :i1]
            acc[1][:, :i1] += p.mT @ q[:, i0:i1]
            acc[2][:, :i1] += (q[:, i0:i1] @ k[:, :i1].mT * w).mT @ do[:, i0:i1]
        if case["state"]:
            t = torch.arange(n, device="cuda", dtype=torch.float64)[:, None]
            before, after = torch.exp(lam * (t + 1)), torch.exp(lam * (n - 1 - t))
            s, whole = st["state"][b].double(), torch.exp(lam * n)
            if grad:
                e = st["dstate"][b].double()
                acc[0] += c * before * (do @ s.mT)
                acc[1] += after * (v @ e.mT)
                acc[2] += after * (k @ e)
                states.append(whole * e + c * (before * q).mT @ do)
            else:
                acc[0] += c * before * (q @ s)
                states.append(whole * s + (after * k).mT @ v)
        for o, a in zip(outs, acc):
            o[at] = a.transpose(0, 1)
    res = tuple(outs) + ((torch.stack(states),) if case["state"] else ())
    return res if len(res) > 1 else res[0]
