"""Linear attention with a decay per head against its float64 oracle: chunked forward and
backward, single tokens, and the run of norm, rotation, attention and gradients together.

Tolerances.  Let M be the operator applied to the absolute values.  Every term q_i k_j v_j of
an output passes at most two roundings to bf16 inside (the weighted product; or the decayed
value and the state), and the output one, each 2^-8 at most: |err| <= 2^-8 |o| + 2 * 2^-8 M,
and fp32 sums add less than 2^-16 M.  Roundings of random values do not line up: each has a
root mean square of at most 2^-8 / sqrt 3 of its value, so four of them give a relative error
of at most 2 * 2^-8 / sqrt 3 = 4.6e-3 in the norm over a tensor, less than the 5e-3 asked.
States handed out in fp32 take the values as a sum of two bf16 numbers (2^-16 at most, root
mean square 2^-18) and fp32 sums: 2^-15 M each, and 1e-5 in the norm.  A single token is fp32
throughout: 2^-8 |o| + 2^-18 M, and 2^-20 M for its state."""
import math

import numpy as np
import pytest
import torch

from oracle import linear as OL
from oracle import qknorm as OQ

pytestmark = pytest.mark.gpu

R = 2.0 ** -8


def _bd():
    from padded_variable_length_b200 import binding as Bd
    Bd.set_wait_limit_ns(500_000_000)  # no legitimate wait inside one CTA comes near this
    return Bd


def f64(t):
    return t.detach().cpu().double().numpy()


def _slopes(H):
    return -torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H)


def _make(rows, H, d, B, state, seed):
    g = torch.Generator().manual_seed(seed)
    t = {n: torch.randn(*rows, H, d, generator=g).to(torch.bfloat16).cuda() for n in ("q", "k", "v", "do")}
    t["state"] = torch.randn(B, H, d, d, generator=g).cuda() if state else None
    t["dstate"] = torch.randn(B, H, d, d, generator=g).cuda() if state else None
    return t


def _places(lengths, packed):
    if not packed:
        return [(b, slice(0, n)) for b, n in enumerate(lengths)]
    ends = np.cumsum(lengths)
    return [(slice(int(e) - n, int(e)),) for e, n in zip(ends, lengths)]


def _compare(got, ref, size, name, state=False):
    got = f64(got)
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    err = np.abs(got - ref)
    bound = 2.0 ** -15 * size if state else R * np.abs(ref) + (2 * R + 2.0 ** -16) * size
    assert np.all(err <= bound + 1e-30), f"{name}: {err.max():.3e} (|ref| {np.abs(ref).max():.3e})"
    if ref.size >= 1000 and np.linalg.norm(ref) > 0:
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= (1e-5 if state else 5e-3), f"{name}: relative error {rel:.2e}"


def _check(t, g, lengths, packed, N, scale=None, ragged=True, seqs=None):
    """Forward and backward of the library against the oracle, sequence by sequence."""
    Bd = _bd()
    q, k, v, do, s0, e = (t[x] for x in ("q", "k", "v", "do", "state", "dstate"))
    d = q.shape[-1]
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    if packed:
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).cuda()
        where = {"cu_seqlens": cu, "max_seqlen": N}
    else:
        where = {"lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda") if ragged else None}
    want_state = s0 is not None
    o, fin = Bd.linear_fwd(q, k, v, g.cuda(), state=s0, return_state=want_state, scale=scale, **where)
    grads = Bd.linear_bwd(q, k, v, do, g.cuda(), state=s0, dstate=e, scale=scale, **where)
    assert Bd.get_status() == 0
    assert (fin is None) == (grads[3] is None) == (not want_state)
    gn = g.double().numpy()
    for b, at in enumerate(_places(lengths, packed)):
        if seqs is not None and b not in seqs:
            continue
        x = [f64(y[at]) for y in (q, k, v, do)]
        st = [None if y is None else f64(y[b]) for y in (s0, e)]
        ax, ast = [np.abs(y) for y in x], [None if y is None else np.abs(y) for y in st]
        ro, rs = OL.forward(*x[:3], gn, sc, st[0])
        mo, ms = OL.forward(*ax[:3], gn, abs(sc), ast[0])
        _compare(o[at], ro, mo, f"o[{b}]")
        rg, mg = OL.backward(*x, gn, sc, *st), OL.backward(*ax, gn, abs(sc), *ast)
        for n, y, r, m in zip(("dq", "dk", "dv"), grads, rg, mg):
            _compare(y[at], r, m, f"{n}[{b}]")
        if want_state:
            _compare(fin[b], rs, ms, f"state[{b}]", state=True)
            _compare(grads[3][b], rg[3], mg[3], f"dstate[{b}]", state=True)
    if not packed:
        for b, n in enumerate(lengths):
            for y in (o, *grads[:3]):
                assert torch.all(y[b, n:] == 0)
    return (o, fin) + tuple(grads)


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[1], [128], [129, 1, 0, 127], [300, 2, 256, 255, 130]])
def test_padded_and_packed(lengths, d, state):
    N, H = max(lengths), 2
    t = _make((len(lengths), N), H, d, len(lengths), state, seed=d + len(lengths))
    pad = _check(t, _slopes(H), lengths, False, N)
    p = {n: (torch.cat([t[n][b, :x] for b, x in enumerate(lengths)]) if n in ("q", "k", "v", "do") else t[n]) for n in t}
    pk = _check(p, _slopes(H), lengths, True, N)
    # the same chunks: the same values to the last bit
    for i, (a, b) in enumerate(zip(pad, pk)):
        if a is not None and i in (0, 2, 3, 4):
            a = torch.cat([a[j, :x] for j, x in enumerate(lengths)])
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("g", [0.0, 0.5, float("nan"), -float("inf"), -60.0, -3.0, -1e-4])
@pytest.mark.parametrize("d", [64, 128])
def test_decays(g, d):
    t = _make((2, 260), 2, d, 2, True, seed=5)
    _check(t, torch.tensor([g, -0.1]), [260, 133], False, 260)


@pytest.mark.parametrize("g", [-1.38, -1.39])  # lambda a little above and below 1/4
def test_large_scores_and_steep_decays(g):
    """Scores of 2^66 and more against weights down to lambda^127: no product overflows on its
    way to a finite output."""
    t = _make((1, 300), 1, 64, 1, False, seed=30)
    t["q"], t["k"] = t["q"] * 2.0 ** 32, t["k"] * 2.0 ** 32
    _check(t, torch.full((1,), g), [300], False, 300, scale=2.0 ** -64)


@pytest.mark.parametrize("scale", [1.0, -0.5, 0.0])
def test_scales(scale):
    t = _make((1, 150), 1, 64, 1, True, seed=6)
    _check(t, _slopes(1), [150], False, 150, scale=scale)


@pytest.mark.parametrize("d", [64, 128])
def test_few_long_sequences_are_split(d):
    """Fewer items than SMs: segments with their own starting states, some sequences shorter
    than one segment, one empty."""
    Bd = _bd()
    assert Bd.linear_workspace_bytes(3, 2500, 2, d) > 0
    assert Bd.linear_workspace_bytes(64, 2500, 16, d) == 0
    t = _make((3, 2500), 2, d, 3, True, seed=7)
    _check(t, torch.tensor([-0.002, -0.3]), [2500, 0, 700], False, 2500)
    t["state"] = t["dstate"] = None
    _check(t, torch.tensor([-0.002, -0.3]), [2433, 128, 640], False, 2500)


@pytest.mark.parametrize("d", [64, 128])
def test_many_items_per_cta(d):
    """More items than SMs, no lengths given, and batches past the sorted size."""
    t = _make((60, 140), 4, d, 60, False, seed=8)
    _check(t, _slopes(4), [140] * 60, False, 140, ragged=False, seqs=[0, 31, 59])
    ln = [(7 * i) % 70 for i in range(600)]
    t = _make((600, 70), 1, d, 600, True, seed=9)
    _check(t, _slopes(1), ln, False, 70, seqs=[0, 1, 9, 300, 599])


def test_pads_may_hold_anything():
    Bd = _bd()
    for d in (64, 128):
        t = _make((2, 200), 2, d, 2, True, seed=10)
        g = _slopes(2).cuda()
        ln = torch.tensor([131, 0], dtype=torch.int32, device="cuda")
        run = lambda: Bd.linear_fwd(t["q"], t["k"], t["v"], g, lengths=ln, state=t["state"], return_state=True) + \
            Bd.linear_bwd(t["q"], t["k"], t["v"], t["do"], g, lengths=ln, state=t["state"], dstate=t["dstate"])
        clean = run()
        for n in ("q", "k", "v", "do"):
            t[n][0, 131:] = float("nan")
            t[n][1] = float("inf")
        assert all(torch.equal(a, b) for a, b in zip(clean, run()))
        # an empty sequence hands its state on
        assert torch.equal(clean[1][1], t["state"][1]) and torch.equal(clean[5][1], t["dstate"][1])


def test_packed_writes_only_its_rows_and_clamps():
    """Rows behind the last sequence stay as they were and may hold NaN; views of wider
    tensors; offsets past the tensor's rows are cut there."""
    Bd = _bd()
    ln, H, d = [70, 0, 200], 2, 64
    T = 300
    base = _make((T,), H, d, 3, False, seed=11)
    for n in ("q", "k", "v", "do"):
        base[n][270:] = float("nan")
    wide = {n: torch.full((T, H, 3, d), 5.0, dtype=torch.bfloat16, device="cuda") for n in ("q", "k", "v", "do", "o", "dq", "dk", "dv")}
    for n in ("q", "k", "v", "do"):
        wide[n][:, :, 1] = base[n]
    v = {n: x[:, :, 1] for n, x in wide.items()}
    cu = torch.tensor([0, 70, 70, 270], dtype=torch.int32, device="cuda")
    g = _slopes(H).cuda()
    Bd.linear_fwd(v["q"], v["k"], v["v"], g, cu_seqlens=cu, max_seqlen=200, out=v["o"])
    Bd.linear_bwd(v["q"], v["k"], v["v"], v["do"], g, cu_seqlens=cu, max_seqlen=200, dq=v["dq"], dk=v["dk"], dv=v["dv"])
    assert Bd.get_status() == 0
    for n in ("o", "dq", "dk", "dv"):
        assert torch.all(wide[n][:, :, 0] == 5) and torch.all(wide[n][:, :, 2] == 5) and torch.all(v[n][270:] == 5)
        assert torch.all(torch.isfinite(v[n]))
    t = {n: base[n][:270].contiguous() for n in ("q", "k", "v", "do")}
    t["state"] = t["dstate"] = None
    want = _check(t, _slopes(H), ln, True, 200)
    for a, n in ((want[0], "o"), (want[2], "dq"), (want[3], "dk"), (want[4], "dv")):
        assert torch.equal(a, v[n][:270])
    bad = torch.tensor([-5, 70, 40, 1 << 30], dtype=torch.int32, device="cuda")
    o = torch.full((270, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    Bd.linear_fwd(t["q"], t["k"], t["v"], g, cu_seqlens=bad, max_seqlen=200, out=o)
    # offsets that break the rules stay inside the tensor: sequences [0, 70), none, and from 40
    # (two sequences then write rows 40 .. 69) the longest allowed, 200 rows, to 240
    assert Bd.get_status() == 0 and torch.equal(o[:40], want[0][:40]) and torch.all(o[240:] == 5)


def test_state_buffers_in_place():
    """The final state may take the place of the starting one; the backward's three passes read
    the states that they are given, so its dstate_out may not, and no call takes a part."""
    Bd = _bd()
    for B, N in ((2, 200), (100, 150), (1, 1500)):
        t = _make((B, N), 2, 64, B, True, seed=12)
        g = _slopes(2).cuda()
        o, fin = Bd.linear_fwd(t["q"], t["k"], t["v"], g, state=t["state"], return_state=True)
        s = t["state"].clone()
        o2, fin2 = Bd.linear_fwd(t["q"], t["k"], t["v"], g, state=s, final_state=s)
        assert fin2 is s and torch.equal(o, o2) and torch.equal(fin, fin2)
        for kw in (dict(dstate_out=t["dstate"]), dict(dstate_out=t["state"])):
            with pytest.raises(Bd.SigattnError) as e:
                Bd.linear_bwd(t["q"], t["k"], t["v"], t["do"], g, state=t["state"], dstate=t["dstate"], **kw)
            assert e.value.code == -1
        two = torch.zeros(2 * t["state"].numel(), device="cuda")
        n = t["state"].numel()
        part = lambda at: two[at:at + n].view_as(t["state"])
        with pytest.raises(Bd.SigattnError):
            Bd.linear_fwd(t["q"], t["k"], t["v"], g, state=part(0), final_state=part(n // 2))
        with pytest.raises(Bd.SigattnError):
            Bd.linear_step(t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], g, part(0), state_out=part(n // 2))
        Bd.linear_fwd(t["q"], t["k"], t["v"], g, state=part(0), final_state=part(n))
    assert Bd.get_status() == 0


def test_shared_heads_are_read_through_zero_strides():
    """One key head for all query heads, as an expanded view: its gradient comes out per head,
    the sum over the heads is the shared one's."""
    Bd = _bd()
    t = _make((2, 150), 3, 64, 2, False, seed=20)
    one = t["k"][:, :, :1].contiguous()
    wide = one.expand(-1, -1, 3, -1)
    g = _slopes(3).cuda()
    a = Bd.linear_fwd(t["q"], wide, t["v"], g)[0]
    b = Bd.linear_fwd(t["q"], wide.contiguous(), t["v"], g)[0]
    assert torch.equal(a, b)
    ga = Bd.linear_bwd(t["q"], wide, t["v"], t["do"], g)
    gb = Bd.linear_bwd(t["q"], wide.contiguous(), t["v"], t["do"], g)
    assert all(torch.equal(x, y) for x, y in zip(ga[:3], gb[:3])) and ga[1].shape == wide.shape
    assert Bd.get_status() == 0


def test_without_tokens():
    Bd = _bd()
    g = _slopes(2).cuda()
    s, e = torch.randn(3, 2, 64, 64, device="cuda"), torch.randn(3, 2, 64, 64, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    where = dict(cu_seqlens=cu, max_seqlen=1)
    o, fin = Bd.linear_fwd(q, q, q, g, state=s, return_state=True, **where)
    *_, ds = Bd.linear_bwd(q, q, q, q, g, state=s, dstate=e, **where)
    assert o.shape == q.shape and torch.equal(fin, s) and torch.equal(ds, e)
    assert torch.all(Bd.linear_fwd(q, q, q, g, return_state=True, **where)[1] == 0)
    assert Bd.linear_step(q, q, q, g, s[:0]).shape == q.shape


def test_packed_rows_of_no_sequence_alone():
    """max_seqlen = 0, all sequences empty: the states go through, the rows stay as they are."""
    Bd = _bd()
    g = _slopes(2).cuda()
    s = torch.randn(3, 2, 64, 64, device="cuda")
    q = torch.randn(5, 2, 64, device="cuda").to(torch.bfloat16)
    where = dict(cu_seqlens=torch.zeros(4, dtype=torch.int32, device="cuda"), max_seqlen=0)
    out = torch.full_like(q, 7.0)
    _, fin = Bd.linear_fwd(q, q, q, g, state=s, return_state=True, out=out, **where)
    *_, ds = Bd.linear_bwd(q, q, q, q, g, state=s, dstate=s, **where)
    assert torch.equal(fin, s) and torch.equal(ds, s) and torch.all(out == 7.0)
    with pytest.raises(Bd.SigattnError):
        Bd.linear_fwd(q, q, q, g, cu_seqlens=where["cu_seqlens"], max_seqlen=-1)


def test_workspace_on_another_stream():
    """A call given its stream keeps its workspace until it has run there, whatever the current
    stream allocates meanwhile."""
    Bd = _bd()
    t = _make((1, 3000), 2, 128, 1, True, seed=21)
    g = _slopes(2).cuda()
    want = Bd.linear_fwd(t["q"], t["k"], t["v"], g, state=t["state"], return_state=True)
    need = Bd.linear_workspace_bytes(1, 3000, 2, 128)
    assert need > 0
    side = torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for i in range(8):
        out, fin = torch.empty_like(want[0]), torch.empty_like(want[1])
        Bd.linear_fwd(t["q"], t["k"], t["v"], g, state=t["state"], out=out, final_state=fin,
                      stream=side if i % 2 else side.cuda_stream)
        torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        outs.append((out, fin))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


@pytest.mark.parametrize("B,N,d", [(40, 300, 64), (2, 3000, 128)])
def test_same_results_on_other_streams_and_in_graphs(B, N, d):
    Bd = _bd()
    t = _make((B, N), 2, d, B, True, seed=13)
    ln = torch.tensor([N - 3 * b for b in range(B)], dtype=torch.int32, device="cuda")
    g = _slopes(2).cuda()
    run = lambda: Bd.linear_fwd(t["q"], t["k"], t["v"], g, lengths=ln, state=t["state"], return_state=True) + \
        Bd.linear_bwd(t["q"], t["k"], t["v"], t["do"], g, lengths=ln, state=t["state"], dstate=t["dstate"])
    want = run()
    same = lambda x: all(torch.equal(a, b) for a, b in zip(want, x))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    again = run()  # at the same time on the current stream
    torch.cuda.synchronize()
    assert same(got) and same(again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(2):
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out)
    assert Bd.get_status() == 0


@pytest.mark.parametrize("B,H,d", [(1, 1, 64), (3, 5, 64), (2, 16, 128), (70, 4, 128)])
def test_step(B, H, d):
    Bd = _bd()
    t = _make((B,), H, d, B, True, seed=14)
    g = _slopes(H)
    g[0] = -float("inf")
    ln = [b % 3 for b in range(B)]
    ln[0] = 1
    lt = torch.tensor(ln, dtype=torch.int32, device="cuda")
    new = torch.full_like(t["state"], 9.0)
    o = Bd.linear_step(t["q"], t["k"], t["v"], g.cuda(), t["state"], lengths=lt, state_out=new)
    for b in range(B):
        if ln[b] == 0:
            assert torch.all(o[b] == 0) and torch.equal(new[b], t["state"][b])
            continue
        x = [f64(t[n][b])[None] for n in ("q", "k", "v")]
        st = f64(t["state"][b])
        ro, rs = OL.forward(*x, g.double().numpy(), 1 / math.sqrt(d), st)
        mo, ms = OL.forward(*map(np.abs, x), g.double().numpy(), 1 / math.sqrt(d), np.abs(st))
        assert np.all(np.abs(f64(o[b]) - ro[0]) <= R * np.abs(ro[0]) + 2.0 ** -18 * mo[0])
        assert np.all(np.abs(f64(new[b]) - rs) <= 2.0 ** -20 * ms)
    # in place, and q / k / v / o as slices of one projection
    wide = torch.full((B, 4, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    for i, n in enumerate(("q", "k", "v")):
        wide[:, i] = t[n]
    s = t["state"].clone()
    o2 = Bd.linear_step(wide[:, 0], wide[:, 1], wide[:, 2], g.cuda(), s, lengths=lt, out=wide[:, 3])
    assert torch.equal(o2, o) and torch.equal(s, new)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_then_tokens(d):
    """A prompt's state carried on token by token gives what the whole sequence gives."""
    Bd = _bd()
    B, n, extra, H = 2, 140, 4, 2
    t = _make((B, n + extra), H, d, B, False, seed=15)
    g = _slopes(H)
    whole = _check(t, g, [n + extra] * B, False, n + extra)[0]
    cut = lambda x: t[x][:, :n]
    o, s = Bd.linear_fwd(cut("q"), cut("k"), cut("v"), g.cuda(), return_state=True)
    steps = [Bd.linear_step(*(t[x][:, n + i] for x in ("q", "k", "v")), g.cuda(), s) for i in range(extra)]
    for b in range(B):
        x = [f64(t[y][b]) for y in ("q", "k", "v")]
        ro, _ = OL.forward(*x, g.double().numpy(), 1 / math.sqrt(d))
        mo, _ = OL.forward(*map(np.abs, x), g.double().numpy(), 1 / math.sqrt(d))
        _compare(o[b], ro[:n], mo[:n], "prompt")
        for i, y in enumerate(steps):
            # the state comes from the chunks (2^-15 M) and the step adds its own rounding
            assert np.all(np.abs(f64(y[b]) - ro[n + i]) <= R * np.abs(ro[n + i]) + 2.0 ** -14 * mo[n + i])
    assert whole.shape == (B, n + extra, H, d)


@pytest.mark.parametrize("N,d", [(400, 64), (3000, 128)])
def test_timeout_is_reported_and_leaves_the_next_call_sound(N, d):
    """With a limit of 1 ns the kernels' waits give up, record it and end; nothing hangs."""
    Bd = _bd()
    t = _make((2, N), 2, d, 2, True, seed=16)
    g = _slopes(2).cuda()
    run = lambda: Bd.linear_fwd(t["q"], t["k"], t["v"], g, state=t["state"], return_state=True) + \
        Bd.linear_bwd(t["q"], t["k"], t["v"], t["do"], g, state=t["state"], dstate=t["dstate"])
    want = run()
    assert Bd.get_status() == 0
    Bd.set_wait_limit_ns(1)
    run()
    assert Bd.get_status() == -6
    Bd.set_wait_limit_ns(500_000_000)
    got = run()
    assert Bd.get_status() == 0 and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("attention", ["linear", "sigmoid"])
def test_together(attention):
    """One layer's path on a packed batch of documents: norm and rotation of q and k, causal
    linear attention (or sigmoid attention over the same rows), and all gradients back to the
    projections and the weights.  Each stage is held to the oracle on that stage's inputs."""
    Bd = _bd()
    ln, H, d = [150, 1, 77], 2, 64
    T = sum(ln)
    t = _make((T,), H, d, 3, False, seed=17)
    gen = torch.Generator().manual_seed(18)
    wq, wk = (1 + 0.2 * torch.randn(2, d, generator=gen)).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in ln]).cuda()
    inv = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).cuda()
    rope = dict(positions=pos, inv_freq=inv)
    yq, yk = Bd.qk_norm_rope(t["q"], t["k"], wq, wk, **rope)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(ln)]).astype(np.int32)).cuda()
    if attention == "linear":
        u = {"q": yq, "k": yk, "v": t["v"], "do": t["do"], "state": None, "dstate": None}
        o, _, dyq, dyk, dv, _ = _check(u, _slopes(H), ln, True, max(ln))
    else:
        plan = Bd.Plan.from_cu_seqlens(cu, max(ln))
        o, _ = Bd.fwd(plan, yq, yk, t["v"])
        dyq, dyk, dv = Bd.bwd(plan, yq, yk, t["v"], o, t["do"])
    dq, dk, dwq, dwk = Bd.qk_norm_rope_bwd(t["q"], t["k"], dyq, dyk, wq, wk, **rope)
    assert Bd.get_status() == 0
    ang = OQ.angles(pos.cpu().numpy()[None], f64(inv), [d // 2])
    for x, dy, w, dx, dw in ((t["q"], dyq, wq, dq, dwq), (t["k"], dyk, wk, dk, dwk)):
        rdx, rdw = OQ.backward(f64(x), f64(dy), f64(w), 1e-6, ang)
        assert np.abs(f64(dx) - rdx).max() <= R * np.abs(rdx).max() + 2.0 ** -14 * np.abs(f64(dy)).max()
        assert np.linalg.norm(f64(dw) - rdw) <= 1e-5 * np.linalg.norm(rdw)
    assert torch.all(torch.isfinite(dv))
