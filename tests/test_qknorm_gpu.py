"""The query / key norm with position rotation against its float64 oracle, forward and
backward.

Tolerances.  An output y (or dx) in bf16 is one rounding, 2^-8 |y|, of a value computed in
fp32: the norm's factor and the weight are relative errors of a few 2^-24, and the rotation
adds a cos and b sin whose factors are off by at most 2^-22, so the fp32 part is below
2^-20 of the row's largest value before it (|z| resp. |r h|, r u mean(h u)).  dw (fp32) sums
products g u over rows, g = a cos t + b sin t of the gradient's pair (a, b): g is off by
2^-22 (|a| + |b|) <= 2^-21 max |dy| of its row whatever it is itself (a and b may cancel, and
in a single row they do: an error relative to |g| cannot be asked), so a product is off by
less than 2^-20 max |dy| |u|, the size summed up below.  Rounding the sums of n values in any
order adds at most n 2^-24 of the sum of sizes and, the errors having either sign, some
sqrt(n) 2^-24: below 2^-18 of it for the n <= 30000 here."""
import numpy as np
import pytest
import torch

from oracle import qknorm as OQ

pytestmark = pytest.mark.gpu

R = 2.0 ** -8
F = 2.0 ** -20


def _bd():
    from padded_variable_length_b200 import binding as Bd
    return Bd


def f64(t):
    return t.detach().cpu().double().numpy()


def _make(B, N, Hq, Hk, d, rot, sections, seed, far=0):
    g = torch.Generator().manual_seed(seed)
    t = {"q": torch.randn(B, N, Hq, d, generator=g) * 2, "k": torch.randn(B, N, Hk, d, generator=g) * 0.3,
         "dyq": torch.randn(B, N, Hq, d, generator=g), "dyk": torch.randn(B, N, Hk, d, generator=g)}
    t = {n: x.to(torch.bfloat16).cuda() for n, x in t.items()}
    t["wq"] = (1 + 0.3 * torch.randn(d, generator=g)).cuda()
    t["wk"] = (1 + 0.3 * torch.randn(d, generator=g)).cuda()
    rope = {}
    if rot:
        pos = torch.randint(-50 if far == 0 else far, 4000 if far == 0 else far + 4000, (len(sections), B, N),
                            generator=g, dtype=torch.int64).to(torch.int32).cuda()
        inv = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
        rope = {"positions": pos, "inv_freq": inv.cuda(), "sections": sections}
    return t, rope


def _angles(rope):
    if not rope:
        return None
    return OQ.angles(rope["positions"].cpu().numpy(), f64(rope["inv_freq"]), rope["sections"])


def _close_rows(got, ref, size, name):
    """|got - ref| <= 2^-8 |ref| + 2^-20 size, size per row."""
    got = f64(got)
    assert np.all(np.isfinite(got)), name
    bad = np.abs(got - ref) - (R * np.abs(ref) + F * size)
    assert bad.max() <= 0, f"{name}: off by {np.abs(got - ref).max():.3e}"


def _check(t, rope, interleaved, lengths, eps=1e-6, norm=True, weights=True):
    Bd = _bd()
    wq, wk = (t["wq"], t["wk"]) if weights else (None, None)
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    yq, yk = Bd.qk_norm_rope(t["q"], t["k"], wq, wk, eps=eps, interleaved=interleaved, lengths=ln, norm=norm, **rope)
    dq, dk, dwq, dwk = Bd.qk_norm_rope_bwd(t["q"], t["k"], t["dyq"], t["dyk"], wq, wk, eps=eps,
                                           interleaved=interleaved, lengths=ln, norm=norm, **rope)
    ang = _angles(rope)
    B, N = t["q"].shape[:2]
    keep = np.ones((B, N), bool) if lengths is None else np.arange(N)[None] < np.array(lengths)[:, None]
    for x, dy, w, y, dx, dw, name in ((t["q"], t["dyq"], wq, yq, dq, dwq, "q"), (t["k"], t["dyk"], wk, yk, dk, dwk, "k")):
        wf = None if w is None else f64(w)
        xs, gs = f64(x)[keep], f64(dy)[keep]
        a = None if ang is None else ang[keep]
        ref = OQ.forward(xs, wf, eps, a, interleaved, norm)
        z = OQ.forward(xs, wf, eps, None, False, norm)
        _close_rows(y[torch.from_numpy(keep)], ref, np.abs(z).max(-1, keepdims=True, initial=0), "y" + name)
        rdx, rdw = OQ.backward(xs, gs, wf, eps, a, interleaved, norm)
        r = 1 / np.sqrt(np.mean(xs * xs, -1, keepdims=True) + eps) if norm else 1.0
        wm = 1.0 if wf is None else np.abs(wf).max()
        size = 4 * r * wm * np.abs(gs).max(-1, keepdims=True, initial=0) * np.maximum(1, np.abs(xs * r).max(-1, keepdims=True, initial=0)) ** 2
        _close_rows(dx[torch.from_numpy(keep)], rdx, size, "d" + name)
        assert torch.all(y[torch.from_numpy(~keep)] == 0) and torch.all(dx[torch.from_numpy(~keep)] == 0)
        if w is None:
            assert dw is None
        else:
            total = (np.abs(gs).max(-1, keepdims=True) * np.abs(xs * r)).reshape(-1, x.shape[-1]).sum(0)
            assert np.all(np.abs(f64(dw) - rdw) <= 2.0 ** -18 * total + 1e-30), name


@pytest.mark.parametrize("d,rot,sections,interleaved", [
    (64, 64, [32], False), (64, 64, [32], True), (128, 128, [64], False), (128, 128, [64], True),
    (64, 32, [5, 11], False), (64, 48, [8, 8, 8], True), (128, 96, [16, 24, 8], False), (128, 16, [2, 2, 2, 2], True),
    (64, 16, [0, 8], False), (128, 112, [56], False), (64, 0, None, False), (128, 0, None, False)])
@pytest.mark.parametrize("heads", [(8, 8), (5, 1), (16, 4)])
def test_matches_oracle(d, rot, sections, interleaved, heads):
    t, rope = _make(3, 37, *heads, d, rot, sections, seed=d + rot + heads[0])
    _check(t, rope, interleaved, [37, 0, 11])


@pytest.mark.parametrize("d", [64, 128])
def test_one_token_and_many(d):
    t, rope = _make(1, 1, 1, 1, d, d, [d // 2], seed=1)
    _check(t, rope, False, None)
    t, rope = _make(2, 5003, 3, 2, d, d, [d // 2], seed=2)
    _check(t, rope, False, [5003, 4999])


@pytest.mark.parametrize("norm,weights,eps", [(True, False, 1e-6), (False, True, 1e-6), (False, False, 0.0), (True, True, 0.5)])
def test_without_norm_or_weights(norm, weights, eps):
    t, rope = _make(2, 19, 4, 2, 64, 64, [32], seed=3)
    _check(t, rope, False, [19, 3], eps=eps, norm=norm, weights=weights)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 5000, -(1 << 31)])
def test_far_positions(far):
    """Positions out to the ends of int32: the oracle's float64 angle p f is itself off by up
    to 2^-53 p f = 2^-22 there, as much as the sines' own error, within the 2^-20 above."""
    t, rope = _make(1, 64, 2, 2, 128, 128, [64], seed=4, far=far)
    _check(t, rope, False, None)


def test_zero_rows():
    """A row of zeros has y = 0, and dx = w g / sqrt(eps)."""
    t, rope = _make(1, 8, 2, 2, 64, 64, [32], seed=5)
    t["q"][:, 3] = 0
    t["k"][:] = 0
    _check(t, rope, False, None)


def test_masked_rows_may_hold_anything():
    Bd = _bd()
    t, rope = _make(2, 9, 4, 4, 64, 64, [32], seed=6)
    ln = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    args = dict(lengths=ln, **rope)
    clean = Bd.qk_norm_rope(t["q"], t["k"], t["wq"], t["wk"], **args)
    gclean = Bd.qk_norm_rope_bwd(t["q"], t["k"], t["dyq"], t["dyk"], t["wq"], t["wk"], **args)
    for n in ("q", "k", "dyq", "dyk"):
        t[n][0, 5:] = float("nan")
        t[n][1] = float("inf")
    dirty = Bd.qk_norm_rope(t["q"], t["k"], t["wq"], t["wk"], **args)
    gdirty = Bd.qk_norm_rope_bwd(t["q"], t["k"], t["dyq"], t["dyk"], t["wq"], t["wk"], **args)
    for a, b in zip(clean + gclean, dirty + gdirty):
        assert torch.equal(a, b)
    # every sequence empty: outputs 0, weight gradients 0
    ln.zero_()
    for x in Bd.qk_norm_rope(t["q"], t["k"], t["wq"], t["wk"], **args) + \
            Bd.qk_norm_rope_bwd(t["q"], t["k"], t["dyq"], t["dyk"], t["wq"], t["wk"], **args):
        assert torch.all(x == 0)


def test_packed_strided_in_place_and_single():
    """Packed tensors as views of a wider projection, outputs written in place, q or k alone."""
    Bd = _bd()
    t, rope = _make(1, 33, 6, 2, 64, 64, [32], seed=7)
    pos = rope.pop("positions")
    want = Bd.qk_norm_rope(t["q"], t["k"], t["wq"], t["wk"], positions=pos, **rope)
    wide = torch.full((33, 10, 64), 7.0, dtype=torch.bfloat16, device="cuda")  # q heads, k heads, v heads
    wide[:, :6], wide[:, 6:8] = t["q"][0], t["k"][0]
    q, k = wide[:, :6], wide[:, 6:8]
    yq, yk = Bd.qk_norm_rope(q, k, t["wq"], t["wk"], positions=pos[:, 0], out_q=q, out_k=k, **rope)
    assert yq.data_ptr() == wide.data_ptr()
    assert torch.equal(wide[:, :6], want[0][0]) and torch.equal(wide[:, 6:8], want[1][0])
    assert torch.all(wide[:, 8:] == 7.0)
    one, none = Bd.qk_norm_rope(t["q"], None, t["wq"], positions=pos[0], **rope)
    assert none is None and torch.equal(one, want[0])
    none, one = Bd.qk_norm_rope(None, t["k"], None, t["wk"], positions=pos, **rope)
    assert none is None and torch.equal(one, want[1])
    # a query broadcast over the batch is read through its zero stride
    q = t["q"].expand(2, -1, -1, -1)
    p2 = pos.expand(1, 2, 33)
    two, _ = Bd.qk_norm_rope(q, None, t["wq"], positions=p2, **rope)
    assert torch.equal(two[0], want[0][0]) and torch.equal(two[1], want[0][0])


def test_weight_gradients_do_not_change_from_run_to_run():
    Bd = _bd()
    t, rope = _make(4, 3001, 8, 8, 64, 64, [32], seed=8)
    a = Bd.qk_norm_rope_bwd(t["q"], t["k"], t["dyq"], t["dyk"], t["wq"], t["wk"], **rope)
    for _ in range(3):
        b = Bd.qk_norm_rope_bwd(t["q"], t["k"], t["dyq"], t["dyk"], t["wq"], t["wk"], **rope)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_other_stream_and_captured():
    Bd = _bd()
    t, rope = _make(2, 50, 4, 4, 128, 128, [64], seed=9)
    run = lambda: Bd.qk_norm_rope(t["q"], t["k"], t["wq"], t["wk"], **rope) + \
        Bd.qk_norm_rope_bwd(t["q"], t["k"], t["dyq"], t["dyk"], t["wq"], t["wk"], **rope)
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    q0 = t["q"].clone()
    t["q"].mul_(2)
    want2 = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want2, out))
    t["q"].copy_(q0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
