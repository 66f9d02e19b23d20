"""Linear attention (and the norm before it) over layouts and lengths that cut across its chunks
and segments: packed sequences in segments, lengths outside of [0, N], views with heads before
tokens.  Values are held to the float64 oracle by test_linear_gpu.py's check, with its bounds."""
import pytest
import torch

from tests.test_linear_gpu import _check, _make, _slopes

pytestmark = pytest.mark.gpu


def _bd():
    from padded_variable_length_b200 import binding as Bd
    Bd.set_wait_limit_ns(500_000_000)
    return Bd


def _pack(t, lengths):
    return {n: torch.cat([x[b, :m] for b, m in enumerate(lengths)]) if n in ("q", "k", "v", "do") else x for n, x in t.items()}


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[700, 0, 2433, 129], [1, 1155], [0, 0, 1700]])
def test_packed_sequences_in_segments(lengths, d, state):
    """First rows that are no multiple of anything, sequences of fewer segments than others, a
    last chunk in a late segment whose rows border on the next sequence's: the oracle's values,
    and the padded batch's (the same chunks and segments) to the last bit."""
    Bd = _bd()
    N, H, B = max(lengths), 2, len(lengths)
    assert Bd.linear_workspace_bytes(B, N, H, d) > 0 and Bd.linear_workspace_bytes(B, N, H, d, True) > 0
    t = _make((B, N), H, d, B, state, seed=N + d)
    g = torch.tensor([-0.002, -0.3])
    packed = _check(_pack(t, lengths), g, lengths, True, N)
    where = dict(lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    pad = Bd.linear_fwd(t["q"], t["k"], t["v"], g.cuda(), state=t["state"], return_state=state, **where) + \
        Bd.linear_bwd(t["q"], t["k"], t["v"], t["do"], g.cuda(), state=t["state"], dstate=t["dstate"], **where)
    assert Bd.get_status() == 0
    for i, (a, b) in enumerate(zip(pad, packed)):
        if i in (0, 2, 3, 4):
            a = torch.cat([a[j, :x] for j, x in enumerate(lengths)])
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("N,H", [(300, 3), (1400, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_outside_of_the_rows_are_clamped(N, H, d):
    Bd = _bd()
    t = _make((4, N), H, d, 4, True, seed=N + d)
    g = _slopes(H).cuda()

    def run(lengths):
        ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        return Bd.linear_fwd(t["q"], t["k"], t["v"], g, lengths=ln, state=t["state"], return_state=True) + \
            Bd.linear_bwd(t["q"], t["k"], t["v"], t["do"], g, lengths=ln, state=t["state"], dstate=t["dstate"])
    want = run([0, N, 101, N])
    got = run([-(1 << 31), (1 << 31) - 1, 101, N + 1])
    assert Bd.get_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # a single token: below 1 is none, above is one
    step = lambda ln: (lambda s: (Bd.linear_step(t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], g, s,
                                                 lengths=torch.tensor(ln, dtype=torch.int32, device="cuda")), s))(t["state"].clone())
    assert all(torch.equal(a, b) for a, b in zip(step([0, 1, 1, 0]), step([-3, 1 << 30, 2, -(1 << 31)])))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [200, 1500])
def test_views_with_heads_before_tokens(N, d, packed):
    """[B, H, N, d] tensors seen as [B, N, H, d]: the same values as dense ones, and new outputs
    in the inputs' order of dimensions."""
    Bd = _bd()
    B, H = 2, 3
    t = _make((B, N), H, d, B, True, seed=N + d)
    if packed:
        ln = [N, N - 77]
        t = _pack(t, ln)
        where = dict(cu_seqlens=torch.tensor([0, N, 2 * N - 77], dtype=torch.int32, device="cuda"), max_seqlen=N)
    else:
        where = dict(lengths=torch.tensor([N - 130, N], dtype=torch.int32, device="cuda"))
    g = _slopes(H).cuda()
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    turned = lambda x: x.transpose(-3, -2).contiguous().transpose(-3, -2)

    def run(q, k, v, do):
        norm = {n: x for n, x in where.items() if n == "lengths"}
        return Bd.qk_norm_rope(q, k, w, w, **norm) + Bd.qk_norm_rope_bwd(q, k, do, v, w, w, **norm) + \
            Bd.linear_fwd(q, k, v, g, state=t["state"], return_state=True, **where) + \
            Bd.linear_bwd(q, k, v, do, g, state=t["state"], dstate=t["dstate"], **where)
    x = [t[n] for n in ("q", "k", "v", "do")]
    y = [turned(a) for a in x]
    assert all(a.stride() != b.stride() for a, b in zip(x, y))
    want, got = run(*x), run(*y)
    assert Bd.get_status() == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b)
        if a.shape == x[0].shape:
            assert b.stride() == y[0].stride()
    # dense inputs into buffers of the other order, and the other way round
    for src, dst in ((x, y), (y, x)):
        o = torch.empty_like(dst[0])
        Bd.linear_fwd(*src[:3], g, state=t["state"], return_state=True, out=o, **where)
        assert torch.equal(o, want[6])
