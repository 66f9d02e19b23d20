"""Packed buffers with more rows than their sequences have: before the first offset, behind the
last, behind a sequence longer than max_seqlen.  What linear attention allocates is 0 there, and
its gradients go on into the norm's weight gradients; what the caller gives stays as it was."""
import numpy as np
import pytest
import torch

from oracle import qknorm as OQ

pytestmark = pytest.mark.gpu


def _bd():
    from padded_variable_length_b200 import binding as Bd
    Bd.set_wait_limit_ns(500_000_000)
    return Bd


def _make(T, H, d, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, H, d, generator=g).to(torch.bfloat16).cuda() for _ in range(4)]


def _leave_nan(like, n):
    """Freed memory of n tensors like this one, full of NaN."""
    torch.cuda.synchronize()
    junk = [torch.full_like(like, float("nan")) for _ in range(n)]
    del junk


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,cu,longest,H", [
    (700, [30, 130, 130, 400, 560], 200, 3),      # before, behind, and a sequence of 270 cut at 200
    (6000, [10, 1500], 1490, 2),                  # one sequence in segments, a long rest
    (5000, [0, 2000, 2000, 4100], 2000, 1),       # segments, and a cut by the second's length
    (300, [300, 300], 5, 2),                      # all rows before the only sequence, an empty one
    (64, [0, 0, 0], 9, 2),                        # no rows in any sequence
    (40, [0, 17, 40], 23, 200)])                  # no rest, many items
def test_new_outputs_are_zero_in_rows_of_no_sequence(T, cu, longest, H, d):
    Bd = _bd()
    q, k, v, do = _make(T, H, d, seed=T + d)
    g = torch.linspace(-0.5, -0.01, H).cuda()
    where = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_seqlen=longest)
    covered = torch.zeros(T, dtype=torch.bool)
    for a, b in zip(cu, cu[1:]):
        covered[a:min(b, a + longest)] = True
    for x in (q, k, v, do):
        x[~covered] = float("nan")
    given = [torch.full_like(q, 5.0) for _ in range(4)]
    Bd.linear_fwd(q, k, v, g, out=given[0], **where)
    Bd.linear_bwd(q, k, v, do, g, dq=given[1], dk=given[2], dv=given[3], **where)
    _leave_nan(q, 4)
    new = [Bd.linear_fwd(q, k, v, g, **where)[0]]
    new += Bd.linear_bwd(q, k, v, do, g, **where)[:3]
    assert Bd.get_status() == 0
    for a, b in zip(given, new):
        assert torch.all(a[~covered] == 5.0) and torch.all(b[~covered] == 0)
        assert torch.equal(a[covered], b[covered]) and torch.all(torch.isfinite(b))
    # some given, some new
    dk = torch.full_like(q, 5.0)
    _leave_nan(q, 2)
    dq, _, dv, _ = Bd.linear_bwd(q, k, v, do, g, dk=dk, **where)
    assert torch.all(dk[~covered] == 5.0) and torch.equal(dq, new[1]) and torch.equal(dv, new[3])


def test_no_sequence_has_a_token():
    """max_seqlen = 0."""
    Bd = _bd()
    q, k, v, do = _make(50, 2, 64, seed=1)
    g = torch.full((2,), -0.1, device="cuda")
    where = dict(cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda"), max_seqlen=0)
    _leave_nan(q, 4)
    assert torch.all(Bd.linear_fwd(q, k, v, g, **where)[0] == 0)
    dk = torch.full_like(q, 5.0)
    dq, _, dv, _ = Bd.linear_bwd(q, k, v, do, g, dk=dk, **where)
    assert torch.all(dq == 0) and torch.all(dv == 0) and torch.all(dk == 5.0)


def test_gradients_go_on_into_the_weights():
    """linear_bwd, then the norm's gradients over the whole buffer: the rest adds nothing.  dw is
    held as in the norm's own tests: 2^-18 of the sum of max |dy| |u| over the rows."""
    Bd = _bd()
    T, H, d, cu = 500, 2, 64, [0, 150, 333]
    q, k, v, do = _make(T, H, d, seed=2)
    g = torch.full((H,), -0.1, device="cuda")
    wq, wk = (1 + 0.2 * torch.randn(2, d, generator=torch.Generator().manual_seed(3))).cuda()
    where = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_seqlen=200)
    yq, yk = Bd.qk_norm_rope(q, k, wq, wk)
    _leave_nan(q, 3)
    dyq, dyk, _, _ = Bd.linear_bwd(yq, yk, v, do, g, **where)
    dq, dk, dwq, dwk = Bd.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk)
    for x, dy, w, dx, dw in ((q, dyq, wq, dq, dwq), (k, dyk, wk, dk, dwk)):
        xs, gs, ws = (t.detach().cpu().double().numpy() for t in (x[:333], dy[:333], w))
        _, ref = OQ.backward(xs, gs, ws, 1e-6)
        u = np.abs(xs) / np.sqrt(np.mean(xs * xs, -1, keepdims=True) + 1e-6)
        size = (np.abs(gs).max(-1, keepdims=True) * u).reshape(-1, d).sum(0)
        assert np.all(np.abs(dw.cpu().double().numpy() - ref) <= 2.0 ** -18 * size)
        assert torch.all(dx[333:] == 0)
