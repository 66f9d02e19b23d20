"""One layer's path with sigmoid attention, packed: norm and rotation of q and k, attention, and
all gradients back to the projections and the weights.  Each stage is held to its float64 oracle
on that stage's own inputs: the norm by test_qknorm_gpu.py's bounds (2^-8 of the value and 2^-20
of its row's size; 2^-18 of the summed sizes for the weights), attention by the bound of all of
its tests (harness.check_close)."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import qknorm as OQ
from tests import harness as Hn
from tests.test_qknorm_gpu import _close_rows, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[150, 1, 77], [300, 0, 129, 256]])
@pytest.mark.parametrize("d,interleaved", [(64, False), (128, True)])
def test_norm_attention_and_gradients(lengths, d, interleaved):
    from padded_variable_length_b200 import binding as Bd
    Bd.set_wait_limit_ns(500_000_000)
    T, H = sum(lengths), 2
    gen = torch.Generator().manual_seed(T + d)
    q, k, v, do = (torch.randn(T, H, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(4))
    wq, wk = (1 + 0.2 * torch.randn(2, d, generator=gen)).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths]).cuda()
    inv = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).cuda()
    rope = dict(positions=pos, inv_freq=inv, interleaved=interleaved)
    ends = np.cumsum([0] + lengths)
    cu = torch.from_numpy(ends.astype(np.int32)).cuda()
    plan = Bd.Plan.from_cu_seqlens(cu, max(lengths))
    bias = Bd.bias_from_counts(torch.cat([torch.full((n,), n, dtype=torch.int32) for n in lengths]).cuda())

    yq, yk = Bd.qk_norm_rope(q, k, wq, wk, **rope)
    o, _ = Bd.fwd(plan, yq, yk, v, bias)
    dyq, dyk, dv = Bd.bwd(plan, yq, yk, v, o, do, bias)
    dq, dk, dwq, dwk = Bd.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, **rope)
    assert Bd.get_status() == 0

    ang = OQ.angles(pos.cpu().numpy()[None], f64(inv), [d // 2])
    for x, dy, w, y, dx, dw, name in ((q, dyq, wq, yq, dq, dwq, "q"), (k, dyk, wk, yk, dk, dwk, "k")):
        xs, gs, ws = f64(x), f64(dy), f64(w)
        z = OQ.forward(xs, ws, 1e-6)
        _close_rows(y, OQ.forward(xs, ws, 1e-6, ang, interleaved), np.abs(z).max(-1, keepdims=True), "y" + name)
        rdx, rdw = OQ.backward(xs, gs, ws, 1e-6, ang, interleaved)
        r = 1 / np.sqrt(np.mean(xs * xs, -1, keepdims=True) + 1e-6)
        most = np.abs(gs).max(-1, keepdims=True)
        _close_rows(dx, rdx, 4 * r * np.abs(ws).max() * most * np.maximum(1, np.abs(xs * r).max(-1, keepdims=True)) ** 2, "d" + name)
        assert np.all(np.abs(f64(dw) - rdw) <= 2.0 ** -18 * (most * np.abs(xs * r)).reshape(-1, d).sum(0)), name

    sc = 1 / math.sqrt(d)
    for n, at in zip(lengths, ends):
        if n == 0:
            continue
        x = [f64(t[at:at + n])[None] for t in (yq, yk, v, do)]
        b = A.bias_from_counts(np.full((1, n), n))
        ref_o, _ = A.forward(*x[:3], b, sc, A.SIGMOID, lengths=np.array([n]))
        ref = A.backward(*x, b, sc, A.SIGMOID, lengths=np.array([n]))
        for got, want, name in zip((o, dyq, dyk, dv), (ref_o, *ref), ("o", "dyq", "dyk", "dv")):
            Hn.check_close(f64(got[at:at + n])[None], want, name)
