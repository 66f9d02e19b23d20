"""The norm over packed buffers with more rows than their sequences: lengths of one entry, the
last offset, says how many are valid.  What the others hold does not matter, NaN included."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (128, 96, True), (64, 0, False)])
@pytest.mark.parametrize("n", [0, 1, 333, 500])
def test_rows_behind_the_count_add_nothing(n, d, rot, interleaved):
    from padded_variable_length_b200 import binding as Bd
    T, H = 500, 3
    g = torch.Generator().manual_seed(n + d)
    q, k, dyq, dyk = (torch.randn(T, H, d, generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    wq, wk = (1 + 0.2 * torch.randn(2, d, generator=g)).cuda()
    rope, cut = {}, {}
    if rot:
        pos = torch.randint(0, 4000, (T,), generator=g, dtype=torch.int32).cuda()
        rope = dict(positions=pos, interleaved=interleaved,
                    inv_freq=10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot).cuda())
        cut = dict(rope, positions=pos[:n])
    # the same rows alone; a batch of no rows gives weight gradients of 0
    want = Bd.qk_norm_rope(q[:n], k[:n], wq, wk, **cut) + \
        Bd.qk_norm_rope_bwd(q[:n], k[:n], dyq[:n], dyk[:n], wq, wk, **cut)
    cu = torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")
    for x in (q, k, dyq, dyk):
        x[n:] = float("nan")
    got = Bd.qk_norm_rope(q, k, wq, wk, lengths=cu[-1:], **rope) + \
        Bd.qk_norm_rope_bwd(q, k, dyq, dyk, wq, wk, lengths=cu[-1:], **rope)
    for a, b in zip(want[:4], got[:4]):
        assert torch.equal(a, b[:n]) and torch.all(b[n:] == 0)
    for a, b, x, dy in zip(want[4:], got[4:], (q, k), (dyq, dyk)):
        # other rows to a block, so sums in another order: each is off by 2^-18 at most of the
        # sum over the rows of max |dy| |u| (see test_qknorm_gpu.py)
        x, dy = x[:n].double(), dy[:n].double()
        u = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        size = (dy.abs().amax(-1, keepdim=True) * u.abs()).sum((0, 1))
        assert torch.all((a - b).abs() <= 2.0 ** -17 * size)
    with pytest.raises(ValueError):
        Bd.qk_norm_rope(q, k, lengths=cu)


def test_sigmoid_attention_over_a_buffer_with_spare_rows():
    """The attention kernels write no row of no sequence: with the count, the norm's gradients
    take none of them up either."""
    from padded_variable_length_b200 import binding as Bd
    T, H, d, n = 400, 2, 64, 277
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(T, H, d, generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    cu = torch.tensor([0, 100, 100, n], dtype=torch.int32, device="cuda")
    plan = Bd.Plan.from_cu_seqlens(cu, 177)
    grads = []
    for rest in (0.0, float("nan")):
        for x in (q, k, v, do):
            x[n:] = rest
        yq, yk = Bd.qk_norm_rope(q, k, w, w, lengths=cu[-1:])
        o, _ = Bd.fwd(plan, yq, yk, v)
        torch.cuda.synchronize()
        out = [torch.full_like(q, float("nan")) for _ in range(3)]
        Bd.bwd(plan, yq, yk, v, o, do, dq=out[0], dk=out[1], dv=out[2])
        grads.append(Bd.qk_norm_rope_bwd(q, k, out[0], out[1], w, w, lengths=cu[-1:]))
    assert Bd.get_status() == 0
    for a, b in zip(*grads):
        assert torch.all(torch.isfinite(a)) and torch.equal(a, b)
