"""The norm in the place of the tensors it is computed from: the same values as elsewhere."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _bf(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("rows", [(2, 300), (1, 1), (400,)])
def test_in_place(rows):
    from padded_variable_length_b200 import binding as Bd
    q, k, dyq, dyk = (_bf(*rows, 3, 64, seed=i) for i in range(4))
    w = torch.linspace(0.5, 1.5, 64, device="cuda")
    y = Bd.qk_norm_rope(q, k, w, w)
    grads = Bd.qk_norm_rope_bwd(q, k, dyq, dyk, w, w)
    same = lambda a, b: all(torch.equal(s, t) for s, t in zip(a, b))
    for one in (False, True):  # both sides, one side
        x = [t.clone() for t in (q, k)]
        assert same(Bd.qk_norm_rope(*x, w, w, out_q=x[0], out_k=None if one else x[1]), y)
        x = [t.clone() for t in (q, k, dyq, dyk)]
        assert same(Bd.qk_norm_rope_bwd(*x, w, w, dq=x[0], dk=None if one else x[1]), grads)
        x = [t.clone() for t in (q, k, dyq, dyk)]
        assert same(Bd.qk_norm_rope_bwd(*x, w, w, dq=x[2], dk=None if one else x[3]), grads)
    with pytest.raises(Bd.SigattnError):
        Bd.qk_norm_rope(q, k, out_q=k)
    with pytest.raises(Bd.SigattnError):
        Bd.qk_norm_rope_bwd(q, k, dyq, dyk, dk=dyq)
    # one tensor on both sides is read twice; its place is neither's
    both = Bd.qk_norm_rope(q, q, w, w)
    assert torch.equal(both[0], y[0]) and torch.equal(both[1], y[0])
    with pytest.raises(Bd.SigattnError):
        Bd.qk_norm_rope(q, q, w, w, out_q=q)
