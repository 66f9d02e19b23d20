"""Attention kernels whose waits give up on batches so short that the copies' warps have issued
everything before anyone gives up: the copies land before shared memory is left, and calls right
behind are sound."""
import pytest
import torch

from padded_variable_length_b200 import workloads as W
from tests import harness as Hn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[100, 0, 37], [128, 200, 256]])
def test_short_batches_give_up_and_the_next_calls_are_sound(lengths, d):
    from padded_variable_length_b200 import binding as Bd
    Bd.set_wait_limit_ns(500_000_000)

    def calls(lengths, d, seed):
        w = W.padded_workload("short", lengths, H=2, d=d, backward=True, seed=seed, npad=max(lengths))
        t, plan, bias = Hn.device_setup(w, W.tensors(w, with_grad=True))
        q, k, v, do = t["q"], t["k"], t["v"], t["do"]
        o, _ = Bd.fwd(plan, q, k, v, bias)
        so, lse = Bd.fwd(plan, q, k, v, None, W.SOFTMAX)
        runs = [lambda: Bd.fwd(plan, q, k, v, bias)[:1], lambda: Bd.fwd(plan, q, k, v, None, W.SOFTMAX),
                lambda: Bd.bwd(plan, q, k, v, o, do, bias),
                lambda: Bd.bwd(plan, q, k, v, so, do, None, W.SOFTMAX, lse)]
        if d == 64:
            # (dQ is summed by reduce-adds, whose order is free)
            runs.append(lambda: Bd.bwd_fused(plan, q, k, v, o, do, bias)[1:])
        return runs

    runs, others = calls(lengths, d, 1), calls([300, 140], 192 - d, 2)
    want, want_other = [f() for f in runs], [f() for f in others]
    assert Bd.get_status() == 0
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))
    for run in runs:
        for other, w in zip(others, want_other):
            try:
                Bd.set_wait_limit_ns(1)
                run()
            finally:
                Bd.set_wait_limit_ns(500_000_000)
            got = other()
            assert Bd.get_status() in (0, -6)
            assert same(got, w)
    for run, w in zip(runs, want):
        got = run()
        assert Bd.get_status() == 0 and same(got, w)
