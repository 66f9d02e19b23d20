"""Attention calls that are given a stream: new outputs and workspaces are in that stream's order,
not in memory that the current stream still writes, and inputs are kept until it has read them."""
import pytest
import torch

from padded_variable_length_b200 import workloads as W
from tests import harness as Hn

pytestmark = pytest.mark.gpu

WAIT = 100_000_000  # cycles, some 50 ms


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op", ["bias", "fwd", "fwd_softmax", "bwd", "bwd_softmax", "bwd_fused"])
def test_new_outputs_are_not_in_memory_that_the_current_stream_still_writes(op, raw):
    from padded_variable_length_b200 import binding as Bd
    w = W.padded_workload("streams", [300, 0, 129], H=2, d=64, backward=True, seed=3, npad=300)
    t, plan, bias = Hn.device_setup(w, W.tensors(w, with_grad=True))
    q, k, v, do = t["q"], t["k"], t["v"], t["do"]
    counts = torch.arange(900, dtype=torch.int32, device="cuda")
    o, _ = Bd.fwd(plan, q, k, v, bias)
    so, lse = Bd.fwd(plan, q, k, v, None, W.SOFTMAX)
    call = {"bias": lambda **kw: (Bd.bias_from_counts(counts, **kw),),
            "fwd": lambda **kw: Bd.fwd(plan, q, k, v, bias, **kw)[:1],
            "fwd_softmax": lambda **kw: Bd.fwd(plan, q, k, v, None, W.SOFTMAX, **kw),
            "bwd": lambda **kw: Bd.bwd(plan, q, k, v, o, do, bias, **kw),
            "bwd_softmax": lambda **kw: Bd.bwd(plan, q, k, v, so, do, None, W.SOFTMAX, lse, **kw),
            # (dQ is summed by reduce-adds, whose order is free)
            "bwd_fused": lambda **kw: Bd.bwd_fused(plan, q, k, v, o, do, bias, **kw)[1:]}[op]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    junk = [torch.empty_like(x) for x in want] + [torch.empty_like(q)]
    for x in junk:
        x.fill_(7.0)
    del junk, x
    got = call(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert Bd.get_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_inputs_are_kept_until_the_stream_has_read_them():
    from padded_variable_length_b200 import binding as Bd
    w = W.padded_workload("streams", [300, 129], H=2, d=64, backward=False, seed=4, npad=300)
    t, plan, bias = Hn.device_setup(w, W.tensors(w, with_grad=False))
    want, _ = Bd.fwd(plan, t["q"], t["k"], t["v"], bias)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    q = t.pop("q")
    Bd.fwd(plan, q, t["k"], t["v"], bias, out=out, stream=side)
    del q
    torch.full_like(want, 9.0)  # the current stream is idle
    side.synchronize()
    assert torch.equal(out, want) and Bd.get_status() == 0
