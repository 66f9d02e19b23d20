"""Calls of the query / key norm and of linear attention that are given a stream: all they do is
in that stream's order, while the current stream is busy with work that it was given before."""
import pytest
import torch

pytestmark = pytest.mark.gpu

WAIT = 100_000_000  # cycles, some 50 ms


def _bd():
    from padded_variable_length_b200 import binding as Bd
    Bd.set_wait_limit_ns(500_000_000)
    return Bd


def _bf(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _handle(side, raw):
    return side.cuda_stream if raw else side


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_states_pass_in_the_streams_order_without_tokens(packed, raw):
    """The states of a call without tokens are written by the side stream just before it."""
    Bd = _bd()
    side = torch.cuda.Stream()
    if packed:
        q = _bf(5, 2, 64)
        where = dict(cu_seqlens=torch.zeros(4, dtype=torch.int32, device="cuda"), max_seqlen=0)
    else:
        q, where = torch.empty(3, 0, 2, 64, dtype=torch.bfloat16, device="cuda"), {}
    g = torch.full((2,), -0.1, device="cuda")
    s, e, fin, ds = (torch.zeros(3, 2, 64, 64, device="cuda") for _ in range(4))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
        s.fill_(3.0)
        e.fill_(5.0)
    Bd.linear_fwd(q, q, q, g, state=s, final_state=fin, stream=_handle(side, raw), **where)
    Bd.linear_bwd(q, q, q, q, g, state=s, dstate=e, dstate_out=ds, stream=_handle(side, raw), **where)
    side.synchronize()
    assert torch.all(fin == 3.0) and torch.all(ds == 5.0)


def test_weight_gradients_without_rows_are_zero_on_the_stream():
    Bd = _bd()
    side = torch.cuda.Stream()
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    seen = torch.ones(64, device="cuda")
    torch.full((64,), float("nan"), device="cuda")  # memory that the gradient could be given
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    dw = Bd.qk_norm_rope_bwd(q, None, q, None, w, stream=side)[2]
    with torch.cuda.stream(side):
        seen.copy_(dw)
    side.synchronize()
    assert torch.all(seen == 0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op", ["norm", "norm_bwd", "linear", "linear_bwd", "step"])
def test_new_outputs_are_not_in_memory_that_the_current_stream_still_writes(op, raw):
    """The current stream has writes to freed buffers of the outputs' sizes ahead of it."""
    Bd = _bd()
    side = torch.cuda.Stream()
    g = torch.full((2,), -0.1, device="cuda")
    x = [_bf(2, 300, 2, 64, seed=i) for i in range(4)]
    y = [_bf(64, 2, 64, seed=i) for i in range(3)]
    s, new = torch.randn(2, 64, 2, 64, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    call = {"norm": lambda **kw: Bd.qk_norm_rope(x[0], x[1], w, w, **kw),
            "norm_bwd": lambda **kw: Bd.qk_norm_rope_bwd(*x, w, w, **kw),
            "linear": lambda **kw: Bd.linear_fwd(*x[:3], g, return_state=True, **kw),
            "linear_bwd": lambda **kw: Bd.linear_bwd(*x, g, **kw)[:3],
            "step": lambda **kw: (Bd.linear_step(*y, g, s, state_out=new, **kw),)}[op]
    want = call()
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    junk = [torch.empty_like(t) for t in want]
    for t in junk:
        t.fill_(7.0)
    del junk, t
    got = call(stream=_handle(side, raw))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert Bd.get_status() == 0


def test_inputs_are_kept_until_the_stream_has_read_them():
    Bd = _bd()
    side = torch.cuda.Stream()
    x = _bf(4, 500, 2, 64)
    want = Bd.qk_norm_rope(x)[0]
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    Bd.qk_norm_rope(x, out_q=out, stream=side)
    size = x.shape
    del x
    other = torch.full(size, 9.0, dtype=torch.bfloat16, device="cuda")  # the current stream is idle
    side.synchronize()
    assert torch.equal(out, want) and torch.all(other == 9.0)
