"""Calls of the norm and of linear attention that their documentation allows and that nothing
else makes: tokens and batch entries that share memory, one tensor as all inputs, values at the
ends of the types, a stream given inside a graph capture, a longest sequence far past the rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _bd():
    from padded_variable_length_b200 import binding as Bd
    Bd.set_wait_limit_ns(500_000_000)
    return Bd


def _bf(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _linear(Bd, q, k, v, do, g, **kw):
    return Bd.linear_fwd(q, k, v, g, **kw)[:1] + Bd.linear_bwd(q, k, v, do, g, **kw)[:3]


@pytest.mark.parametrize("N", [70, 1300])
@pytest.mark.parametrize("shared", [0, 1, 2, (0, 1), (0, 1, 2)])
def test_inputs_that_share_memory(shared, N):
    """A zero stride along batch entries (0), tokens (1), heads (2)."""
    Bd = _bd()
    shape, dims = (2, N, 3, 64), shared if isinstance(shared, tuple) else (shared,)
    one = _bf(*(1 if i in dims else n for i, n in enumerate(shape)), seed=1).expand(shape)
    q, v, do = (_bf(*shape, seed=i) for i in (2, 3, 4))
    g = torch.full((3,), -0.05, device="cuda")
    for place in range(3):
        wide, dense = [q, q, v, do], [q, q, v, do]
        wide[place], dense[place] = one, one.contiguous()
        got, want = _linear(Bd, *wide, g), _linear(Bd, *dense, g)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    a, b = Bd.qk_norm_rope(one, q), Bd.qk_norm_rope(one.contiguous(), q)
    assert torch.equal(a[0], b[0]) and a[0].shape == shape
    a, b = Bd.qk_norm_rope_bwd(one, q, one, do), Bd.qk_norm_rope_bwd(one.contiguous(), q, one.contiguous(), do)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert Bd.get_status() == 0


def test_one_tensor_as_every_input():
    Bd = _bd()
    x, g = _bf(2, 300, 2, 64, seed=5), torch.full((2,), -0.05, device="cuda")
    got, want = _linear(Bd, x, x, x, x, g), _linear(Bd, *(x.clone() for _ in range(4)), g)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and Bd.get_status() == 0


def test_longest_sequence_far_past_the_rows():
    """max_seqlen only bounds: the plan of segments goes by it, the values by the lengths."""
    Bd = _bd()
    q, k, v, do = (_bf(500, 2, 64, seed=i) for i in range(4))
    g = torch.full((2,), -0.05, device="cuda")
    cu = torch.tensor([0, 200, 500], dtype=torch.int32, device="cuda")
    want = _linear(Bd, q, k, v, do, g, cu_seqlens=cu, max_seqlen=300)
    for longest in (301, 100_000, (1 << 31) - 257):
        got = _linear(Bd, q, k, v, do, g, cu_seqlens=cu, max_seqlen=longest)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and Bd.get_status() == 0
    with pytest.raises(Bd.SigattnError):
        Bd.linear_fwd(q, k, v, g, cu_seqlens=cu, max_seqlen=(1 << 31) - 1)


def test_norm_at_the_ends_of_the_types():
    Bd = _bd()
    x = _bf(4, 2, 64, seed=6)
    x[0] = 0
    x[1] = 1e19  # its squares pass fp32
    x[2] = x[2] * 1e15
    x[3] = x[3] * 1e-30
    y = Bd.qk_norm_rope(x)[0].double()
    assert torch.all(y[:2] == 0)
    ref = x[2:].double() / (x[2:].double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
    assert torch.all((y[2:] - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * ref.abs().amax(-1, keepdim=True))
    y = Bd.qk_norm_rope(x, eps=0.0)[0]
    assert torch.all(torch.isnan(y[0])) and not torch.any(torch.isnan(y[2]))


def test_stream_given_inside_a_capture():
    """The capture's own stream, and one forked off it, by object and by handle."""
    Bd = _bd()
    q, k, v, do = (_bf(2, 1300, 2, 64, seed=i) for i in range(4))
    g, w = torch.full((2,), -0.05, device="cuda"), torch.ones(64, device="cuda")

    def run(stream):
        y = Bd.qk_norm_rope(q, k, w, w, stream=stream)
        o, s = Bd.linear_fwd(y[0], y[1], v, g, return_state=True, stream=stream)
        grads = Bd.linear_bwd(y[0], y[1], v, do, g, stream=stream)[:3]
        return (o, s) + grads + Bd.qk_norm_rope_bwd(q, k, grads[0], grads[1], w, w, stream=stream)
    want = run(None)
    for raw in (False, True):
        own, forked = torch.cuda.Stream(), torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=own):
            here = torch.cuda.current_stream()
            a = run(here.cuda_stream if raw else here)
            forked.wait_stream(here)
            b = run(forked.cuda_stream if raw else forked)
            here.wait_stream(forked)
        for _ in range(2):
            for x in a + b:
                x.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for got in (a, b) for x, y in zip(got, want))
    assert Bd.get_status() == 0
