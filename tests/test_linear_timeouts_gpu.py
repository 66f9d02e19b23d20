"""Linear attention whose waits give up: every copy has landed and every arrival has been seen
before a CTA ends, so that whatever runs next in its shared memory is sound.

The calls differ in what is in flight when the first wait gives up: sequences of one chunk and
of fewer chunks than stages, where the copies' warp has issued everything and gone on before
anyone else gives up; longer ones, where it gives up itself; segments, whose states come from
the kernel without outputs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _calls(Bd, B, N, H, d, packed, state):
    g = torch.Generator().manual_seed(B + N + d)
    rows = (B * N,) if packed else (B, N)
    q, k, v, do = (torch.randn(*rows, H, d, generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    s, e = (torch.randn(B, H, d, d, generator=g).cuda() if state else None for _ in range(2))
    decay = -torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).cuda()
    where = {}
    if packed:
        where = {"cu_seqlens": (N * torch.arange(B + 1)).to(torch.int32).cuda(), "max_seqlen": N}
    return lambda: (Bd.linear_fwd(q, k, v, decay, state=s, return_state=state, **where)
                    + Bd.linear_bwd(q, k, v, do, decay, state=s, dstate=e, **where))


@pytest.mark.parametrize("B,N,H,d,packed,state", [
    (2, 100, 2, 64, False, True), (3, 128, 2, 128, True, False), (2, 250, 2, 64, True, True),
    (2, 256, 3, 128, False, False), (90, 200, 2, 64, True, False), (1, 1300, 2, 64, False, True),
    (2, 1600, 1, 128, True, False)])
def test_other_calls_are_sound_after_waits_that_gave_up(B, N, H, d, packed, state):
    from padded_variable_length_b200 import binding as Bd
    Bd.set_wait_limit_ns(500_000_000)
    run = _calls(Bd, B, N, H, d, packed, state)
    others = [_calls(Bd, *x) for x in ((3, 300, 2, 192 - d, False, True), (1, 1200, 1, d, True, False), (160, 40, 1, d, False, False))]
    want = [f() for f in [run] + others]
    assert Bd.get_status() == 0
    same = lambda a, b: all(x is None and y is None or torch.equal(x, y) for x, y in zip(a, b))
    for i, other in enumerate(others):
        try:
            Bd.set_wait_limit_ns(1)
            for _ in range(3):
                run()
        finally:
            Bd.set_wait_limit_ns(500_000_000)
        # right behind, on the same stream: other layouts in the shared memory just left
        got = other()
        assert Bd.get_status() in (0, -6)
        assert same(got, want[1 + i])
    got = run()
    assert Bd.get_status() == 0 and same(got, want[0])
