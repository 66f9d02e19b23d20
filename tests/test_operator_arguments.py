"""Refusals of the query / key norm and of linear attention, without a device: the C entry
points answer bad arguments before any CUDA call, the binding raises before it calls in."""
import ctypes

import pytest
import torch

from padded_variable_length_b200 import binding as Bd

P, S3, S2 = ctypes.c_void_p, ctypes.c_int64 * 3, ctypes.c_int64 * 2
INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3
OKS = S3(512, 64, 64)


def _qk(B=2, N=8, Hq=2, Hk=2, d=64, q=P(16), qs=OKS, k=P(16), norm=1, eps=1e-6, rot=32, il=0, axes=1, sec=(16,),
        inv=P(16), pos=P(16), sa=0, sb=8, yq=P(16), yk=P(16)):
    c = None if sec is None else (ctypes.c_int32 * len(sec))(*sec)
    return Bd.lib.sigattn_qk_norm_rope(B, N, Hq, Hk, d, None, q, qs, k, OKS, None, None, norm, eps, rot, il, axes, c,
                                       inv, pos, sa, sb, yq, OKS, yk, OKS, None)


@pytest.mark.parametrize("kw,code", [
    ({"B": 0}, INVALID), ({"N": 0}, INVALID), ({"Hq": -1}, INVALID), ({"Hq": 0, "Hk": 0}, INVALID), ({"q": None}, INVALID),
    ({"k": None}, INVALID), ({"yq": None}, INVALID), ({"norm": 2}, INVALID), ({"eps": -1.0}, INVALID),
    ({"eps": float("nan")}, INVALID), ({"rot": -16}, INVALID), ({"il": 2}, INVALID), ({"d": 96}, UNSUPPORTED),
    ({"rot": 24}, UNSUPPORTED), ({"rot": 80}, UNSUPPORTED), ({"sec": (15,)}, INVALID), ({"sec": (17, -1), "axes": 2}, INVALID),
    ({"sec": None}, INVALID), ({"axes": 0}, INVALID), ({"axes": 5, "sec": (4, 3, 3, 3, 3)}, UNSUPPORTED), ({"inv": None}, INVALID),
    ({"pos": None}, INVALID), ({"sa": -1}, INVALID), ({"q": P(8)}, ALIGNMENT), ({"qs": S3(512, 60, 64)}, ALIGNMENT),
    ({"qs": S3(-512, 64, 64)}, INVALID), ({"B": 1 << 20, "N": 1 << 20}, UNSUPPORTED), ({"yk": P(24)}, ALIGNMENT)])
def test_qk_norm_rope_refuses(kw, code):
    assert _qk(**kw) == code


def test_qk_norm_rope_bwd_refuses():
    n = ctypes.c_size_t()
    size = Bd.lib.sigattn_qk_norm_rope_bwd_workspace_size
    assert size(2, 8, 64, ctypes.byref(n)) == 0 and n.value == 2 * 2 * 64 * 4
    assert size(2, 8, 64, None) == INVALID and size(0, 8, 64, ctypes.byref(n)) == INVALID
    assert size(2, 8, 80, ctypes.byref(n)) == UNSUPPORTED

    def call(dy=P(16), dq=P(16), dw=P(16), ws=P(16), nb=1 << 20):
        return Bd.lib.sigattn_qk_norm_rope_bwd(2, 8, 2, 0, 64, None, P(16), OKS, None, OKS, dy, OKS, None, OKS, P(16),
                                               None, 1, 1e-6, 0, 0, 0, None, None, None, 0, 0, dq, OKS, None, OKS, dw,
                                               None, ws, nb, None)
    assert call(dy=None) == INVALID and call(dq=None) == INVALID
    assert call(ws=None) == INVALID and call(nb=16) == INVALID and call(ws=P(8)) == ALIGNMENT


def _fwd(B=2, N=8, T=0, H=2, d=64, ln=None, cu=None, g=P(16), scale=1.0, q=P(16), qs=OKS, s=None, o=P(16), f=None,
         ws=None, nb=0):
    return Bd.lib.sigattn_linear_fwd(B, N, T, H, d, ln, cu, g, scale, q, qs, P(16), OKS, P(16), OKS, s, o, OKS, f, ws,
                                     nb, None)


@pytest.mark.parametrize("kw,code", [
    ({"B": 0}, INVALID), ({"N": 0}, INVALID), ({"H": 0}, INVALID), ({"cu": P(16), "T": 0}, INVALID), ({"g": None}, INVALID),
    ({"scale": float("inf")}, INVALID), ({"ln": P(16), "cu": P(16), "T": 9}, INVALID), ({"q": None}, INVALID),
    ({"o": None}, INVALID), ({"d": 32}, UNSUPPORTED), ({"B": 1 << 20, "H": 1 << 10}, UNSUPPORTED), ({"q": P(24)}, ALIGNMENT),
    ({"qs": S3(512, 64, 4)}, ALIGNMENT), ({"qs": S3(0, -64, 64)}, INVALID), ({"s": P(20)}, ALIGNMENT), ({"f": P(20)}, ALIGNMENT),
    ({"N": 4096}, INVALID), ({"N": 4096, "ws": P(16), "nb": 64}, INVALID), ({"N": 4096, "ws": P(8), "nb": 1 << 40}, ALIGNMENT)])
def test_linear_fwd_refuses(kw, code):
    assert _fwd(**kw) == code


def test_linear_bwd_and_step_refuse():
    def bwd(N=8, do=P(16), dk=P(16), s=None, e=None, ds=None, ws=None, nb=0):
        return Bd.lib.sigattn_linear_bwd(2, N, 0, 2, 64, None, None, P(16), 1.0, P(16), OKS, P(16), OKS, P(16), OKS, do,
                                         OKS, s, e, P(16), OKS, dk, OKS, P(16), OKS, ds, ws, nb, None)
    assert bwd(do=None) == INVALID and bwd(dk=None) == INVALID and bwd(N=4096) == INVALID
    assert bwd(s=P(4)) == ALIGNMENT and bwd(e=P(4)) == ALIGNMENT and bwd(ds=P(4)) == ALIGNMENT

    def step(B=2, H=2, d=64, g=P(16), scale=1.0, q=P(2), s2=S2(1, 1), st=P(16), so=P(16), o=P(2)):
        return Bd.lib.sigattn_linear_step(B, H, d, None, g, scale, q, s2, P(2), S2(1, 1), P(2), S2(1, 1), st, so, o,
                                          S2(1, 1), None)
    for kw in ({"B": 0}, {"H": 0}, {"g": None}, {"scale": float("nan")}, {"q": None}, {"st": None}, {"so": None}, {"o": None},
               {"s2": S2(-1, 1)}):
        assert step(**kw) == INVALID
    assert step(d=96) == UNSUPPORTED and step(B=1 << 20, H=1 << 20) == UNSUPPORTED
    assert step(st=P(8)) == ALIGNMENT and step(so=P(8)) == ALIGNMENT


def test_workspace_goes_by_the_items():
    for back, passes in ((False, 1), (True, 3)):
        assert Bd.linear_workspace_bytes(64, 16384, 16, 128, back) == 0   # enough items
        assert Bd.linear_workspace_bytes(1, 512, 1, 128, back) == 0       # too short to split
        n = Bd.linear_workspace_bytes(1, 16384, 2, 128, back)
        assert n > 0 and n % (passes * 2 * 128 * 128 * 4) == 0
    for bad in ((0, 8, 2, 64), (2, 0, 2, 64), (2, 8, 0, 64), (2, 8, 2, 80)):
        with pytest.raises(Bd.SigattnError):
            Bd.linear_workspace_bytes(*bad)


def test_binding_refuses_before_calling():
    q = torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16)
    g = torch.zeros(2)
    with pytest.raises(ValueError):  # not on a GPU
        Bd.qk_norm_rope(q, q)
    with pytest.raises(ValueError):
        Bd.qk_norm_rope(None, None)
    with pytest.raises(ValueError):
        Bd.qk_norm_rope(q.float(), None)
    with pytest.raises(ValueError):
        Bd.linear_fwd(q, q, q, g)
    with pytest.raises(ValueError):
        Bd.linear_fwd(q.float(), q, q, g)
    with pytest.raises(ValueError):
        Bd.linear_step(q[:, 0], q[:, 0], q[:, 0], g, torch.zeros(2, 2, 64, 64))
    with pytest.raises(ValueError):
        Bd.linear_step(q, q, q, g, torch.zeros(2, 2, 64, 64))


@pytest.mark.parametrize("same", ["q", "k", "v"])
def test_linear_output_that_is_an_input_is_refused(same):
    at = {n: P(1 << 20 | i << 12) for i, n in enumerate(("q", "k", "v", "do", "dq", "dk", "dv"))}
    t = lambda n: (at[n], OKS)
    assert Bd.lib.sigattn_linear_fwd(2, 8, 0, 2, 64, None, None, P(16), 1.0, *t("q"), *t("k"), *t("v"), None, at[same], OKS,
                                     None, None, 0, None) == INVALID
    assert Bd.lib.sigattn_linear_step(2, 2, 64, None, P(16), 1.0, at["q"], S2(1, 1), at["k"], S2(1, 1), at["v"], S2(1, 1),
                                      P(16), P(16), at[same], S2(1, 1), None) == INVALID
    for out in ("dq", "dk", "dv"):
        for other in (same, "do", *({"dq", "dk", "dv"} - {out})):
            outs = [at[other] if n == out else at[n] for n in ("dq", "dk", "dv")]
            assert Bd.lib.sigattn_linear_bwd(2, 8, 0, 2, 64, None, None, P(16), 1.0, *t("q"), *t("k"), *t("v"), *t("do"), None,
                                             None, outs[0], OKS, outs[1], OKS, outs[2], OKS, None, None, 0, None) == INVALID
