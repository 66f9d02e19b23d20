"""The norm's outputs may take the place of the tensors that they are computed from, of no other:
the others are refused before any CUDA call (no device needed)."""
import ctypes

import pytest

from padded_variable_length_b200 import binding as Bd

P, S3 = ctypes.c_void_p, ctypes.c_int64 * 3
S, WIDE = S3(512, 64, 64), S3(1024, 128, 64)
AT = {n: P(1 << 20 | i << 16) for i, n in enumerate(("q", "k", "dyq", "dyk", "a", "b"))}
INVALID = -1


def _fwd(yq, yk, ys=S):
    return Bd.lib.sigattn_qk_norm_rope(2, 8, 2, 2, 64, None, AT["q"], S, AT["k"], S, None, None, 1, 1e-6, 0, 0, 0, None, None,
                                       None, 0, 0, AT[yq], ys, AT[yk], S, None)


def _bwd(dq, dk, ys=S):
    return Bd.lib.sigattn_qk_norm_rope_bwd(2, 8, 2, 2, 64, None, AT["q"], S, AT["k"], S, AT["dyq"], S, AT["dyk"], S, None,
                                           None, 1, 1e-6, 0, 0, 0, None, None, None, 0, 0, AT[dq], ys, AT[dk], S, None, None,
                                           None, 0, None)


@pytest.mark.parametrize("yq,yk", [("k", "b"), ("a", "q"), ("a", "a"), ("k", "q")])
def test_forward_refuses(yq, yk):
    assert _fwd(yq, yk) == INVALID


def test_forward_refuses_its_own_place_with_other_strides():
    assert _fwd("q", "b", WIDE) == INVALID


@pytest.mark.parametrize("dq,dk", [("k", "b"), ("dyk", "b"), ("a", "q"), ("a", "dyq"), ("a", "a"), ("dyk", "dyq")])
def test_backward_refuses(dq, dk):
    assert _bwd(dq, dk) == INVALID


@pytest.mark.parametrize("dq", ["q", "dyq"])
def test_backward_refuses_its_own_place_with_other_strides(dq):
    assert _bwd(dq, "b", WIDE) == INVALID
