"""The linear attention calls that end in _ex refuse zero_rest of outputs that they do not have
(no device needed)."""
import ctypes

import pytest

from padded_variable_length_b200 import binding as Bd

P, S3 = ctypes.c_void_p, ctypes.c_int64 * 3
S = S3(0, 128, 64)


@pytest.mark.parametrize("rest", [2, 4, 3, -1, 8])
def test_forward(rest):
    assert Bd.lib.sigattn_linear_fwd_ex(2, 8, 16, 2, 64, None, P(16), P(16), 1.0, P(16), S, P(32), S, P(48), S, None,
                                        P(64), S, None, rest, None, 0, None) == -1


@pytest.mark.parametrize("rest", [8, 9, -1, 1 << 20])
def test_backward(rest):
    assert Bd.lib.sigattn_linear_bwd_ex(2, 8, 16, 2, 64, None, P(16), P(16), 1.0, P(16), S, P(32), S, P(48), S, P(64), S,
                                        None, None, P(80), S, P(96), S, P(112), S, None, rest, None, 0, None) == -1
