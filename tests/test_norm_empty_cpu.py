"""No tokens: arrays over tokens may be null (an empty tensor has no address), whatever
the norms have besides; checked without a GPU, as far as the search for one."""
import ctypes

import pytest

from test_fp8_norm_refusals_cpu import OK_PTR, arr, b  # noqa: F401  (b: the fixture)


@pytest.mark.parametrize("gate_rows", [0, 4])
@pytest.mark.parametrize("eight", [False, True])
def test_forward(b, gate_rows, eight):  # noqa: F811
    d = b.make_norm_params(0, 512, b.NORM_KINDS["rms"], b.NORM_KINDS["rms"], gate_rows, 2)
    none = arr(None, None)
    status = b.library().tpmlp_norm_forward(
        ctypes.byref(d), none, none, OK_PTR, None, None, OK_PTR, None, none, None if eight else none, None,
        None, None, None)
    assert status != b.TPMLP_ERR_INVALID_ARG
    # what does not go by tokens is still looked at
    status = b.library().tpmlp_norm_forward(
        ctypes.byref(d), none, none, None, None, None, OK_PTR, None, none, None if eight else none, None,
        None, None, None)
    assert status == b.TPMLP_ERR_INVALID_ARG
