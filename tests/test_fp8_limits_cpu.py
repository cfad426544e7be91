"""The largest sizes of the 8-bit linear layers: what the products round up to tiles in 32
bits is taken, what would pass 2^31 is refused."""
import pytest

from test_fp8_norm_refusals_cpu import _linear, b  # noqa: F401  (b: the fixture)

MOST = 2 ** 31 - 256


@pytest.mark.parametrize("split", ["column", "row"])
@pytest.mark.parametrize("which", range(3))
def test_largest_sizes(b, split, which):  # noqa: F811
    def dims(n):
        d = [16, 16, 16]
        d[which] = n
        return b.make_linear_dims(*d, 1)
    size = b.tpmlp_fp8_linear_workspace_bytes
    assert size(dims(MOST)) > 0
    # the next size of its kind, and the largest below 2^31
    for n in ((MOST + 1, 2 ** 31 - 1) if which == 0 else (MOST + 16, 2 ** 31 - 16)):
        assert size(dims(n)) == 0
        for back in (False, True):
            assert _linear(b, split, back, dims=dims(n)) == b.TPMLP_ERR_UNSUPPORTED
