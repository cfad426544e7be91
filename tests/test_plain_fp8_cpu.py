"""The plain 64-bit forms of the 8-bit calls against torch's own casts and
hand-worked values (CPU)."""
import pytest
import torch

import plain_fp8 as plain


@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_round8_is_the_cast(fmt, dtype):
    top = plain.FORMATS[fmt][0]
    x = torch.cat([torch.randn(20000) * 3, torch.randn(5000) * 1e-3, torch.randn(5000) * 100,
                   torch.tensor([0.0, top, -top, 2.0 ** -9, 3 * 2.0 ** -10, 2.0 ** -17])])
    x = x.clamp(-top, top)
    assert torch.equal(plain.round8(x.double(), fmt), x.to(dtype).double())


def test_scale_by_hand():
    a = torch.tensor([448.0, 449.0, 447.0, 224.0, 0.0, 1e-44, float("inf"), float("nan")],
                     dtype=torch.float64)
    s = plain.scale_of(a, "e4m3")
    assert s[:4].tolist() == [1.0, 2.0, 1.0, 0.5]
    assert s[4:6].tolist() == [2.0 ** -119] * 2 and torch.isnan(s[6:]).all()
    assert plain.scale_of(torch.tensor([57344.0, 57345.0], dtype=torch.float64), "e5m2").tolist() == [1.0, 2.0]


def test_groups_by_hand():
    x = torch.zeros(130, 129)
    x[0, 0], x[129, 128], x[1, 128] = 448.0, 896.0, 3.0
    q, s = plain.quantize(x, "e4m3", 1)
    assert s.shape == (130, 2) and s[0, 0] == 1 and s[129, 1] == 2 and q[129, 128] == 448
    q, s = plain.quantize(x, "e4m3", 0)
    assert s.shape == (2, 129) and s[0, 0] == 1 and s[1, 128] == 2
    q, s = plain.quantize_block(x, "e4m3")
    assert s.tolist()[0][0] == 1 and s.tolist()[1][1] == 2 and s.shape == (2, 2)
    assert torch.equal(plain.block_value(q, s), x.double())
    assert torch.equal(plain.rows_value(*(lambda a, b: (a, b.T))(*plain.quantize(x, "e4m3", 1))), x.double())
