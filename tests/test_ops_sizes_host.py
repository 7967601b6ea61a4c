"""Sizes that do not fit the C interface's 32-bit fields are refused, not cut (no GPU needed)."""

import pytest

import quantized_moe_decode_gemv_gb300 as pkg
from tests.test_ops_streams_host import Tensor, linear

WIDE = 2 ** 32 + 256


@pytest.mark.parametrize("field", ["in_features", "out_features", "group_size", "max_tokens"])
def test_linear_config(field):
    kw = dict(in_features=256, out_features=96, group_size=64, max_tokens=4)
    pkg.QLinearConfig(**kw).to_c()
    for v in (WIDE, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(pkg.MoEError) as err:
            pkg.QLinearConfig(**{**kw, field: v}).to_c()
        assert err.value.status == 1
    with pytest.raises(TypeError):
        pkg.QLinearConfig(**{**kw, field: 64.0}).to_c()


@pytest.mark.parametrize("field", ["in_features", "out_features", "max_tokens"])
def test_gated_config(field):
    kw = dict(in_features=256, out_features=96, max_tokens=4)
    pkg.GatedConfig(**kw).to_c()
    for v in (WIDE, 2 ** 31):
        with pytest.raises(pkg.MoEError) as err:
            pkg.GatedConfig(**{**kw, field: v}).to_c()
        assert err.value.status == 1


def test_rows():
    op = linear()
    op.forward(Tensor(3, 64))
    with pytest.raises(pkg.MoEError) as err:
        op.forward(Tensor(2 ** 32 + 3, 64))
    assert err.value.status == 1
