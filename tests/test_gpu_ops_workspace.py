"""What the operator handles keep on the device."""
import pytest
import torch

from tests import ops_reference as ref
from tests.test_gpu_ops import make_block, make_linear, rows, want_block, want_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def test_a_serving_block_of_few_rows_holds_no_split_sums(pkg):
    op, x, up, gate, _ = make_block(pkg, 16, 512, 16384, "bf16", "swiglu", False)
    assert op.device_bytes() < 4096
    for T in (1, 8, 16):
        want, e, *_ = want_block(x[:T], up, gate, "bf16", "swiglu")
        ref.check(op(x[:T], up, gate), want, e, "bf16", "block")


def test_a_block_holds_one_tile_an_sm_at_most(pkg):
    cfg = pkg.GatedConfig(in_features=4096, out_features=8192, max_tokens=4096)
    assert pkg.GatedBlock(cfg).device_bytes() <= 152 * 128 * 256 * 4 + 4096


def test_a_projection_holds_the_split_sums_of_its_plans(pkg):
    """4096 rows of 4096 x 4096: 9 MB of codes and scales and less than 24 MB beside them."""
    op, _, _, _ = make_linear(pkg, 4096, 4096, "nvfp4", 16, "bf16", "none", False, 4096)
    assert op.device_bytes() < (9 + 24) << 20
    op.close()
    for T in (17, 40, 129, 300):   # splits of K, up to the handle's last row
        op, _, w, _ = make_linear(pkg, 1026, 4096, "affine", 64, "bf16", "none", False, T, seed=2)
        x = rows(T, 4096, "bf16", T)
        want, e = want_linear(x, None, w, None, "affine", 64, "bf16", "none")
        ref.check(op(x), want, e, "bf16", "split")
        assert op.last_launch_count() == 2
        op.close()
