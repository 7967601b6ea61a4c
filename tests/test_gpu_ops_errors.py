"""A call that fails leaves nothing behind: the next calls of the library and of
torch run as if it had not been made."""
import pytest
import torch

from tests import ops_reference as ref
from tests.test_gpu_ops import make_linear, rows, want_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def test_no_room_for_a_workspace(pkg):
    """A workspace of 2^56 bytes is refused by the allocator; what follows is not."""
    import moe_inputs as mi
    spec = mi.SPECS["tiny"]
    layer = pkg.MoELayer(pkg.MoEConfig.from_spec(spec, max_tokens=4), pkg.upload_arrays(mi.make_layer(spec, 0).arrays()))
    x = rows(4, spec.hidden, "bf16", 0)
    before = layer(x)
    live = pkg.load_library().moe_debug_live_allocations()
    huge = pkg.GatedConfig(in_features=8, out_features=1 << 24, max_tokens=2 ** 31 - 1, training=True)
    for _ in range(2):
        with pytest.raises(pkg.MoEError) as err:
            pkg.GatedBlock(huge)
        assert err.value.status == 7
        assert pkg.load_library().moe_debug_live_allocations() == live
        assert torch.equal(layer(x), before)
        op, _, w, _ = make_linear(pkg, 96, 256, "affine", 64, "bf16", "none", False, 32)
        y = rows(3, 256, "bf16", 1)
        want, e = want_linear(y, None, w, None, "affine", 64, "bf16", "none")
        ref.check(op(y), want, e, "bf16", "after a failure")
        op.close()
        assert pkg.load_library().moe_debug_live_allocations() == live
    assert torch.ones(4, device="cuda").sum().item() == 4


def test_saved_buffers_that_overlap_are_refused(pkg):
    """C entry: pre-activations kept over x, out, a weight or each other."""
    T, K, N = 20, 64, 64
    op = pkg.GatedBlock(pkg.GatedConfig(in_features=K, out_features=N, max_tokens=T, training=True))
    lib = pkg.load_library()
    buf = torch.zeros(1 << 16, device="cuda")
    at = {n: buf.data_ptr() + 4 * i * 4096 for i, n in enumerate(("x", "out", "gate", "up", "sg", "su"))}

    def call(**other):
        p = {**at, **other}
        return lib.moe_gated_forward(op.handle, p["x"], K, T, p["gate"], p["up"], p["out"], N, p["sg"], p["su"], None)

    assert call() == 0
    for a, b in (("sg", "x"), ("sg", "out"), ("su", "out"), ("su", "up"), ("sg", "gate"), ("su", "gate"), ("su", "sg")):
        assert call(**{a: at[b]}) == 1, (a, b)
    assert call(su=at["sg"] + 4 * T * N) == 0     # one behind the other
    torch.cuda.synchronize()
