"""What a handle of the orthogonalised update holds, against what its header says."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def pad(n):
    return (n + 31) // 32 * 32


def stated(n, rows, cols):
    """(bytes without K splits, most with them)"""
    m, sms = min(rows, cols), torch.cuda.get_device_properties(0).multi_processor_count
    x = n * (4 * rows + 2 * pad(rows)) * pad(cols)
    a = n * (4 * m * pad(m) + 8 * pad(m) + 12)
    sums = 12 * min(n * -(-rows * -(-cols // 8) // 1024), 8 * sms + n)
    small = 64 + 4 * 3 * 8 * sms      # the status word and the splits' counters
    return x + a + sums + small, x + a + sums + small + 3 * 2 * 4 * 128 * 128 * sms


@pytest.mark.parametrize("n,rows,cols", [(65536, 16, 16), (5000, 64, 64), (300, 200, 300), (1, 64, 256), (1, 1024, 4096), (1, 7168, 2048),
                                         (3, 512, 300), (1, 8192, 4096), (20, 1000, 1000)])
def test_a_handle_holds_what_is_stated(pkg, n, rows, cols):
    op = pkg.Orthogonalizer(pkg.OrthoConfig(rows=rows, cols=cols, max_matrices=n))
    without, most = stated(n, rows, cols)
    assert op.device_bytes() <= (without if n >= 300 else most)    # (many matrices: no splits)
    op.close()


@pytest.mark.parametrize("rows,cols,sizes", [(40, 24, (700, 1, 152, 33)), (300, 520, (70, 1, 9, 64, 2)), (256, 136, (2000, 1, 3, 1216, 500))])
def test_norms_of_fewer_matrices_than_the_handle_holds(pkg, rows, cols, sizes):
    """The partial sums of a call lie where its number of matrices puts them."""
    most = max(sizes)
    g = torch.randn(most, rows, cols, device="cuda") * torch.logspace(-6, 6, most, device="cuda")[:, None, None]
    op = pkg.Orthogonalizer(pkg.OrthoConfig(rows=rows, cols=cols, max_matrices=most, dtype="fp32", steps=1, coefficients=(1.0, 0.0, 0.0),
                                            eps=0.0))
    want = g.double() / g.double().flatten(1).norm(dim=1)[:, None, None]
    for n in sizes:
        got = op(g[most - n:])
        # the identity: what is left is X, rounded once; sums of squares by chains of at most 64 additions,
        # 2^-19 after the root, the factor in two fp32 parts, X's two terms 2^-22: below 2^-18
        assert ((got.double() - want[most - n:]).abs() <= (2.0 ** -8 + 2.0 ** -18) * want[most - n:].abs() + 2.0 ** -36).all()
    assert op.device_status() == 0
