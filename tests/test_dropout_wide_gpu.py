"""Dropout of tensors so large that a thread takes four eights, every element
against the 64-bit form and under the tolerances of test_adapter_gpu.py.
"""

import pytest

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402
from test_adapter_gpu import E32, OFFSET, SEED, U, keep_of, randn  # noqa: E402
from test_block_gpu import near  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


SWITCH = 8 * 256 * 2048   # elements up to which a thread takes one eight


@pytest.mark.parametrize("shape", [(SWITCH,), (SWITCH + 1,), (SWITCH + 7,), (SWITCH + 8,), (SWITCH + 8192,),
                                   (SWITCH + 3 * 8192 - 8,), (2049, 2053), (3, 1000, 2001)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.9])
def test_dropout_of_four_eights(shape, p):
    x, r = randn(1, *shape), randn(2, *shape)
    keep = keep_of(shape, p)
    ref = x.double() * keep
    y = wq.dropout(x, p, SEED, OFFSET)
    near(y, ref, U * ref.abs() * (1 + 2 ** -9) + 2.0 ** -25, "dropout")
    assert not y[keep == 0].any()
    assert torch.equal(wq.dropout_backward(x, p, SEED, OFFSET), y)
    z = wq.dropout(x, p, SEED, OFFSET, residual=r)
    sum64 = ref + r.double()
    near(z, sum64, U * sum64.abs() * (1 + 2 ** -9) + 4 * E32 * (ref.abs() + sum64.abs()) + 2.0 ** -25, "residual")
    r2, x2 = r.clone(), x.clone()
    assert wq.dropout(x, p, SEED, OFFSET, residual=r2, out=r2) is r2 and torch.equal(r2, z)
    assert torch.equal(wq.dropout(x2, p, SEED, OFFSET, residual=r, out=x2), z)
    assert torch.equal(wq.dropout(x, p, SEED, OFFSET, out=x), y)


def test_four_eights_leave_the_neighbours_alone():
    n, pad = SWITCH + 8197, 64
    buf = torch.full((n + 2 * pad,), 7.0, device="cuda").half()
    x = randn(1, n)
    wq.dropout(x, 0.3, SEED, OFFSET, out=buf[pad:pad + n])
    assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()
    assert torch.equal(buf[pad:pad + n], wq.dropout(x, 0.3, SEED, OFFSET))
