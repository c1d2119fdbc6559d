"""Outputs so large that a block of the adapters' second product has several tiles
of columns (that these sizes do is tested in test_adapter_grids.py), every
element against the 64-bit forms and under the tolerances of test_adapter_gpu.py.
"""

import pytest

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402
from test_adapter_gpu import OFFSET, SEED, Pool, check_backward, check_forward, make_slots, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


# ranks of every width, columns that end in a tile's middle, in fewer than eight
# of it, and with it; two to eight tiles to a block; rows in runs, mixed, absent
FORWARD = [
    # M, K, N, R, L, slots, add, p
    (2100, 64, 8201, 24, 3, "random", True, 0.0),
    (2100, 96, 8201, 64, 1, None, True, 0.1),
    (2117, 64, 8192, 128, 4, "runs", False, 0.0),
    (2053, 64, 8195, 33, 2, "other", False, 0.3),
    (4111, 64, 8195, 16, 3, "runs", True, 0.2),
    (4100, 32, 8704, 64, 70, "random", True, 0.0),
    (8200, 64, 8197, 48, 4, "runs", True, 0.0),
    (16500, 32, 8199, 7, 2, "random", True, 0.0),
]
BACKWARD = [
    (2100, 8224, 72, 24, 3, "random", True, 0.1),
    (2100, 8224, 65, 64, 1, None, True, 0.0),
    (2117, 8192, 72, 128, 4, "runs", False, 0.2),
    (2100, 8224, 7, 17, 2, "other", True, 0.3),
    (4111, 8704, 40, 16, 3, "runs", True, 0.2),
    (4100, 8224, 64, 64, 4, "runs", True, 0.05),
    (8200, 4128, 64, 128, 2, "random", False, 0.0),
]


@pytest.mark.parametrize("M,K,N,R,L,kind,add,p", FORWARD)
def test_forward_of_several_tiles(M, K, N, R, L, kind, add, p):
    P, x, slots = Pool(11, L, R, N, K), randn(1, M, K), make_slots(kind, M, L)
    base = randn(2, M, N) if add else None
    drop = dict(p=p, seed=SEED, offset=OFFSET)
    y, hidden = wq.adapters(x, *P.args, slots=slots, base=base, save_hidden=True, **drop)
    check_forward(P, x, slots, base, p, y, hidden, "forward")
    if add:
        wq.adapters(x, *P.args, slots=slots, base=base, out=base, **drop)
        assert torch.equal(base, y)


@pytest.mark.parametrize("M,K,N,R,L,kind,add,p", BACKWARD)
def test_backward_of_several_tiles(M, K, N, R, L, kind, add, p):
    P, x, slots = Pool(21, L, R, N, K), randn(3, M, K), make_slots(kind, M, L)
    dy, hidden = randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    add = randn(6, M, K, sigma=0.1) if add else None
    drop = dict(p=p, seed=SEED, offset=OFFSET)
    got = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, dx_add=add, **drop)
    check_backward(P, dy, x, hidden, slots, add, p, *got, "backward")
    if add is not None:
        wq.adapters_backward(dy, None, None, *P.args, slots=slots, dx_add=add, out=add, need_weights=False, **drop)
        assert torch.equal(add, got[0])
