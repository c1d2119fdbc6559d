"""Neighbouring rows of very different magnitude: every row's h is brought into
fp16's range by itself, whatever its neighbours hold.  Sums of a row do not depend
on the others, so a batch gives the bits of its rows' own calls, and stays within
the tolerances of test_adapter_gpu.py.
"""

import pytest

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402
from test_adapter_gpu import OFFSET, SEED, Pool, check_backward, check_forward, make_slots, randn  # noqa: E402

pytestmark = pytest.mark.gpu

# powers of two that a row is scaled by, in turn, none of them next to its like
FACTORS = [2.0 ** k for k in (0, 10, -12, 13, -6, 7, 13, -13, 3, -10, 12)]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


def scaled_rows(t, first):
    f = [FACTORS[(first + m) % len(FACTORS)] for m in range(t.shape[0])]
    return (t.float() * torch.tensor(f, device="cuda").unsqueeze(1)).half()


# one launch (up to 16 rows, four to an adapter, rank 16, K 4096) and two
SIZES = [(2, 64, 40, 4, 1, None), (4, 4096, 4096, 16, 1, None), (3, 1056, 130, 9, 1, None), (4, 96, 520, 16, 2, "random"),
         (16, 4096, 1032, 16, 4, "runs"), (16, 512, 257, 12, 5, "random"), (13, 2080, 520, 16, 40, "random"),
         (16, 256, 136, 7, 16, "random"), (40, 512, 264, 16, 1, None), (16, 4128, 264, 16, 8, "random"),
         (70, 256, 520, 48, 3, "random"), (150, 128, 130, 128, 2, "runs")]


@pytest.mark.parametrize("M,K,N,R,L,kind", SIZES)
@pytest.mark.parametrize("first", [0, 3])
def test_forward(M, K, N, R, L, kind, first):
    P, x, slots = Pool(11, L, R, N, K), scaled_rows(randn(1, M, K), first), make_slots(kind, M, L)
    P.scales.mul_(0.25)
    y, hidden = wq.adapters(x, *P.args, slots=slots, save_hidden=True)
    check_forward(P, x, slots, None, 0.0, y, hidden, "far rows")
    if M > 16:
        return
    for m in range(M):   # alone
        at = None if slots is None else slots[m:m + 1].clone()
        y1, h1 = wq.adapters(x[m:m + 1].clone(), *P.args, slots=at, save_hidden=True)
        if K <= 4096:    # (otherwise ranges of K may meet in another order)
            assert torch.equal(h1[0], hidden[m]) and torch.equal(y1[0], y[m]), m


@pytest.mark.parametrize("M,K,N,R,L,kind", SIZES)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_dx(M, K, N, R, L, kind, p):
    P, slots = Pool(21, L, R, N, K), make_slots(kind, M, L)
    dy = scaled_rows(randn(4, M, N), 1)
    P.scales.mul_(0.25)
    dx, _, _ = wq.adapters_backward(dy, None, None, *P.args, slots=slots, p=p, seed=SEED, offset=OFFSET, need_weights=False)
    check_backward(P, dy, None, None, slots, None, p, dx, None, None, "far rows")
