"""Calls that wq_adapter.h allows and no other file makes: no slots with a pool of
several, ranks of 1 and 2, a chance that rounds to none, more windows of rows and
more adapters than one launch takes.  References and tolerances of
test_adapter_gpu.py."""

import pytest

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402
from test_adapter_gpu import (E32, OFFSET, SEED, Pool, check_backward, check_forward, keep_of, make_slots,  # noqa: E402
                              randn, split_error)
from test_block_gpu import near  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


def both(P, M, K, N, R, slots, p, add, what):
    x, dy, hidden = randn(1, M, K), randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    base, dx_add = (randn(2, M, N), randn(6, M, K, sigma=0.1)) if add else (None, None)
    drop = dict(p=p, seed=SEED, offset=OFFSET)
    y, h = wq.adapters(x, *P.args, slots=slots, base=base, save_hidden=True, **drop)
    check_forward(P, x, slots, base, p, y, h, what)
    got = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, dx_add=dx_add, **drop)
    check_backward(P, dy, x, hidden, slots, dx_add, p, *got, what)


# (the reference takes a pool's first adapter where there are no slots)
@pytest.mark.parametrize("M,K,N,R,L", [(1, 64, 40, 16, 5), (16, 512, 136, 8, 1000), (7, 96, 7, 3, 4), (70, 256, 130, 24, 3),
                                       (300, 128, 264, 128, 2)])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_no_slots_take_the_first_of_several(M, K, N, R, L, p):
    P = Pool(11, L, R, N, K)
    P.down[1:], P.up[1:] = float("nan"), float("nan")      # nobody's
    x, dy, hidden, base = randn(1, M, K), randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32), randn(2, M, N)
    drop = dict(p=p, seed=SEED, offset=OFFSET)
    y, h = wq.adapters(x, *P.args, base=base, save_hidden=True, **drop)
    check_forward(P, x, None, base, p, y, h, "no slots")
    dx, ddown, dup = wq.adapters_backward(dy, x, hidden, *P.args, dx_add=x, **drop)
    check_backward(P, dy, x, hidden, None, x, p, dx, ddown, dup, "no slots")
    assert not ddown[1:].any() and not dup[1:].any()


@pytest.mark.parametrize("M,K,N,R,L,kind", [(1, 64, 40, 1, 1, None), (3, 4096, 130, 2, 3, "random"), (16, 96, 520, 1, 16, "random"),
                                            (40, 4128, 257, 1, 2, "runs"), (150, 512, 1032, 2, 3, "random"), (9, 64, 3, 1, 2, "random")])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_ranks_of_one_and_two(M, K, N, R, L, kind, p):
    both(Pool(11, L, R, N, K), M, K, N, R, make_slots(kind, M, L), p, True, "small rank")


@pytest.mark.parametrize("M,K,N", [(4, 512, 136), (100, 512, 136)])
def test_a_chance_that_rounds_to_none(M, K, N):
    P, x, dy = Pool(11, 1, 16, N, K), randn(1, M, K), randn(4, M, N)
    p = 2.0 ** -17 * 0.99
    y, h = wq.adapters(x, *P.args, save_hidden=True)
    y2, h2 = wq.adapters(x, *P.args, save_hidden=True, p=p, seed=SEED, offset=OFFSET)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    for a, b in zip(wq.adapters_backward(dy, x, h, *P.args),
                    wq.adapters_backward(dy, x, h, *P.args, p=p, seed=SEED, offset=OFFSET)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind,p", [("runs", 0.0), ("random", 0.1)])
def test_more_windows_than_one_launch_takes(kind, p):
    """65519 windows of 64 rows to a launch of the first product."""
    M, K, N, R, L = 65519 * 64 + 100, 32, 9, 3, 3
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    P, slots = Pool(11, L, R, N, K), make_slots(kind, M, L)
    x, dy = randn(1, M, K), randn(4, M, N, sigma=0.1)
    drop = dict(p=p, seed=SEED, offset=OFFSET)
    y, h = wq.adapters(x, *P.args, slots=slots, save_hidden=True, **drop)
    check_forward(P, x, slots, None, p, y, h, "windows")
    hidden = randn(5, M, R, dtype=torch.float32)
    got = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, **drop)
    check_backward(P, dy, x, hidden, slots, None, p, *got, "windows")
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,p", [(200, 0.0), (40000, 0.2)])
def test_more_adapters_than_one_launch_takes(M, p):
    """32767 adapters to a launch of the gradients (half of them at ranks above 64)."""
    K, N, R, L = 32, 9, 2, 33001
    P, slots = Pool(11, L, R, N, K), make_slots("random", M, L)
    slots[-1], slots[0] = L - 1, 32767
    x, dy, hidden = randn(1, M, K), randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    y, h = wq.adapters(x, *P.args, slots=slots, p=p, seed=SEED, offset=OFFSET, save_hidden=True)
    # y, with each row's own adapter gathered
    used = slots >= 0
    at = slots.clamp(min=0).long()
    xd = x.double() * (keep_of((M, K), p) if p else 1.0) * used.unsqueeze(1)
    down, up, s = P.down[at].double(), P.up[at].double(), P.scales[at].double().unsqueeze(1)
    hd = (down * xd.unsqueeze(1)).sum(2)
    eh = 2 * (K + 64) * E32 * (down * xd.unsqueeze(1)).abs().sum(2) + 4 * E32 * hd.abs()
    near(h, hd, eh + 2.0 ** -149, "hidden")
    ref = s * (hd.unsqueeze(2) * up).sum(1)
    tol = s.abs() * (((eh + split_error(hd, 1)).unsqueeze(2) + 2 * (2 * R + 64) * E32 * hd.abs().unsqueeze(2)) * up.abs()).sum(1)
    near(y, ref, tol + 2.0 ** -11 * 1.01 * ref.abs() + 4 * E32 * ref.abs() + 2.0 ** -25, "y")
    # the gradients of the adapters that occur, summed row by row
    _, ddown, dup = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, p=p, seed=SEED, offset=OFFSET, need_dx=False)
    g = dy.double() * used.unsqueeze(1)
    dh = (up * g.unsqueeze(1)).sum(2)
    first = 2 * (N + 64) * E32 * (up * g.unsqueeze(1)).abs().sum(2)
    most = max(int(torch.bincount(at[used]).max()), 1)
    n = 2 * (2 * most + 64) * E32

    def summed(rows):
        out = torch.zeros(L, *rows.shape[1:], dtype=torch.float64, device="cuda")
        return out.index_add_(0, at[used], rows[used])

    def widest(v):   # the largest of an adapter's rows, a bound of every group of 32's
        out = torch.zeros(L, R, dtype=torch.float64, device="cuda")
        return out.scatter_reduce_(0, at[used].unsqueeze(1).expand(-1, R), v[used].abs(), "amax")[at]

    for got, hh, err, src, what in ((ddown, dh, first, xd, "ddown"), (dup, hidden.double(), 0.0, g, "dup")):
        ref = summed(s.unsqueeze(2) * hh.unsqueeze(2) * src.unsqueeze(1))
        e = 2.0 ** -22 * hh.abs() + 2.0 ** -38 * widest(hh) + err + n * hh.abs()
        tol = summed((s.unsqueeze(2) * e.unsqueeze(2) * src.unsqueeze(1)).abs()) + 8 * E32 * ref.abs()
        near(got, ref, tol + 2.0 ** -149, what)
