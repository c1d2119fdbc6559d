"""Infinities in the operands that meet h, dh or hidden: up in y, down in dx, x
in ddown, dy in dup.  The formula makes an infinity of the sum's sign of one,
NaN of two of opposite signs and of one beside a zero; the kernels have to make
the same, although they multiply by h in two parts, of which the second may be
zero or of the other sign.

The references are sums of elementwise products in 64 bits, which follow the
same rules.  Finite elements are compared under the tolerances of
test_adapter_gpu.py; where |h| meets an infinity it is of the size of its row's
or column's others, so that its first part is not zero.
"""

import pytest

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402
from test_adapter_gpu import E32, OFFSET, SEED, U, Pool, keep_of, make_slots, randn, rows_of  # noqa: E402
from test_block_gpu import near  # noqa: E402

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


def product(a, b):
    """a [m][n] . b [n][k] and the sum of the finite products' magnitudes, in 64
    bits, product by product."""
    out, size = torch.zeros(2, a.shape[0], b.shape[1], dtype=torch.float64, device="cuda")
    for i in range(a.shape[1]):
        term = a[:, i:i + 1].double() * b[i:i + 1].double()
        out += term
        size += torch.where(term.isfinite(), term.abs(), 0.0)
    return out, size


def same(got, ref, size, terms, half, what):
    """Non-finite where the reference is, and the same; else within the
    tolerance of that many terms in two parts (and of half a step of fp16)."""
    got = got.double()
    for name, of in (("nan", torch.isnan), ("+inf", lambda t: t == INF), ("-inf", lambda t: t == -INF)):
        wrong = of(got) != of(ref)
        assert not wrong.any(), f"{what}: {name} at {wrong.nonzero()[:3].tolist()}: {got[wrong][:3]} for {ref[wrong][:3]}"
    fine = ref.isfinite()
    tol = (2.0 ** -21 + 2 * (2 * terms + 64) * E32) * size + (U * ref.abs() + 2.0 ** -25 if half else 2.0 ** -149)
    near(got[fine], ref[fine], tol[fine], what)


def with_infinities(t):
    """Of either sign in the last dimension, alone, two of one sign and two of
    opposite signs in a column of the sum."""
    t = t.clone()
    t[..., 0, ::5] = INF
    t[..., -1, 1::7] = -INF
    t[..., 0, 2::9] = -INF
    t[..., t.shape[-2] // 2, 2::18] = -INF
    return t


SIZES = [
    # M, K, N, R, L, slots: one launch, two, the rank's 16, 32, 64 and 128, rows by list and all of one adapter's
    (3, 64, 8, 16, 2, "random"), (3, 64, 7, 4, 2, "random"), (16, 96, 137, 5, 9, "random"), (4, 128, 520, 16, 1, None),
    (40, 64, 7, 16, 1, None), (40, 64, 8, 16, 1, None), (150, 160, 130, 12, 3, "runs"), (150, 96, 136, 24, 3, "random"),
    (100, 64, 72, 32, 1, None), (131, 96, 264, 33, 2, "runs"), (300, 64, 137, 64, 1, None), (90, 96, 200, 128, 2, "random"),
    (70, 64, 7, 100, 2, "random"), (600, 64, 520, 64, 3, "runs"),
]


@pytest.mark.parametrize("M,K,N,R,L,kind", SIZES)
@pytest.mark.parametrize("add", [True, False])
def test_up(M, K, N, R, L, kind, add):
    P, x, slots = Pool(11, L, R, N, K), randn(1, M, K), make_slots(kind, M, L)
    up = with_infinities(P.up)
    base = randn(2, M, N) if add else None
    y, hidden = wq.adapters(x, P.down, up, P.scales, slots=slots, base=base, save_hidden=True)
    assert hidden.isfinite().all()
    assert torch.equal(hidden, wq.adapters(x, *P.args, slots=slots, base=base, save_hidden=True)[1])
    for a, rows in rows_of(slots, M, L):
        if not len(rows):
            continue
        ref, size = product(hidden[rows], up[a])
        s = P.scales[a].double()
        ref, size = s * ref, s.abs() * size
        if add:
            ref, size = ref + base[rows].double(), size + base[rows].double().abs()
        same(y[rows], ref, size, R, True, f"y of adapter {a}")


@pytest.mark.parametrize("M,K,N,R,L,kind", SIZES)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_down_in_dx(M, K, N, R, L, kind, p):
    P, slots = Pool(21, L, R, N, K), make_slots(kind, M, L)
    down, dy, add = with_infinities(P.down), randn(4, M, N, sigma=0.1), randn(6, M, K, sigma=0.1)
    dx, _, _ = wq.adapters_backward(dy, None, None, down, P.up, P.scales, slots=slots, p=p, seed=SEED, offset=OFFSET,
                                    dx_add=add, need_weights=False)
    keep = keep_of((M, K), p) if p else torch.ones(M, K, dtype=torch.float64, device="cuda")
    for a, rows in rows_of(slots, M, L):
        if not len(rows):
            continue
        dh, first = product(dy[rows], P.up[a].T)
        error = 2 * (N + 64) * E32 * first
        ref, size = product(dh, down[a])
        _, more = product(error, down[a])
        s, k = P.scales[a].double(), keep[rows]
        # dropped elements are zero whatever they hold
        ref = torch.where(k > 0, s * ref * k, 0.0) + add[rows].double()
        size = (s.abs() * (size + more / 2.0 ** -21)) * k + add[rows].double().abs()
        same(dx[rows], ref, size, R, True, f"dx of adapter {a}")


@pytest.mark.parametrize("M,K,N,R,L,kind", SIZES)
def test_dy_in_dup(M, K, N, R, L, kind):
    """A gradient that has left fp16's range, as a loss scale too large makes."""
    P, x, slots = Pool(31, L, R, N, K), randn(3, M, K), make_slots(kind, M, L)
    dy, hidden = randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    hidden[:, ::2] = hidden[:, ::2].half().float()      # no second part
    dy[M // 2, ::3] = INF
    dy[0, 1::3] = -INF
    dy[M - 1, ::6] = -INF
    _, ddown, dup = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, need_dx=False)
    for a, rows in rows_of(slots, M, L):
        if not len(rows):
            assert not dup[a].any() and not ddown[a].any()
            continue
        ref, size = product(hidden[rows].T, dy[rows])
        s = P.scales[a].double()
        same(dup[a], s * ref, s.abs() * size, len(rows), False, f"dup of adapter {a}")


@pytest.mark.parametrize("M,K,N,R,L,kind", SIZES)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_x_in_ddown(M, K, N, R, L, kind, p):
    P, x, slots = Pool(41, L, R, N, K), randn(3, M, K), make_slots(kind, M, L)
    dy, hidden = randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    x[M // 2, ::3] = INF
    x[0, 1::3] = -INF
    x[M - 1, ::6] = -INF
    _, ddown, _ = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, p=p, seed=SEED, offset=OFFSET, need_dx=False)
    keep = keep_of((M, K), p) if p else torch.ones(M, K, dtype=torch.float64, device="cuda")
    xd = torch.where(keep > 0, x.double() * keep, 0.0)
    for a, rows in rows_of(slots, M, L):
        if not len(rows):
            continue
        dh, first = product(dy[rows], P.up[a].T)
        error = 2 * (N + 64) * E32 * first
        ref, size = product(dh.T, xd[rows])
        _, more = product(error.T, xd[rows])
        s = P.scales[a].double()
        same(ddown[a], s * ref, s.abs() * (size + more / 2.0 ** -21), len(rows), False, f"ddown of adapter {a}")


def test_far_rows_of_a_long_list():
    """The infinity is in the last of several ranges of rows, whose sums meet in
    another kernel; finite columns keep their bits."""
    M, K, N, R = 2048, 256, 264, 16
    P, x = Pool(51, 1, R, N, K), randn(3, M, K)
    dy, hidden = randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    want = wq.adapters_backward(dy, x, hidden, *P.args, need_dx=False)
    dy[M - 2, 7] = INF
    _, ddown, dup = wq.adapters_backward(dy, x, hidden, *P.args, need_dx=False)
    assert torch.equal(dup[0, :, 7], torch.sign(hidden[M - 2] * P.scales) * INF)
    others = torch.arange(N, device="cuda") != 7
    assert torch.equal(dup[:, :, others], want[2][:, :, others])
    assert not ddown.isfinite().any()      # (the whole of that row's dh is an infinity)
