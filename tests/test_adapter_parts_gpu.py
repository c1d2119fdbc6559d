"""The two fp16 numbers in which h, dh and hidden enter their second products.

Exact cases: h's are whole numbers of 12 to 16 bits, of which the first number
holds 11, met by weights of 1, 0 and -1 that cancel what pairs of them share.  All
products and sums are whole numbers below 2^24, so that every order of fp32
additions is exact, and the results are below 2048, exact in fp16.  The oracle
without the second numbers gives other results in every case.

Bounds: h is scaled by a power of two so that its largest magnitude lies in [2^13,
2^14).  The first number is off by at most 2^-11 of its value (2^-25, half fp16's
smallest step, where that is more), the second by 2^-11 of the rest (or 2^-25): an
element is off by at most 2^-22 of itself or 2^-25 / 2^13 = 2^-38 of the largest.
The largest is its row's in y and dx; in ddown and dup it is its column's among 32
rows that follow one another in the adapter's.
"""

import pytest

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402
from test_adapter_gpu import E32, OFFSET, SEED, U, make_slots, randn, rows_of  # noqa: E402
from test_block_gpu import near  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def integers(g, low, high, *shape):
    return torch.randint(low, high, shape, generator=g, device="cuda")


def shared_by_pairs(g, n, *rest):
    """[n][...] whole numbers, 1 to 15 of 2048 each that 2 i and 2 i + 1 share, and
    their own 0 to 15 (low, high)."""
    high = integers(g, 1, 16, (n + 1) // 2, *rest).repeat_interleave(2, 0)[:n]
    return integers(g, 0, 16, n, *rest), high


def cancelling(g, n, cols):
    """[n][cols] of 1, 0 and -1: 2 i + 1 the negative of 2 i, a last odd one 0."""
    v = integers(g, -1, 2, n // 2, cols).repeat_interleave(2, 0)
    v[1::2] *= -1
    return torch.cat([v, v.new_zeros(n % 2, cols)])


def first_part(h, dim):
    """h rounded to one fp16 number, as it is scaled."""
    scale = torch.exp2(13 - torch.floor(torch.log2(h.abs().amax(dim, keepdim=True).clamp(min=1))))
    return (h * scale).half().double() / scale


SIZES = [
    # M, C (the long side), rank, adapters, slots: one launch and two, ranks in every width, whole and odd
    (1, 520, 16, 1, None), (9, 130, 12, 3, "random"), (40, 520, 16, 2, "random"), (70, 264, 17, 1, None),
    (100, 640, 24, 3, "runs"), (65, 1025, 31, 1, None), (150, 512, 32, 4, "random"), (33, 200, 33, 2, "random"),
    (100, 1032, 48, 1, None), (200, 520, 63, 3, "runs"), (129, 520, 64, 1, None), (90, 96, 65, 2, "random"),
    (64, 648, 100, 2, "runs"), (300, 520, 128, 1, None), (2100, 8201, 64, 3, "random"),
]


@pytest.mark.parametrize("M,N,R,L,kind", SIZES)
def test_forward(M, N, R, L, kind):
    g, slots, K = generator(M + R), make_slots(kind, M, L), 32
    factor = 1 + integers(g, 0, 2, M)               # rows of different magnitude
    x, down, up = torch.zeros(M, K), torch.zeros(L, R, K), torch.zeros(L, R, N)
    x, down, up = (t.cuda().half() for t in (x, down, up))
    x[:, 7], x[:, 20] = factor, 2048 * factor
    for a in range(L):
        down[a, :, 7], down[a, :, 20] = shared_by_pairs(g, R)
        up[a] = cancelling(g, R, N)
    y, hidden = wq.adapters(x, down, up, torch.ones(L, device="cuda"), slots=slots, save_hidden=True)
    differs = False
    for a, rows in rows_of(slots, M, L):
        h = x[rows].double() @ down[a].double().T
        assert torch.equal(hidden[rows].double(), h)
        assert torch.equal(y[rows].double(), h @ up[a].double())
        if len(rows):
            differs |= not torch.equal(first_part(h, 1) @ up[a].double(), h @ up[a].double())
    assert differs


@pytest.mark.parametrize("M,K,R,L,kind", [(M, (C + 31) // 32 * 32, R, L, kind) for M, C, R, L, kind in SIZES])
def test_dx(M, K, R, L, kind):
    g, slots, N = generator(M + R), make_slots(kind, M, L), 40
    factor = 1 + integers(g, 0, 2, M)
    dy, down, up = (t.cuda().half() for t in (torch.zeros(M, N), torch.zeros(L, R, K), torch.zeros(L, R, N)))
    dy[:, 7], dy[:, 20] = factor, 2048 * factor
    for a in range(L):
        up[a, :, 7], up[a, :, 20] = shared_by_pairs(g, R)
        down[a] = cancelling(g, R, K)
    ones = torch.ones(L, device="cuda")
    dx, _, _ = wq.adapters_backward(dy, None, None, down, up, ones, slots=slots, need_weights=False)
    # doubled where it is kept, which is exact too
    dropped, _, _ = wq.adapters_backward(dy, None, None, down, up, ones, slots=slots, need_weights=False, p=0.5, seed=SEED,
                                         offset=OFFSET)
    assert torch.equal(dropped, wq.dropout_backward(dx, 0.5, SEED, OFFSET))
    differs = False
    for a, rows in rows_of(slots, M, L):
        h = dy[rows].double() @ up[a].double().T
        assert torch.equal(dx[rows].double(), h @ down[a].double())
        if len(rows):
            differs |= not torch.equal(first_part(h, 1) @ down[a].double(), h @ down[a].double())
    assert differs


# rows of an adapter at most 120: with the factors' 2^17 below 2^24
@pytest.mark.parametrize("M,R,L,kind", [(100, 16, 1, None), (120, 5, 1, None), (200, 17, 3, "random"), (120, 32, 1, None),
                                        (77, 33, 1, None), (110, 64, 1, None), (300, 63, 5, "random"), (120, 128, 1, None),
                                        (99, 101, 1, None)])
def test_gradients(M, R, L, kind):
    g, slots, K, N = generator(M + R), make_slots(kind, M, L), 160, 137
    low, high = shared_by_pairs(g, M)
    x, dy, hidden = torch.zeros(M, K), torch.zeros(M, N), torch.zeros(M, R)
    x, dy, hidden = x.cuda().half(), dy.cuda().half(), hidden.cuda()
    up, down = torch.zeros(L, R, N, device="cuda").half(), torch.zeros(L, R, K, device="cuda").half()
    factor = 1 + integers(g, 0, 2, L, R)
    for a, rows in rows_of(slots, M, L):
        n = len(rows)
        assert n <= 120
        if not n:
            continue
        low, high = shared_by_pairs(g, n)
        up[a, :, 7], up[a, :, 20] = factor[a], 2048 * factor[a]
        x[rows] = cancelling(g, n, K).half()
        dy[rows] = cancelling(g, n, N).half()
        dy[rows, 7], dy[rows, 20] = low.half(), high.half()
        low, high = shared_by_pairs(g, n, R)
        hidden[rows] = (low + 2048 * high).float()
    ones = torch.ones(L, device="cuda")
    # the dy of dh = low + 2048 high: its other columns meet zeros of up
    _, ddown, dup = wq.adapters_backward(dy, x, hidden, down, up, ones, slots=slots, need_dx=False)
    differs = [False, False]
    for a, rows in rows_of(slots, M, L):
        if not len(rows):
            continue
        d, h, xa, da = dy[rows].double() @ up[a].double().T, hidden[rows].double(), x[rows].double(), dy[rows].double()
        assert torch.equal(ddown[a].double(), d.T @ xa)
        whole = da.clone()
        whole[:, 7] = whole[:, 20] = 0
        assert torch.equal((h.T @ whole)[:, :7], dup[a].double()[:, :7])
        assert torch.equal((h.T @ whole)[:, 21:], dup[a].double()[:, 21:])
        differs[0] |= not torch.equal(first_part(d, 0).T @ xa, d.T @ xa)
        differs[1] |= not torch.equal(first_part(h, 0).T @ whole, h.T @ whole)
    assert all(differs)


def error_of(h, dim):
    """The bound of the header, element by element."""
    return torch.maximum(2.0 ** -22 * h.abs(), 2.0 ** -38 * h.abs().amax(dim, keepdim=True).expand_as(h))


@pytest.mark.parametrize("M,R", [(96, 8), (128, 24), (150, 64), (128, 128)])
def test_small_rows_beside_large_ones_in_the_gradients(M, R):
    """Some rows' hidden and dh are 10^11 times the others', whose x and dy are the
    large ones: the small rows decide the sums, off by the stated bound, 32 rows
    at a time."""
    K, N = 96, 72
    x, dy = randn(1, M, K, sigma=0.01), randn(2, M, N, sigma=1.0)
    up, down = randn(3, 1, R, N, sigma=0.3), randn(4, 1, R, K)
    hidden = randn(5, M, R, dtype=torch.float32) * 1e-5
    # dup: hidden of three rows is large where their dy is small; rows 32 to 63 have none such
    far = torch.tensor([3, 70, 71], device="cuda")
    hidden[far] *= 1e11
    dy[far] = 0
    dy[far, 5] = 2.0 ** -20
    _, _, dup = wq.adapters_backward(dy, x, hidden, down, up, torch.ones(1, device="cuda"), need_dx=False)
    h, d = hidden.double(), dy.double()
    error = torch.cat([error_of(p, 0) for p in h.split(32)])
    ref = h.T @ d
    tol = error.T @ d.abs() + 2 * (2 * M + 64) * E32 * (h.abs().T @ d.abs()) + 4 * E32 * ref.abs() + 2.0 ** -149
    near(dup[0], ref, tol, "dup")
    # ddown: dh of the far rows is large, their x tiny; the others' dh is 10^-11 of it
    dy = randn(6, M, N, sigma=2.0 ** -20)
    dy[far] = randn(7, 3, N, sigma=3e4).clamp(-6e4, 6e4)
    x = randn(8, M, K, sigma=2e4).clamp(-6e4, 6e4)
    x[far] = 0
    x[far, 9] = 2.0 ** -14
    _, ddown, _ = wq.adapters_backward(dy, x, hidden, down, up, torch.ones(1, device="cuda"), need_dx=False)
    d, u, xa = dy.double(), up[0].double(), x.double()
    dh = d @ u.T
    first = 2 * (N + 64) * E32 * (d.abs() @ u.abs().T) + 4 * E32 * dh.abs()
    error = torch.cat([error_of(p, 0) for p in dh.split(32)]) * (1 + 2.0 ** -10) + first
    ref = dh.T @ xa
    tol = error.T @ xa.abs() + 2 * (2 * M + 64) * E32 * ((dh.abs() + first).T @ xa.abs()) + 8 * E32 * ref.abs() + 2.0 ** -149
    near(ddown[0], ref, tol, "ddown")


@pytest.mark.parametrize("M,R", [(3, 16), (40, 16), (70, 48), (100, 128)])
def test_small_elements_beside_large_ones_in_a_row(M, R):
    """One element of h is 10^10 times its row's others and meets zeros of up: what
    is left of the others stays within the stated bound."""
    K, N = 64, 136
    x, down, up = randn(1, M, K), randn(2, 1, R, K, sigma=2.0 ** -12), randn(3, 1, R, N, sigma=100.0)
    down[0, 2] = randn(4, K, sigma=3e4).clamp(-6e4, 6e4)
    up[0, 2, ::2] = 0
    scale = torch.full((1,), 0.125, device="cuda")
    y, hidden = wq.adapters(x, down, up, scale, save_hidden=True)
    h, u = hidden.double(), up[0].double()
    ref = 0.125 * (h @ u)
    tol = 0.125 * (error_of(h, 1) @ u.abs() + 2 * (2 * R + 64) * E32 * (h.abs() @ u.abs())) + 4 * E32 * ref.abs()
    fits = ref.abs() < 6e4
    assert fits[:, ::2].all()
    near(torch.where(fits, y.double(), 0.0), torch.where(fits, ref, 0.0), tol + U * (ref.abs() + tol) + 2.0 ** -25, "y")


@pytest.mark.parametrize("M,R,N", [(3, 16, 264), (40, 16, 264), (70, 48, 136), (128, 128, 72)])
def test_subnormal_operands(M, R, N):
    """The matrix cores align a product by its operands' exponents, and an fp16
    subnormal's is 2^-14 whatever its leading bit: the sums' rounding counts it
    so, in y with a subnormal up and in dup with a subnormal dy."""
    g, K = generator(M + R), 64
    least = lambda t: torch.where(t != 0, t.abs().clamp(min=2.0 ** -14), 0.0)  # noqa: E731
    up = (integers(g, -1023, 1024, 1, R, N).double() * 2.0 ** -24).half()
    x, down = randn(1, M, K), randn(2, 1, R, K)
    y, hidden = wq.adapters(x, down, up, torch.full((1,), 1024.0, device="cuda"), save_hidden=True)
    h, u = hidden.double(), up[0].double()
    ref = 1024 * (h @ u)
    tol = 1024 * (error_of(h, 1) @ u.abs() + 2 * (2 * R + 64) * E32 * (h.abs() @ least(u))) + 4 * E32 * ref.abs()
    near(y, ref, tol + U * (ref.abs() + tol) + 2.0 ** -25, "y")
    dy = (integers(g, -1023, 1024, M, N).double() * 2.0 ** -24).half()
    _, _, dup = wq.adapters_backward(dy, x, hidden, down, up, torch.full((1,), 1024.0, device="cuda"), need_dx=False)
    d, error = dy.double(), torch.cat([error_of(p, 0) for p in h.split(32)])
    ref = 1024 * (h.T @ d)
    tol = 1024 * (error.T @ d.abs() + 2 * (2 * M + 64) * E32 * (h.abs().T @ least(d))) + 4 * E32 * ref.abs() + 2.0 ** -149
    near(dup[0], ref, tol, "dup")
