"""Low-rank adapters and dropout (wq_adapter.h) on the GPU against plain 64-bit
implementations.

Tolerances, per element, with u = 2^-11 (half a step of fp16), e = 2^-24 (half
a step of fp32):

- products: fp32 accumulation of n terms in any order and grouping, each
  addition rounded (matrix cores may truncate where they align: 2 e each):
  2 (n + 64) e sum |a b|, 64 for the partial sums that meet at the end;
- dropout's factor and the scale: a rounding each of the factor itself and of
  the product with it, 4 e of the result together;
- the first product enters the second in two fp16 numbers.  The first is off by
  at most 2^-11 of its value, the second by 2^-11 of the rest: 2^-22; scaled
  so that the largest value of its row (of its column within some rows, in the
  gradients) is at least 2^8, fp16's smallest half step 2^-25 adds at most
  2^-33 of that largest value.  The two parts double the terms of the second
  product;
- stored fp16: u |y| + 2^-25 (half the smallest subnormal step).
"""

import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402
from test_block_gpu import make_layer, near  # noqa: E402

pytestmark = pytest.mark.gpu

U, E32 = 2.0 ** -11, 2.0 ** -24
SEED, OFFSET = 0x9A3C5E7F12345678, 0x0123456789ABCDEF


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


def randn(seed, *shape, sigma=1.0, dtype=torch.float16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(dtype)


def make_slots(kind, M, L, seed=5):
    g = np.random.default_rng([seed, M, L])
    if kind is None:
        return None
    if kind == "runs":        # ragged runs, one adapter each, some without one
        ends = np.sort(g.integers(0, M + 1, size=5))
        s = np.zeros(M, dtype=np.int32)
        for i, (a, b) in enumerate(zip(np.r_[0, ends], np.r_[ends, M])):
            s[a:b] = -1 if i == 2 else g.integers(0, L)
    elif kind == "random":    # any order, an eighth without one
        s = g.integers(0, L, size=M).astype(np.int32)
        s[g.random(M) < 0.125] = -1
    elif kind == "none":
        s = np.full(M, -1, dtype=np.int32)
    else:                     # numbers that are no adapter's, far ones among them
        s = g.choice(np.array([-2147483648, -7, L, L + 1, 2147483647, 0, L - 1], dtype=np.int64), size=M).astype(np.int32)
    return torch.from_numpy(s).cuda()


def keep_of(shape, p, seed=SEED, offset=OFFSET):
    """(kept as float64, with its factor) on the GPU."""
    keep, factor = O.drop_keep(shape, p, seed, offset)
    return torch.from_numpy(keep).cuda().double() * factor


class Pool:
    def __init__(self, seed, L, R, N, K):
        self.down, self.up = randn(seed, L, R, K, sigma=K ** -0.5), randn(seed + 1, L, R, N, sigma=0.05)
        self.scales = randn(seed + 2, L, dtype=torch.float32)
        self.args = (self.down, self.up, self.scales)


def rows_of(slots, M, L):
    if slots is None:
        return [(0, torch.arange(M, device="cuda"))]
    return [(a, (slots == a).nonzero().flatten()) for a in range(L)]


def split_error(h, dim):
    """Of h in two fp16 numbers, scaled by the largest along dim."""
    return 2.0 ** -22 * h.abs() + 2.0 ** -33 * h.abs().amax(dim, keepdim=True)


def check_forward(P, x, slots, base, p, y, hidden, what):
    M, K = x.shape
    L, R, N = P.up.shape
    xd = x.double() * (keep_of((M, K), p) if p else 1.0)
    ref, tol = torch.zeros(M, N, dtype=torch.float64, device="cuda"), torch.zeros(M, N, dtype=torch.float64, device="cuda")
    h, eh = (torch.zeros(M, R, dtype=torch.float64, device="cuda") for _ in range(2))
    for a, rows in rows_of(slots, M, L):
        if not len(rows):
            continue
        down, up, s = P.down[a].double(), P.up[a].double(), P.scales[a].double()
        h[rows] = xd[rows] @ down.T
        eh[rows] = 2 * (K + 64) * E32 * (xd[rows].abs() @ down.abs().T) + 4 * E32 * h[rows].abs()
        ha = h[rows]
        ref[rows] = s * (ha @ up)
        tol[rows] = s.abs() * ((eh[rows] + split_error(ha, 1)) @ up.abs()
                               + 2 * (2 * R + 64) * E32 * ((ha.abs() + eh[rows]) @ up.abs())) + 4 * E32 * ref[rows].abs()
    if base is not None:
        ref = ref + base.double()
        tol = tol + E32 * ref.abs()
    near(y, ref, tol + U * (ref.abs() + tol) + 2.0 ** -25, what + " y")
    if hidden is not None:
        assert hidden.dtype == torch.float32
        near(hidden, h, eh + 2.0 ** -149, what + " hidden")


def check_backward(P, dy, x, hidden, slots, add, p, dx, ddown, dup, what):
    M, N = dy.shape
    L, R, K = P.down.shape
    keep = keep_of((M, K), p) if p else None
    ref, tol = (torch.zeros(M, K, dtype=torch.float64, device="cuda") for _ in range(2))
    dyd = dy.double()
    for a, rows in rows_of(slots, M, L):
        if not len(rows):
            if ddown is not None:
                assert not ddown[a].any() and not dup[a].any(), what
            continue
        down, up, s = P.down[a].double(), P.up[a].double(), P.scales[a].double()
        g = dyd[rows]
        dh = g @ up.T
        eh = 2 * (N + 64) * E32 * (g.abs() @ up.abs().T) + 4 * E32 * dh.abs()
        ref[rows] = s * (dh @ down)
        tol[rows] = s.abs() * ((eh + split_error(dh, 1)) @ down.abs()
                               + 2 * (2 * R + 64) * E32 * ((dh.abs() + eh) @ down.abs())) + 4 * E32 * ref[rows].abs()
        if ddown is not None:
            n = 2 * (2 * len(rows) + 64) * E32
            xa = x[rows].double() * (1.0 if keep is None else keep[rows])
            r = s * (dh.T @ xa)
            t = s.abs() * ((eh + split_error(dh, 0)).T @ xa.abs() + n * ((dh.abs() + eh).T @ xa.abs())) + 8 * E32 * r.abs()
            near(ddown[a], r, t + 2.0 ** -149, f"{what} ddown[{a}]")
            ha = hidden[rows].double()
            r = s * (ha.T @ g)
            t = s.abs() * (split_error(ha, 0).T @ g.abs() + n * (ha.abs().T @ g.abs())) + 8 * E32 * r.abs()
            near(dup[a], r, t + 2.0 ** -149, f"{what} dup[{a}]")
    if keep is not None:
        ref, tol = ref * keep, tol * keep + 4 * E32 * (ref * keep).abs()
    if add is not None:
        ref = ref + add.double()
        tol = tol + E32 * ref.abs()
    if dx is not None:
        near(dx, ref, tol + U * (ref.abs() + tol) + 2.0 ** -25, what + " dx")


# M across the row tiles and their borders; K that ends inside a step; N odd,
# below a vector, across column tiles; ranks odd, at and beyond the products'
# 16s and 32s; adapters' rows in runs, mixed, absent
CASES = [
    # M, K, N, R, L, slots, add, p
    (1, 32, 1, 1, 1, None, True, 0.0),
    (1, 4096, 4096, 16, 1, None, True, 0.0),
    (1, 4128, 5001, 128, 3, "random", False, 0.25),
    (2, 64, 7, 3, 2, "random", True, 0.0),
    (5, 96, 8, 8, 40, "random", True, 0.1),
    (15, 160, 130, 12, 4, "random", False, 0.0),
    (16, 4096, 1032, 16, 32, "random", True, 0.0),
    (17, 4128, 257, 17, 3, "runs", True, 0.5),
    (31, 1056, 129, 31, 5, "random", True, 0.0),
    (33, 2080, 512, 32, 3, "runs", False, 0.05),
    (64, 11008, 640, 64, 9, "random", True, 0.0),
    (65, 288, 1025, 33, 2, "other", True, 0.1),
    (100, 1024, 96, 65, 4, "runs", False, 0.0),
    (129, 256, 1001, 127, 3, "runs", True, 0.3),
    (173, 4128, 5001, 12, 6, "runs", False, 0.1),
    (200, 512, 264, 8, 7, "none", True, 0.1),
    (200, 512, 264, 8, 7, "none", False, 0.0),
    (257, 2048, 2056, 16, 64, "random", True, 0.0),
    (311, 4128, 5001, 8, 6, "runs", True, 0.0),
    (513, 1024, 1024, 24, 1, None, True, 0.1),
    (777, 736, 1111, 48, 2, "other", False, 0.2),
    (1500, 320, 520, 128, 2, "runs", True, 0.1),
    (2048, 1024, 768, 16, 3, "runs", True, 0.05),
    (4099, 128, 72, 4, 1000, "random", True, 0.0),
]


@pytest.mark.parametrize("M,K,N,R,L,kind,add,p", CASES)
def test_forward(M, K, N, R, L, kind, add, p):
    P, x, slots = Pool(11, L, R, N, K), randn(1, M, K), make_slots(kind, M, L)
    base = randn(2, M, N) if add else None
    y, hidden = wq.adapters(x, *P.args, slots=slots, base=base, p=p, seed=SEED, offset=OFFSET, save_hidden=True)
    check_forward(P, x, slots, base, p, y, hidden, "forward")
    again = wq.adapters(x, *P.args, slots=slots, base=base, p=p, seed=SEED, offset=OFFSET)
    assert torch.equal(again, y)
    if base is not None:
        wq.adapters(x, *P.args, slots=slots, base=base, p=p, seed=SEED, offset=OFFSET, out=base)
        assert torch.equal(base, y)


# the form of one launch: rows, ranks and K up to its limits and past them, N
# whose last tile has fewer than eight columns of its own
@pytest.mark.parametrize("M,K,N,R,L,kind,add", [
    (1, 32, 8, 1, 1, None, True), (2, 64, 9, 16, 3, "other", False), (3, 4096, 129, 5, 2, "random", True),
    (4, 4096, 4096, 16, 1, None, True), (4, 1056, 135, 9, 4, "runs", True), (5, 512, 640, 16, 1, None, True),
    (8, 4096, 12288, 16, 8, "random", True), (13, 2080, 1000, 12, 40, "random", False), (16, 4096, 385, 16, 16, "random", True),
    (16, 4096, 513, 16, 4, "none", True), (16, 4096, 512, 16, 4, "runs", False), (16, 4128, 512, 16, 16, "random", True),
    (16, 4096, 512, 17, 16, "random", True), (17, 4096, 512, 16, 16, "random", True), (6, 3200, 131, 3, 1000, "random", True)])
def test_a_few_rows(M, K, N, R, L, kind, add):
    P, x, slots = Pool(15, L, R, N, K), randn(1, M, K), make_slots(kind, M, L)
    base = randn(2, M, N) if add else None
    y, hidden = wq.adapters(x, *P.args, slots=slots, base=base, save_hidden=True)
    check_forward(P, x, slots, base, 0.0, y, hidden, "few rows")
    assert torch.equal(wq.adapters(x, *P.args, slots=slots, base=base), y)
    if add:
        assert torch.equal(wq.adapters(x, *P.args, slots=slots, base=base, out=base), y)


def test_rows_in_another_order():
    """A permutation of the rows and their slots is one of the outputs, whatever
    fragments the rows share (the sums' order does not depend on them)."""
    M, K, N, R, L = 190, 1024, 600, 16, 5
    P, x, slots = Pool(16, L, R, N, K), randn(1, M, K), make_slots("runs", M, L)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    perm = torch.randperm(M, generator=g, device="cuda")
    y, h = wq.adapters(x, *P.args, slots=slots, save_hidden=True)
    y2, h2 = wq.adapters(x[perm].contiguous(), *P.args, slots=slots[perm].contiguous(), save_hidden=True)
    assert torch.equal(y[perm], y2) and torch.equal(h[perm], h2)


@pytest.mark.parametrize("M,K,N,R,L,kind,add,p", CASES)
def test_backward(M, K, N, R, L, kind, add, p):
    P, x, slots = Pool(21, L, R, N, K), randn(3, M, K), make_slots(kind, M, L)
    dy, hidden = randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    dx_add = randn(6, M, K, sigma=0.1) if add else None
    drop = dict(p=p, seed=SEED, offset=OFFSET)
    got = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, dx_add=dx_add, **drop)
    check_backward(P, dy, x, hidden, slots, dx_add, p, *got, "backward")
    dx, none, none_too = wq.adapters_backward(dy, None, None, *P.args, slots=slots, dx_add=dx_add, need_weights=False, **drop)
    assert none is None and none_too is None and torch.equal(dx, got[0])
    none, ddown, dup = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, need_dx=False, **drop)
    assert none is None and torch.equal(ddown, got[1]) and torch.equal(dup, got[2])
    if add:
        wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, dx_add=dx_add, out=dx_add, **drop)
        assert torch.equal(dx_add, got[0])


@pytest.mark.parametrize("magnitude", [1e-12, 1e-5, 3e4, 1e12])
def test_hidden_values_far_from_one(magnitude):
    """The first product's values leave fp16's range on both sides: it is
    scaled into it, row by row and column by column."""
    M, K, N, R, L = 70, 256, 200, 16, 2
    P, x, slots = Pool(31, L, R, N, K), randn(1, M, K), make_slots("random", M, L)
    hidden = randn(5, M, R, dtype=torch.float32) * magnitude
    hidden[:, 3] *= 1e6
    dy = randn(4, M, N, sigma=0.1)
    P.scales.mul_(1e-6 / magnitude)
    got = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots)
    check_backward(P, dy, x, hidden, slots, None, 0.0, *got, "far")
    # forward: large and small products from large and small inputs
    P.scales.fill_(1.0)
    f = min(max(magnitude, 1e-4), 30.0)
    x = (x.float() * f).half()
    P.down.copy_((P.down.float() * 100).half() if magnitude > 1 else P.down)
    P.scales.div_(f * (100 if magnitude > 1 else 1))
    y, h = wq.adapters(x, *P.args, slots=slots, save_hidden=True)
    check_forward(P, x, slots, None, 0.0, y, h, "far")


def test_a_far_row_leaves_the_others_their_precision():
    """One row's gradient is 10^10 times the others': dx is scaled row by row."""
    M, K, N, R = 40, 128, 96, 8
    P, x = Pool(41, 1, R, N, K), randn(1, M, K)
    dy = randn(4, M, N, sigma=1e-4)
    dy[17] = 3e4
    P.scales.fill_(1e-3)
    hidden = randn(5, M, R, dtype=torch.float32)
    got = wq.adapters_backward(dy, x, hidden, *P.args)
    check_backward(P, dy, x, hidden, None, None, 0.0, *got, "far row")


@pytest.mark.parametrize("M,R", [(3, 8), (40, 16), (200, 64)])
def test_rows_are_independent(M, R):
    """Infinities and NaN in one row, and in an adapter that only this row
    takes, stay in it (forward, dx), and in that adapter's gradients."""
    K, N, L = 256, 200, 3
    P, x = Pool(51, L, R, N, K), randn(1, M, K)
    slots = make_slots("random", M, 2)
    base, dy, hidden = randn(2, M, N), randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    bad = M // 2
    slots[bad] = 2
    want = wq.adapters(x, *P.args, slots=slots, base=base, save_hidden=True)
    wb = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots)
    for value in (float("inf"), float("nan")):
        x2, dy2, h2, down2, up2 = (t.clone() for t in (x, dy, hidden, P.down, P.up))
        for t in (x2, dy2, h2):
            t[bad, ::3] = value
        down2[2, :, ::5] = value
        up2[2, :, ::7] = value
        got = wq.adapters(x2, down2, up2, P.scales, slots=slots, base=base, save_hidden=True)
        gb = wq.adapters_backward(dy2, x2, h2, down2, up2, P.scales, slots=slots)
        others = torch.arange(M, device="cuda") != bad
        for a, b in zip(got + gb[:1], want + wb[:1]):
            assert torch.equal(a[others], b[others])
            assert not torch.isfinite(a[bad]).all()
        for a, b in zip(gb[1:], wb[1:]):
            assert torch.equal(a[:2], b[:2])
            assert not torch.isfinite(a[2]).all()


def test_infinite_products_as_the_formula_has_them():
    """x of one infinity and an adapter of positive weights: y is +inf, not NaN."""
    K, N, R = 64, 40, 4
    down, up = torch.full((1, R, K), 0.5, device="cuda").half(), torch.full((1, R, N), 0.25, device="cuda").half()
    x = torch.ones(3, K, device="cuda").half()
    x[1, 5] = float("inf")
    y, h = wq.adapters(x, down, up, torch.ones(1, device="cuda"), save_hidden=True)
    assert (y[1] == float("inf")).all() and (h[1] == float("inf")).all()
    assert (y[0] == R * 0.5 * K * 0.25).all() and (y[2] == y[0]).all()
    dy = torch.ones(3, N, device="cuda").half()
    dx, ddown, dup = wq.adapters_backward(dy, x.abs().clamp(max=2), h, down, up, torch.ones(1, device="cuda"))
    assert (dup == float("inf")).all() and torch.isfinite(ddown).all() and torch.isfinite(dx).all()


def test_rows_without_an_adapter_pass_through():
    M, K, N, R, L = 50, 128, 99, 8, 2
    P, x, base = Pool(61, L, R, N, K), randn(1, M, K), randn(2, M, N)
    x[7] = float("nan")
    slots = torch.full((M,), 1, dtype=torch.int32, device="cuda")
    slots[5:20] = -1
    y, h = wq.adapters(x, *P.args, slots=slots, base=base, save_hidden=True)
    assert torch.equal(y[5:20], base[5:20]) and not h[5:20].any()
    y = wq.adapters(x, *P.args, slots=slots)
    assert not y[5:20].any()
    add = randn(3, M, K)
    dy = randn(4, M, N)
    dy[8] = float("inf")
    dx, ddown, dup = wq.adapters_backward(dy, x, h, *P.args, slots=slots, dx_add=add)
    assert torch.equal(dx[5:20], add[5:20])
    assert torch.isfinite(ddown).all() and torch.isfinite(dup).all() and not ddown[0].any() and not dup[0].any()


# --------------------------------------------------------------- dropout ----

@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (1000, 3), (64, 4096), (257, 1001), (3, 5, 7, 11)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9, 2.0 ** -17 * 1.01, 0.9999])
def test_dropout(shape, p):
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
    if p == 0:
        assert torch.equal(y, x)


def test_dropout_of_infinities():
    x = torch.full((4096,), float("nan"), device="cuda").half()
    x[::2] = float("inf")
    keep = keep_of((4096,), 0.5) > 0
    y = wq.dropout(x, 0.5, SEED, OFFSET)
    assert not y[~keep].any() and not torch.isfinite(y[keep]).any()


def test_every_threshold_is_the_generators():
    """The mask at many chances shows the draws themselves: ones are kept up to
    their own draw."""
    n = 4096
    draws = torch.from_numpy(O.drop_halves(0, n, SEED, OFFSET).astype(np.int64)).cuda()
    x = torch.ones(n, device="cuda").half()
    for t in (1, 2, 255, 256, 257, 32767, 32768, 40000, 65534):
        assert torch.equal(wq.dropout(x, t / 65536, SEED, OFFSET) != 0, draws >= t), t


def test_seeds_and_offsets_make_other_masks():
    x = torch.ones(1 << 16, device="cuda").half()
    masks = [wq.dropout(x, 0.5, s, o) != 0 for s, o in ((0, 0), (1, 0), (1 << 32, 0), (0, 1), (0, 1 << 32), ((1 << 64) - 1, 0))]
    for i, a in enumerate(masks):
        assert abs(a.float().mean().item() - 0.5) < 0.01
        for b in masks[:i]:
            assert 0.48 < (a == b).float().mean().item() < 0.52


def test_step_is_added_to_the_offset():
    x = randn(1, 1000)
    step = torch.tensor([5], dtype=torch.int64, device="cuda")
    assert torch.equal(wq.dropout(x, 0.3, 7, 10, step=step), wq.dropout(x, 0.3, 7, 15))
    step.fill_(-3)     # modulo 2^64
    assert torch.equal(wq.dropout(x, 0.3, 7, 1, step=step), wq.dropout(x, 0.3, 7, (1 << 64) - 2))


def test_dropout_past_32_bit_offsets():
    """More than 2^32 elements (the generator's upper counter word is past
    zero from element 2^35 on: the oracle's pins cover it)."""
    n = (1 << 32) + 1029
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 5 * n:
        pytest.skip("not enough memory")
    x = torch.empty(n, dtype=torch.float16, device="cuda").fill_(1)
    wq.dropout(x, 0.25, SEED, OFFSET, out=x)
    for first in (0, (1 << 31) - 512, (1 << 32) - 1024, (1 << 32) + 8):
        m = min(n - first, 2048)
        want = torch.from_numpy(O.drop_halves(first, m, SEED, OFFSET) >= 16384).cuda()
        assert torch.equal(x[first:first + m] != 0, want), first
    del x
    torch.cuda.empty_cache()


def test_dropout_inside_the_adapters_is_dropout():
    """adapters of dropout's output is adapters with dropout, where 1 / (1 - p)
    is a power of two: then nothing is rounded on the way."""
    M, K, N, R, L = 77, 288, 104, 16, 2
    P, x, slots = Pool(71, L, R, N, K), randn(1, M, K), make_slots("random", M, L)
    dropped = wq.dropout(x, 0.5, SEED, OFFSET)
    y, h = wq.adapters(x, *P.args, slots=slots, p=0.5, seed=SEED, offset=OFFSET, save_hidden=True)
    y2, h2 = wq.adapters(dropped, *P.args, slots=slots, save_hidden=True)
    assert torch.equal(h, h2) and torch.equal(y, y2)
    dy = randn(4, M, N, sigma=0.1)
    a = wq.adapters_backward(dy, x, h, *P.args, slots=slots, p=0.5, seed=SEED, offset=OFFSET)
    b = wq.adapters_backward(dy, dropped, h, *P.args, slots=slots)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    # doubled after one rounding and before it: the same but where the undoubled value is subnormal
    doubled = wq.dropout_backward(b[0], 0.5, SEED, OFFSET)
    big = doubled.abs() > 2.0 ** -12
    assert torch.equal(a[0][big], doubled[big])


# ------------------------------------------------------------- gradients ----

def test_gradient_against_differences():
    """Central differences of sum(y * dy) in 64 bits from the forward kernel's
    formula agree with the backward kernel along random directions."""
    M, K, N, R, L, p = 37, 96, 70, 6, 3, 0.25
    P, x, slots = Pool(81, L, R, N, K), randn(1, M, K), make_slots("random", M, L)
    dy = randn(4, M, N, sigma=0.1)
    keep = keep_of((M, K), p)
    one = (slots.unsqueeze(1) == torch.arange(L, device="cuda", dtype=torch.int32)).double()

    def loss(x, down, up):
        h = torch.stack([(x * keep) @ down[a].T for a in range(L)], 1) * one.unsqueeze(2)
        y = sum((h[:, a] @ up[a]) * P.scales[a].double() for a in range(L))
        return (y * dy.double()).sum()

    at = [x.double(), P.down.double(), P.up.double()]
    _, hidden = wq.adapters(x, *P.args, slots=slots, p=p, seed=SEED, offset=OFFSET, save_hidden=True)
    grads = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, p=p, seed=SEED, offset=OFFSET)
    for i in range(3):
        v = randn(90 + i, *at[i].shape, dtype=torch.float64)
        # the loss is linear in each argument: the difference has no error but rounding
        plus, minus = list(at), list(at)
        plus[i], minus[i] = at[i] + 0.5 * v, at[i] - 0.5 * v
        want = (loss(*plus) - loss(*minus)).item()
        got = (grads[i].double() * v).sum().item()
        # dx is rounded to fp16: u of every term, and products' errors far below it
        room = (U * 1.01 * grads[i].double().abs() * v.abs()).sum().item() + 2.0 ** -25 * v.abs().sum().item()
        assert abs(got - want) <= room, (i, got, want, room)


def test_adapted_layer_forward_and_backward():
    """A quantized layer with its adapters, a training step's calls in a row:
    forward on the layer's output, both backward passes, against 64 bits on
    the same intermediate values."""
    M, K, N, R, L, p = 150, 512, 328, 16, 3, 0.1
    Lay = make_layer(91, N, K, 4, 128)
    packed, scales, zeros, bits, gs = Lay["args"]
    base = wq.QuantizedLinear(packed, scales, zeros, bits, gs, K)
    P, x, slots = Pool(95, L, R, N, K), randn(1, M, K), make_slots("runs", M, L)
    layer = wq.AdaptedLinear(base, *P.args)
    bias, res = randn(7, N), randn(8, M, N)
    drop = dict(p=p, seed=SEED, offset=OFFSET)
    y, hidden = layer(x, slots, bias=bias, residual=res, save_hidden=True, **drop)
    z = base.forward_act(x, bias=bias, residual=res)
    check_forward(P, x, slots, z, p, y, hidden, "layer")
    dy = randn(4, M, N, sigma=0.1)
    dx, ddown, dup = layer.backward(dy, x, hidden, slots, **drop)
    dz = base.backward(dy)[0]
    check_backward(P, dy, x, hidden, slots, dz, p, dx, ddown, dup, "layer")
    # a decode batch of the same layer, and the block's residual dropped
    y1 = layer(x[:4], slots[:4])
    check_forward(P, x[:4], slots[:4], base.forward_act(x[:4]), 0.0, y1, None, "decode")
    out = wq.dropout(y, 0.1, SEED, OFFSET + 1, residual=res)
    assert torch.isfinite(out).all()
    assert ddown.shape == P.down.shape and dup.shape == P.up.shape


# ------------------------------------------------- streams, graphs, memory ----

def test_graph_replay():
    """Forward and backward captured once and replayed with other inputs and
    another step, eager work between the replays."""
    M, K, N, R, L, p = 130, 512, 264, 16, 3, 0.2
    P, x, slots = Pool(101, L, R, N, K), randn(1, M, K), make_slots("runs", M, L)
    base, dy = randn(2, M, N), randn(4, M, N, sigma=0.1)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def calls(step=step, offset=9):
        drop = dict(p=p, seed=SEED, offset=offset, step=step)
        y, h = wq.adapters(x, *P.args, slots=slots, base=base, save_hidden=True, **drop)
        return (y, h) + wq.adapters_backward(dy, x, h, *P.args, slots=slots, dx_add=x, **drop) + \
            (wq.dropout(y, 0.3, SEED, offset, step=step, residual=base),)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for i in range(4):
        x.copy_(randn(200 + i, M, K))
        slots.copy_(make_slots("random" if i % 2 else "runs", M, L, seed=i))
        step.fill_(1000 * i)
        torch.cuda.synchronize()
        graph.replay()
        want = calls(None, 9 + 1000 * i)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    M, K, N, R, L = 300, 1024, 520, 32, 4
    sets = []
    for i in range(2):
        P, x, slots = Pool(110 + 5 * i, L, R, N, K), randn(1 + i, M, K), make_slots("random", M, L, seed=i)
        sets.append((P, x, slots, randn(4 + i, M, N, sigma=0.1), randn(6 + i, M, R, dtype=torch.float32)))

    def calls(P, x, slots, dy, h):
        return (wq.adapters(x, *P.args, slots=slots),) + wq.adapters_backward(dy, x, h, *P.args, slots=slots)

    want = [calls(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.parametrize("M,K,N,R,L", [(1, 32, 9, 3, 1), (33, 96, 130, 12, 2), (130, 160, 257, 40, 3)])
def test_neighbouring_memory_is_left_alone(M, K, N, R, L):
    """Outputs and the workspace lie between guard words, whole; the smallest
    workspace is enough whatever it holds."""
    P, x, slots = Pool(121, L, R, N, K), randn(1, M, K), make_slots("random", M, L)
    dy, hidden = randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    PAD = 64   # elements on each side

    def guarded(n, dtype, fill):
        buf = torch.full((n + 2 * PAD,), fill, dtype=dtype, device="cuda")
        return buf, buf[PAD:PAD + n]

    def untouched(buf, fill):
        return bool((buf[:PAD] == fill).all() and (buf[-PAD:] == fill).all())

    want = wq.adapters(x, *P.args, slots=slots, save_hidden=True) + wq.adapters_backward(dy, x, hidden, *P.args, slots=slots)
    for fill in (7, 255):
        need = [wq.adapters_workspace_size(e, M, N, K, R, L) for e in ("adapters", "adapters_backward")]
        ws = [guarded(n, torch.uint8, fill) for n in need]
        y, h, dx = guarded(M * N, torch.float16, 7), guarded(M * R, torch.float32, 7), guarded(M * K, torch.float16, 7)
        wq.adapters(x, *P.args, slots=slots, out=y[1].view(M, N), hidden=h[1].view(M, R), workspace=ws[0][1])
        _, ddown, dup = wq.adapters_backward(dy, x, hidden, *P.args, slots=slots, out=dx[1].view(M, K), workspace=ws[1][1])
        assert all(untouched(b, 7) for b, _ in (y, h, dx)) and all(untouched(b, fill) for b, _ in ws)
        for a, b in zip((y[1].view(M, N), h[1].view(M, R), dx[1].view(M, K), ddown, dup), want):
            assert torch.equal(a, b)
    # gradients' own buffers, through the library's entry point
    import ctypes
    gd, gu = guarded(L * R * K, torch.float32, 7), guarded(L * R * N, torch.float32, 7)
    v = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    code = wq.lib().wq_adapters_backward(v(dy), v(x), v(hidden), v(P.down), v(P.up), v(P.scales), v(slots), 0.0, 0, 0, None,
                                         None, None, v(gd[1]), v(gu[1]), M, N, K, R, L, v(ws[1][1]), need[1], None)
    torch.cuda.synchronize()
    assert code == 0 and untouched(gd[0], 7) and untouched(gu[0], 7)
    assert torch.equal(gd[1].view(L, R, K), want[3]) and torch.equal(gu[1].view(L, R, N), want[4])
    n = M * N
    buf, view = guarded(n, torch.float16, 7)
    wq.dropout(want[0].view(-1), 0.3, 1, out=view)
    assert untouched(buf, 7) and torch.equal(view, wq.dropout(want[0].view(-1), 0.3, 1))


def test_empty_batches():
    P = Pool(131, 2, 8, 40, 64)
    x, dy, h = torch.empty(0, 64, device="cuda").half(), torch.empty(0, 40, device="cuda").half(), torch.empty(0, 8, device="cuda")
    y, hidden = wq.adapters(x, *P.args, save_hidden=True)
    assert y.shape == (0, 40) and hidden.shape == (0, 8)
    dx, ddown, dup = wq.adapters_backward(dy, x, h, *P.args, slots=torch.empty(0, dtype=torch.int32, device="cuda"))
    assert dx.shape == (0, 64) and not ddown.any() and not dup.any() and ddown.shape == P.down.shape
    assert wq.dropout(x, 0.5, 1).shape == (0, 64)


def test_activations_past_32_bit_offsets():
    """More than 2^32 bytes and 2^31 elements of x, y and dx: sampled rows, the
    last ones among them, and a gradient over all rows of ones."""
    M, K, N, R = (1 << 16) + 37, 32768 + 32, 32768 + 8, 4
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    P = Pool(141, 1, R, N, K)
    x = torch.empty(M, K, dtype=torch.float16, device="cuda")
    for i in range(0, M, 4096):
        x[i:i + 4096] = randn(i, min(4096, M - i), K)
    y = wq.adapters(x, *P.args)
    rows = torch.cat([torch.arange(0, M, 5003), torch.arange(M - 40, M)]).cuda()
    check_forward(P, x[rows], None, None, 0.0, y[rows], None, "far rows")
    dx = x.clone()
    wq.adapters_backward(y, None, None, *P.args, dx_add=dx, out=dx, need_weights=False)
    check_backward(P, y[rows], None, None, None, x[rows], 0.0, dx[rows], None, None, "far rows")
    del dx
    hidden = torch.ones(M, R, device="cuda")
    x.fill_(1)
    P.scales.fill_(1)
    y.zero_()
    y[-3:] = 1
    _, ddown, dup = wq.adapters_backward(y, x, hidden, *P.args, need_dx=False)
    assert (dup == 3).all()
    want = 3 * P.up.double().sum(2)          # every column of ddown[r]: three rows' dh
    tol = 3 * 2 * (N + 64) * E32 * P.up.double().abs().sum(2) + 2.0 ** -20 * want.abs()
    near(ddown[:, :, -1], want, tol, "far ddown")
    near(ddown[:, :, 0], want, tol, "far ddown")
    del x, y
    torch.cuda.empty_cache()


def test_pool_past_32_bit_offsets():
    """A pool of more than 2^31 elements on either side; its last adapter."""
    L, R, K, N, M = 1100, 128, 16384, 16392, 21
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough memory")
    down, up = (torch.zeros(L, R, c, dtype=torch.float16, device="cuda") for c in (K, N))
    small = Pool(151, 2, R, N, K)
    down[-2:], up[-2:] = small.down, small.up
    scales = torch.ones(L, device="cuda")
    small.scales.fill_(1)
    x, dy, h = randn(1, M, K), randn(4, M, N, sigma=0.1), randn(5, M, R, dtype=torch.float32)
    s = make_slots("random", M, 2)
    slots = torch.where(s >= 0, s + (L - 2), s)
    y, hidden = wq.adapters(x, down, up, scales, slots=slots, save_hidden=True)
    check_forward(small, x, s, None, 0.0, y, hidden, "far pool")
    dx, ddown, dup = wq.adapters_backward(dy, x, h, down, up, scales, slots=slots)
    check_backward(small, dy, x, h, s, None, 0.0, dx, ddown[-2:], dup[-2:], "far pool")
    assert not ddown[:-2].any() and not dup[:-2].any()
    del down, up, ddown, dup
    torch.cuda.empty_cache()


def test_another_current_device_and_stream():
    """The tensors' device and torch's current stream on it are used."""
    P, x = Pool(161, 1, 8, 40, 64), randn(1, 9, 64)
    want = wq.adapters(x, *P.args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = wq.adapters(x, *P.args)
        z = wq.dropout(got, 0.5, 3)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(z, wq.dropout(want, 0.5, 3))
