"""The feed-forward block's products (wq_block.h) on the GPU against plain
64-bit implementations.

Layers are random codes, scales and zero-points packed by the oracle; the
reference multiplies the oracle's dequantized weights (fp16 values) in
float64.  Tolerances, per element, with u = 2^-11 (half a step of fp16), e =
2^-24 (half a step of fp32):

- products: fp32 accumulation of n terms in any order, each addition rounded
  (matrix cores may truncate where they align: 2 e each), err <= 2 (n + 8) e
  sum |a b|, called E below;
- activations: slopes at most 1.2, so E enters act(z) 1.2 times.  The kernels
  evaluate e^v by a hardware exponential: v log2(e) rounded (relative error of
  e^v up to |v| 1.5 e) and 2^x within 2 e; with the division and products
  after it act(v) is within 32 e (1 + |v|) |act(v)| for |v| <= 16, and below
  -16 under 2^-18 in magnitude on both sides; both are covered by
  2^-18 (|act(v)| + 2^-6);
- stored fp16: u |y| + 2^-25 (half the smallest subnormal step).
"""

import ctypes

import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402

pytestmark = pytest.mark.gpu

U, E32 = 2.0 ** -11, 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


def make_layer(seed, N, K, bits, gs, sym=False, act_order=False):
    """Random packed layer; w: float64 [N][K] in original channel order."""
    g = np.random.default_rng([seed, N, K, bits])
    top = (1 << bits) - 1
    codes = g.integers(0, top + 1, size=(N, K), dtype=np.uint8)
    G = 1 if gs == -1 else K // gs
    scales = (0.1 / (top + 1) * (0.5 + g.random((N, G)))).astype(np.float16)
    zeros = None if sym else g.integers(0, top + 1, size=(N, G), dtype=np.uint8)
    perm = g.permutation(K).astype(np.int32) if act_order else None
    z = np.full((N, G), 1 << (bits - 1)) if sym else zeros
    n = K // G
    q = codes.astype(np.float64) - np.repeat(z.astype(np.float64), n, axis=1)
    w = (q * np.repeat(scales.astype(np.float64), n, axis=1)).astype(np.float16).astype(np.float64)
    packed = O.pack(codes, bits).view(np.int32)
    if perm is not None:
        back = np.empty_like(w)
        back[:, perm] = w
        w = back
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return dict(args=(dev(packed), dev(scales), dev(zeros), bits, gs), perm=dev(perm), w=dev(w))


def randn(seed, *shape, sigma=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).half()


def act64(v, kind):
    """act and its derivative in float64, from their formulas."""
    if kind == "none":
        return v, torch.ones_like(v)
    if kind == "relu":
        return v.clamp(min=0), (v > 0).double()
    if kind == "gelu":
        cdf = torch.special.ndtr(v)
        return v * cdf, cdf + v * torch.exp(-v * v / 2) / (2 * np.pi) ** 0.5
    if kind == "gelu_tanh":
        c = (2 / np.pi) ** 0.5
        t = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    s = torch.sigmoid(v)
    return v * s, s * (1 + v * (1 - s))


def near(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what + ": not finite"
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), f"{what}: off by {(got - ref).abs().max().item():.3e}, over by {over.max().item():.3e}"


def product(x, w, bias):
    x = x.double()
    z = x @ w.T
    e = 2 * (w.shape[1] + 8) * E32 * (x.abs() @ w.abs().T)
    if bias is not None:
        z = z + bias.double()
        e = e + E32 * z.abs()
    return z, e


def act_tol(a):
    return 2.0 ** -18 * (a.abs() + 2.0 ** -6)


def stored(v):
    return U * v.abs() + 2.0 ** -25


def check_linear(L, x, bias, residual, act, y, preact, what):
    z, e = product(x, L["w"], bias)
    a, _ = act64(z, act)
    ref = a + (0 if residual is None else residual.double())
    tol = 1.2 * e + act_tol(a) + E32 * ref.abs()
    near(y, ref, tol + stored(ref.abs() + tol), what + " y")
    if preact is not None:
        near(preact, z, e + stored(z.abs() + e), what + " preact")


def check_gated(L, x, bias, act, h, preact, what):
    z, e = product(x, L["w"], bias)
    n = h.shape[1]
    a, _ = act64(z[:, :n], act)
    ea = 1.2 * e[:, :n] + act_tol(a)
    u, eu = z[:, n:], e[:, n:]
    ref = a * u
    tol = ea * u.abs() + a.abs() * eu + ea * eu + E32 * ref.abs()
    near(h, ref, tol + stored(ref.abs() + tol), what + " h")
    if preact is not None:
        near(preact, z, e + stored(z.abs() + e), what + " preact")


# M across the decode kernel's row fragments, the tiles of 64, 128 and 256
# rows and their borders; N across 16-, 128- and 256-wide tiles, odd ones
# among them; K that ends inside a 64-, 128- or 256-deep step.
FWD = [
    # M, N, K, bits, gs, sym, act_order, act, bias, residual
    (1, 16, 32, 4, 32, False, False, "none", False, False),
    (1, 1, 64, 4, 64, True, False, "silu", True, True),
    (1, 4096, 1024, 4, 128, False, False, "none", True, True),
    (2, 33, 288, 3, 32, False, True, "gelu", True, False),
    (7, 520, 2080, 2, 32, True, False, "relu", False, True),
    (15, 257, 320, 8, 160, False, False, "gelu_tanh", True, True),
    (16, 64, 8192, 4, 128, False, False, "none", False, True),       # K split, few tiles
    (17, 48, 8192, 8, -1, False, False, "silu", True, False),        # two row fragments, K split
    (32, 1000, 544, 4, 32, False, True, "silu", True, True),
    (33, 255, 96, 4, 96, False, False, "gelu", True, True),
    (33, 300, 8224, 3, 32, False, False, "gelu", True, True),        # split tiles
    (64, 256, 4096, 4, 128, True, False, "none", False, False),
    (65, 511, 224, 2, 32, False, True, "relu", True, True),
    (129, 1025, 160, 8, 32, False, False, "gelu_tanh", False, True),
    (257, 770, 1120, 3, -1, False, False, "silu", True, False),
    (300, 4104, 352, 4, 32, False, False, "gelu", True, True),
    (512, 33000, 96, 4, 32, False, False, "silu", True, True),       # many tiles
    (1030, 16384, 64, 2, 64, False, False, "none", False, True),
    (1030, 16391, 64, 8, 64, False, False, "gelu", True, True),      # rows not 16-byte aligned
]


@pytest.mark.parametrize("M,N,K,bits,gs,sym,ao,act,bias,res", FWD)
def test_linear_act(M, N, K, bits, gs, sym, ao, act, bias, res):
    L = make_layer(1, N, K, bits, gs, sym, ao)
    x = randn(2, M, K)
    b = randn(3, N, sigma=0.3) if bias else None
    r = randn(4, M, N) if res else None
    y, z = wq.linear_act(x, *L["args"], perm=L["perm"], bias=b, residual=r, act=act, save_preact=True)
    check_linear(L, x, b, r, act, y, z, "linear")
    # without the pre-activations, in place over the residual
    out = None if r is None else r.clone()
    y2 = wq.linear_act(x, *L["args"], perm=L["perm"], bias=b, residual=out, act=act, out=out)
    assert torch.equal(y2, y)


@pytest.mark.parametrize("M,N,K,bits,gs,sym,ao,act,bias,res", FWD)
def test_gated(M, N, K, bits, gs, sym, ao, act, bias, res):
    L = make_layer(5, 2 * N, K, bits, gs, sym, ao)
    x = randn(6, M, K)
    b = randn(7, 2 * N, sigma=0.3) if bias else None
    h, z = wq.gated(x, *L["args"], perm=L["perm"], bias=b, act=act, save_preact=True)
    check_gated(L, x, b, act, h, z, "gated")
    assert torch.equal(wq.gated(x, *L["args"], perm=L["perm"], bias=b, act=act), h)


BWD = [
    # M, N, K, bits, gs, sym, act_order, act, add, dbias
    (1, 1, 32, 4, 32, False, False, "none", False, True),
    (1, 5, 64, 2, 64, True, False, "silu", True, True),
    (1, 4096, 1024, 4, 128, False, False, "none", True, False),
    (3, 33, 288, 3, 32, False, True, "gelu", True, True),
    (16, 8192, 64, 4, 64, False, False, "relu", False, True),        # split over the weight rows
    (31, 257, 320, 8, 160, False, False, "gelu_tanh", True, True),
    (64, 64, 544, 4, 32, False, False, "silu", False, False),
    (65, 130, 96, 4, 96, False, True, "none", True, True),
    (100, 4104, 256, 3, -1, False, False, "silu", True, True),
    (129, 250, 224, 2, 32, False, False, "relu", True, False),
    (130, 63, 8224, 8, 32, True, False, "gelu", False, True),
    (257, 520, 2080, 4, 32, False, True, "silu", True, True),
    (300, 65, 4128, 4, 32, False, False, "gelu_tanh", True, True),
    (512, 96, 33024, 4, 128, False, False, "silu", True, False),     # many tiles
    (1030, 72, 16416, 3, 96, False, False, "none", True, True),
    (1031, 71, 16384, 2, 64, False, False, "gelu", False, True),
]


def dz_ref(op, dy, z, act):
    d = dy.double()
    n = d.shape[1]
    if z is None:
        return d, torch.zeros_like(d)
    z = z.double()
    a, s = act64(z[:, :n], act)
    # slopes: sums of up to three terms of size 1 + |v|, each within the
    # activation's error
    es = 2.0 ** -18 * (1 + z[:, :n].abs()) if act not in ("none", "relu") else torch.zeros_like(s)
    if op == "linear":
        return d * s, d.abs() * es
    u = z[:, n:]
    return (torch.cat([d * u * s, d * a], 1),
            torch.cat([(d * u).abs() * (es + 2 * E32 * s.abs()), d.abs() * (act_tol(a) + E32 * a.abs())], 1))


def check_backward(op, L, dy, z, act, add, dx, dz, dbias, what):
    ref, e = dz_ref(op, dy, z, act)
    if dz is not None:
        near(dz, ref, e + stored(ref.abs() + e), what + " dz")
    else:  # the operand may differ by its rounding and error
        dz = ref
    if dbias is not None:
        t = e.sum(0) + (dy.shape[0] + 2) * E32 * (ref.abs() + e).sum(0)
        near(dbias, ref.sum(0), t, what + " dbias")
    # the product itself, on the fp16 operand the kernel wrote
    w = L["w"]
    dxr = dz.double() @ w
    t = 2 * (w.shape[0] + 8) * E32 * (dz.double().abs() @ w.abs())
    if dz is ref:
        t = t + (e + stored(ref.abs() + e)) @ w.abs()
    if add is not None:
        dxr = dxr + add.double()
        t = t + E32 * dxr.abs()
    near(dx, dxr, t + stored(dxr.abs() + t), what + " dx")


@pytest.mark.parametrize("op", ["linear", "gated"])
@pytest.mark.parametrize("M,N,K,bits,gs,sym,ao,act,add,db", BWD)
def test_backward(op, M, N, K, bits, gs, sym, ao, act, add, db):
    rows = 2 * N if op == "gated" else N
    f = wq.gated_backward if op == "gated" else wq.linear_act_backward
    L = make_layer(11, rows, K, bits, gs, sym, ao)
    dy = randn(12, M, N)
    z = randn(13, M, rows, sigma=2.0) if op == "gated" or act != "none" else None
    r = randn(14, M, K) if add else None
    dx, dz, dbias = f(dy, z, *L["args"], perm=L["perm"], act=act, dx_add=r, need_dbias=db)
    assert (dbias is not None) == db
    check_backward(op, L, dy, z, act, r, dx, dz, dbias, op)
    # without dz and dbias, in place over dx_add: the same dx
    out = None if r is None else r.clone()
    dx2, none, none2 = f(dy, z, *L["args"], perm=L["perm"], act=act, dx_add=out, need_dz=False, out=out)
    assert none is None and none2 is None and torch.equal(dx2, dx)


@pytest.mark.parametrize("entry,M,N,K,ao", [
    ("linear_act", 8, 64, 8192, False), ("linear_act", 40, 300, 8192, True), ("gated", 8, 64, 8192, True),
    ("gated", 100, 130, 8192, False), ("linear_act_backward", 20, 8192, 256, False),
    ("linear_act_backward", 20, 4100, 288, True), ("gated_backward", 70, 4100, 256, False)])
def test_smallest_workspace(entry, M, N, K, ao):
    """With only the part of the workspace that cannot be left out the results
    hold; one byte less is refused.  What the workspace held does not matter."""
    is_gated, back = entry.startswith("gated"), entry.endswith("backward")
    rows = 2 * N if is_gated else N
    L = make_layer(21, rows, K, 4, 32, False, ao)
    full = wq.block_workspace_size(entry, M, N, K, 4, ao)
    r256 = lambda b: (b + 255) // 256 * 256  # noqa: E731
    if not back:
        least = r256(M * K * 2) if ao else 0
        x = randn(22, M, K)
        call = lambda ws: getattr(wq, entry)(x, *L["args"], perm=L["perm"], act="silu", workspace=ws)  # noqa: E731
    else:
        tiles = -(-M // 64) * -(-K // 256)
        least = r256(M * ((rows + 7) // 8 * 8) * 2) + (tiles * 64 * 256 * 4 if ao else 0)
        dy, z = randn(23, M, N), randn(24, M, rows)
        call = lambda ws: getattr(wq, entry)(dy, z, *L["args"], perm=L["perm"], act="silu", need_dz=False,  # noqa: E731
                                             workspace=ws)[0]
    assert full > least, "the shape has to have an optional part"
    tensor = lambda n, v: torch.full((n,), v, dtype=torch.uint8, device="cuda")  # noqa: E731
    a, b = call(tensor(full, 0xFF)), call(tensor(full, 0x3C))
    assert torch.equal(a, b)
    c = call(tensor(max(least, 1), 0xFF))
    for y in (a, c):
        if not back:
            (check_gated(L, x, None, "silu", y, None, entry) if is_gated else
             check_linear(L, x, None, None, "silu", y, None, entry))
        else:
            check_backward("gated" if is_gated else "linear", L, dy, z, "silu", None, y, None, None, entry)
    if least:
        with pytest.raises(wq.WQError) as err:
            call(tensor(least - 1, 0))
        assert err.value.status == wq.WQ_ERR_ARG


@pytest.mark.parametrize("M", [3, 40, 300])
def test_rows_are_independent(M):
    """NaN and infinities in some rows leave the others bit for bit."""
    N, K = 136, 288
    L = make_layer(31, 2 * N, K, 4, 32)
    x = randn(32, M, K)
    h, z = wq.gated(x, *L["args"], save_preact=True)
    bad = x.clone()
    bad[1, 5], bad[M - 1, K - 1] = float("nan"), float("inf")
    h2, z2 = wq.gated(bad, *L["args"], save_preact=True)
    keep = [m for m in range(M) if m not in (1, M - 1)]
    assert torch.equal(h2[keep], h[keep]) and torch.equal(z2[keep], z[keep])
    assert torch.isnan(z2[1]).all()
    inf_ref = bad[M - 1].double() @ L["w"].T
    fin = ~torch.isnan(inf_ref)
    assert torch.equal(z2[M - 1].double()[fin], inf_ref[fin]) and torch.isnan(z2[M - 1][~fin]).all()
    dh = randn(33, M, N)
    dx, dz, _ = wq.gated_backward(dh, z, *L["args"])
    dhb = dh.clone()
    dhb[1, 3], dhb[M - 1, N - 1] = float("nan"), float("inf")
    dx2, dz2, _ = wq.gated_backward(dhb, z, *L["args"])
    assert torch.equal(dx2[keep], dx[keep]) and torch.equal(dz2[keep], dz[keep])
    assert torch.isnan(dx2[1]).all()


@pytest.mark.parametrize("act", ACTS)
def test_activation_limits(act):
    """Pre-activations at the ends of fp16's range, at infinities and NaN: the
    derivative and the activation take their limits, NaN stays NaN."""
    inf = float("inf")
    v = torch.tensor([0.0, -0.0, 1e-7, -1e-7, 20.0, -20.0, 90.0, -90.0, 65504.0, -65504.0, inf, -inf, float("nan")],
                     device="cuda").half()
    n = v.numel()
    L = make_layer(41, 2 * n, 32, 8, 32)
    z = torch.cat([v, torch.ones_like(v)]).view(1, 2 * n).contiguous()
    dh = torch.ones(1, n, device="cuda").half()
    _, dz, _ = wq.gated_backward(dh, z, *L["args"], act=act)
    dg, du = dz[0, :n].double(), dz[0, n:].double()
    a, s = act64(v.double(), act)
    far = v.double().abs() >= 90
    a = torch.where(far & (v > 0), v.double(), torch.where(far & (act != "none"), torch.zeros_like(a), a))
    if act == "none":
        a = v.double()
    s = torch.where(far, (v > 0).double() if act != "none" else torch.ones_like(s), s)
    ok = ~torch.isnan(v)
    fin = ok & torch.isfinite(a)
    assert ((du - a).abs()[fin] <= (act_tol(a) + stored(a))[fin]).all()
    assert torch.equal(du[ok & ~torch.isfinite(a)], a[ok & ~torch.isfinite(a)])
    assert ((dg - s).abs()[ok] <= (2.0 ** -18 * (1 + v.double().abs().clamp(max=100)) + stored(s))[ok]).all()
    assert torch.isnan(du[~ok]).all()
    assert torch.isnan(dg[~ok]).all() or act == "none"


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradient_against_differences(act):
    """dx of the whole block against central differences of its 64-bit loss
    sum(c * y).  The kernel's gradient is taken at fp16 pre-activations and
    passes fp16 dh and dz: each rounding moves the directional derivative by
    at most u of the sum of the magnitudes along its path, of which there are
    five (g's and u's rounding with slope and curvature, both bounded by
    1.2 + |z|; dh, dz, dx); the difference quotient's own error, of the order
    of eps^2 = 1e-8, is far below the sixth u."""
    M, I, K, N = 5, 32, 64, 32
    gu, down = make_layer(51, 2 * I, K, 4, 32), make_layer(52, N, I, 4, 32)
    x, c = randn(54, M, K), randn(55, M, N)
    mlp = wq.QuantizedGatedMLP(wq.QuantizedLinear(*gu["args"][:3], 4, 32, K),
                               wq.QuantizedLinear(*down["args"][:3], 4, 32, I), act=act)
    y, z = mlp(x, save=True)
    dx, dz, dh = mlp.backward(c, z)
    v = dx.double()  # the steepest direction

    def loss(xx):
        zz = xx @ gu["w"].T
        return (c.double() * ((act64(zz[:, :I], act)[0] * zz[:, I:]) @ down["w"].T)).sum()

    eps = 1e-4
    diff = (loss(x.double() + eps * v) - loss(x.double() - eps * v)) / (2 * eps)
    got = (v * v).sum()
    zz = (x.double() @ gu["w"].T).abs()
    dhm = c.double().abs() @ down["w"].abs()
    path = torch.cat([dhm * zz[:, I:] * (1.2 + zz[:, :I]), dhm * (zz[:, :I] + 1.2)], 1) @ gu["w"].abs()
    tol = 6 * U * (path * v.abs()).sum()
    assert (got - diff).abs() <= tol, (got.item(), diff.item(), tol.item())
    # the bound has to bite: a gradient that misses one factor would fail
    assert tol < 0.5 * got


def test_block_forward_backward_run():
    """Gate/up, down with the residual, and back, as a user runs them, on odd
    sizes with act-order, an AWQ scale and mixed widths."""
    M, K, I = 45, 288, 416
    gu, down = make_layer(61, 2 * I, K, 4, 32, act_order=True), make_layer(62, K, I, 3, 32)
    mlp = wq.QuantizedGatedMLP(wq.QuantizedLinear(*gu["args"][:3], 4, 32, K, perm=gu["perm"]),
                               wq.QuantizedLinear(*down["args"][:3], 3, 32, I))
    x = randn(63, M, K)
    y, z = mlp(x, residual=x, save=True)
    h = wq.gated(x, *gu["args"], perm=gu["perm"])
    check_gated(gu, x, None, "silu", h, z, "run")
    check_linear(down, h, None, x, "none", y, None, "run")
    assert torch.equal(y, mlp(x, residual=x))
    dy = randn(64, M, K)
    dx, dz, dh = mlp.backward(dy, z, dx_add=dy)
    check_backward("linear", down, dy, None, "none", None, dh, dy, None, "run down")
    check_backward("gated", gu, dh, z, "silu", dy, dx, dz, None, "run gate/up")
    s = (0.5 + torch.rand(K, device="cuda")).half()
    scaled = wq.QuantizedLinear(*gu["args"][:3], 4, 32, K, perm=gu["perm"], act_scale=s)
    y2, z2 = scaled.forward_act(x, act="gelu", save_preact=True)
    xs = wq.scale_act(x, s)
    check_linear(gu, xs, None, None, "gelu", y2, z2, "scaled")
    d2 = randn(65, M, 2 * I)
    dx2, dz2, _ = scaled.backward(d2, z2, act="gelu")
    plain = wq.linear_act_backward(d2, z2, *gu["args"], perm=gu["perm"], act="gelu")[0]
    assert torch.equal(dx2, wq.scale_act(plain, s))
    with pytest.raises(ValueError, match="AWQ scale"):
        scaled.backward(d2, z2, act="gelu", dx_add=x)


def test_empty_problems():
    L = make_layer(71, 48, 64, 4, 32)
    none = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    assert wq.linear_act(none, *L["args"]).shape == (0, 48)
    assert wq.gated(none, *L["args"]).shape == (0, 24)
    dx, dz, db = wq.linear_act_backward(none[:, :48].contiguous(), None, *L["args"], need_dbias=True)
    assert dx.shape == (0, 64) and torch.equal(db, torch.zeros(48, device="cuda"))
    # no weight rows: dx is an empty sum, or dx_add
    zero = (torch.empty((0, 8), dtype=torch.int32, device="cuda"), torch.empty((0, 2), dtype=torch.float16, device="cuda"),
            None, 4, 32)
    dy = torch.empty((7, 0), dtype=torch.float16, device="cuda")
    assert wq.linear_act(randn(72, 7, 64), *zero).shape == (7, 0)
    assert torch.equal(wq.linear_act_backward(dy, None, *zero)[0], torch.zeros(7, 64, device="cuda").half())
    add = randn(73, 7, 64)
    assert torch.equal(wq.linear_act_backward(dy, None, *zero, dx_add=add)[0], add)


@pytest.mark.parametrize("M", [1, 200])
def test_graph_replay(M):
    """Forward and backward captured once, replayed on new inputs between
    eager work: every replay equals the eager result."""
    K, I = 1024, 520
    gu = make_layer(81, 2 * I, K, 4, 128, act_order=True)
    x, dy = randn(83, M, K), randn(84, M, I)
    bias = randn(85, 2 * I)

    def step(x, dy):
        h, z = wq.gated(x, *gu["args"], perm=gu["perm"], bias=bias, save_preact=True)
        dx, dz, db = wq.gated_backward(dy, z, *gu["args"], perm=gu["perm"], dx_add=x, need_dbias=True)
        return h, z, dx, dz, db

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(x, dy)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(x, dy)
    for k in range(4):
        x.copy_(randn(90 + k, M, K))
        dy.copy_(randn(95 + k, M, I))
        graph.replay()
        got = [t.clone() for t in outs]
        want = step(x, dy)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own do not disturb each
    other."""
    L = make_layer(101, 1030, 4096, 4, 128)
    xs = [randn(102 + i, 150, 4096) for i in range(2)]
    ref = [wq.linear_act(x, *L["args"], act="gelu") for x in xs]
    dref = [wq.linear_act_backward(r, r, *L["args"], act="gelu")[0] for r in ref]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                y = wq.linear_act(xs[i], *L["args"], act="gelu")
                outs[i].append((y, wq.linear_act_backward(y, y, *L["args"], act="gelu")[0]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, ref[i]) and torch.equal(d, dref[i]) for y, d in outs[i])


def test_neighbouring_memory_is_left_alone():
    """Outputs inside larger buffers: nothing before or after them changes."""
    M, N, K = 37, 131, 160
    L = make_layer(111, 2 * N, K, 4, 32)
    x, dh = randn(112, M, K), randn(113, M, N)

    def inside(rows, cols):
        n = rows * cols
        whole = torch.full((64 + n + 64,), 7.0, dtype=torch.float16, device="cuda")
        return whole, whole[64:64 + n].view(rows, cols)

    wh, h = inside(M, N)
    wz, z = inside(M, 2 * N)
    wq.gated(x, *L["args"], out=h, preact=z)
    wd, dx = inside(M, K)
    wq.gated_backward(dh, z, *L["args"], out=dx)
    for w in (wh, wz, wd):
        assert (w[:64] == 7).all() and (w[-64:] == 7).all()
    check_gated(L, x, None, "silu", h, z, "inside")


def test_outputs_past_32_bit_offsets():
    """M * N past 2^31 values: sampled rows of y and of dx against 64 bits."""
    M, N, K = 70000, 32768, 64
    L = make_layer(121, N, K, 4, 32)
    x = randn(122, M, K)
    y = wq.linear_act(x, *L["args"], act="silu")
    rows = torch.tensor([0, 1, 32767, 65535, 65536, 69998, 69999], device="cuda")
    check_linear(L, x[rows], None, None, "silu", y[rows], None, "far rows")
    dx, dz, _ = wq.linear_act_backward(y, y, *L["args"], act="silu")
    check_backward("linear", L, y[rows], y[rows], "silu", None, dx[rows], dz[rows], None, "far rows")


def test_weights_past_32_bit_offsets():
    """Packed weights of more than 4 GiB, one token and a tile of rows."""
    N, K = (1 << 21) + 40, 4128
    g = torch.Generator(device="cuda")
    g.manual_seed(131)
    packed = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda", dtype=torch.int32)
    scales = torch.full((N, K // 32), 0.01, dtype=torch.float16, device="cuda")
    rows = torch.tensor([0, 77, 2 ** 20 + 3, N - 40, N - 1], device="cuda")
    q = (packed[rows].unsqueeze(-1) >> (4 * torch.arange(8, device="cuda", dtype=torch.int32))) & 15
    w = ((q.view(5, K).double() - 8) * scales[0, 0].double()).half().double()
    for M in (1, 65):
        x = randn(132, M, K)
        y = wq.linear_act(x, packed, scales, None, 4, 32)
        check_linear(dict(w=w), x, None, None, "none", y[:, rows].contiguous(), None, "far weights")
        # a gradient that is zero but at those rows
        dy = torch.zeros((M, N), dtype=torch.float16, device="cuda")
        dy[:, rows] = randn(133, M, 5)
        dx = wq.linear_act_backward(dy, None, packed, scales, None, 4, 32)[0]
        ref = dy[:, rows].double() @ w
        t = 2 * 64 * E32 * (dy[:, rows].double().abs() @ w.abs())
        near(dx, ref, t + stored(ref.abs() + t), "far weights dx")


def test_unaligned_pointers_are_refused_with_device_memory():
    L = make_layer(141, 64, 64, 4, 32)
    buf = torch.zeros(4 * 64 + 8, dtype=torch.float16, device="cuda")
    x = buf[4:4 + 4 * 64].view(4, 64)
    with pytest.raises(wq.WQError) as e:
        wq.linear_act(x, *L["args"])
    assert e.value.status == wq.WQ_ERR_ARG
    with pytest.raises(wq.WQError):
        wq.linear_act(randn(142, 4, 64), *L["args"], bias=buf[4:68])


def test_preact_must_not_be_the_output():
    L = make_layer(151, 64, 64, 4, 32)
    y = torch.empty((4, 64), dtype=torch.float16, device="cuda")
    p = ctypes.c_void_p
    st = wq.lib().wq_linear_act(p(randn(152, 4, 64).data_ptr()), p(L["args"][0].data_ptr()),
                                p(L["args"][1].data_ptr()), p(L["args"][2].data_ptr()), None, None, None, 0,
                                p(y.data_ptr()), p(y.data_ptr()), 4, 64, 64, 4, 32, None, 0, None)
    assert st == wq.WQ_ERR_ARG


@pytest.mark.parametrize("M,K", [(1, 32), (5, 96), (20, 160), (40, 96), (200, 32)])
@pytest.mark.parametrize("bits,N", [(8, 48), (8, 47), (4, 48)])
def test_codes_past_k_stay_out(M, K, bits, N):
    """Where K ends inside a kernel's step, the words behind a row are the next
    row's.  Every other row holds codes whose distance from the zero-point
    overflows fp16 with the scale of the row before it: that row's outputs
    stay finite and right.  (Zero times infinity would be NaN.)"""
    G, top, zero = K // 32, (1 << bits) - 1, 1 << (bits - 1)
    codes = np.full((N, K), zero, dtype=np.uint8)
    codes[0::2] += np.arange(K, dtype=np.uint8) % 2      # weights 0 and s
    codes[1::2] = top                                    # (top - zero) s > 65504
    s = np.float16(65504 / (top - zero) * 1.01)
    scales = np.full((N, G), s, dtype=np.float16)
    assert float(s) * (top - zero) > 65520  # rounds to infinity
    x = (randn(161, M, K, sigma=1.0) / 4096).contiguous()
    y = wq.linear_act(x, torch.from_numpy(O.pack(codes, bits).view(np.int32)).cuda(), torch.from_numpy(scales).cuda(),
                      torch.full((N, G), zero, dtype=torch.uint8, device="cuda"), bits, 32)
    w = torch.from_numpy((codes[0::2].astype(np.float64) - zero) * float(s)).cuda()
    check_linear(dict(w=w), x, None, None, "none", y[:, 0::2].contiguous(), None, "even rows")


# tiles beyond one per compute unit: whole rounds of whole tiles, and a last
# round cut along the sum
@pytest.mark.parametrize("op,M,N,K,bits,gs,ao", [
    ("linear", 300, 36002, 3200, 4, 32, False),      # 2 x 141 tiles of 256 rows, 26 of them cut
    ("linear", 1100, 17800, 3200, 4, 128, False),    # 5 x 70, 94 of them cut
    ("gated", 1100, 8001, 2080, 8, 32, True),
    ("linear_backward", 1100, 2085, 14400, 4, 64, False),
    ("linear_backward", 300, 2500, 36032, 3, 32, False),
    ("linear_backward", 300, 3200, 25600, 4, 128, False),  # 3 x 100 of 128 rows, 44 of them cut
    ("gated_backward", 1100, 1043, 14400, 4, 32, True)])
def test_rounds_of_whole_and_cut_tiles(op, M, N, K, bits, gs, ao):
    """Large products whose tiles fill the machine more than once, sampled
    columns against 64 bits, and the same call without a workspace to cut any
    tile: equal but for the order of the sums."""
    gated, back = op.startswith("gated"), op.endswith("backward")
    rows = 2 * N if gated else N
    L = make_layer(171, rows, K, bits, gs, False, ao)
    pick = torch.arange(0, M, 37, device="cuda")
    if not back:
        x = randn(172, M, K)
        least = (M * K * 2 + 255) // 256 * 256 if ao else 1
        small = torch.empty(least, dtype=torch.uint8, device="cuda")
        for ws in (None, small):
            if gated:
                h, z = wq.gated(x, *L["args"], perm=L["perm"], save_preact=True, workspace=ws)
                check_gated(L, x[pick], None, "silu", h[pick], z[pick], op)
            else:
                y, z = wq.linear_act(x, *L["args"], perm=L["perm"], act="gelu", save_preact=True, workspace=ws)
                check_linear(L, x[pick], None, None, "gelu", y[pick], z[pick], op)
        return
    dy = randn(173, M, N)
    z = randn(174, M, rows) if gated else None
    f = wq.gated_backward if gated else wq.linear_act_backward
    ld = (rows + 7) // 8 * 8
    least = (M * ld * 2 + 255) // 256 * 256 + (-(-M // 64) * -(-K // 256) * 64 * 1024 if ao else 0)
    small = torch.empty(least, dtype=torch.uint8, device="cuda")
    for ws in (None, small):
        dx, dz, _ = f(dy, z, *L["args"], perm=L["perm"], workspace=ws)
        check_backward("gated" if gated else "linear", L, dy[pick], None if z is None else z[pick],
                       "silu" if gated else "none", None, dx[pick], dz[pick] if gated else dy[pick], None, op)


@pytest.mark.parametrize("M", [1, 16, 17, 32])
@pytest.mark.parametrize("N,K,gs,bits", [(48, 4128, 32, 4), (47, 4096, 128, 4), (4100, 8192, 32, 3), (33, 65536, 32, 4),
                                         (130, 2080, 32, 8)])
def test_decode_batches_however_scales_lie(M, N, K, gs, bits):
    """Scales that start off 16 bytes, that do not fill whole 16 bytes, or too
    many of them to stay in LDS take another way to the decode kernel, with
    the same sums: bit for bit."""
    for f, rows in ((wq.linear_act, N), (wq.gated, 2 * N)):
        L = make_layer(181, rows, K, bits, gs)
        p, s, z = L["args"][:3]
        x = randn(182, M, K)
        y = f(x, p, s, z, bits, gs)
        if f is wq.gated:
            check_gated(L, x, None, "silu", y, None, "decode")
        else:
            check_linear(L, x, None, None, "none", y, None, "decode")
        ws = torch.empty(s.numel() + 1, dtype=s.dtype, device="cuda")
        wz = torch.empty(z.numel() + 1, dtype=z.dtype, device="cuda")
        s2, z2 = ws[1:].view_as(s).copy_(s), wz[1:].view_as(z).copy_(z)
        assert torch.equal(f(x, p, s2, z2, bits, gs), y)


def test_decode_without_workspace():
    """A decode batch whose K has to be split falls back where there is no room
    for the partial sums."""
    M, N, K = 20, 64, 8192
    L = make_layer(191, N, K, 4, 128)
    x = randn(192, M, K)
    assert wq.block_workspace_size("linear_act", M, N, K, 4, False) > 0
    y = wq.linear_act(x, *L["args"], workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    check_linear(L, x, None, None, "none", y, None, "no room")


@pytest.mark.parametrize("M", [3, 70])
def test_subnormal_weights_and_inputs(M):
    """fp16's subnormals count: weights below 2^-14 (scales of a few steps of
    2^-24) times ordinary inputs, and ordinary weights times subnormal
    inputs, forward and backward."""
    N, K = 144, 288
    L = make_layer(201, N, K, 4, 32)
    p, s, z, bits, gs = L["args"]
    tiny = (torch.arange(1, s.numel() + 1, device="cuda") % 37 + 1).view_as(s) * 2.0 ** -24
    q = torch.from_numpy(O.unpack(p.cpu().numpy().view(np.uint32), 4, K)).cuda().double()
    w = ((q - z.double().repeat_interleave(32, 1)) * tiny.double().repeat_interleave(32, 1)).half().double()
    x, dy = randn(202, M, K, sigma=1000.0), randn(203, M, N, sigma=1000.0)
    T = dict(w=w)
    y = wq.linear_act(x, p, tiny.half(), z, bits, gs)
    assert y.abs().max() > 2.0 ** -10
    check_linear(T, x, None, None, "none", y, None, "tiny weights")
    dx, dz, _ = wq.linear_act_backward(dy, None, p, tiny.half(), z, bits, gs)
    check_backward("linear", T, dy, None, "none", None, dx, dy, None, "tiny weights")
    x, dy = randn(204, M, K, sigma=2.0 ** -18), randn(205, M, N, sigma=2.0 ** -18)
    check_linear(L, x, None, None, "none", wq.linear_act(x, *L["args"]), None, "tiny inputs")
    dx, dz, _ = wq.linear_act_backward(dy, None, *L["args"])
    check_backward("linear", L, dy, None, "none", None, dx, dy, None, "tiny inputs")
