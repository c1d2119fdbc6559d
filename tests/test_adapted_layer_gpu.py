"""AdaptedLinear over every kind of quantized layer: bits, groups, symmetric
codes, act-order and an AWQ input scale, whose division is the layer's alone: the
adapters take x itself.  Under the tolerances of test_adapter_gpu.py beside the
layer's own output and gradient, which tests of their own hold."""

import pytest

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402
from test_adapter_gpu import OFFSET, SEED, Pool, check_backward, check_forward, make_slots, randn  # noqa: E402
from test_block_gpu import make_layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


def layer_of(N, K, bits, gs, sym, act_order, awq):
    Lay = make_layer(91, N, K, bits, gs, sym=sym, act_order=act_order)
    packed, scales, zeros, bits, gs = Lay["args"]
    s = (randn(92, K).abs() + 0.5).half() if awq else None
    return wq.QuantizedLinear(packed, scales, zeros, bits, gs, K, perm=Lay["perm"], act_scale=s), Lay["w"], s


@pytest.mark.parametrize("bits,gs,sym,act_order,awq", [(4, 128, False, False, True), (4, 128, False, True, False),
                                                       (4, 32, True, True, True), (3, 64, False, False, True),
                                                       (8, -1, False, False, False), (3, 128, True, True, False)])
@pytest.mark.parametrize("M,p", [(1, 0.0), (9, 0.0), (33, 0.25), (150, 0.1)])
def test_forward_and_backward(bits, gs, sym, act_order, awq, M, p):
    K, N, R, L = 512, 328, 16, 3
    base, w, s = layer_of(N, K, bits, gs, sym, act_order, awq)
    P, x, slots = Pool(95, L, R, N, K), randn(1, M, K), make_slots("random", M, L)
    layer = wq.AdaptedLinear(base, *P.args)
    bias, res, drop = randn(7, N), randn(8, M, N), dict(p=p, seed=SEED, offset=OFFSET)
    z = base.forward_act(x, bias=bias, residual=res)
    if awq:   # of the scaled x, the adapters' of x (the two differ)
        scaled = wq.scale_act(x, s)
        assert not torch.equal(scaled, x)
        plain = scaled.double() @ w.T + bias.double() + res.double()
        assert (z.double() - plain).abs().max() <= 0.01 * plain.abs().max()
    y, hidden = layer(x, slots, bias=bias, residual=res, save_hidden=True, **drop)
    check_forward(P, x, slots, z, p, y, hidden, "layer")
    dy = randn(4, M, N, sigma=0.1)
    dz = base.backward(dy)[0]
    dx, ddown, dup = layer.backward(dy, x, hidden, slots, **drop)
    check_backward(P, dy, x, hidden, slots, dz, p, dx, ddown, dup, "layer")
    dx2, none, none_too = layer.backward(dy, x, hidden, slots, need_weights=False, **drop)
    assert torch.equal(dx2, dx) and none is None and none_too is None


def test_empty_batch():
    base, _, _ = layer_of(328, 512, 4, 128, False, True, True)
    P = Pool(95, 3, 16, 328, 512)
    layer = wq.AdaptedLinear(base, *P.args)
    x, slots = torch.empty(0, 512, device="cuda").half(), torch.empty(0, dtype=torch.int32, device="cuda")
    y, hidden = layer(x, slots, save_hidden=True)
    assert y.shape == (0, 328) and hidden.shape == (0, 16)
    dx, ddown, dup = layer.backward(y, x, hidden, slots)
    assert dx.shape == (0, 512) and not ddown.any() and not dup.any()


def test_graph_replay():
    """A training step's calls on one layer, captured once, with other inputs and
    other masks in every replay."""
    M, K, N, R, L = 70, 512, 328, 16, 3
    base, _, _ = layer_of(N, K, 4, 128, False, False, True)
    P, x, slots, dy = Pool(95, L, R, N, K), randn(1, M, K), make_slots("runs", M, L), randn(4, M, N, sigma=0.1)
    layer, step = wq.AdaptedLinear(base, *P.args), torch.zeros(1, dtype=torch.int64, device="cuda")

    def calls(step, offset):
        drop = dict(p=0.2, seed=SEED, offset=offset, step=step)
        y, h = layer(x, slots, save_hidden=True, **drop)
        return (y, h) + layer.backward(dy, x, h, slots, **drop)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls(step, 9)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(step, 9)
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
