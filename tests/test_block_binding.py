"""What the feed-forward block's Python functions refuse before the library is
called, on the CPU (tensors without memory)."""

import ctypes

import pytest

import weight_only_int4_wq_amd as wq

torch = pytest.importorskip("torch")


def meta(*shape, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device="meta")


FORWARD, BACKWARD = (wq.linear_act, wq.gated), (wq.linear_act_backward, wq.gated_backward)
WIDE = 1 << 32


def call(fn, M, N, K, **more):
    """fn on a 2-bit layer of one group, N output columns."""
    is_gated = fn in (wq.gated, wq.gated_backward)
    rows = 2 * N if is_gated else N
    layer = (meta(rows, K // 16, dtype=torch.int32), meta(rows, 1), None, 2, -1)
    if fn in FORWARD:
        return fn(meta(M, K), *layer, **more)
    return fn(meta(M, N), meta(M, rows), *layer, **more)


@pytest.mark.parametrize("fn", FORWARD + BACKWARD)
@pytest.mark.parametrize("M,N,K", [(1, 2, WIDE + 64), (1, WIDE + 2, 32), (WIDE + 3, 2, 32), (1, 2, 1 << 31),
                                   (1 << 31, 2, 32)])
def test_sizes_that_a_32_bit_integer_would_wrap(fn, M, N, K):
    """A size that 32 bits turn into another, valid one."""
    assert ctypes.c_int32(WIDE + 64).value == 64
    with pytest.raises(ValueError, match="2\\^31"):
        call(fn, M, N, K)


@pytest.mark.parametrize("entry", ["linear_act", "gated", "linear_act_backward", "gated_backward"])
def test_workspace_of_sizes_that_a_32_bit_integer_would_wrap(entry):
    assert wq.block_workspace_size(entry, 33, 64, 4096, 4, True) > 0
    for M, N, K in ((WIDE + 33, 64, 4096), (33, WIDE + 64, 4096), (33, 64, WIDE + 4096)):
        with pytest.raises(ValueError, match="2\\^31"):
            wq.block_workspace_size(entry, M, N, K, 4, True)


def needs(t):
    return t.requires_grad_()


@pytest.mark.parametrize("fn", FORWARD + BACKWARD)
def test_a_lost_gradient_is_said(fn, recwarn):
    """The functions record nothing for autograd: a tensor that requires a
    gradient is accepted with a warning, and without one where no graph is
    recorded.  (The calls end at the check for GPU tensors.)"""
    rows = 4 if fn in (wq.gated, wq.gated_backward) else 2
    layer = (meta(rows, 4, dtype=torch.int32), meta(rows, 1), None, 2, -1)
    if fn in FORWARD:
        cases = [((needs(meta(3, 64)), *layer), {}), ((meta(3, 64), *layer), dict(bias=needs(meta(rows))))]
        if fn is wq.linear_act:
            cases.append(((meta(3, 64), *layer), dict(residual=needs(meta(3, 2)))))
        plain = (meta(3, 64), *layer)
    else:
        z = meta(3, rows)
        cases = [((needs(meta(3, 2)), z, *layer), {}), ((meta(3, 2), needs(meta(3, rows)), *layer), {}),
                 ((meta(3, 2), z, *layer), dict(dx_add=needs(meta(3, 64))))]
        plain = (meta(3, 2), z, *layer)
    for args, more in cases:
        more.update(act="silu")
        with pytest.warns(UserWarning, match="no gradient"), pytest.raises(ValueError, match="GPU tensors"):
            fn(*args, **more)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU tensors"):
            fn(*args, **more)
    with pytest.raises(ValueError, match="GPU tensors"):
        fn(*plain, act="silu")
    assert len(recwarn) == 0


def test_a_gradient_lost_at_the_awq_scale_is_said():
    """Where the AWQ scale is applied first, its result would hide that x
    requires a gradient."""
    layer = wq.QuantizedLinear(meta(4, 4, dtype=torch.int32), meta(4, 1), None, 2, -1, 64, act_scale=meta(64))
    for f in (layer.forward_act, wq.QuantizedGatedMLP(layer, wq.QuantizedLinear(
            meta(5, 2, dtype=torch.int32), meta(5, 1), None, 32, -1, 2))):
        with pytest.warns(UserWarning, match="no gradient"), pytest.raises(ValueError, match="GPU tensors"):
            f(needs(meta(3, 64)))


def test_wrong_types_are_still_named():
    layer = (meta(2, 4, dtype=torch.int32), meta(2, 1), None, 2, -1)
    with pytest.raises(ValueError, match="bias must be a torch tensor"):
        wq.linear_act(meta(3, 64), *layer, bias=[0.0, 0.0])
    with pytest.raises(ValueError, match="dx_add must be a torch tensor"):
        wq.linear_act_backward(meta(3, 2), None, *layer, dx_add=1.0)


class OnDevice:
    """Stands for a tensor on GPU `index`."""
    requires_grad = False

    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.mark.parametrize("index", [0, 1])
def test_the_awq_scale_runs_on_the_tensors_device(index, monkeypatch):
    """Like the products themselves: the tensors' device is the current one
    while the library is called, whichever was current before."""
    current = [0]

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    seen = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(wq, "scale_act", lambda x, s: seen.append(current[0]))
    layer = wq.QuantizedLinear(meta(4, 4, dtype=torch.int32), meta(4, 1), None, 2, -1, 64, act_scale=meta(64))
    layer._scaled(OnDevice(index))
    assert seen == [index] and current == [0]


def test_sizes_whose_sum_alone_is_large():
    """Large sizes that each fit in 32 bits go to the library's own checks."""
    with pytest.raises(ValueError, match="GPU tensors"):
        call(wq.linear_act, 1 << 30, 1 << 21, 1 << 22)
    with pytest.raises(ValueError, match="GPU tensors"):
        call(wq.linear_act, (1 << 31) - 1, 1 << 21, 1 << 22)
