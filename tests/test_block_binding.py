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
