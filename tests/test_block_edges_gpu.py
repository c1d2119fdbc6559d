"""The feed-forward block's products at the ends of what their header allows,
on the GPU against plain 64-bit implementations, with the layers, references
and tolerances of the other sizes' tests."""

import pytest

torch = pytest.importorskip("torch")
import weight_only_int4_wq_amd as wq  # noqa: E402
from test_block_gpu import check_backward, check_gated, check_linear, make_layer, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wq.lib()


def test_more_pieces_than_a_launch_holds():
    """Act-order's gradient of 2^20 rows by 16384 channels: 2^24 groups of four
    rows of a tile and some more, of which a launch takes 2^24 - 1 at a time.
    Sampled rows, the first, the last and those of the last groups among them."""
    M, N, K = (1 << 20) + 5, 8, 16384
    torch.cuda.empty_cache()
    need = wq.block_workspace_size("linear_act_backward", M, N, K, 4, True) + 2 * M * K
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip("not enough memory")
    L = make_layer(301, N, K, 4, 128, act_order=True)
    dy = randn(302, M, N)
    dx, _, _ = wq.linear_act_backward(dy, None, *L["args"], perm=L["perm"])
    rows = torch.cat([torch.arange(0, M, 9973), torch.arange(M - 300, M)]).cuda()
    check_backward("linear", L, dy[rows], None, "none", None, dx[rows], dy[rows], None, "far pieces")
    del dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K", [(20, 262144 + 4096), (2, 524288 + 4096)])
def test_decode_batches_of_very_long_rows(M, K):
    """Rows longer than the decode kernel's ranges hold."""
    N = 17
    L = make_layer(311, 2 * N, K, 4, 128)
    x = randn(312, M, K)
    y = wq.linear_act(x, *L["args"], act="relu")
    check_linear(L, x, None, None, "relu", y, None, "long rows")
    check_gated(L, x, None, "silu", wq.gated(x, *L["args"]), None, "long rows")
