"""The adapters' grids where a kernel counts on them, on the CPU (the recorder
of test_adapter_launches.py)."""

import pytest

from test_adapter_launches import pytestmark as _marks, run  # noqa: F401

pytestmark = list(_marks)


def test_one_launch_has_blocks_for_every_adapter(run):  # noqa: F811
    """A block of the one-launch form takes one adapter's rows, 16 at most: there
    are as many in y as adapters can occur, and no such launch for more rows."""
    calls = [dict(M=M, L=L, N=N, K=K, slots=True) for M in range(1, 19) for L in (1, 2, 3, 4, 5, 16, 17, 1000)
             for N, K in ((8, 32), (4096, 4096), (12288, 4096), (640, 4128))]
    ones = 0
    for a, got in zip(calls, run([("wq_adapters", c) for c in calls])):
        assert got["status"] == 0
        one = a["M"] <= 16 and a["M"] <= 4 * a["L"] and a["K"] <= 4096
        assert len(got["launches"]) == (1 if one else 2), a
        if one:
            ones += 1
            assert got["launches"][0]["gy"] == min(a["L"], a["M"]), a
    assert ones > 200


@pytest.mark.parametrize("entry", ["wq_adapters", "wq_adapters_backward"])
def test_the_wide_cases_have_several_tiles_to_a_block(run, entry):  # noqa: F811
    """The cases of test_adapter_wide_gpu.py reach the loop over column tiles of the
    second product: its launch has fewer blocks in y than there are 512s of
    columns."""
    import test_adapter_wide_gpu as wide
    forward = entry == "wq_adapters"
    cases = wide.FORWARD if forward else wide.BACKWARD
    calls = [(entry, dict(M=M, K=K, N=N, R=R, L=L, slots=kind is not None, add=add, p=p))
             for M, K, N, R, L, kind, add, p in cases]
    for case, got in zip(cases, run(calls)):
        C = case[2] if forward else case[1]
        at = 1 + (not forward and case[2] < 8)   # (a narrow dy has its lists made by a launch of their own)
        launch = got["launches"][at]
        assert launch["bx"] == 256 and launch["gx"] == -(-case[0] // 64), (case, got)
        assert launch["gy"] < -(-C // 512), (case, launch)
