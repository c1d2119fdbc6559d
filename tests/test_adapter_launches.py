"""What the adapters' and dropout's entry points ask of the HIP runtime, on the
CPU: the recorder of the block's launches stands in for the runtime.  The calls
pass made-up device addresses, which nothing follows."""

import json
import shutil
import subprocess
import sys
import textwrap

import pytest

import weight_only_int4_wq_amd as wq
from test_block_launches import RECORDER, ROOT

torch = pytest.importorskip("torch")

pytestmark = [
    pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes made-up device addresses"),
    pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler"),
]

RUNNER = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
import weight_only_int4_wq_amd as wq
class Launch(ctypes.Structure):
    _fields_ = [("fn", ctypes.c_void_p)] + [(n, ctypes.c_uint32) for n in ("gx", "gy", "gz", "bx", "by", "bz")] + \
        [("lds", ctypes.c_uint64)]
out = []
for entry, a in json.loads(sys.stdin.read()):
    rec.recorded_clear()
    at = lambda n: (n + 1) << 50
    M, N, K, R, L, p = (a.get(k, d) for k, d in (("M", 1), ("N", 64), ("K", 64), ("R", 16), ("L", 1), ("p", 0.0)))
    slots = at(0) if a.get("slots") else None
    tail = [M, N, K, R, L]
    if entry == "wq_dropout":
        need, args = 0, [at(1), at(2) if a.get("add") else None, p, 1, 2, None, at(3), a["n"]]
    elif entry == "wq_adapters":
        need = wq.lib().wq_adapters_workspace_size(*tail, int(p > 0))
        args = [at(1), at(2), at(3), at(4), slots, at(5) if a.get("add") else None, p, 1, 2, None, at(6), None, *tail,
                at(7) if need else None, need]
    else:
        need = wq.lib().wq_adapters_backward_workspace_size(*tail)
        w = a.get("weights", True)
        args = [at(1), at(2), at(3), at(4), at(5), at(6), slots, p, 1, 2, None, None, at(8) if a.get("dx", True) else None,
                at(9) if w else None, at(10) if w else None, *tail, at(11), need]
    status = getattr(wq.lib(), entry)(*args, None)
    q = ctypes.POINTER(Launch)()
    n = rec.recorded_launches(ctypes.byref(q))
    out.append({"status": status, "workspace": need,
                "launches": [{f: getattr(q[i], f) for f, _ in Launch._fields_} for i in range(n)]})
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    wq.lib()
    where = tmp_path_factory.mktemp("recorder")
    (where / "recorder.c").write_text(RECORDER)
    lib = str(where / "librecorder.so")
    r = subprocess.run(["gcc", "-std=c99", "-O1", "-shared", "-fPIC", str(where / "recorder.c"), "-o", lib],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    (where / "runner.py").write_text(textwrap.dedent(RUNNER))

    def go(calls):
        r = subprocess.run([sys.executable, str(where / "runner.py"), lib, ROOT], input=json.dumps(calls),
                           capture_output=True, text=True, timeout=100)
        assert r.returncode == 0, r.stderr[-2000:]
        return json.loads(r.stdout.splitlines()[-1])

    return go


def within_limits(got):
    assert got["status"] == 0 and 0 < len(got["launches"]) < 200
    for q in got["launches"]:
        assert 0 < q["gx"] * q["bx"] < 1 << 32 and 0 < q["gy"] <= 65535 and 0 < q["gz"] <= 65535, q
        assert q["bx"] * q["by"] * q["bz"] <= 1024 and q["lds"] <= 65536


BIG = 1 << 22
SIZES = [dict(M=M, N=N, K=K, R=R, L=L, slots=slots, p=p)
         for M, N, K, L in ((1, 1, 32, 1), (1, BIG, BIG, 1), (5, 7, 64, 1 << 20), (16, 8, 64, 70000), (64, 129, 96, 64),
                            (300, 4096, 4096, 1 << 20), (4099, 72, 64, 33000), ((1 << 22) + 1, 130, 64, 3),
                            (1 << 28, 9, 64, 2), (1 << 28, 3, 32, 40000))
         for R in (1, 17, 128) for slots in (False, True) for p in (0.0, 0.5)]


@pytest.mark.parametrize("entry", ["wq_adapters", "wq_adapters_backward"])
def test_launches_stay_within_limits(run, entry):
    for size, got in zip(SIZES, run([(entry, s) for s in SIZES])):
        try:
            within_limits(got)
        except AssertionError as e:
            raise AssertionError(f"{size}: {e}")


def test_backward_launches_what_is_asked_for(run):
    size = dict(M=500, N=4096, K=4096, R=16, L=1)
    both, dx, weights = run([("wq_adapters_backward", {**size, **m}) for m in ({}, dict(weights=False), dict(dx=False))])
    assert len(both["launches"]) >= len(weights["launches"]) > len(dx["launches"]) == 2


def test_dropout_launches(run):
    calls = [dict(n=n, add=add, p=0.1) for n in (1, 8, 2049, (1 << 22) * 8, (1 << 33) + 5, 1 << 40) for add in (0, 1)]
    for a, got in zip(calls, run([("wq_dropout", c) for c in calls])):
        within_limits(got)
        done = sum(q["gx"] * q["bx"] for q in got["launches"])
        per = 8 if a["n"] <= 8 * 256 * 2048 else 32    # elements of a thread
        assert done * per >= a["n"] > (done - 256) * per


def test_one_launch_for_a_few_rows(run):
    """One launch and no workspace for up to four rows to an adapter without
    dropout; two otherwise."""
    got = run([("wq_adapters", {**dict(N=4096, K=4096), **m}) for m in (
        dict(M=1), dict(M=16, L=16, slots=True), dict(M=4), dict(M=5), dict(M=1, p=0.1), dict(M=1, R=17),
        dict(M=1, K=4128), dict(M=17, L=16, slots=True))])
    assert [len(g["launches"]) for g in got] == [1, 1, 1, 2, 2, 2, 2, 2]
    assert [g["workspace"] > 0 for g in got] == [False] * 3 + [True] * 5
