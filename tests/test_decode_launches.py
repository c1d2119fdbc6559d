"""The matrix-core decode kernel's shared-memory limit, as the recorder of the
HIP calls sees it on the CPU (made-up device addresses, which nothing
follows)."""

import json
import subprocess
import sys

from test_block_launches import RECORDER, ROOT, pytestmark  # noqa: F401

# a device of 256 compute units and 160 KB of shared memory
DEVICE = r"""
int hipGetDevice(int *dev) { *dev = 0; return 0; }
int hipDeviceGetAttribute(int *v, int attr, int dev) {
    *v = attr == 63 ? 256 : attr == 74 ? 160 * 1024 : 0;
    return 0;
}
"""

RUNNER = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
import weight_only_int4_wq_amd as wq
class Attribute(ctypes.Structure):
    _fields_ = [("fn", ctypes.c_void_p), ("attr", ctypes.c_int), ("value", ctypes.c_int)]
out = []
for M in (2, 8, 16):
    for K in (2048, 4096, 8192, 11008):
        for gs in (32, 128):
            rec.recorded_clear()
            need = wq.lib().wq_workspace_size(M, 4096, K, 4, 0)
            st = wq.lib().wq_gemv(1 << 40, 2 << 40, 3 << 40, None, None, 4 << 40, M, 4096, K, 4, gs, 5 << 40, need, None)
            p = ctypes.POINTER(Attribute)()
            n = rec.recorded_attributes(ctypes.byref(p))
            out.append([st, [[p[i].fn, p[i].value] for i in range(n)]])
print(json.dumps(out))
"""


def test_decode_kernels_limit_does_not_depend_on_the_call(tmp_path):
    (tmp_path / "recorder.c").write_text(RECORDER + DEVICE)
    lib = str(tmp_path / "librecorder.so")
    subprocess.run(["gcc", "-std=c99", "-O1", "-shared", "-fPIC", str(tmp_path / "recorder.c"), "-o", lib], check=True)
    (tmp_path / "runner.py").write_text(RUNNER)
    r = subprocess.run([sys.executable, str(tmp_path / "runner.py"), lib, ROOT], capture_output=True, text=True,
                       timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    limits = {}
    for status, attributes in json.loads(r.stdout.splitlines()[-1]):
        assert status == 0
        for fn, value in attributes:
            limits.setdefault(fn, set()).add(value)
    assert limits, "none of the layers takes more than 64 KB"
    assert all(len(v) == 1 for v in limits.values()), limits
