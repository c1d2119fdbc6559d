"""What the feed-forward block's entry points ask of the HIP runtime, on the
CPU: a small library that records kernel attributes and launches, and runs
nothing, stands in for the runtime's functions.  The calls pass made-up device
addresses, which nothing follows."""

import json
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

import weight_only_int4_wq_amd as wq

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = [
    pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes made-up device addresses"),
    pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler"),
]

RECORDER = r"""
#include <stddef.h>
#include <stdint.h>
typedef struct { uint32_t x, y, z; } dim;
typedef struct { const void *fn; uint32_t gx, gy, gz, bx, by, bz; uint64_t lds; } launch;
typedef struct { const void *fn; int attr, value; } attribute;
static launch launches[256];
static attribute attributes[256];
static int n_launches, n_attributes;
static struct { dim g, b; size_t lds; void *s; } next;
int __hipPushCallConfiguration(dim g, dim b, size_t lds, void *s) {
    next.g = g; next.b = b; next.lds = lds; next.s = s;
    return 0;
}
int __hipPopCallConfiguration(dim *g, dim *b, size_t *lds, void **s) {
    *g = next.g; *b = next.b; *lds = next.lds; *s = next.s;
    return 0;
}
int hipLaunchKernel(const void *fn, dim g, dim b, void **args, size_t lds, void *s) {
    if (n_launches < 256) launches[n_launches++] = (launch){fn, g.x, g.y, g.z, b.x, b.y, b.z, lds};
    return 0;
}
int hipFuncSetAttribute(const void *fn, int attr, int value) {
    if (n_attributes < 256) attributes[n_attributes++] = (attribute){fn, attr, value};
    return 0;
}
int hipGetLastError(void) { return 0; }
int recorded_launches(const launch **p) { *p = launches; return n_launches; }
int recorded_attributes(const attribute **p) { *p = attributes; return n_attributes; }
void recorded_clear(void) { n_launches = n_attributes = 0; }
"""

# Runs in a process of its own, where the recorder is loaded before the HIP
# runtime: `calls` is a list of (entry, arguments by name); prints what each
# returned and recorded.
RUNNER = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
import weight_only_int4_wq_amd as wq
class Launch(ctypes.Structure):
    _fields_ = [("fn", ctypes.c_void_p)] + [(n, ctypes.c_uint32) for n in ("gx", "gy", "gz", "bx", "by", "bz")] + \
        [("lds", ctypes.c_uint64)]
class Attribute(ctypes.Structure):
    _fields_ = [("fn", ctypes.c_void_p), ("attr", ctypes.c_int), ("value", ctypes.c_int)]
def recorded(kind, struct):
    p = ctypes.POINTER(struct)()
    n = getattr(rec, "recorded_" + kind)(ctypes.byref(p))
    return [{f: getattr(p[i], f) for f, _ in struct._fields_} for i in range(n)]
ORDER = {
    "wq_linear_act": "x packed scales zeros perm bias residual act y preact M N K bits gs ws wsb",
    "wq_gated": "x packed scales zeros perm bias act y preact M N K bits gs ws wsb",
    "wq_linear_act_backward": "dy preact act packed scales zeros perm add dx dz dbias M N K bits gs ws wsb",
    "wq_gated_backward": "dy preact act packed scales zeros perm add dx dz dbias M N K bits gs ws wsb",
}
out = []
for entry, given in json.loads(sys.stdin.read()):
    rec.recorded_clear()
    a = dict.fromkeys("x packed scales zeros perm bias residual y preact dy add dx dz dbias ws".split())
    a.update(act=0, M=1, N=64, K=128, bits=4, gs=32, wsb=0)
    a.update(given)
    need = getattr(wq.lib(), entry + "_workspace_size")(a["M"], a["N"], a["K"], a["bits"], int(a["perm"] is not None))
    if a["wsb"] == "queried":
        a["wsb"] = need
    status = getattr(wq.lib(), entry)(*[a[n] for n in ORDER[entry].split()], None)
    out.append({"status": status, "workspace": need, "launches": recorded("launches", Launch),
                "attributes": recorded("attributes", Attribute)})
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """run([(entry, arguments), ...]) -> what each call returned and recorded."""
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


def at(n):
    """Array n's made-up address, 1 TiB from the others."""
    return (n + 1) << 40


FORWARD = dict(x=at(0), packed=at(1), scales=at(2), y=at(3), ws=at(4), wsb="queried")
BACKWARD = dict(dy=at(0), packed=at(1), scales=at(2), dx=at(3), ws=at(4), wsb="queried")


def test_kernel_attributes_do_not_depend_on_the_call(run):
    """A kernel's shared-memory limit belongs to the process: calls from two
    threads that set it to what each of them needs could lower it under each
    other's launch.  Every call that sets a kernel's limit sets the same, and
    none launches more than that."""
    got = run([(entry, {**args, "M": M, "N": N, "K": K, "bits": bits, "gs": gs, **more})
               for entry, args, more in (("wq_linear_act", FORWARD, {}), ("wq_gated", FORWARD, {}),
                                         ("wq_linear_act_backward", BACKWARD, {}))
               for M in (1, 8, 20, 100) for N in (4096, 4128) for K in (1024, 2048, 4096, 8192) for bits in (4, 8)
               for gs in (32, 128, -1)])
    limits, most = {}, {}
    for call in got:
        assert call["status"] == 0
        for a in call["attributes"]:
            limits.setdefault((a["fn"], a["attr"]), set()).add(a["value"])
        for k in call["launches"]:
            most[k["fn"]] = max(most.get(k["fn"], 0), k["lds"])
    assert limits
    changing = {k: sorted(v) for k, v in limits.items() if len(v) > 1}
    assert not changing, changing
    for (fn, _), v in limits.items():
        assert most.get(fn, 0) <= max(v)


# ------------------------------------------------------ overlapping arrays --

M, N, K, GS = 4, 64, 128, 32


def sizes(gated):
    """Bytes of each array of 4 rows, 128 channels in, 64 out."""
    rows = 2 * N if gated else N
    g = K // GS
    return dict(x=M * K * 2, packed=rows * K // 2, scales=rows * g * 2, zeros=rows * g, perm=K * 4, bias=rows * 2,
                residual=M * N * 2, y=M * N * 2, preact=M * rows * 2, dy=M * N * 2, add=M * K * 2, dx=M * K * 2,
                dz=M * rows * 2, dbias=rows * 4, ws=1 << 20)


ENTRIES = {
    "wq_linear_act": ("y preact ws", "x packed scales zeros perm bias residual"),
    "wq_gated": ("y preact ws", "x packed scales zeros perm bias"),
    "wq_linear_act_backward": ("dx dz dbias ws", "dy preact packed scales zeros perm add"),
    "wq_gated_backward": ("dx dz dbias ws", "dy preact packed scales zeros perm add"),
}


@pytest.mark.parametrize("entry", ENTRIES)
def test_what_is_written_lies_apart(run, entry):
    """Every array that a call writes, the workspace among them, against every
    other array: one on top of the other, its last 16 bytes in the other and
    its first 16 in the other are refused before anything is launched; right
    behind the other and right before it is fine."""
    written, read = (s.split() for s in ENTRIES[entry])
    n = sizes(entry.startswith("wq_gated"))
    apart = {a: at(i) for i, a in enumerate(written + read)}
    apart.update(wsb=n["ws"], M=M, N=N, K=K, gs=GS, act=1)
    names, bad, good = [], [], []
    for i, w in enumerate(written):
        for other in written[i + 1:] + read:
            base = apart[other]
            for where in (base, base + n[other] - 16, base - n[w] + 16):
                names.append((w, other, where - base))
                bad.append((entry, {**apart, w: where}))
            good += [(entry, {**apart, w: base + n[other]}), (entry, {**apart, w: base - n[w]})]
    whole = {("y", "residual", 0), ("dx", "add", 0)}       # updates in place
    got = run(bad)
    for name, call, r in zip(names, bad, got):
        if name in whole:
            assert r["status"] == 0 and r["launches"], name
        else:
            assert r["status"] == 1 and not r["launches"], (name, call, r)
    for call, r in zip(good, run(good)):
        assert r["status"] == 0 and r["launches"], (call, r)


def test_empty_sums_lie_apart_too(run):
    """No weight rows: dx is dx_add, copied; half on top of it would be read
    after it was written."""
    size = M * K * 2
    for where, status in ((0, 0), (size, 0), (size - 16, 1), (16 - size, 1)):
        r, = run([("wq_linear_act_backward", dict(M=M, N=0, K=K, gs=GS, dx=at(0) + where, add=at(0)))])
        assert r["status"] == status, where


# --------------------------------------------------------------- launches --

def test_launches_stay_within_the_runtimes_limits(run):
    """Fewer than 2^32 threads in x and 2^16 blocks in y, up to the largest
    sizes: what a launch past them leaves undone, earlier kernels have begun."""
    big = [(1 << 20, 8, 16384), (1 << 21, 16, 16384), ((1 << 30) - 5, 16, 32), (1 << 30, 1, 32), (1 << 26, 1030, 64),
           (70000, 32768, 64), (33, 1 << 21, 4096), (257, 2048, 1 << 22), (1, 1 << 21, 1 << 22), (32, 1 << 21, 32)]
    calls = [(entry, {**(BACKWARD if entry.endswith("backward") else FORWARD), **more, "M": m, "N": n, "K": k,
                      "perm": at(7) if perm else None})
             for entry in ENTRIES for m, n, k in big for perm in (False, True)
             for more in ([dict(act=1, preact=at(8), dbias=at(9)), dict(act=1, preact=at(8))]
                          if entry.endswith("backward") else [{}])]
    far = {a: (i + 1) << 56 for i, a in enumerate("x dy packed scales y dx ws perm preact dbias".split())}
    calls = [(e, {k: far[k] if k in far and v is not None else v for k, v in a.items()}) for e, a in calls]
    for call, r in zip(calls, run(calls)):
        assert r["status"] == 0 and r["launches"], call
        for k in r["launches"]:
            assert 0 < k["gx"] * k["bx"] < 1 << 32 and 0 < k["gy"] < 1 << 16 and k["gz"] == 1, (call, k)


def test_what_no_launch_covers_is_refused_first(run):
    """More tiles than a launch holds: refused before the first kernel."""
    calls = [("wq_linear_act", {**FORWARD, "perm": (9 << 56), "M": 1 << 30, "N": 1 << 22, "K": 32}),
             ("wq_gated", {**FORWARD, "perm": (9 << 56), "M": 1 << 30, "N": 1 << 21, "K": 32}),
             ("wq_linear_act_backward", {**BACKWARD, "act": 1, "preact": 9 << 56, "M": 1 << 30, "N": 8, "K": 1 << 22})]
    far = {a: (i + 1) << 56 for i, a in enumerate("x dy packed scales y dx".split())}
    for e, a in calls:
        a.update({k: v for k, v in far.items() if k in a}, ws=8 << 56, wsb=1 << 52)
    for call, r in zip(calls, run(calls)):
        assert r["status"] == 1 and not r["launches"], (call, r["status"], len(r["launches"]))


@pytest.mark.parametrize("entry", ["wq_linear_act", "wq_gated"])
def test_decode_batches_of_very_long_rows_are_cut(run, entry):
    """Rows too long for the decode kernel's 64 ranges take the tile kernel;
    with exactly the workspace that was asked for it cuts them."""
    shapes = [(20, 262144 + 4096), (32, 1 << 20), (1, 524288 + 4096), (16, 1 << 22)]
    got = run([(entry, {**FORWARD, "M": m, "N": 48, "K": k, "gs": 128, "perm": perm}) for m, k in shapes
               for perm in (None, at(7))])
    for (m, k), r in zip([s for s in shapes for _ in range(2)], got):
        assert r["status"] == 0
        assert max(launch["gx"] for launch in r["launches"][-2:]) >= 8, (m, k, r)
    # one channel block less and the decode kernel takes them, in 64 ranges
    for m, k in ((20, 262144), (1, 524288)):
        r, = run([(entry, {**FORWARD, "M": m, "N": 48, "K": k, "gs": 128})])
        assert r["status"] == 0 and r["launches"][0]["gy"] == 64
