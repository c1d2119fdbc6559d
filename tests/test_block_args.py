"""Argument checks of the feed-forward block's entry points, on the CPU: the C
ABI's refusals (no kernel is launched: every call fails its checks, or is
empty) and the binding's."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

import weight_only_int4_wq_amd as wq

torch = pytest.importorskip("torch")

OK, ARG, UNSUPPORTED = 0, 1, 2
FAKE = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10008)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 1 << 40

# made-up device addresses: only where no GPU could follow them
fake_pointers = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes made-up device addresses")


def header_names():
    src = open(os.path.join(ROOT, "include", "wq_block.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return set(re.findall(r"^\s*(?:wq_status|size_t)\s+(wq_[a-z_0-9]+)\s*\(", src, flags=re.M))


def test_header_and_library_agree():
    names = header_names()
    assert len(names) == 8
    for n in names:
        assert hasattr(wq.lib(), n), n
        assert n in wq._SIG, n


def test_header_is_plain_c(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use_block.c"
    src.write_text("#include <wq_block.h>\ntypedef void (*fn_t)(void);\nconst fn_t fns[] = {\n" +
                   "".join(f"    (fn_t)&{n},\n" for n in sorted(header_names())) + "};\n")
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                        "-c", str(src), "-o", str(tmp_path / "use_block.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_activation_numbers_match_the_header():
    src = open(os.path.join(ROOT, "include", "wq_block.h")).read()
    got = {k.lower(): int(v) for k, v in re.findall(r"WQ_ACT_([A-Z_]+) = (\d+)", src)}
    assert got == wq.ACTIVATIONS


def forward(name, x=FAKE, packed=FAKE, scales=FAKE, zeros=None, perm=None, bias=None, res=None, act=0, y=FAKE,
            preact=None, M=4, N=64, K=128, bits=4, gs=32, ws=None, wsb=0):
    tail = [act, y, preact, M, N, K, bits, gs, ws, wsb, None]
    head = [x, packed, scales, zeros, perm, bias]
    return getattr(wq.lib(), name)(*head, *([] if name == "wq_gated" else [res]), *tail)


def backward(name, dy=FAKE, preact=FAKE, act=4, packed=FAKE, scales=FAKE, perm=None, add=None,
             dx=ctypes.c_void_p(0x20000), dz=ctypes.c_void_p(0x30000), db=None, M=4, N=64, K=128, bits=4, gs=32,
             ws=None, wsb=0):
    return getattr(wq.lib(), name)(dy, preact, act, packed, scales, None, perm, add, dx, dz, db, M, N, K, bits, gs, ws,
                                   wsb, None)


@fake_pointers
@pytest.mark.parametrize("name", ["wq_linear_act", "wq_gated"])
@pytest.mark.parametrize("M", [4, 100])
def test_forward_refusals(name, M):
    for bad in (dict(x=None), dict(packed=None), dict(scales=None), dict(y=None), dict(x=MIS), dict(packed=MIS),
                dict(y=MIS), dict(bias=MIS), dict(preact=MIS), dict(ws=MIS, wsb=BIG), dict(perm=MIS, ws=FAKE, wsb=BIG),
                dict(act=-1), dict(act=5), dict(K=100), dict(K=0), dict(N=-1), dict(gs=48), dict(gs=96), dict(gs=0),
                dict(preact=FAKE), dict(K=(1 << 22) + 32), dict(N=(1 << 22) + 2), dict(perm=FAKE),
                dict(perm=FAKE, ws=FAKE, wsb=M * 128 * 2 - 1)):
        assert forward(name, **{"M": M, **bad}) == ARG, bad
    assert forward(name, M=-1) == ARG
    for bits in (0, 1, 5, 16):
        assert forward(name, M=M, bits=bits) == UNSUPPORTED
    assert forward(name, M=0, x=None, y=None) == OK
    assert forward(name, M=M, N=0, y=None) == OK
    if name == "wq_linear_act":
        assert forward(name, M=M, res=MIS) == ARG
    else:
        assert forward(name, M=M, N=(1 << 21) + 1) == ARG   # 2 I weight rows


@fake_pointers
@pytest.mark.parametrize("name", ["wq_linear_act_backward", "wq_gated_backward"])
def test_backward_refusals(name):
    for bad in (dict(dy=None), dict(preact=None), dict(packed=None), dict(scales=None), dict(dx=None), dict(dy=MIS),
                dict(preact=MIS), dict(packed=MIS), dict(add=MIS), dict(dx=MIS), dict(dz=MIS), dict(db=MIS),
                dict(ws=MIS, wsb=BIG), dict(perm=MIS, ws=FAKE, wsb=BIG), dict(act=-1), dict(act=5), dict(K=100),
                dict(gs=48), dict(gs=0), dict(M=-1), dict(N=-1), dict(dz=FAKE), dict(dz=None),
                dict(perm=FAKE), dict(perm=FAKE, ws=FAKE, wsb=4 * 128 * 4 - 1), dict(dz=None, ws=FAKE, wsb=255),
                dict(M=100, db=FAKE)):
        assert backward(name, **bad) == ARG, bad
    assert backward(name, dz=ctypes.c_void_p(0x20000)) == ARG           # dz is dx
    for bits in (0, 1, 5, 16):
        assert backward(name, bits=bits) == UNSUPPORTED
    assert backward(name, M=0, dy=None, preact=None, dx=None, dz=None) == OK
    if name == "wq_linear_act_backward":
        # without an activation preact is not read, but rows that are not 16-byte aligned need a copy
        assert backward(name, act=0, preact=None, N=65) == ARG


@fake_pointers
def test_workspace_sizes():
    r256 = lambda b: (b + 255) // 256 * 256  # noqa: E731
    size = wq.block_workspace_size
    for M in (1, 20, 40, 300):
        plain, perm = (size("linear_act", M, 96, 4096, 4, p) for p in (False, True))
        assert perm - plain == r256(M * 4096 * 2)
        assert plain % (M * 96 * 4 if M <= 32 else 64 * 256 * 4) == 0
        plain, perm = (size("gated", M, 96, 4096, 4, p) for p in (False, True))
        assert perm - plain == r256(M * 4096 * 2) and plain % (M * 192 * 4 if M <= 32 else 64 * 256 * 4) == 0
        for entry, rows in (("linear_act_backward", 99), ("gated_backward", 198)):
            assert size(entry, M, 99, 4096, 4, False) >= r256(M * ((rows + 7) // 8 * 8) * 2)
            assert size(entry, M, 99, 4096, 4, True) >= r256(M * ((rows + 7) // 8 * 8) * 2) + -(-M // 64) * 64 * 4096 * 4
    for entry in ("linear_act", "gated", "linear_act_backward", "gated_backward"):
        assert size(entry, 0, 96, 4096, 4, True) == 0
        assert size(entry, 4, 0, 4096, 4, True) == 0
        assert size(entry, 4, 96, 4100, 4, True) == 0
        assert size(entry, 4, 96, 4096, 5, True) == 0


# ------------------------------------------------------------- binding ----

def meta(*shape, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device="meta")


def layer(N, K, bits=4, gs=32):
    return (meta(N, K * bits // 32, dtype=torch.int32), meta(N, K // gs), meta(N, K // gs, dtype=torch.uint8), bits, gs)


@pytest.mark.parametrize("fn,rows", [(wq.linear_act, 64), (wq.gated, 128)])
def test_binding_forward_checks(fn, rows):
    L = layer(rows, 96)
    x = meta(4, 96)
    with pytest.raises(ValueError, match="GPU tensors"):
        fn(x, *L)
    for bad, word in ((dict(bias=meta(rows - 1)), "bias"), (dict(out=meta(4, 63)), "out"),
                      (dict(preact=meta(4, rows - 1)), "preact"), (dict(act="tanh"), "act"),
                      (dict(perm=meta(95, dtype=torch.int32)), "perm"), (dict(perm=meta(96)), "perm"),
                      (dict(workspace=meta(4)), "workspace")):
        with pytest.raises(ValueError, match=word):
            fn(x, *L, **bad)
    for bad, word in ((meta(4, 64), "columns"), (meta(96, 4).t(), "contiguous"), (meta(4, 96, dtype=torch.float32), "x must be"),
                      (torch.empty(4, 96, dtype=torch.float16), "device|is on")):
        with pytest.raises(ValueError, match=word):
            fn(bad, *L)
    with pytest.raises(ValueError, match="bits"):
        fn(x, *L[:3], 5, 32)
    if fn is wq.linear_act:
        with pytest.raises(ValueError, match="residual"):
            fn(x, *L, residual=meta(4, 63))
    else:
        with pytest.raises(ValueError, match="even"):
            fn(x, *layer(127, 96))


@pytest.mark.parametrize("fn,rows", [(wq.linear_act_backward, 64), (wq.gated_backward, 128)])
def test_binding_backward_checks(fn, rows):
    L = layer(rows, 96)
    dy, z = meta(4, 64), meta(4, rows)
    with pytest.raises(ValueError, match="GPU tensors"):
        fn(dy, z, *L, act="silu")
    with pytest.raises(ValueError, match="preact is required"):
        fn(dy, None, *L, act="silu")
    for bad, word in ((dict(dx_add=meta(4, 64)), "dx_add"), (dict(out=meta(3, 96)), "out"), (dict(act="x"), "act")):
        with pytest.raises(ValueError, match=word):
            fn(dy, z, *L, **{"act": "silu", **bad})
    with pytest.raises(ValueError, match="preact"):
        fn(dy, meta(4, rows + 1), *L, act="silu")
    with pytest.raises(ValueError, match="columns"):
        fn(meta(4, 63), z, *L, act="silu")


def test_gated_mlp_checks_its_layers():
    mk = lambda N, K: wq.QuantizedLinear(*layer(N, K)[:3], 4, 32, K)  # noqa: E731
    wq.QuantizedGatedMLP(mk(256, 64), mk(64, 128))
    with pytest.raises(ValueError, match="twice"):
        wq.QuantizedGatedMLP(mk(128, 64), mk(64, 128))
    with pytest.raises(ValueError, match="act"):
        wq.QuantizedGatedMLP(mk(256, 64), mk(64, 128), act="swish")


@fake_pointers
def test_overlapping_arrays_are_refused():
    """Outputs on top of inputs, whole or in part: 4 rows of 128 channels in,
    64 out."""
    at = lambda b: ctypes.c_void_p(0x100000 + b)  # noqa: E731
    x, y, z, far = at(0), at(0x10000), at(0x20000), at(0x40000)
    for name, rows in (("wq_linear_act", 64), ("wq_gated", 128)):
        for bad in (dict(y=x), dict(y=at(4 * 128 * 2 - 16)), dict(preact=y), dict(preact=at(0x10000 + 4 * 64 * 2 - 16)),
                    dict(preact=at(0x10000 - 4 * rows * 2 + 16)), dict(preact=x)):
            assert forward(name, **{"x": x, "y": y, "preact": z, **bad}) == ARG, bad
    for bad in (dict(res=z), dict(res=at(0x10000 + 16))):
        assert forward("wq_linear_act", **{"x": x, "y": y, "preact": z, **bad}) == ARG, bad
    for name in ("wq_linear_act_backward", "wq_gated_backward"):
        good = dict(dy=x, preact=y, dx=z, dz=far)
        for bad in (dict(dx=x), dict(dx=at(4 * 64 * 2 - 16)), dict(dx=y), dict(dz=x), dict(dz=y), dict(dz=z),
                    dict(add=far), dict(add=at(0x20000 + 16))):
            assert backward(name, **{**good, **bad}) == ARG, bad
