"""Argument checks of the adapters' and dropout's entry points, on the CPU: the
C ABI's refusals (no kernel is launched: every call fails its checks, or is
empty) and the binding's; and the pins of the dropout oracle."""

import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import oracle as O
import weight_only_int4_wq_amd as wq

torch = pytest.importorskip("torch")

OK, ARG, UNSUPPORTED = 0, 1, 2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 1 << 50

# made-up device addresses: only where no GPU could follow them
fake_pointers = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes made-up device addresses")


def at(b):
    return ctypes.c_void_p(0x10000000 * (b + 1))


def off(b, n):
    return ctypes.c_void_p(0x10000000 * (b + 1) + n)


def header_names():
    src = open(os.path.join(ROOT, "include", "wq_adapter.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return set(re.findall(r"^\s*(?:wq_status|size_t)\s+(wq_[a-z_0-9]+)\s*\(", src, flags=re.M))


def test_header_and_library_agree():
    names = header_names()
    assert len(names) == 5
    for n in names:
        assert hasattr(wq.lib(), n), n
        assert n in wq._SIG, n


def test_header_is_plain_c(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "use_adapter.c"
    src.write_text("#include <wq_adapter.h>\ntypedef void (*fn_t)(void);\nconst fn_t fns[] = {\n" +
                   "".join(f"    (fn_t)&{n},\n" for n in sorted(header_names())) + "};\n")
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                        "-c", str(src), "-o", str(tmp_path / "use_adapter.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


M_, N_, K_, R_, L_ = 5, 72, 64, 8, 3


def forward(x=at(0), down=at(1), up=at(2), scales=at(3), slots=at(4), base=at(5), p=0.1, seed=1, offset=2, step=at(6),
            y=at(7), hidden=at(8), M=M_, N=N_, K=K_, R=R_, L=L_, ws=at(9), wsb=BIG):
    return wq.lib().wq_adapters(x, down, up, scales, slots, base, p, seed, offset, step, y, hidden, M, N, K, R, L, ws, wsb,
                                None)


def backward(dy=at(0), x=at(1), hidden=at(2), down=at(3), up=at(4), scales=at(5), slots=at(6), p=0.1, seed=1, offset=2,
             step=at(7), add=at(8), dx=at(9), ddown=at(10), dup=at(11), M=M_, N=N_, K=K_, R=R_, L=L_, ws=at(12), wsb=BIG):
    return wq.lib().wq_adapters_backward(dy, x, hidden, down, up, scales, slots, p, seed, offset, step, add, dx, ddown,
                                         dup, M, N, K, R, L, ws, wsb, None)


def dropout(x=at(0), res=at(1), p=0.1, seed=1, offset=2, step=at(2), y=at(3), n=100):
    return wq.lib().wq_dropout(x, res, p, seed, offset, step, y, n, None)


SIZES = (dict(M=-1), dict(M=(1 << 30) + 1), dict(N=0), dict(N=-1), dict(N=(1 << 22) + 1), dict(K=0), dict(K=48),
         dict(K=(1 << 22) + 32), dict(R=0), dict(R=-1), dict(L=0), dict(L=(1 << 22) + 1))
CHANCES = (dict(p=-0.1), dict(p=1.0), dict(p=1.5), dict(p=float("nan")), dict(p=1 - 2.0 ** -18))


@fake_pointers
def test_forward_refusals():
    for bad in SIZES + CHANCES + (dict(x=None), dict(down=None), dict(up=None), dict(scales=None), dict(y=None),
                                  dict(ws=None), dict(wsb=0)):
        assert forward(**bad) == ARG, bad
    for i, name in enumerate(["x", "down", "up", "scales", "slots", "base", "step", "y", "hidden", "ws"]):
        by = {"scales": 2, "slots": 2, "step": 4}.get(name, 8)
        assert forward(**{name: off(i, by)}) == ARG, name
    need = wq.adapters_workspace_size("adapters", M_, N_, K_, R_, L_)
    assert need > 0
    assert forward(wsb=need - 1) == ARG
    assert forward(R=129) == UNSUPPORTED
    assert forward(M=0, x=None, y=None, ws=None, wsb=0) == OK


@fake_pointers
def test_forward_overlaps():
    ny, nh = M_ * N_ * 2, M_ * R_ * 4
    for name, i in dict(x=0, down=1, up=2, scales=3, slots=4, step=6, hidden=8, ws=9).items():
        assert forward(y=at(i)) == ARG, name
    for name, i in dict(x=0, down=1, up=2, scales=3, slots=4, base=5, step=6, y=7, ws=9).items():
        assert forward(hidden=at(i)) == ARG, name
        if name != "ws":
            assert forward(ws=at(i)) == ARG, name
    assert forward(base=off(7, 16)) == ARG and forward(base=off(7, -16)) == ARG   # part of y, not y
    assert forward(hidden=off(7, (ny - 1) // 16 * 16)) == ARG
    assert forward(hidden=off(7, -(nh // 16) * 16 + 16)) == ARG


@fake_pointers
def test_backward_refusals():
    for bad in SIZES + CHANCES + (dict(dy=None), dict(x=None), dict(hidden=None), dict(down=None), dict(up=None),
                                  dict(scales=None), dict(ddown=None), dict(dup=None), dict(ws=None), dict(wsb=0)):
        assert backward(**bad) == ARG, bad
    names = ["dy", "x", "hidden", "down", "up", "scales", "slots", "step", "add", "dx", "ddown", "dup", "ws"]
    for i, name in enumerate(names):
        by = {"scales": 2, "slots": 2, "step": 4}.get(name, 8)
        assert backward(**{name: off(i, by)}) == ARG, name
    need = wq.adapters_workspace_size("adapters_backward", M_, N_, K_, R_, L_)
    assert need > 0
    assert backward(wsb=need - 1) == ARG
    assert backward(R=129) == UNSUPPORTED
    assert backward(M=0, dy=None, x=None, hidden=None, dx=None, ddown=None, dup=None, ws=None, wsb=0) == OK
    assert backward(dx=None, ddown=None, dup=None) == OK           # nothing is asked for


@fake_pointers
def test_backward_overlaps():
    for name, i in dict(dx=9, ddown=10, dup=11, ws=12).items():
        for other, j in dict(dy=0, x=1, hidden=2, down=3, up=4, scales=5, slots=6, step=7, add=8, dx=9, ddown=10, dup=11,
                             ws=12).items():
            if j != i and (name, other) != ("dx", "add"):
                assert backward(**{name: at(j)}) == ARG, (name, other)
    assert backward(add=off(9, 16)) == ARG
    assert backward(M=0, dup=at(10)) == ARG


@fake_pointers
def test_dropout_refusals():
    for bad in CHANCES + (dict(x=None), dict(y=None), dict(n=-1), dict(n=1 << 62), dict(x=off(0, 8)), dict(y=off(3, 2)),
                          dict(res=off(1, 8)), dict(step=off(2, 4)), dict(y=off(0, 16)), dict(y=off(1, 16)),
                          dict(y=at(2))):
        assert dropout(**bad) == ARG, bad
    assert dropout(n=0, x=None, y=None, res=None) == OK


def test_workspace_sizes():
    size = wq.adapters_workspace_size
    for entry in ("adapters", "adapters_backward"):
        assert size(entry, 0, 64, 64, 8, 1) == 0
        for bad in ((4, 0, 64, 8, 1), (4, 64, 48, 8, 1), (4, 64, 64, 0, 1), (4, 64, 64, 129, 1), (4, 64, 64, 8, 0)):
            assert size(entry, *bad) == 0
        for M in (1, 33, 5000):
            assert size(entry, M, 4096, 4096, 16, 4) >= M * 16 * 4
        for i in range(5):
            wrapped = [4, 64, 64, 8, 1]
            wrapped[i] += 1 << 32
            with pytest.raises(ValueError, match="2\\^31"):
                size(entry, *wrapped)


# ------------------------------------------------------------- binding ----

def meta(*shape, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device="meta")


def pool(L=3, R=8, N=72, K=64):
    return meta(L, R, K), meta(L, R, N), meta(L, dtype=torch.float32)


F32, I32, I64 = torch.float32, torch.int32, torch.int64


def test_binding_forward_checks():
    x = meta(5, 64)
    with pytest.raises(ValueError, match="GPU tensors"):
        wq.adapters(x, *pool(), slots=meta(5, dtype=I32), base=meta(5, 72), p=0.1, save_hidden=True)
    for bad, word in ((dict(slots=meta(4, dtype=I32)), "slots"), (dict(slots=meta(5, dtype=I64)), "slots"),
                      (dict(base=meta(5, 71)), "base"), (dict(base=meta(5, 72, dtype=F32)), "base"),
                      (dict(out=meta(4, 72)), "out"), (dict(hidden=meta(5, 7, dtype=F32)), "hidden"),
                      (dict(hidden=meta(5, 8)), "hidden"), (dict(workspace=meta(4)), "workspace"), (dict(p=1.0), "p must"),
                      (dict(p=-0.5), "p must"), (dict(p=float("nan")), "p must"), (dict(p=1 - 2.0 ** -18), "p must"),
                      (dict(seed=-1), "seed"), (dict(offset=1 << 64), "offset"), (dict(step=meta(2, dtype=I64)), "step"),
                      (dict(step=meta(1, dtype=I32)), "step"), (dict(base=[1.0]), "base"), (dict(slots=[0] * 5), "slots")):
        with pytest.raises(ValueError, match=word):
            wq.adapters(x, *pool(), **bad)
    down, up, scales = pool()
    for args, word in (((meta(5, 60), down, up, scales), "down|channels"), ((x, down, meta(3, 7, 72), scales), "up"),
                       ((x, down, up[:2], scales), "up"), ((x, down, up, scales[:2]), "scales"),
                       ((x, down, up, meta(3)), "scales"), ((x, down[0], up, scales), "down"),
                       ((x, down, up[0], scales), "up"), ((x, None, up, scales), "down"), ((x, down, None, scales), "up"),
                       ((x, down.transpose(1, 2), up, scales), "down|rank"), ((None, down, up, scales), "x "),
                       ((meta(64, 5).t(), down, up, scales), "contiguous"),
                       ((meta(5, 64, dtype=F32), down, up, scales), "x must be"),
                       ((torch.empty(5, 64, dtype=torch.float16), down, up, scales), "is on"),
                       ((x, *pool(R=129)), "ranks"), ((x, *pool(L=0)), "at least"), ((x, *pool(N=0)), "at least"),
                       ((meta(5, 48), *pool(K=48)), "multiple of 32")):
        with pytest.raises(ValueError, match=word):
            wq.adapters(*args)


def test_binding_backward_checks():
    good = dict(dy=meta(5, 72), x=meta(5, 64), hidden=meta(5, 8, dtype=F32))
    call = lambda **more: wq.adapters_backward(**{**good, **dict(zip(("down", "up", "scales"), pool())), **more})  # noqa: E731
    with pytest.raises(ValueError, match="GPU tensors"):
        call()
    with pytest.raises(ValueError, match="GPU tensors"):
        call(x=None, hidden=None, need_weights=False)
    for bad, word in ((dict(x=None), "x is required"), (dict(hidden=None), "hidden is required"), (dict(x=meta(4, 64)), "x "),
                      (dict(hidden=meta(5, 8)), "hidden"), (dict(dx_add=meta(5, 72)), "dx_add"), (dict(out=meta(5, 72)), "out"),
                      (dict(need_dx=False, out=meta(5, 64)), "needs dx"), (dict(need_dx=False, dx_add=meta(5, 64)), "needs dx"),
                      (dict(dy=meta(5, 71)), "up"), (dict(down=meta(3, 64)), "down"), (dict(up=meta(3, 8, 64)), "up"),
                      (dict(p=1.0), "p must"), (dict(step=meta(1)), "step"), (dict(slots=meta(6, dtype=I32)), "slots")):
        with pytest.raises(ValueError, match=word):
            call(**bad)


def test_binding_dropout_checks():
    x = meta(5, 7, 3)
    with pytest.raises(ValueError, match="GPU tensors"):
        wq.dropout(x, 0.1, 1, residual=meta(5, 7, 3))
    with pytest.raises(ValueError, match="GPU tensors"):
        wq.dropout_backward(x, 0.1, 1)
    for bad, word in ((dict(residual=meta(5, 7, 4)), "residual"), (dict(out=meta(5, 7, 3, dtype=F32)), "out"),
                      (dict(p=1), "p must"), (dict(seed=1 << 64), "seed"), (dict(offset=-1), "offset"),
                      (dict(step=meta(1, dtype=F32)), "step")):
        with pytest.raises(ValueError, match=word):
            wq.dropout(**{"x": x, "p": 0.1, "seed": 1, **bad})
    for bad in (meta(5, 7, dtype=F32), meta(5, 7).t(), None):
        with pytest.raises(ValueError):
            wq.dropout(bad, 0.1, 1)


@pytest.mark.parametrize("M,N,K,L", [((1 << 32) + 3, 72, 64, 3), (5, (1 << 32) + 72, 64, 3), (5, 72, (1 << 32) + 64, 3),
                                     (5, 72, 64, (1 << 32) + 3)])
def test_sizes_that_a_32_bit_integer_would_wrap(M, N, K, L):
    with pytest.raises(ValueError, match="2\\^31"):
        wq.adapters(meta(M, K), *pool(L, 8, N, K))
    with pytest.raises(ValueError, match="2\\^31"):
        wq.adapters_backward(meta(M, N), meta(M, K), meta(M, 8, dtype=F32), *pool(L, 8, N, K))


def test_a_lost_gradient_is_said(recwarn):
    def needs(t):
        return t.requires_grad_()

    x, dy, h = meta(5, 64), meta(5, 72), meta(5, 8, dtype=F32)
    for i in range(4):
        args = [meta(5, 64), *pool()]
        needs(args[i])
        with pytest.warns(UserWarning, match="no gradient"), pytest.raises(ValueError, match="GPU tensors"):
            wq.adapters(*args)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU tensors"):
            wq.adapters(*args)
    with pytest.warns(UserWarning, match="no gradient"), pytest.raises(ValueError, match="GPU tensors"):
        wq.adapters(x, *pool(), base=needs(meta(5, 72)))
    for args, more in (((needs(meta(5, 72)), x, h), {}), ((dy, needs(meta(5, 64)), h), {}),
                       ((dy, x, h), dict(dx_add=needs(meta(5, 64))))):
        with pytest.warns(UserWarning, match="no gradient"), pytest.raises(ValueError, match="GPU tensors"):
            wq.adapters_backward(*args, *pool(), **more)
    for more in (dict(x=needs(meta(8))), dict(x=meta(8), residual=needs(meta(8)))):
        with pytest.warns(UserWarning, match="no gradient") as w, pytest.raises(ValueError, match="GPU tensors"):
            wq.dropout(p=0.1, seed=1, **more)
        assert w[0].filename == __file__
    with pytest.warns(UserWarning, match="no gradient") as w, pytest.raises(ValueError, match="GPU tensors"):
        wq.adapters(needs(meta(5, 64)), *pool())
    assert w[0].filename == __file__
    with pytest.raises(ValueError, match="GPU tensors"):
        wq.adapters(x, *pool())
    assert len(recwarn) == 0


def test_adapted_linear_checks_its_pool():
    base = wq.QuantizedLinear(meta(72, 8, dtype=I32), meta(72, 2), None, 4, 32, 64)
    wq.AdaptedLinear(base, *pool())
    for bad, word in ((pool(K=96), "base layer"), (pool(N=71), "base layer"), ((meta(3, 8, 64), meta(3, 7, 72), None), "rank"),
                      ((meta(8, 64), meta(3, 8, 72), None), "rank")):
        with pytest.raises(ValueError, match=word):
            wq.AdaptedLinear(base, *bad)


# -------------------------------------------------------------- oracle ----

@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_the_generator_gives_its_published_answers(counter, key, words):
    """The known answers published with the generator: zeros, ones, and the
    digits of pi."""
    got = O.philox4x32(np.array([counter], dtype=np.uint32), key)
    assert tuple(int(v) for v in got[0]) == words


def test_the_generator_in_whole_numbers():
    """The same words from Python's integers, ten rounds written out."""
    def words(c, k):
        c, k = list(c), list(k)
        for _ in range(10):
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32) ^ c[1] ^ k[0], b % 2 ** 32, (a >> 32) ^ c[3] ^ k[1], a % 2 ** 32]
            k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
        return c

    g = np.random.default_rng(3)
    c = g.integers(0, 1 << 32, size=(50, 4), dtype=np.uint64).astype(np.uint32)
    for row in c:
        key = (int(row[0]) ^ 0x12345678, int(row[3]))
        assert [int(v) for v in O.philox4x32(row[None], key)[0]] == words([int(v) for v in row], key)


def test_order_of_the_draws():
    """Eight to a block, low half first, the stream in the counter's upper
    words."""
    seed, offset = 0x1234567890ABCDEF, 0xFEDCBA9876543210
    d = O.drop_halves(16, 21, seed, offset)
    for i in range(21):
        g = (16 + i) // 8
        w = O.philox4x32(np.array([[g, 0, offset & 0xFFFFFFFF, offset >> 32]], dtype=np.uint32),
                         (seed & 0xFFFFFFFF, seed >> 32))[0]
        assert d[i] == (int(w[i % 8 // 2]) >> (16 * (i % 2))) & 0xFFFF
    far = O.drop_halves(1 << 36, 8, seed, 0)
    w = O.philox4x32(np.array([[0, 2, 0, 0]], dtype=np.uint32), (seed & 0xFFFFFFFF, seed >> 32))[0]
    assert [int(v) for v in far[::2]] == [int(v) & 0xFFFF for v in w]
    keep, factor = O.drop_keep((30, 40), 0.25, 5, 6)
    assert factor == 4 / 3 and 0.7 < keep.mean() < 0.8
    assert O.drop_keep((3, 5), 0.0, 5, 6)[0].all()


@pytest.mark.parametrize("index", [0, 1])
def test_the_tensors_device_is_current_during_the_call(index, monkeypatch):
    """The library runs on the tensors' device and its current stream, whichever
    device was current before."""
    current, seen = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Library:
        @staticmethod
        def wq_dropout(*args):
            seen.append((current[0], *args))
            return 0

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 70 + i, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(wq, "_lib", Library)
    wq._on_device("wq_dropout", torch.device("cuda", index), (5, 6))
    assert seen == [(index, 5, 6, 70 + index)] and current == [0]
