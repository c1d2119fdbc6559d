"""Low-rank adapters beside a quantized layer, forward and backward, and dropout, as cases to measure.

Four operators on fp16 activations:

- adapters:           y[m] = base[m] + s[a] * (x'[m] . down[a]^T) . up[a], a = slots[m]: rows of many requests at
                      once, each with its own adapter or none (a slot that is no adapter's number);
- adapters backward:  dh[m] = s[a] * dy[m] . up[a]^T, dx[m] = dropout'(dh[m] . down[a]) + add[m],
                      ddown[a] = sum over the rows of a of dh[m]^T x'[m], dup[a] = s[a] * sum of hidden[m]^T dy[m];
- dropout:            y = (kept ? x / (1 - p) : 0) + residual, and its backward pass on dy with the same seed;

x' = dropout(x) in training, x otherwise; hidden[m] = x'[m] . down[a]^T is kept for the backward pass.

Which elements are kept: elements are numbered in row-major order, eight of them share one Philox4x32-10 block
(counter: the eight's number in 64 bits, then `offset` in 64 bits; key: the seed), element i of the eight takes the
low (i even) or high (i odd) 16 bits of word i / 2, and is kept where they are at least t = round(p * 65536).  The
kept ones are divided by 1 - t / 65536.
"""

import math
import random

import torch

own = False


def _adapters(name, op, M, K, N, rank, adapters, requests, **more):
    """requests: runs of rows with one adapter each; 0: every row takes the only adapter, no slots are given."""
    c = {"name": name, "op": op, "M": M, "K": K, "N": N, "rank": rank, "adapters": adapters, "requests": requests,
         "none": False, "add": True, "save": False, "p": 0.0}
    c.update(more)
    return c


def _dropout(name, op, rows, cols, p, **more):
    c = {"name": name, "op": op, "M": rows, "K": cols, "p": p, "add": False}
    c.update(more)
    return c


def listed():
    return [
        # one token of one request through an attention output projection with its adapter: latency
        _adapters("adapters 1 token", "adapters", 1, 4096, 4096, 16, 1, 0),
        # a decode batch on the fused query, key and value projections, every request with another adapter
        _adapters("adapters 16 requests", "adapters", 16, 4096, 12288, 16, 32, 16),
        # a large decode batch on the down projection, long rows, four requests to an adapter, some without one
        _adapters("adapters 128 requests", "adapters", 128, 11008, 4096, 64, 24, 128, none=True),
        # the prompts of five requests in one batch
        _adapters("adapters 2048 tokens", "adapters", 2048, 4096, 4096, 16, 8, 5),
        # ragged prompts, odd rank and column count, no projection's output to add to, kept for training
        _adapters("adapters 173 tokens ragged", "adapters", 173, 4128, 5001, 12, 6, 7, none=True, add=False, save=True),
        # a training step's forward pass through an up projection, dropout on the adapter's input
        _adapters("adapters training 4096", "adapters", 4096, 4096, 11008, 64, 1, 0, save=True, p=0.05),
        # the backward pass of a square projection in a training step
        _adapters("backward 2048", "adapters_backward", 2048, 4096, 4096, 16, 1, 0, p=0.1),
        # its largest form: a down projection, four adapters trained in one batch
        _adapters("backward 4096 of 4", "adapters_backward", 4096, 11008, 4096, 64, 4, 4, p=0.05),
        # a short ragged batch of many small adapters, odd column count, some rows without one
        _adapters("backward 311 ragged", "adapters_backward", 311, 4128, 5001, 8, 6, 9, none=True, add=False),
        # a decode-sized tensor: latency
        _dropout("dropout 64 rows", "dropout", 64, 4096, 0.1),
        # a block's output dropped onto the residual stream
        _dropout("dropout 2048 rows residual", "dropout", 2048, 4096, 0.1, add=True),
        # the gradient of a wide activation, element count that is no multiple of eight
        _dropout("dropout backward 8191", "dropout_backward", 8191, 11005, 0.25),
    ]


def _used(case):
    """Adapters that some row takes."""
    if not case["requests"]:
        return 1
    q = case["requests"]
    return min(case["adapters"], q - q // 4 if case["none"] else q)


def _rows(case):
    """Rows with an adapter, up to the raggedness of the runs."""
    q = case["requests"]
    return case["M"] * ((q - q // 4) / q if q and case["none"] else 1.0)


def work(case):
    M, K = case["M"], case["K"]
    if case["op"].startswith("dropout"):
        return {"bytes": M * K * (6.0 if case["add"] else 4.0), "flops": M * K * (2.0 if case["add"] else 1.0)}
    N, R = case["N"], case["rank"]
    b = 2.0 * _used(case) * R * (K + N) + 4.0 * case["adapters"] + (4.0 * M if case["requests"] else 0.0)
    f = 2.0 * _rows(case) * R * (K + N)
    if case["op"] == "adapters":
        b += 2.0 * M * (K + N) + (2.0 * M * N if case["add"] else 0.0) + (4.0 * M * R if case["save"] else 0.0)
        return {"bytes": b, "flops": f}
    b += 2.0 * M * (N + 2 * K) + 4.0 * M * R + (2.0 * M * K if case["add"] else 0.0)
    b += 4.0 * case["adapters"] * R * (K + N)                  # the gradients of every adapter
    return {"bytes": b, "flops": 2.0 * f}


def draw(rng):
    """One row to 4096, layers from 64 to 11264 channels, ranks 1 to 128, up to 32 adapters; dropout up to 2^26 elements."""

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["adapters", "adapters", "adapters_backward", "adapters_backward", "dropout", "dropout_backward"])
        p = rng.choice([0.01, 0.05, 0.1, 0.1, 0.3, 0.5, round(rng.uniform(0.001, 0.9), 4)])
        if op.startswith("dropout"):
            n, cols = log_int(1, 1 << 26), log_int(1, 16384)
            c = _dropout("", op, max(1, n // cols), cols, p, add=op == "dropout" and rng.random() < 0.5)
        else:
            M, adapters = log_int(1, 4096), log_int(1, 32)
            c = _adapters("", op, M, 32 * log_int(2, 352), log_int(64, 11264),
                          rng.choice([4, 8, 16, 16, 32, 64, 128, log_int(1, 128)]), adapters,
                          0 if adapters == 1 and rng.random() < 0.5 else min(M, rng.choice([M, log_int(1, 64)])),
                          none=rng.random() < 0.3, add=rng.random() < 0.7, p=rng.choice([0.0, p]))
            c["save"] = op == "adapters" and rng.random() < 0.4
        del c["name"]
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def prepare(case, seed):
    """The activations, the adapters' pool and the batch's slots, on the GPU."""
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = random.Random(seed)

    def normal(*shape, sigma=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * sigma).half()

    s = dict(case)
    M, K = case["M"], case["K"]
    s["seed"], s["offset"] = host.getrandbits(63), host.getrandbits(40)
    if case["op"].startswith("dropout"):
        s["x"] = normal(M, K)
        s["add_v"] = normal(M, K) if case["add"] else None
        return s
    N, R, L, q = case["N"], case["rank"], case["adapters"], case["requests"]
    s["down"] = normal(L, R, K, sigma=K ** -0.5)
    s["up"] = normal(L, R, N, sigma=0.02)
    s["scales"] = 0.5 + 1.5 * torch.rand(L, generator=g, device=dev)
    s["slots"] = None
    if q:
        ends = sorted(host.sample(range(1, M), q - 1)) + [M]   # ragged runs, one row each where q = M
        pool, slots, at, took = host.sample(range(L), L), [], 0, 0
        for i, end in enumerate(ends):
            if case["none"] and i % 4 == 3:
                slot = -1
            else:
                slot, took = pool[took % L], took + 1
            slots += [slot] * (end - at)
            at = end
        s["slots"] = torch.tensor(slots, dtype=torch.int32).to(dev)
    s["x"] = normal(M, K)
    if case["op"] == "adapters":
        s["add_v"] = normal(M, N) if case["add"] else None
    else:
        s["dy"] = normal(M, N, sigma=0.1)
        s["hidden"] = torch.randn(M, R, generator=g, device=dev)
        if s["slots"] is not None:
            s["hidden"].mul_((s["slots"] >= 0).unsqueeze(1))
        s["add_v"] = normal(M, K, sigma=0.1) if case["add"] else None
    return s


# ------------------------------------------------------------- plain form --

_MASK = 0xFFFFFFFF


def _philox(groups, seed, offset):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) of the counters (group, offset): int64 [groups][4] words."""
    n = torch.arange(groups, device="cuda", dtype=torch.int64)
    c0, c1 = n & _MASK, n >> 32
    c2 = torch.full_like(n, offset & _MASK)
    c3 = torch.full_like(n, offset >> 32)
    k0, k1 = seed & _MASK, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # (modulo 2^64: all the bits of both products)
        c0, c1, c2, c3 = ((b >> 32) & _MASK) ^ c1 ^ k0, b & _MASK, ((a >> 32) & _MASK) ^ c3 ^ k1, a & _MASK
        k0, k1 = (k0 + 0x9E3779B9) & _MASK, (k1 + 0xBB67AE85) & _MASK
    return torch.stack((c0, c1, c2, c3), 1)


def _threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def _drop(s, v):
    """dropout of v [rows][cols] in 32 bits."""
    t = _threshold(s["p"])
    if t == 0:
        return v
    w = _philox((v.numel() + 7) // 8, s["seed"], s["offset"])
    u = torch.stack((w & 0xFFFF, w >> 16), 2).view(-1)[: v.numel()].view_as(v)
    return torch.where(u >= t, v * (65536.0 / (65536 - t)), torch.zeros_like(v))


def _member(s):
    """1 where row m takes adapter a, as [M][adapters][1]."""
    a = torch.arange(s["adapters"], device="cuda", dtype=torch.int32)
    slots = torch.zeros(s["M"], device="cuda", dtype=torch.int32) if s["slots"] is None else s["slots"]
    return (slots.unsqueeze(1) == a).float().unsqueeze(2)


def _forward(s):
    M, K, N, R, L = s["M"], s["K"], s["N"], s["rank"], s["adapters"]
    one = _member(s)
    h = (_drop(s, s["x"].float()) @ s["down"].float().view(L * R, K).t()).view(M, L, R) * one
    y = (h * s["scales"].view(1, L, 1)).view(M, L * R) @ s["up"].float().view(L * R, N)
    if s["add_v"] is not None:
        y = y + s["add_v"].float()
    out = {"y": y.half()}
    if s["save"]:
        out["hidden"] = h.sum(1)
    return out


def _backward(s):
    M, K, N, R, L = s["M"], s["K"], s["N"], s["rank"], s["adapters"]
    take = _member(s) * s["scales"].view(1, L, 1)
    dy, down, up = s["dy"].float(), s["down"].float().view(L * R, K), s["up"].float().view(L * R, N)
    dh = ((dy @ up.t()).view(M, L, R) * take).view(M, L * R)
    dx = _drop(s, dh @ down)
    if s["add_v"] is not None:
        dx = dx + s["add_v"].float()
    ddown = dh.t() @ _drop(s, s["x"].float())
    dup = (s["hidden"].unsqueeze(1) * take).view(M, L * R).t() @ dy
    return {"dx": dx.half(), "ddown": ddown.view(L, R, K), "dup": dup.view(L, R, N)}


def _run_own(s):
    import weight_only_int4_wq_amd as wq

    if s["op"] == "dropout":
        return {"y": wq.dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["add_v"])}
    if s["op"] == "dropout_backward":
        return {"dx": wq.dropout_backward(s["x"], s["p"], s["seed"], s["offset"])}
    if s["op"] == "adapters":
        r = wq.adapters(s["x"], s["down"], s["up"], s["scales"], slots=s["slots"], base=s["add_v"], p=s["p"],
                        seed=s["seed"], offset=s["offset"], save_hidden=s["save"])
        return {"y": r[0], "hidden": r[1]} if s["save"] else {"y": r}
    dx, ddown, dup = wq.adapters_backward(s["dy"], s["x"], s["hidden"], s["down"], s["up"], s["scales"],
                                          slots=s["slots"], p=s["p"], seed=s["seed"], offset=s["offset"],
                                          dx_add=s["add_v"])
    return {"dx": dx, "ddown": ddown, "dup": dup}


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "adapters":
        return _forward(state)
    if state["op"] == "adapters_backward":
        return _backward(state)
    y = _drop(state, state["x"].float())
    if state["add_v"] is not None:
        y = y + state["add_v"].float()
    return {"y" if state["op"] == "dropout" else "dx": y.half()}


# ---------------------------------------------------------------- 64 bits --

def _product(a, m):
    """The 64-bit product of 32-bit words a (held in int64) and the number m, from 16-bit halves: its high and low word."""
    a0, a1, m0, m1 = a % 65536, a // 65536, m % 65536, m // 65536
    low = a0 * m0
    mid = a1 * m0 + low // 65536
    other = a0 * m1 + mid % 65536
    return a1 * m1 + mid // 65536 + other // 65536, (other % 65536) * 65536 + low % 65536


def _kept(rows, cols, t, seed, offset):
    """Truth values [rows][cols]: the elements that dropout keeps."""
    n = rows * cols
    at = torch.arange(-(-n // 8), device="cuda")
    word = [at % 2 ** 32, at // 2 ** 32, torch.full_like(at, offset % 2 ** 32), torch.full_like(at, offset // 2 ** 32)]
    for r in range(10):
        key = [(seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        high0, low0 = _product(word[0], 0xD2511F53)
        high1, low1 = _product(word[2], 0xCD9E8D57)
        word = [high1.bitwise_xor(word[1]).bitwise_xor(key[0]), low1, high0.bitwise_xor(word[3]).bitwise_xor(key[1]), low0]
    keep = torch.empty(at.numel(), 8, dtype=torch.bool, device="cuda")
    for i in range(8):
        half = word[i // 2] // 65536 if i % 2 else word[i // 2] % 65536
        keep[:, i] = half >= t
    return keep.flatten()[:n].reshape(rows, cols)


def exact(case, seed):
    s = prepare(case, seed)
    t = math.floor(case["p"] * 65536 + 0.5)
    x = s["x"].double()
    keep = None
    if t:
        keep = _kept(case["M"], case["K"], t, s["seed"], s["offset"]).double() / (1 - t / 65536)
        x = x * keep
    if case["op"].startswith("dropout"):
        if s["add_v"] is not None:
            x = x + s["add_v"].double()
        return {"y" if case["op"] == "dropout" else "dx": x}
    sets = [(a, (s["slots"] == a).nonzero().flatten()) for a in range(case["adapters"])] if s["slots"] is not None \
        else [(0, torch.arange(case["M"], device="cuda"))]
    forward = case["op"] == "adapters"
    wide = case["N"] if forward else case["K"]
    out = torch.zeros(case["M"], wide, dtype=torch.float64, device="cuda")
    hidden = torch.zeros(case["M"], case["rank"], dtype=torch.float64, device="cuda")
    ddown, dup = torch.zeros(s["down"].shape, dtype=torch.float64, device="cuda"), torch.zeros(
        s["up"].shape, dtype=torch.float64, device="cuda")
    for a, rows in sets:
        down, up, scale = s["down"][a].double(), s["up"][a].double(), s["scales"][a].double()
        if forward:
            hidden[rows] = x[rows].matmul(down.T)
            out[rows] = hidden[rows].matmul(up) * scale
        else:
            dy = s["dy"][rows].double()
            dh = dy.matmul(up.T) * scale
            out[rows] = dh.matmul(down)
            ddown[a] = dh.T.matmul(x[rows])
            dup[a] = s["hidden"][rows].double().T.matmul(dy) * scale
    if not forward and keep is not None:
        out = out * keep
    if s["add_v"] is not None:
        out = out + s["add_v"].double()
    if forward:
        return {"y": out, "hidden": hidden} if case["save"] else {"y": out}
    return {"dx": out, "ddown": ddown, "dup": dup}
