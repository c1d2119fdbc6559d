"""The products of a quantized feed-forward block, forward and backward, as cases to measure.

Four operators on weights that stay packed at 2, 3, 4 or 8 bits per code:

- linear:           y = act(x . W^T + bias) + residual, z = x . W^T + bias kept for training;
- linear backward:  dz = dy * act'(z), dx = dz . W (+ add), dbias = sum of dz over the rows;
- gated:            h = act(x . Wg^T + bg) * (x . Wu^T + bu), the gate rows stacked over the up rows;
- gated backward:   dg = dh * u * act'(g), du = dh * act(g), dx = [dg du] . W (+ add), dbias;

with W = fp16((q - z) * s) per group of input channels, in the packed channel
order (`perm`: packed column j holds original channel perm[j]).
"""

import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _case(name, op, M, N, K, bits=4, group=128, **more):
    """N: output columns of the linear layer; of one projection for the gated block."""
    c = {"name": name, "op": op, "M": M, "N": N, "K": K, "bits": bits, "group": group, "act": "none", "sym": False,
         "perm": False, "bias": False, "add": False, "save": False}
    c.update(more)
    return c


def listed():
    return [
        # one token through an attention output projection onto the residual stream: latency
        _case("linear 1 token", "linear", 1, 4096, 4096, bias=True, add=True),
        # a decode batch through the down projection, long rows
        _case("linear 16 tokens", "linear", 16, 4096, 11008, add=True),
        # a prompt through the down projection
        _case("linear 2048 tokens", "linear", 2048, 4096, 11008, add=True),
        # a short ragged prompt, 3-bit act-order codes in small groups, odd column count, kept for training
        _case("linear 173 tokens 3-bit", "linear", 173, 5001, 4128, 3, 32, act="gelu", perm=True, bias=True, save=True),
        # the down projection's input gradient in a training step
        _case("linear backward 2048", "linear_backward", 2048, 4096, 11008),
        # a plain two-layer block's first product backward: 8-bit codes, odd column count, bias gradient
        _case("linear backward 311 8-bit", "linear_backward", 311, 5001, 4096, 8, 128, act="gelu", bias=True, add=True),
        # one token through gate and up
        _case("gated 1 token", "gated", 1, 11008, 4096, act="silu"),
        # a decode batch on the wide layer
        _case("gated 8 tokens", "gated", 8, 14336, 8192, act="silu"),
        # a ragged chunk of 2-bit symmetric codes, channel count that ends inside a tile
        _case("gated 45 tokens 2-bit", "gated", 45, 1401, 2080, 2, 32, act="gelu_tanh", sym=True, bias=True, save=True),
        # a prompt or a training step's forward pass
        _case("gated 2048 tokens", "gated", 2048, 11008, 4096, act="silu", save=True),
        # its backward pass, the residual stream's gradient added
        _case("gated backward 2048", "gated_backward", 2048, 11008, 4096, act="silu", add=True),
        # a few rows backward through act-order codes with one group per column
        _case("gated backward 77 act-order", "gated_backward", 77, 2751, 4096, 4, -1, act="silu", perm=True, bias=True),
    ]


def _flops(case):
    return 2.0 * case["M"] * case["N"] * case["K"] * (2 if case["op"].startswith("gated") else 1)


def draw(rng):
    """M from one token to 2048, layers from a few hundred to 11264 channels."""

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = max(_flops(c) for c in listed())
    while True:
        group = rng.choice([32, 64, 128, 128, 256, -1])
        unit = 32 if group == -1 else group
        c = _case("", rng.choice(["linear", "linear_backward", "gated", "gated_backward"]), log_int(1, 2048),
                  log_int(64, 11264), unit * max(1, log_int(256, 11264) // unit), rng.choice([2, 3, 4, 4, 8]), group,
                  act=rng.choice(ACTS[1:]), sym=rng.random() < 0.3, perm=rng.random() < 0.25, bias=rng.random() < 0.5,
                  add=rng.random() < 0.5, save=rng.random() < 0.5)
        del c["name"]
        if c["op"].startswith("linear") and rng.random() < 0.5:
            c["act"] = "none"
        if c["op"] == "gated":
            c["add"] = False
        if c["op"].endswith("backward"):
            c["save"] = False
        if _flops(c) <= most:
            return c


def _pack(q, bits):
    """Codes [N][K] as int32 words: a little-endian bitstream per row."""
    N, K = q.shape
    if bits == 3:
        b = (q.view(N, K, 1) >> torch.arange(3, device=q.device, dtype=torch.int32)) & 1
        b = b.view(N, K * 3 // 32, 32)
        per, bits = 32, 1
    else:
        per = 32 // bits
        b = q.view(N, K * bits // 32, per)
    sh = bits * torch.arange(per, device=q.device, dtype=torch.int64)
    w = (b.to(torch.int64) << sh).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def prepare(case, seed):
    """A layer's packed weights and the tensors of one pass, on the GPU."""
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    M, N, K, bits = case["M"], case["N"], case["K"], case["bits"]
    gated = case["op"].startswith("gated")
    rows = 2 * N if gated else N
    G = 1 if case["group"] == -1 else K // case["group"]
    mid, top = 1 << (bits - 1), (1 << bits) - 1

    def normal(*shape, sigma=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * sigma).half()

    # weights of standard deviation 0.02: codes spread over five deviations
    q = (torch.randn(rows, K, generator=g, device=dev) * ((top + 1) / 5.0) + mid).round_().clamp_(0, top)
    s = dict(case)
    s["packed"] = _pack(q.to(torch.int32), bits)
    del q
    s["scales"] = (0.02 * 5.0 / (top + 1) * (0.75 + 0.5 * torch.rand(rows, G, generator=g, device=dev))).half()
    s["zeros"] = None
    if not case["sym"]:
        spread = 1 if bits < 4 else 2
        z = torch.randint(-spread, spread + 1, (rows, G), generator=g, device=dev) + mid
        s["zeros"] = z.clamp(0, top).to(torch.uint8)
    s["perm"] = torch.randperm(K, generator=g, device=dev).to(torch.int32) if case["perm"] else None
    if case["op"] in ("linear", "gated"):
        s["x"] = normal(M, K)
        s["bias_v"] = normal(rows, sigma=0.1) if case["bias"] else None
        s["add_v"] = normal(M, N) if case["add"] else None
    else:
        s["dy"] = normal(M, N, sigma=0.1)
        need = gated or case["act"] != "none"
        s["preact"] = normal(M, rows, sigma=1.3) if need else None
        s["add_v"] = normal(M, K, sigma=0.1) if case["add"] else None
    return s


# ------------------------------------------------------------- plain form --

def _weights(s):
    """fp16((q - z) * s) in 32 bits, rows in packed channel order."""
    p, bits, K = s["packed"], s["bits"], s["K"]
    N = p.shape[0]
    if bits == 3:
        w = p.view(N, K // 32, 3).to(torch.int64) & 0xFFFFFFFF
        w = torch.cat([w, torch.zeros_like(w[..., :1])], dim=-1)
        at = 3 * torch.arange(32, device=p.device)
        lo, off = at // 32, at % 32
        q = ((w[..., lo] >> off) | (w[..., lo + 1] << (32 - off))) & 7
        q = q.view(N, K)
    else:
        sh = bits * torch.arange(32 // bits, device=p.device, dtype=torch.int32)
        q = ((p.unsqueeze(-1) >> sh) & ((1 << bits) - 1)).view(N, K)
    G = s["scales"].shape[1]
    q = q.view(N, G, K // G).float()
    z = float(1 << (bits - 1)) if s["zeros"] is None else s["zeros"].float().unsqueeze(-1)
    return ((q - z) * s["scales"].float().unsqueeze(-1)).half().float().view(N, K)


_TANH_C = math.sqrt(2.0 / math.pi)


def _act(v, kind):
    if kind == "none":
        return v
    if kind == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if kind == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if kind == "gelu_tanh":
        return v * torch.sigmoid(2.0 * _TANH_C * (v + 0.044715 * v * v * v))
    return v * torch.sigmoid(v)


def _act_grad(v, kind):
    if kind == "none":
        return torch.ones_like(v)
    if kind == "relu":
        return (v > 0).to(v.dtype)
    if kind == "gelu":
        return 0.5 * torch.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = torch.sigmoid(2.0 * _TANH_C * (v + 0.044715 * v * v * v))
        return t + v * t * (1.0 - t) * 2.0 * _TANH_C * (1.0 + 3.0 * 0.044715 * v * v)
    t = torch.sigmoid(v)
    return t * (1.0 + v * (1.0 - t))


def _forward(s, w):
    x = s["x"].float()
    if s["perm"] is not None:
        x = x[:, s["perm"].long()]
    z = x @ w.t()
    if s["bias_v"] is not None:
        z = z + s["bias_v"].float()
    if s["op"] == "gated":
        gate, up = z[:, : s["N"]], z[:, s["N"]:]
        out = _act(gate, s["act"]) * up
    else:
        out = _act(z, s["act"])
        if s["add_v"] is not None:
            out = out + s["add_v"].float()
    out = {"out": out.half()}
    if s["save"]:
        out["preact"] = z.half()
    return out


def _backward(s, w):
    dy = s["dy"].float()
    if s["op"] == "gated_backward":
        z = s["preact"].float()
        gate, up = z[:, : s["N"]], z[:, s["N"]:]
        dz = torch.cat([dy * up * _act_grad(gate, s["act"]), dy * _act(gate, s["act"])], dim=1)
    elif s["act"] == "none":
        dz = dy
    else:
        dz = dy * _act_grad(s["preact"].float(), s["act"])
    dx = dz @ w
    if s["perm"] is not None:
        dx = torch.empty_like(dx).index_copy_(1, s["perm"].long(), dx)
    if s["add_v"] is not None:
        dx = dx + s["add_v"].float()
    out = {"dx": dx.half()}
    if s["preact"] is not None:
        out["dz"] = dz.half()
    if s["bias"]:
        out["dbias"] = dz.sum(0)
    return out


def _run_own(s):
    import weight_only_int4_wq_amd as wq

    layer = (s["packed"], s["scales"], s["zeros"], s["bits"], s["group"])
    if s["op"] == "linear":
        r = wq.linear_act(s["x"], *layer, perm=s["perm"], bias=s["bias_v"], residual=s["add_v"], act=s["act"],
                          save_preact=s["save"])
        return {"out": r[0], "preact": r[1]} if s["save"] else {"out": r}
    if s["op"] == "gated":
        r = wq.gated(s["x"], *layer, perm=s["perm"], bias=s["bias_v"], act=s["act"], save_preact=s["save"])
        return {"out": r[0], "preact": r[1]} if s["save"] else {"out": r}
    f = wq.gated_backward if s["op"] == "gated_backward" else wq.linear_act_backward
    dx, dz, dbias = f(s["dy"], s["preact"], *layer, perm=s["perm"], act=s["act"], dx_add=s["add_v"],
                      need_dbias=s["bias"])
    out = {"dx": dx}
    if s["preact"] is not None:
        out["dz"] = dz
    if s["bias"]:
        out["dbias"] = dbias
    return out


def run(state):
    if own:
        return _run_own(state)
    w = _weights(state)
    return _forward(state, w) if "x" in state else _backward(state, w)


def work(case):
    M, N, K, bits = case["M"], case["N"], case["K"], case["bits"]
    gated = case["op"].startswith("gated")
    rows = 2 * N if gated else N
    G = 1 if case["group"] == -1 else K // case["group"]
    b = rows * K * bits / 8 + rows * G * (2 if case["sym"] else 3) + (4 * K if case["perm"] else 0)
    if case["op"] in ("linear", "gated"):
        b += 2 * M * K + 2 * M * N                       # x, out
        b += 2 * rows if case["bias"] else 0
        b += 2 * M * N if case["add"] else 0
        b += 2 * M * rows if case["save"] else 0
    else:
        b += 2 * M * N + 2 * M * K                       # dy, dx
        b += 4 * M * rows if gated or case["act"] != "none" else 0   # z in, dz out
        b += 4 * rows if case["bias"] else 0
        b += 2 * M * K if case["add"] else 0
    return {"bytes": b, "flops": _flops(case)}


# ---------------------------------------------------------------- 64 bits --

def _exact_weights(s):
    bits, K = s["bits"], s["K"]
    by = s["packed"].view(torch.uint8)
    by = torch.cat([by, torch.zeros_like(by[:, :1])], dim=1)
    first = torch.arange(K, device=by.device) * bits
    at, off = first // 8, (first % 8).to(torch.int32)
    two = by[:, at].to(torch.int32) + 256 * by[:, at + 1].to(torch.int32)
    q = torch.bitwise_and(two >> off, 2 ** bits - 1)
    del two
    n = K // s["scales"].shape[1]
    sc = s["scales"].double().repeat_interleave(n, dim=1)
    if s["zeros"] is None:
        q = q - 2 ** (bits - 1)
    else:
        q = q - s["zeros"].to(torch.int32).repeat_interleave(n, dim=1)
    w = (q.double() * sc).half().double()
    if s["perm"] is not None:  # to original channel order
        back = torch.empty_like(w)
        back[:, s["perm"].long()] = w
        return back
    return w


def _exact_act(v, kind):
    """(act(v), act'(v))"""
    if kind == "none":
        return v, torch.ones_like(v)
    if kind == "relu":
        return v.clamp(min=0), torch.where(v > 0, 1.0, 0.0).double()
    if kind == "gelu":
        cdf = torch.special.ndtr(v)
        return v * cdf, cdf + v * torch.exp(-v * v / 2) * (2 * math.pi) ** -0.5
    if kind == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (v + 0.044715 * v ** 3))
        return v / 2 * (1 + t), (1 + t) / 2 + v / 2 * (1 - t * t) * c * (1 + 0.134145 * v ** 2)
    e = 1 / (1 + torch.exp(-v))
    return v * e, e + v * e * (1 - e)


def exact(case, seed):
    s = prepare(case, seed)
    w = _exact_weights(s)
    N = s["N"]
    if "x" in s:
        z = s["x"].double().matmul(w.T)
        if s["bias_v"] is not None:
            z += s["bias_v"].double()
        if s["op"] == "gated":
            out = _exact_act(z[:, :N], s["act"])[0] * z[:, N:]
        else:
            out = _exact_act(z, s["act"])[0]
        if s["add_v"] is not None:
            out = out + s["add_v"].double()
        return {"out": out, "preact": z} if s["save"] else {"out": out}
    dy = s["dy"].double()
    dz = dy
    if s["preact"] is not None:
        z = s["preact"].double()
        a, da = _exact_act(z[:, :N], s["act"])
        dz = dy * da
        if s["op"] == "gated_backward":
            dz = torch.cat((dz * z[:, N:], dy * a), 1)
    out = {"dx": dz.matmul(w)}
    if s["add_v"] is not None:
        out["dx"] += s["add_v"].double()
    if s["preact"] is not None:
        out["dz"] = dz
    if s["bias"]:
        out["dbias"] = dz.sum(dim=0)
    return out
