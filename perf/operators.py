"""Cases that measure the linear-layer operators of this library.

Operators (X is p x q, W is r x q, Y is p x r, all row-major with a row stride):

  linear      Y = R + D(act(X W^T + b)), optionally with Z = X W^T + b
  linear_bwd  dX, dW, db of the same layer from dY, X, W and Z
  dropout     Y = R + D(X)
  linear_i8   Y = R + act(s t (Q V^T) + b): X quantised by rows to int8 Q with scales s, the
              int8 weights V with row scales t made beforehand

D drops with a counter-based generator (Philox4x32-10: Salmon, Moraes, Dror and Shaw, "Parallel
random numbers: as easy as 1, 2, 3", 2011): element (i, j) takes the 16-bit lane j % 8 of the
block with counter (i ceil(r / 8) + j / 8, offset) and key seed, is kept where that lane is at
least T = rint(2^16 p), and is scaled by 2^16 / (2^16 - T).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def case(name, op, type, p, q, r, act="none", bias=False, residual=False, drop=0.0, keep_z=False, pad=0):
    return {"name": name, "op": op, "type": type, "p": p, "q": q, "r": r, "act": act, "bias": bias,
            "residual": residual, "drop": drop, "keep_z": keep_z, "pad": pad}


def listed():
    return [
        # one new token through a feed-forward block's first product, while serving
        case("linear_token", "linear", "bf16", 1, 2048, 8192, act="gelu", bias=True),
        # one new token of each of 37 sequences through its second product, added to the stream
        case("linear_tokens", "linear", "f16", 37, 8192, 2048, bias=True, residual=True),
        # a vocabulary-like odd width and a ragged batch, rows inside a wider buffer, training
        case("linear_ragged", "linear", "bf16", 777, 1999, 4099, act="silu", bias=True, residual=True, drop=0.1, pad=5),
        # a training step's forward pass, the pre-activation kept for the gradient
        case("linear_train", "linear", "bf16", 8192, 2048, 8192, act="gelu", bias=True, keep_z=True),
        # gradients of a small layer, where launches count
        case("backward_small", "linear_bwd", "f16", 256, 256, 1024, act="gelu_tanh", bias=True, drop=0.1),
        # gradients at odd sizes
        case("backward_ragged", "linear_bwd", "bf16", 1537, 1001, 2049, act="relu", bias=True, pad=3),
        # a training step's gradients of linear_train
        case("backward_train", "linear_bwd", "bf16", 8192, 2048, 8192, act="gelu", bias=True),
        # dropout of a few rows
        case("dropout_small", "dropout", "f16", 16, 1, 2048, drop=0.1, residual=True),
        # dropout and residual of a long batch of activations
        case("dropout_large", "dropout", "bf16", 16384, 1, 8192, drop=0.1, residual=True),
        # one new token through int8 weights: their bytes are the work
        case("i8_token", "linear_i8", "bf16", 1, 8192, 8192, bias=True, residual=True),
        # a ragged batch of tokens through int8 weights
        case("i8_tokens", "linear_i8", "f16", 203, 2048, 8191, act="silu", bias=True),
        # a long prompt through int8 weights
        case("i8_prompt", "linear_i8", "bf16", 8192, 2048, 8192, act="gelu", bias=True),
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        # half of the sizes are multiples of 64 where they can be, as most layers' are
        return max(lo, v // 64 * 64) if v >= 128 and rng.random() < 0.5 else v

    op = rng.choice(["linear", "linear_bwd", "dropout", "linear_i8"])
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    drop = rng.choice([0.0, 0.1, 0.25])
    some = lambda: rng.random() < 0.5  # noqa: E731
    pad = rng.choice([0, 0, 8, 5])
    if op == "dropout":
        p, r = size(1, 16384), size(64, 8192)
        return case("", op, rng.choice(["bf16", "f16", "f32"]), p, 1, r, drop=rng.choice([0.1, 0.25, 0.5]), residual=some(), pad=pad) | {"name": None}
    p, q, r = size(1 if op != "linear_bwd" else 64, 8192), size(256, 8192), size(256, 8192)
    while p * q * r > 8192 * 2048 * 8192:
        p = max(1, p // 2)
    c = case("", op, rng.choice(["bf16", "f16"]), p, q, r, act=act, bias=some() or op == "linear_bwd", residual=some() and op != "linear_bwd",
             drop=drop if op != "linear_i8" else 0.0, keep_z=op == "linear" and some(), pad=pad)
    return c | {"name": None}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, p, q, r, pad = TYPES[case["type"]], case["p"], case["q"], case["r"], case["pad"]

    def normal(rows, cols, scale=1.0, at=0.0):
        wide = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).add_(at).to(dt)
        return wide[:, :cols]

    s = {"case": dict(case), "drop": case["drop"], "seed": 0x5DEECE66D + 2 * seed, "offset": (1 << 33) + seed}
    if case["op"] == "dropout":
        s["x"] = normal(p, r)
        s["residual"] = normal(p, r, 2.0) if case["residual"] else None
        return s
    s["x"] = normal(p, q)
    if case["op"] == "linear_i8":
        # weights quantised once, row by row, as a serving program loads them
        w = torch.randn(r, q, generator=gen, device="cuda", dtype=torch.float32) / math.sqrt(q)
        top = w.abs().amax(1)
        s["wq"] = torch.round(w * (127.0 / top)[:, None]).to(torch.int8)
        s["ws"] = top / 127.0
    else:
        s["w"] = normal(r, q, 1.0 / math.sqrt(q))
    s["bias"] = (torch.randn(r, generator=gen, device="cuda") * 0.1).to(dt) if case["bias"] else None
    if case["op"] == "linear_bwd":
        s["dy"] = normal(p, r, 0.05)
        s["z"] = normal(p, r) if case["act"] != "none" else None
    else:
        s["residual"] = normal(p, r, 2.0) if case["residual"] else None
    return s


# ---- the plain form ---------------------------------------------------------------
def kept(p, r, drop, seed, offset, device):
    """Whether each element of a p x r matrix is kept, and the scale of those that are."""
    low = 0xFFFFFFFF
    blocks = torch.arange(p * ((r + 7) // 8), device=device, dtype=torch.int64)
    c0, c1 = blocks & low, blocks >> 32
    c2, c3 = torch.full_like(blocks, offset & low), torch.full_like(blocks, offset >> 32 & low)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    words = torch.stack([c0, c1, c2, c3], 1)
    lanes = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(p, -1)[:, :r]
    t = int(round(65536 * drop))
    return lanes >= t, 65536.0 / (65536 - t)


def dropped(v, s):
    if s["drop"] == 0.0:
        return v
    keep, scale = kept(v.shape[0], v.shape[1], s["drop"], s["seed"], s["offset"], v.device)
    return torch.where(keep, v * scale, torch.zeros_like(v))


def activated(a, act):
    if act == "relu":
        return torch.where(a > 0, a, torch.zeros_like(a))
    if act == "gelu":
        return 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a)))
    if act == "silu":
        return a / (1.0 + torch.exp(-a))
    return a


def slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        g = 1.0 / (1.0 + torch.exp(-z))
        return g * (1.0 + z * (1.0 - g))
    return torch.ones_like(z)


def run_plain(s):
    c, x = s["case"], s["x"].float()
    dt = TYPES[c["type"]]
    if c["op"] == "dropout":
        y = dropped(x, s)
        return (y if s["residual"] is None else s["residual"].float() + y).to(dt)
    if c["op"] == "linear_bwd":
        dz = dropped(s["dy"].float(), s)
        if c["act"] != "none":
            dz = dz * slope(s["z"].float(), c["act"])
        return (dz @ s["w"].float()).to(dt), (dz.t() @ x).to(dt), dz.sum(0).to(dt)
    if c["op"] == "linear_i8":
        top = x.abs().amax(1, keepdim=True)
        qx = torch.where(top > 0, torch.round(x * (127.0 / top)), torch.zeros_like(x))
        a = (qx @ s["wq"].float().t()) * (top / 127.0) * s["ws"]
    else:
        a = x @ s["w"].float().t()
    if s["bias"] is not None:
        a = a + s["bias"].float()
    y = dropped(activated(a, c["act"]), s)
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return (y.to(dt), a.to(dt)) if c["keep_z"] else y.to(dt)


# ---- the library's operators --------------------------------------------------------
def run_own(s):
    from fp64_gemm_emulation_amd import binding as oz
    c = s["case"]
    drop = {"dropout": s["drop"], "seed": s["seed"], "offset": s["offset"]}
    if c["op"] == "dropout":
        return oz.dropout_add(s["x"], s["residual"], **drop)
    if c["op"] == "linear_bwd":
        return oz.linear_backward(s["dy"], s["x"], s["w"], z=s["z"], activation=c["act"], **drop)
    if c["op"] == "linear_i8":
        return oz.linear_i8(s["x"], s["wq"], s["ws"], bias=s["bias"], activation=c["act"], residual=s["residual"])
    return oz.linear(s["x"], s["w"], bias=s["bias"], activation=c["act"], residual=s["residual"], return_z=c["keep_z"], **drop)


def run(state):
    return run_own(state) if own else run_plain(state)


def work(case):
    p, q, r = case["p"], case["q"], case["r"]
    e = TYPES[case["type"]].itemsize
    if case["op"] == "dropout":
        return {"bytes": e * p * r * (3 if case["residual"] else 2), "flops": 2 * p * r}
    if case["op"] == "linear_bwd":
        planes = 2 if case["act"] != "none" else 1
        return {"bytes": e * (planes * p * r + 2 * p * q + 2 * r * q + r), "flops": 4 * p * q * r}
    out = 1 + bool(case["residual"]) + bool(case["keep_z"])
    weights = r * q + 4 * r if case["op"] == "linear_i8" else e * r * q
    return {"bytes": e * (p * q + out * p * r + (r if case["bias"] else 0)) + weights, "flops": 2 * p * q * r}


# ---- the definition in 64 bits --------------------------------------------------------
def mask64(c, s):
    """D's factor for every element, by unsigned 64-bit arithmetic on the host."""
    p, r = c["p"], c["r"]
    if c["drop"] == 0.0:
        return 1.0
    u = np.uint64
    half, word = u(32), u(0xFFFFFFFF)
    per_row = -(-r // 8)
    n = np.arange(p * per_row, dtype=np.uint64)
    ctr = [n & word, n >> half, np.full_like(n, s["offset"] & 0xFFFFFFFF), np.full_like(n, s["offset"] >> 32)]
    key = [s["seed"] & 0xFFFFFFFF, (s["seed"] >> 32) & 0xFFFFFFFF]
    for i in range(10):
        first, second = u(0xD2511F53) * ctr[0], u(0xCD9E8D57) * ctr[2]
        ka = u((key[0] + i * 0x9E3779B9) % 2 ** 32)
        kb = u((key[1] + i * 0xBB67AE85) % 2 ** 32)
        ctr = [(second >> half) ^ ctr[1] ^ ka, second & word, (first >> half) ^ ctr[3] ^ kb, first & word]
    lanes = np.empty((n.size, 8), dtype=np.uint16)
    for i, w in enumerate(ctr):
        lanes[:, 2 * i] = (w & u(0xFFFF)).astype(np.uint16)
        lanes[:, 2 * i + 1] = (w >> u(16)).astype(np.uint16)
    t = round(c["drop"] * 65536)
    keep = torch.from_numpy(lanes.reshape(p, 8 * per_row)[:, :r] >= t).cuda()
    return keep.double() * (65536 / (65536 - t))


def phi64(v):
    return torch.special.ndtr(v)


def act64(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return v * phi64(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * v * (1 + 0.044715 * v ** 2))
    return v * torch.sigmoid(v) if act == "silu" else v


def dact64(v, act):
    if act == "relu":
        return torch.heaviside(v, torch.zeros((), dtype=v.dtype, device=v.device))
    if act == "gelu":
        return phi64(v) + v * torch.exp(-v ** 2 / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(8 / math.pi)
        g = torch.sigmoid(k * v * (1 + 0.044715 * v ** 2))
        return g + v * g * (1 - g) * k * (1 + 0.134145 * v ** 2)
    if act == "silu":
        g = torch.sigmoid(v)
        return g + v * g * (1 - g)
    return torch.ones_like(v)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "dropout":
        y = x * mask64(case, s)
        return y if s["residual"] is None else y + s["residual"].double()
    if case["op"] == "linear_bwd":
        g = s["dy"].double() * mask64(case, s)
        if case["act"] != "none":
            g = g * dact64(s["z"].double(), case["act"])
        return torch.matmul(g, s["w"].double()), torch.matmul(g.t().contiguous(), x), g.sum(dim=0)
    if case["op"] == "linear_i8":
        step = x.abs().max(dim=1, keepdim=True).values / 127
        levels = torch.nan_to_num(x / step).round()
        a = torch.matmul(levels * step, (s["wq"].double() * s["ws"].double()[:, None]).t())
    else:
        a = torch.matmul(x, s["w"].double().t())
    if s["bias"] is not None:
        a = a + s["bias"].double()
    y = act64(a, case["act"]) * mask64(case, s)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return (y, a) if case["keep_z"] else y
