"""Cases that measure the operators around the linear layers.

Operators (tokens are rows, all matrices row-major with a row stride):

  norm          H = X + R, rounded to its type; Y = H (mean(H^2) + eps)^(-1/2) w, by rows; with
                "i8" the rows of Y are quantised to int8 with one scale each, and returned as
                the values the levels stand for
  norm_bwd      dX (which is dR too) and dw of the same from dY, H and the gradient that
                reaches H from its other uses
  adapters      Y = R + act(X W^T + b + c_a (X A_a^T) B_a^T), a = index[i] the low-rank adapter of
                token i's request, or -1 for none
  logprobs      of the logits' rows: l_t - lse for the given token t (0 for t = -1, a padded place),
                lse = log sum exp l, the entropy, and the largest log probabilities with their tokens
  logprobs_bwd  the logits' gradient from those of the log probability and of the entropy
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def norm(name, type, p, q, residual=False, i8=False, pad=0):
    return {"name": name, "op": "norm", "type": type, "p": p, "q": q, "residual": residual, "i8": i8, "pad": pad}


def norm_bwd(name, type, p, q, stream=True, pad=0):
    return {"name": name, "op": "norm_bwd", "type": type, "p": p, "q": q, "stream": stream, "pad": pad}


def adapters(name, type, p, q, r, n, k, requests, act="none", bias=False, residual=False, pad=0):
    return {"name": name, "op": "adapters", "type": type, "p": p, "q": q, "r": r, "n": n, "k": k, "requests": requests,
            "act": act, "bias": bias, "residual": residual, "pad": pad}


def logprobs(name, type, p, v, top=0, entropy=False, masked=False, pad=0):
    return {"name": name, "op": "logprobs", "type": type, "p": p, "v": v, "top": top, "entropy": entropy, "masked": masked,
            "pad": pad}


def logprobs_bwd(name, type, p, v, entropy=False, masked=False, pad=0):
    return {"name": name, "op": "logprobs_bwd", "type": type, "p": p, "v": v, "entropy": entropy, "masked": masked, "pad": pad}


def listed():
    return [
        # one new token before a product with int8 weights
        norm("norm_token_i8", "bf16", 1, 8192, residual=True, i8=True),
        # a ragged batch of tokens before a product with int8 weights, rows inside a wider buffer
        norm("norm_ragged_i8", "f16", 777, 1999, residual=True, i8=True, pad=5),
        # a training step's activations, the sum kept for the residual stream
        norm("norm_train", "bf16", 16384, 8192, residual=True),
        # gradient of a small layer, where launches count
        norm_bwd("norm_bwd_small", "f16", 256, 1024),
        # gradient of norm_train
        norm_bwd("norm_bwd_train", "bf16", 16384, 8192),
        # one new token of one request through a shared projection and its adapter
        adapters("adapters_token", "bf16", 1, 2048, 8192, 32, 16, 1, act="gelu", bias=True),
        # one new token of each of 37 requests, with adapters of their own
        adapters("adapters_tokens", "f16", 37, 8192, 2048, 64, 32, 37, residual=True),
        # the prompts of 24 requests in one batch
        adapters("adapters_prompt", "bf16", 8192, 2048, 8192, 16, 64, 24, act="gelu", bias=True),
        # sampling: log probabilities and alternatives of a few new tokens
        logprobs("logprobs_tokens", "bf16", 16, 131072, top=20, entropy=True, masked=True),
        # scoring of a training batch's tokens, with their entropy
        logprobs("logprobs_train", "bf16", 4096, 131072, entropy=True),
        # gradient over a ragged batch in 32 bits
        logprobs_bwd("logprobs_bwd_ragged", "f32", 203, 32003, entropy=True, masked=True, pad=3),
        # gradient of logprobs_train
        logprobs_bwd("logprobs_bwd_train", "bf16", 4096, 131072, entropy=True),
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        # half of the sizes are multiples of 64 where they can be, as most layers' are
        return max(lo, v // 64 * 64) if v >= 128 and rng.random() < 0.5 else v

    some = lambda: rng.random() < 0.5  # noqa: E731
    pad = rng.choice([0, 0, 8, 5])
    op = rng.choice(["norm", "norm_bwd", "adapters", "logprobs", "logprobs_bwd"])
    if op in ("norm", "norm_bwd"):
        type, p, q = rng.choice(["bf16", "f16", "f32"]), size(1, 16384), size(64, 8192)
        if type == "f32":
            p = max(1, p // 2)
        if op == "norm":
            c = norm(None, type, p, q, residual=some(), i8=some() and type != "f32", pad=pad)
        else:
            c = norm_bwd(None, type, p, q, stream=some(), pad=pad)
    elif op == "adapters":
        p, q, r, k, n = size(1, 8192), size(256, 8192), size(256, 8192), rng.choice([4, 8, 16, 24, 32, 64]), size(1, 64)
        while p * q * r > 8192 * 2048 * 8192:
            p = max(1, p // 2)
        # a few prompts, or one new token of each request
        requests = p if p <= 64 and some() else min(p, rng.randint(1, 24))
        c = adapters(None, rng.choice(["bf16", "f16"]), p, q, r, n, k, requests, act=rng.choice(["none", "gelu", "silu"]),
                     bias=some(), residual=some(), pad=pad)
    else:
        type, p, v = rng.choice(["bf16", "f16", "f32"]), size(1, 4096), size(1000, 131072)
        if type == "f32":
            p = max(1, p // 2)
        if op == "logprobs":
            c = logprobs(None, type, p, v, top=rng.choice([0, 1, 5, 20, 64]), entropy=some(), masked=some(), pad=pad)
        else:
            c = logprobs_bwd(None, type, p, v, entropy=some(), masked=some(), pad=pad)
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, p, pad = TYPES[case["type"]], case["p"], case["pad"]

    def normal(rows, cols, scale=1.0, pad=pad):
        wide = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dt)
        return wide[:, :cols]

    s = {"case": dict(case)}
    if case["op"] in ("norm", "norm_bwd"):
        q = case["q"]
        s["w"] = (1.0 + 0.2 * torch.randn(q, generator=gen, device="cuda")).to(dt)
        if case["op"] == "norm":
            s["x"] = normal(p, q)
            s["residual"] = normal(p, q, 2.0) if case["residual"] else None
        else:
            s["h"] = normal(p, q, 2.0)
            s["dy"] = normal(p, q, 0.05)
            s["dh"] = normal(p, q, 0.05) if case["stream"] else None
    elif case["op"] == "adapters":
        q, r, n, k = case["q"], case["r"], case["n"], case["k"]
        s["x"], s["w"] = normal(p, q), normal(r, q, 1.0 / math.sqrt(q))
        s["a"] = normal(n * k, q, 1.0 / math.sqrt(q), pad=0).view(n, k, q)
        s["b"] = normal(n * r, k, 0.5 / math.sqrt(k), pad=0).view(n, r, k)
        s["c"] = torch.rand(n, generator=gen, device="cuda") + 0.5
        # each request's tokens lie together; one request in eight or so has no adapter
        m = case["requests"]
        which = torch.randint(0, n, (m,), generator=gen, device="cuda", dtype=torch.int32)
        which[torch.rand(m, generator=gen, device="cuda") < 0.125] = -1
        if p == m:
            s["index"] = which
        else:
            cuts = torch.randint(1, p, (m - 1,), generator=gen, device="cuda").sort().values
            s["index"] = which[torch.searchsorted(cuts, torch.arange(p, device="cuda"), right=True)]
        s["bias"] = (torch.randn(r, generator=gen, device="cuda") * 0.1).to(dt) if case["bias"] else None
        s["residual"] = normal(p, r, 2.0) if case["residual"] else None
    else:
        v = case["v"]
        s["logits"] = normal(p, v, 2.5)
        rows = torch.arange(p, device="cuda")
        s["tokens"] = torch.randint(0, v, (p,), generator=gen, device="cuda")
        at = s["logits"][rows, s["tokens"]] + 6.0  # most given tokens are likely ones
        if case["masked"]:
            # a vocabulary mask: tokens that may not follow
            s["logits"][:, torch.rand(v, generator=gen, device="cuda") < 0.05] = -math.inf
        s["logits"][rows, s["tokens"]] = at
        s["tokens"][torch.rand(p, generator=gen, device="cuda") < 0.02] = -1
        if case["op"] == "logprobs_bwd":
            # what the forward call left: each row's lse and entropy
            lse, entropy = statistics(s["logits"].double())
            s["lse"], s["h"] = lse.float(), entropy.float()
            s["dlp"] = torch.randn(p, generator=gen, device="cuda") / 64
            s["dh"] = torch.randn(p, generator=gen, device="cuda") / 512 if case["entropy"] else None
    return s


def statistics(l):
    """lse and entropy of each row."""
    u = l - l.amax(1, keepdim=True)
    e = torch.exp(u)
    total = e.sum(1)
    entropy = torch.log(total) - (e * torch.where(e > 0, u, torch.zeros_like(u))).sum(1) / total
    return l.amax(1) + torch.log(total), entropy


# ---- the plain form ---------------------------------------------------------------
def activated(a, act):
    if act == "gelu":
        return 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5)))
    if act == "silu":
        return a / (1.0 + torch.exp(-a))
    return a


def largest(l, top):
    """Tokens of each row's largest logits, the lowest of equal ones first: keys that hold the
    value's order above the negated token's."""
    bits = (l + 0.0).view(torch.int32).to(torch.int64)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    keys = (order << 32) + (0xFFFFFFFF - torch.arange(l.shape[1], device=l.device))
    return 0xFFFFFFFF - (torch.topk(keys, top, dim=1).values & 0xFFFFFFFF)


def run_plain(s):
    c = s["case"]
    dt = TYPES[c["type"]]
    if c["op"] == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = (h + s["residual"].float()).to(dt).float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].float()
        if c["i8"]:
            top = y.abs().amax(1, keepdim=True)
            y = torch.round(y * (127.0 / top)) * (top / 127.0)
        return (y.to(dt), h.to(dt)) if c["residual"] else y.to(dt)
    if c["op"] == "norm_bwd":
        h, dy = s["h"].float(), s["dy"].float()
        rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        g, n = dy * s["w"].float(), h * rstd
        dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return dx.to(dt), (dy * n).sum(0).to(dt)
    if c["op"] == "adapters":
        x, n, k = s["x"].float(), c["n"], c["k"]
        # every adapter's first product, those of other requests' adapters set to zero
        t = (x @ s["a"].float().view(n * k, -1).t()).view(-1, n, k) * s["c"][:, None]
        t = t * (s["index"][:, None] == torch.arange(n, device=x.device))[:, :, None]
        a = x @ s["w"].float().t() + t.view(-1, n * k) @ s["b"].float().transpose(1, 2).reshape(n * k, -1)
        if s["bias"] is not None:
            a = a + s["bias"].float()
        y = activated(a, c["act"])
        return (y if s["residual"] is None else s["residual"].float() + y).to(dt)
    l, given = s["logits"].float(), s["tokens"] >= 0
    t = s["tokens"].clamp(min=0)[:, None]
    if c["op"] == "logprobs_bwd":
        p = torch.exp(l - s["lse"][:, None])
        d = -p * (s["dlp"] * given)[:, None]
        d.scatter_add_(1, t, (s["dlp"] * given)[:, None])
        if s["dh"] is not None:
            d = d - s["dh"][:, None] * p * (torch.where(p > 0, l - s["lse"][:, None], torch.zeros_like(l)) + s["h"][:, None])
        return d.to(dt)
    lse, entropy = statistics(l)
    out = {"logprobs": torch.where(given, l.gather(1, t)[:, 0] - lse, torch.zeros_like(lse)), "lse": lse}
    if c["entropy"]:
        out["entropy"] = entropy
    if c["top"]:
        out["top_tokens"] = largest(l, c["top"])
        out["top_logprobs"] = l.gather(1, out["top_tokens"]) - lse[:, None]
    return out


# ---- the library's operators --------------------------------------------------------
def run_own(s):
    from fp64_gemm_emulation_amd import binding as oz
    c = s["case"]
    if c["op"] == "norm" and c["i8"]:
        levels, scale, *h = oz.rms_norm_i8(s["x"], s["w"], residual=s["residual"], eps=EPS)
        y = torch.empty(levels.shape, dtype=TYPES[c["type"]], device=levels.device)
        torch.mul(levels, scale[:, None], out=y)
        return (y, *h) if h else y
    if c["op"] == "norm":
        return oz.rms_norm(s["x"], s["w"], residual=s["residual"], eps=EPS)
    if c["op"] == "norm_bwd":
        return oz.rms_norm_backward(s["dy"], s["h"], s["w"], dh=s["dh"], eps=EPS)
    if c["op"] == "adapters":
        return oz.linear_adapters(s["x"], s["w"], s["a"], s["b"], s["index"], scale=s["c"], bias=s["bias"],
                                  activation=c["act"], residual=s["residual"])
    if c["op"] == "logprobs_bwd":
        return oz.token_logprobs_backward(s["dlp"], s["logits"], s["tokens"], s["lse"], dentropy=s["dh"],
                                          entropy=s["h"] if c["entropy"] else None)
    got = oz.token_logprobs(s["logits"], s["tokens"], top=c["top"], entropy=c["entropy"])
    out = {"logprobs": got.logprobs, "lse": got.lse}
    if c["entropy"]:
        out["entropy"] = got.entropy
    if c["top"]:
        out["top_tokens"], out["top_logprobs"] = got.top_tokens, got.top_logprobs
    return out


def run(state):
    return run_own(state) if own else run_plain(state)


def work(case):
    p, e = case["p"], TYPES[case["type"]].itemsize
    if case["op"] == "norm":
        pq = p * case["q"]
        out = (1 if case["i8"] else e) * pq + (4 * p if case["i8"] else 0)
        return {"bytes": e * pq * (3 if case["residual"] else 1) + out + e * case["q"], "flops": 5 * pq}
    if case["op"] == "norm_bwd":
        return {"bytes": e * (p * case["q"] * (4 if case["stream"] else 3) + 2 * case["q"]), "flops": 10 * p * case["q"]}
    if case["op"] == "adapters":
        q, r, k = case["q"], case["r"], case["k"]
        used = min(case["n"], case["requests"])
        out = 2 if case["residual"] else 1
        return {"bytes": e * (p * q + r * q + out * p * r + used * k * (q + r) + (r if case["bias"] else 0)) + 4 * p,
                "flops": 2 * p * q * r + 2 * p * k * (q + r)}
    pv = p * case["v"]
    if case["op"] == "logprobs_bwd":
        return {"bytes": 2 * e * pv + 20 * p, "flops": 6 * pv}
    return {"bytes": e * pv + p * (16 + 12 * case["top"]), "flops": 5 * pv}


# ---- the definition in 64 bits --------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:
            # the sum is rounded to its type before the norm
            h = (h + s["residual"].double()).to(TYPES[case["type"]]).double()
        y = h / torch.sqrt((h ** 2).sum(dim=1, keepdim=True) / case["q"] + EPS) * s["w"].double()
        if case["i8"]:
            step = y.abs().max(dim=1, keepdim=True).values / 127
            y = (y / step).round() * step
        return (y, h) if case["residual"] else y
    if case["op"] == "norm_bwd":
        h, dy, w = s["h"].double(), s["dy"].double(), s["w"].double()
        power = (h ** 2).sum(dim=1, keepdim=True) / case["q"] + EPS
        dx = dy * w / power.sqrt() - h * (dy * w * h).sum(dim=1, keepdim=True) / case["q"] / power ** 1.5
        if case["stream"]:
            dx = dx + s["dh"].double()
        return dx, (dy * h / power.sqrt()).sum(dim=0)
    if case["op"] == "adapters":
        x = s["x"].double()
        a = torch.matmul(x, s["w"].double().t())
        for i in range(case["n"]):
            rows = (s["index"] == i).nonzero()[:, 0]
            if len(rows):
                a[rows] += torch.matmul(torch.matmul(x[rows], s["a"][i].double().t()), s["b"][i].double().t()) * s["c"][i].double()
        if case["bias"]:
            a = a + s["bias"].double()
        if case["act"] == "gelu":
            a = a * torch.special.ndtr(a)
        elif case["act"] == "silu":
            a = a * torch.sigmoid(a)
        return a + s["residual"].double() if case["residual"] else a
    given, rows = s["tokens"] >= 0, torch.arange(case["p"], device="cuda")
    t = s["tokens"].clamp(min=0)
    if case["op"] == "logprobs_bwd":
        logp = torch.log_softmax(s["logits"].double(), dim=1)
        p = logp.exp()
        dlp = torch.where(given, s["dlp"].double(), 0.0)
        d = -dlp[:, None] * p
        d[rows, t] += dlp
        if case["entropy"]:
            plogp = torch.special.xlogy(p, p)
            d -= s["dh"].double()[:, None] * (plogp - p * plogp.sum(dim=1, keepdim=True))
        return d
    l = s["logits"].double()
    lse = torch.logsumexp(l, dim=1)
    out = {"logprobs": torch.where(given, l[rows, t] - lse, 0.0), "lse": lse}
    if case["entropy"]:
        out["entropy"] = torch.special.entr((l - lse[:, None]).exp()).sum(dim=1)
    if case["top"]:
        out["top_tokens"] = None
        out["top_logprobs"] = torch.topk(l, case["top"], dim=1).values - lse[:, None]
    return out
