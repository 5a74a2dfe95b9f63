"""Plain 64-bit forms of the linear-layer operators, on torch tensors of any device, and the
error bounds the tests hold the kernels to.

Bounds.  A product of depth q in 32-bit accumulators is off by at most about (q + 16) 2^-23
times the product of the magnitudes (each of the q additions rounds once, or truncates, at
2^-23 of a partial sum that the magnitudes bound).  Activations have slopes up to 1.13 and are
evaluated in f32 to a few 2^-22 of |a| + 1.  Dropout multiplies all that by its scale.  The
result is then rounded once: half a unit in the last place, 2^-8 (bf16) or 2^-11 (f16) of it,
or half the smallest subnormal.  In the gradients dZ is rounded to the type before the
products, which adds the same 2^-8 or 2^-11 of the products of the magnitudes.
"""
import math

import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def philox(counter, key):
    """Philox4x32-10 of one counter (4 words) and key (2 words), in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def draws(rows, cols, seed, offset, row0=0):
    """The 16-bit draw of every element of rows row0 .. row0 + rows - 1 of a matrix of cols columns."""
    per_row = -(-cols // 8)
    n = np.arange(row0 * per_row, (row0 + rows) * per_row, dtype=np.uint64)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [n & low, n >> half, np.full_like(n, offset & 0xFFFFFFFF), np.full_like(n, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    u = np.stack([w for x in c for w in (x & np.uint64(0xFFFF), x >> np.uint64(16))], 1).astype(np.int64)
    return u.reshape(rows, per_row * 8)[:, :cols]


def keep_and_scale(rows, cols, drop, device="cpu"):
    """(bool mask, scale) of drop = (probability, seed, offset); drop may be None."""
    if drop is None or drop[0] == 0.0:
        return torch.ones(rows, cols, dtype=torch.bool, device=device), 1.0
    t = int(np.rint(drop[0] * 65536))
    keep = torch.from_numpy(draws(rows, cols, drop[1], drop[2]) >= t).to(device)
    return keep, 65536.0 / (65536 - t) if t < 65536 else 0.0


def dropped(v, drop):
    keep, scale = keep_and_scale(v.shape[0], v.shape[1], drop, v.device)
    return torch.where(keep, v * scale, torch.zeros_like(v)), scale


def activate(a, act):
    if act == "relu":
        return torch.where(a <= 0, torch.zeros_like(a), a)
    if act == "gelu":
        return a * 0.5 * torch.erfc(-a / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    if act == "silu":
        return a * torch.sigmoid(a)
    return a


def slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 0.134145 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def rounding(y, dtype):
    return UNIT[dtype] * y.abs() + TINY[dtype]


def linear(x, w, bias=None, act="none", residual=None, drop=None):
    """(y, z, bound of y, bound of z) in 64 bits."""
    x64, w64, dt = x.double(), w.double(), x.dtype
    a = x64 @ w64.t()
    err = (x.shape[1] + 16) * 2.0 ** -23 * (x64.abs() @ w64.abs().t())
    if bias is not None:
        a = a + bias.double()
        err = err + 2.0 ** -23 * a.abs()
    y, scale = dropped(activate(a, act), drop)
    bound = scale * (1.2 * err + (2.0 ** -20 * (1 + a.abs()) if act != "none" else 0.0))
    if residual is not None:
        y = y + residual.double()
        bound = bound + 2.0 ** -23 * y.abs()
    return y, a, bound * 1.01 + rounding(y, dt), err * 1.01 + rounding(a, dt)


def linear_backward(dy, x, w, z=None, act="none", drop=None):
    """(dx, dw, db) and their bounds in 64 bits."""
    dt = dy.dtype
    dz, scale = dropped(dy.double(), drop)
    dz_err = torch.zeros_like(dz)
    if act != "none":
        dz_err = 2.0 ** -19 * dz.abs() * (1 + z.double().abs())
        dz = dz * slope(z.double(), act)
    rounded = dz_err + (rounding(dz, dt) if act != "none" or drop is not None else 0.0)
    x64, w64 = x.double(), w.double()
    dx, dw, db = dz @ w64, dz.t() @ x64, dz.sum(0)
    p, r = dz.shape
    ex = rounded @ w64.abs() + (r + 16) * 2.0 ** -23 * (dz.abs() @ w64.abs())
    ew = rounded.t() @ x64.abs() + (p + 16) * 2.0 ** -23 * (dz.abs().t() @ x64.abs())
    eb = dz_err.sum(0) + (p + 16) * 2.0 ** -23 * dz.abs().sum(0)
    return (dx, dw, db), (ex * 1.02 + rounding(dx, dt), ew * 1.02 + rounding(dw, dt), eb * 1.02 + rounding(db, dt))


def quantize(x):
    """(int8 levels, f32 scales) by the rule of ozaki2_quantize_rows, in its 32-bit steps."""
    x = x.float()
    m = x.abs().amax(1) if x.shape[1] else x.new_zeros(x.shape[0])
    live = (m >= 1e-36) & torch.isfinite(m)
    inv = torch.where(live, torch.full_like(m, 127.0) / m, torch.zeros_like(m))
    levels = torch.where(live[:, None], torch.round(x * inv[:, None]), torch.zeros_like(x)).to(torch.int8)
    # (a division by a tensor: by a Python number torch multiplies by the reciprocal on a GPU)
    step = m / torch.full_like(m, 127.0)
    scale = torch.where(torch.isfinite(m), torch.where(live, step, torch.zeros_like(m)), torch.full_like(m, math.nan))
    return levels, scale


def linear_i8(x, v, t, bias=None, act="none", residual=None):
    """(y, bound) in 64 bits from the quantised operands."""
    dt = x.dtype
    levels, s = quantize(x)
    a = (levels.double() @ v.double().t()) * s.double()[:, None] * t.double()
    err = 4 * 2.0 ** -24 * a.abs()  # the conversion of the sum and the two scalings
    if bias is not None:
        a = a + bias.double()
        err = err + 2.0 ** -23 * a.abs()
    y = activate(a, act)
    bound = 1.2 * err + (2.0 ** -20 * (1 + a.abs()) if act != "none" else 0.0)
    if residual is not None:
        y = y + residual.double()
        bound = bound + 2.0 ** -23 * y.abs()
    return y, bound * 1.01 + rounding(y, dt)


def assert_within(got, want, bound, what):
    """Every element within its bound; NaN and Inf where, and only where, they belong."""
    top = torch.finfo(got.dtype).max
    got = got.double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)} != {tuple(want.shape)}"
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    other = ~fine & ~torch.isnan(want)
    assert torch.equal(got[other], want[other]), f"{what}: infinities differ"
    # a value past the type's range rounds to infinity
    past = torch.isinf(got) & (torch.sign(got) == torch.sign(want)) & (want.abs() + bound >= top)
    off = torch.where(past, torch.zeros_like(want), (got - want).abs() - bound)[fine]
    assert not (off > 0).any(), f"{what}: {int((off > 0).sum())} of {want.numel()} elements out of bounds, by up to {off.max().item():.3e}"
