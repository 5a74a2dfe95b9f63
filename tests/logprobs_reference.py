"""Log probabilities of tokens and their gradient in 64 bits, on torch tensors of any device, and the
error bounds the tests hold the kernels to.

Bounds, in units u = 2^-24.  With d = l - m, m the row's maximum: exp(d) is off by (|d| + 3) u of
itself (d is rounded, then multiplied, then the exponential's own error), and at most v / 256 + 100 additions,
rescalings and joins round each sum (256 threads take a row at least).  So s = sum exp(d) is off
by E = (v / 256 + 103) u + A u, relative, with A = sum p |d|; log s adds 3 u of itself, and
l - m - log s a rounding of each step.  The entropy log s - t / s has t = sum exp(d) d of one sign,
off by (v / 256 + 104) u of itself and by sum p d^2 of its factors.  In the gradient p = exp(l - lse) is off
by what lse is rounded by, |lse| u (where the kernel works lse out anew, by E), and by (2 |log p| + 4) u.
"""
import math
from typing import NamedTuple

import torch

from tests.linear_reference import rounding

U = 2.0 ** -24


class Row(NamedTuple):
    d: torch.Tensor      # l - max
    logs: torch.Tensor   # log sum exp(d)
    lse: torch.Tensor
    entropy: torch.Tensor
    bad: torch.Tensor    # rows with NaN or +Inf
    none: torch.Tensor   # rows of -Inf alone
    err: torch.Tensor    # of log s
    err_h: torch.Tensor  # of the entropy


def rows(l):
    l = l.double()
    p, v = l.shape
    bad = (torch.isnan(l) | (l == math.inf)).any(1)
    none = (l == -math.inf).all(1)
    l = torch.where((bad | none)[:, None], torch.zeros_like(l), l)
    m = l.amax(1)
    d = l - m[:, None]
    e = d.exp()
    s = e.sum(1)
    dz = torch.where(e > 0, d, torch.zeros_like(d))
    t, b = (e * dz).sum(1) / s, (e * dz * dz).sum(1) / s
    logs = s.log()
    n = v / 256 + 103
    err = (n - t) * U + 4 * U * logs
    err_h = err + (n + 4) * U * -t + U * (b - t) + 4 * U * (logs - t)
    nan, inf = torch.full_like(s, math.nan), torch.full_like(s, -math.inf)
    fix = lambda x, empty: torch.where(bad, nan, torch.where(none, empty, x))  # noqa: E731
    return Row(d, logs, fix(m + logs, inf), fix(logs - t, torch.zeros_like(s)), bad, none, err, err_h)


def given(r, tokens):
    """(log probabilities of the tokens, bounds)"""
    v = r.d.shape[1]
    z = r.d.gather(1, tokens.clamp(0, v - 1)[:, None])[:, 0] - r.logs
    z = torch.where(r.none, torch.full_like(z, -math.inf), z)
    z = torch.where(r.bad | (tokens >= v), torch.full_like(z, math.nan), z)
    z = torch.where(tokens < 0, torch.zeros_like(z), z)
    return z, r.err + 4 * U * torch.nan_to_num(z.abs(), posinf=0.0) + 2 * U * r.logs


def largest(l, top):
    """Indices of the largest logits: a stable sort, NaN as -Inf."""
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l).double()
    return torch.sort(l, dim=1, descending=True, stable=True).indices[:, :top]


def top_values(r, which):
    z = r.d.gather(1, which) - r.logs[:, None]
    z = torch.where(r.none[:, None], torch.full_like(z, -math.inf), z)
    z = torch.where(r.bad[:, None], torch.full_like(z, math.nan), z)
    return z, r.err[:, None] + 4 * U * torch.nan_to_num(z.abs(), posinf=0.0) + 2 * U * r.logs[:, None]


def backward(l, tokens, dlp=None, dh=None):
    """(gradient, bound); lse and the entropy are taken to be given rounded to f32."""
    dt, r, v = l.dtype, rows(l), l.shape[1]
    z = r.d - r.logs[:, None]
    p = z.exp()
    z = torch.where(p > 0, z, torch.zeros_like(z))
    out, weight = torch.zeros_like(p), torch.zeros_like(p)
    if dlp is not None:
        dlp = torch.where(tokens < 0, torch.zeros_like(dlp), dlp).double()
        hot = torch.zeros_like(p).scatter_(1, tokens.clamp(0, v - 1)[:, None], 1.0)
        out = dlp[:, None] * (hot - p)
        weight = dlp.abs()[:, None] * p
    if dh is not None:
        h = r.entropy[:, None]
        out = out - dh.double()[:, None] * p * (z + h)
        weight = weight + dh.double().abs()[:, None] * p * (z.abs() + h)
    lse = torch.where(r.lse.abs() <= 64, r.lse.abs() * U, r.err)[:, None]
    bound = weight * (lse + (2 * z.abs() + 8) * U) + 4 * U * out.abs()
    if dh is not None:
        bound = bound + dh.double().abs()[:, None] * p * (lse + 4 * U * (z.abs() + h))
    bad = r.bad | (tokens >= v) if dlp is not None else r.bad
    out = torch.where(bad[:, None], torch.full_like(out, math.nan), out)
    out = torch.where((r.none & ~bad)[:, None], torch.zeros_like(out), out)
    bound = torch.nan_to_num(bound)
    return out, bound * 1.01 + rounding(out, dt) + 2.0 ** -126
