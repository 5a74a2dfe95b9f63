"""The norm and its gradient in 64 bits, on torch tensors of any device, and the error bounds the
tests hold the kernels to.

Bounds, in units u = 2^-24 (an f32 operation rounds within u of its result).  A row's sum of
squares goes through at most 32 additions in a thread, 6 over a wave and 16 over the waves, all of
positive numbers: 54 u.  The norm takes its root (half of that), and a division, a root and an
addition (3 u): rstd is off by 31 u, and y = h rstd w, two or three products, by 34 u; the bound
takes 48 u.  A row's mean of g n is off by 54 u of the mean of |g n| for its sum and 36 u for
its factors; dx adds the errors of both terms of the bracket, each at most 128 u of its own
magnitude.  dw adds p products, each off by 34 u, in at most p + 16 roundings.  Results are then
rounded once, by half a step of the type.
"""
import torch

from tests.linear_reference import rounding

U = 2.0 ** -24


def hidden(x, residual):
    """x + residual as one rounded 32-bit sum, rounded to the type (the sum of two 16-bit numbers
    is rounded twice here as in the kernel)."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm(h, w, eps):
    """(y unrounded, its bound before rounding) in 64 bits."""
    h64 = h.double()
    y = h64 / (h64.square().mean(1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.double()
    return y, 48 * U * y.abs()


def rms_norm(h, w, eps):
    y, err = norm(h, w, eps)
    return y, err * 1.01 + rounding(y, h.dtype)


def backward(dy, h, w, dh, eps):
    """((dx, dw), bounds) in 64 bits."""
    dt, p, q = dy.dtype, *dy.shape
    h, dy = h.double(), dy.double()
    g = dy if w is None else dy * w.double()
    rstd = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    n = h * rstd
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    err = 128 * U * rstd * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        err = err + U * dx.abs()
    dw = (dy * n).sum(0)
    err_w = (p + 16 + 36) * U * (dy * n).abs().sum(0)
    return (dx, dw), (err * 1.01 + rounding(dx, dt), err_w * 1.01 + rounding(dw, dt))
