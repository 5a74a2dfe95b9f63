"""The product with adapters in 64 bits, on torch tensors of any device, and the error bounds the
tests hold the kernels to.

Bounds, beside those of the product (tests/linear_reference.py): S = scale X A^T is summed like a
product of depth q, joined from up to 16 parts and rounded to the type before it meets B (half
a step of it; products of few rows leave that out), whose product with it has depth k.
"""
import torch

from tests.linear_reference import TINY, UNIT, activate, rounding


def linear_adapters(x, w, a, b, index, scale=None, bias=None, act="none", residual=None):
    """(y, bound) in 64 bits."""
    x64, w64, dt = x.double(), w.double(), x.dtype
    q, k = x.shape[1], a.shape[1]
    z = x64 @ w64.t()
    err = (q + 16) * 2.0 ** -23 * (x64.abs() @ w64.abs().t())
    for j in set(index.tolist()) & set(range(a.shape[0])):
        at = (index == j).nonzero()[:, 0]
        c = 1.0 if scale is None else scale[j].double()
        aj, bj, xj = a[j].double(), b[j].double(), x64[at]
        s = c * (xj @ aj.t())
        serr = abs(c) * (q + 34) * 2.0 ** -23 * (xj.abs() @ aj.abs().t()) + UNIT[dt] * s.abs() + TINY[dt]
        z[at] += s @ bj.t()
        err[at] += 1.01 * (serr @ bj.abs().t()) + (k + 16) * 2.0 ** -23 * (s.abs() @ bj.abs().t())
    err = err + 2.0 ** -23 * z.abs()
    if bias is not None:
        z = z + bias.double()
        err = err + 2.0 ** -23 * z.abs()
    y = activate(z, act)
    bound = 1.2 * err + (2.0 ** -20 * (1 + z.abs()) if act != "none" else 0.0)
    if residual is not None:
        y = y + residual.double()
        bound = bound + 2.0 ** -23 * y.abs()
    return y, bound * 1.01 + rounding(y, dt)
