"""A feed-forward block trained in bfloat16 and served from int8 weights.

    x  = tokens + D(positions)                       dropout_add
    h  = gelu(x W1^T + b1)                           linear, pre-activation kept
    y  = x + D(h W2^T + b2)                          linear, dropout and residual in its epilogue

Training takes the gradients with linear_backward (the masks are made anew from seed and
offset), weights are held in float32 and rounded to bfloat16 for each step.  Serving quantises
the trained weights by rows and runs single tokens through linear_i8.  The emulated FP64 product
(dgemm) of the same weights is the yardstick of what bfloat16 and int8 cost in accuracy.

    python3 examples/feed_forward.py [--tokens 2048] [--width 1024] [--hidden 4096] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp64_gemm_emulation_amd import binding as oz  # noqa: E402


class FeedForward:
    """Weights in float32; compute copies in `dtype`."""

    def __init__(self, width, hidden, dropout, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda rows, cols: torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5  # noqa: E731
        self.master = {"w1": new(hidden, width), "b1": torch.zeros(hidden, device="cuda"),
                       "w2": new(width, hidden), "b2": torch.zeros(width, device="cuda")}
        self.moments = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in self.master.items()}
        self.dropout, self.dtype, self.seed = dropout, dtype, seed
        self.refresh()

    def refresh(self):
        for name, value in self.master.items():
            setattr(self, name, value.to(self.dtype))

    def drop(self, step, place):
        """Another mask for each step and place: the generator's offset."""
        return dict(dropout=self.dropout, seed=self.seed, offset=3 * step + place)

    def forward(self, tokens, positions, step):
        x = oz.dropout_add(positions, tokens, **self.drop(step, 0))
        h, z = oz.linear(x, self.w1, bias=self.b1, activation="gelu", return_z=True)
        y = oz.linear(h, self.w2, bias=self.b2, residual=x, **self.drop(step, 1))
        return y, (x, h, z)

    def backward(self, dy, saved, step):
        """Gradients of the weights, of the tokens and of the positions."""
        x, h, z = saved
        dh, dw2, db2 = oz.linear_backward(dy, h, self.w2, **self.drop(step, 1))
        dx, dw1, db1 = oz.linear_backward(dh, x, self.w1, z=z, activation="gelu")
        dx += dy                                             # the residual's path
        return {"w1": dw1, "b1": db1, "w2": dw2, "b2": db2}, dx, oz.dropout_add(dx, **self.drop(step, 0))

    def update(self, grads, rate, step):
        """Adam on the float32 weights."""
        for name, grad in grads.items():
            first, second = self.moments[name]
            grad = grad.float()
            first.lerp_(grad, 0.1)
            second.lerp_(grad * grad, 0.05)
            self.master[name] -= rate * (first / (1 - 0.9 ** (step + 1))) / ((second / (1 - 0.95 ** (step + 1))).sqrt() + 1e-8)
        self.refresh()

    def quantized(self):
        return {"w1": oz.quantize_rows(self.master["w1"]), "w2": oz.quantize_rows(self.master["w2"])}

    def serve_i8(self, x, q):
        h = oz.linear_i8(x, *q["w1"], bias=self.b1, activation="gelu")
        return oz.linear_i8(h, *q["w2"], bias=self.b2, residual=x)

    def serve(self, x):
        return oz.linear(oz.linear(x, self.w1, bias=self.b1, activation="gelu"), self.w2, bias=self.b2, residual=x)

    def serve_f64(self, x):
        """The block in double precision, its products emulated on int8 matrix cores: W x for
        the tokens as columns."""
        mul = lambda w, a: oz.dgemm(oz.colmajor(w.double()), oz.colmajor(a), s=15)  # noqa: E731
        x = x.double().t()
        a = mul(self.master["w1"], x) + self.master["b1"].double()[:, None]
        h = 0.5 * a * torch.erfc(-a * 0.5 ** 0.5)
        return (x + mul(self.master["w2"], h) + self.master["b2"].double()[:, None]).t()


def run(tokens=2048, width=1024, hidden=4096, steps=20, rate=1e-3, dropout=0.1):
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    x, positions = new(tokens, width).bfloat16(), (0.1 * new(tokens, width)).bfloat16()
    teacher = new(width, width) * width ** -0.5
    target = x.float() + 0.5 * torch.tanh(x.float() @ teacher.t())
    block = FeedForward(width, hidden, dropout)
    losses = []
    for step in range(steps):
        y, saved = block.forward(x, positions, step)
        err = y.float() - target
        losses.append(err.square().mean())
        grads, _, _ = block.backward((err * (2.0 / tokens)).bfloat16(), saved, step)
        block.update(grads, rate, step)
    one = x[:1].contiguous()
    q = block.quantized()
    exact = block.serve_f64(one) - one.double()       # what the block adds to the stream
    off = lambda y: ((y.double() - one.double() - exact).norm() / exact.norm()).item()  # noqa: E731
    return {"losses": [v.item() for v in losses], "bf16": off(block.serve(one)), "int8": off(block.serve_i8(one, q))}


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 2048), ("width", 1024), ("hidden", 4096), ("steps", 20)):
        p.add_argument(f"--{name}", type=int, default=value)
    out = run(**vars(p.parse_args()))
    print("loss " + " ".join(f"{v:.4f}" for v in out["losses"]))
    print(f"one token against the emulated FP64 block: bfloat16 {out['bf16']:.2e}, int8 weights {out['int8']:.2e}")


if __name__ == "__main__":
    main()
