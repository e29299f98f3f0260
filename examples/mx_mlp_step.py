"""Half a gated MLP's training step in MX form.

h = silu(z) * u, y = h w^T and, from dL/dy, the gradients of z, u and w, as a
training step runs them with this library: h goes to the product in 4 bits,
z and u are kept for the backward pass as 8-bit MX blocks (2.06 bytes an
element of h instead of 4), gradients are cast to E5M2 in both directions by
one read, and the weight gradient is added to a 32-bit sum.

    python examples/mx_mlp_step.py

Prints how far the output and each gradient are from the same step in 32 bits
without any cast.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tensor_scaling_cast_gb300 import fp8q as F  # noqa: E402


class HalfMLP:
    """The weights w [hidden, ffn] in MX form and what a step needs between its passes."""

    def __init__(self, w: torch.Tensor, tokens: int):
        hidden, ffn = w.shape
        new, dev = F.MXMatrix.allocate, w.device
        self.w4, self.w8, self.w8t = new(hidden, ffn, F.E2M1), new(hidden, ffn), new(ffn, hidden)
        F.mx_cast_ex(w, F.E2M1, F.MX_CEIL, 0, F.MX_ROWWISE, self.w4.q, self.w4.e8m0)
        F.mx_cast_dual(w, F.E4M3, F.MX_CEIL, 0, self.w8.q, self.w8.e8m0, self.w8t.q, self.w8t.e8m0)
        self.z, self.u, self.h4 = new(tokens, ffn), new(tokens, ffn), new(tokens, ffn, F.E2M1)
        self.dy, self.dyt = new(tokens, hidden, F.E5M2), new(hidden, tokens, F.E5M2)
        self.h8, self.h8t = new(tokens, ffn), new(ffn, tokens)
        self.dh, self.h = (torch.empty(tokens, ffn, dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.dw = torch.zeros(hidden, ffn, device=dev)               # summed over steps

    def forward(self, z, u):
        y = torch.empty(z.shape[0], self.w4.shape[0], dtype=z.dtype, device=z.device)
        F.mx_act_forward(F.MX_ACT_SILU, z, u, z_saved=self.z, u_saved=self.u, h_mx=self.h4, rule=F.MX_CEIL)
        F.mx_matmul(self.h4, self.w4, y)
        return y

    def backward(self, dy):
        F.mx_cast_dual(dy, F.E5M2, F.MX_CEIL, 0, self.dy.q, self.dy.e8m0, self.dyt.q, self.dyt.e8m0)
        F.mx_matmul(self.dy, self.w8t, self.dh)                      # dh = dy w
        dz, du = torch.empty_like(self.dh), torch.empty_like(self.dh)
        F.mx_act_backward(F.MX_ACT_SILU, self.z, self.u, self.dh, dz, du, h=self.h)
        F.mx_cast_dual(self.h, F.E4M3, F.MX_CEIL, 0, self.h8.q, self.h8.e8m0, self.h8t.q, self.h8t.e8m0)
        F.mx_matmul(self.dyt, self.h8t, self.dw, add=self.dw)        # dw += dy^T h
        return dz, du


def main(tokens=1024, ffn=4096, hidden=1024, seed=0, quiet=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z, u = torch.randn(tokens, 2 * ffn, generator=gen, device="cuda").bfloat16().split(ffn, 1)
    w = (torch.randn(hidden, ffn, generator=gen, device="cuda") * 0.02).bfloat16()
    dy = (torch.randn(tokens, hidden, generator=gen, device="cuda") * 1e-3).bfloat16()
    mlp = HalfMLP(w, tokens)
    y = mlp.forward(z, u)
    dz, du = mlp.backward(dy)
    leaves = [t.detach().float().requires_grad_() for t in (z, u, w)]
    want = (torch.nn.functional.silu(leaves[0]) * leaves[1]) @ leaves[2].T
    want.backward(dy.float())
    off = {name: ((got.float() - ref).norm() / ref.norm()).item()
           for name, got, ref in (("y", y, want.detach()), ("dz", dz, leaves[0].grad), ("du", du, leaves[1].grad),
                                  ("dw", mlp.dw, leaves[2].grad))}
    if not quiet:
        print(f"{tokens} tokens, {hidden} x {ffn}: relative difference to 32 bits "
              + ", ".join(f"{k} {v:.3f}" for k, v in off.items()))
    return off


if __name__ == "__main__":
    main()
