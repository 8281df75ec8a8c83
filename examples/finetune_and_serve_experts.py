#!/usr/bin/env python3
"""Unquantised experts trained and then served, on the tiny workload's routing.

* ``step``: one step on bf16 SwiGLU experts.  The layer's routing and buckets
  give rows and offsets; the gate and up product has SwiGLU in its epilogue, the
  gradient goes back through it, and the experts' gradients are clipped together by
  their global norm.
* ``serve``: the trained experts as a layer, for a few tokens at a time.

Run it on a GPU:  python examples/finetune_and_serve_experts.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_layer_sigmoid_amd as mx  # noqa: E402
from examples.shared_and_finetuned_experts import Buffers, bucket  # noqa: E402

MOST = 32   # tokens of one call of the few-token layer


class Experts:
    """G SwiGLU experts w1 [G, 2F, H], w2 [G, H, F] in bf16, and what a step on
    ``rows`` bucketed rows needs; rows in no group are left at zero."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, rows: int):
        self.w1, self.w2 = w1.clone(), w2.clone()
        self.G, F2, self.H = w1.shape
        self.F, self.rows = F2 // 2, rows
        e = lambda *n, t=torch.bfloat16: torch.zeros(*n, dtype=t, device=w1.device)  # noqa: E731
        self.up = mx.Linear(rows, F2, self.H, groups=self.G)
        self.down = mx.Linear(rows, self.H, self.F, groups=self.G)
        self.up_dw = mx.Linear(rows, F2, self.H, groups=self.G, out_type="f32")
        self.down_dw = mx.Linear(rows, self.H, self.F, groups=self.G, out_type="f32")
        self.pre, self.act, self.o = e(rows, F2), e(rows, self.F), e(rows, self.H)
        self.dact, self.dz, self.dx = e(rows, self.F), e(rows, F2), e(rows, self.H)
        self.dw1, self.dw2 = e(*w1.shape, t=torch.float32), e(*w2.shape, t=torch.float32)
        self.grads = mx.GradList([self.dw1, self.dw2])   # clipped in place
        self.norm = e(1, t=torch.float32)
        need = [mx.moe_linear_act_workspace_bytes(self.up)]
        need += [mx.moe_linear_workspace_bytes(d) for d in (self.up, self.down)] + [mx.moe_grad_workspace_bytes(2), 256]
        self.scratch = torch.empty(max(need), dtype=torch.uint8, device=w1.device)

    def forward(self, x, offsets) -> torch.Tensor:
        """o = (silu(gate) * up) w2^T with [gate | up] = x w1^T; x holds the rows."""
        mx.moe_grouped_linear_act(self.up, x, self.w1, self.act, self.scratch, act="silu", gated=True, pre=self.pre,
                                  offsets=offsets)
        mx.moe_grouped_linear(self.down, self.act, self.w2, self.o, self.scratch, offsets=offsets)
        return self.o

    def backward(self, x, do, offsets) -> torch.Tensor:
        """The gradients of <o, do>: dw1, dw2 (f32), and the rows' returned."""
        mx.moe_grouped_linear_dw(self.down_dw, do, self.act, self.dw2, self.scratch, offsets=offsets)
        mx.moe_grouped_linear_dx(self.down, do, self.w2, self.dact, self.scratch, offsets=offsets)
        mx.moe_grouped_linear_act_backward(self.up, self.dact, self.pre, self.dz, self.scratch, act="silu", gated=True,
                                           offsets=offsets)
        mx.moe_grouped_linear_dw(self.up_dw, self.dz, x, self.dw1, self.scratch, offsets=offsets)
        mx.moe_grouped_linear_dx(self.up, self.dz, self.w1, self.dx, self.scratch, offsets=offsets)
        return self.dx

    def clip(self, max_norm: float) -> torch.Tensor:
        mx.moe_grad_clip(self.grads, max_norm, self.norm, self.scratch)
        return self.norm

    def update(self, rate: float) -> None:
        self.w1.copy_(self.w1.float() - rate * self.dw1)
        self.w2.copy_(self.w2.float() - rate * self.dw2)


def mix(o, tokens, w, T: int) -> torch.Tensor:
    """y[t] = sum over t's rows of w * o."""
    return torch.zeros(T, o.shape[1], device=o.device).index_add_(0, tokens, o.float() * w[:, None])


def step(ex: Experts, x, tokens, w, offsets, target, rate: float, max_norm: float):
    """A gradient step on 0.5 |y - target|^2; (loss, norm before clipping)."""
    rows = x[tokens]
    err = mix(ex.forward(rows, offsets), tokens, w, x.shape[0]) - target
    ex.backward(rows, (err[tokens] * w[:, None]).bfloat16(), offsets)
    norm = ex.clip(max_norm)
    ex.update(rate)
    return 0.5 * err.square().sum(), norm


def serve(ex: Experts, b: Buffers) -> torch.Tensor:
    """The layer on the experts, MOST tokens a call."""
    out = torch.empty_like(b.x)
    f = lambda n: getattr(b.d, n)  # noqa: E731
    for t in range(0, f("T"), MOST):
        n = min(MOST, f("T") - t)
        d = mx.Dims(T=n, T_max=n, H=f("H"), F=f("F"), E=f("E"), k=f("k"), P_total=f("P_total"), p0=f("p0"),
                    P_local=f("P_local"), R_max=f("R_max"), token_id_base=f("token_id_base") + t)
        mx.moe_forward_a16w16(d, b.x[t:t + n], b.logits[t:t + n], ex.w1, ex.w2, b.rep_count, b.rep_slots, out[t:t + n],
                              mx.a16w16_workspace(d))
    return out


def main() -> None:
    b = Buffers()
    H, F, G = b.d.H, b.d.F, b.d.P_local
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    r = lambda *n: (torch.randn(*n, generator=g, device="cuda") * 0.05).bfloat16()  # noqa: E731
    tokens, w, offsets = bucket(b)
    ex = Experts(r(G, 2 * F, H), r(G, H, F), tokens.numel())
    target = torch.randn(b.d.T, H, generator=g, device="cuda")
    for i in range(3):
        loss, norm = step(ex, b.x, tokens, w, offsets, target, 0.1, 1.0)
        print(f"step {i}: loss {float(loss):.6g}, gradient norm {float(norm):.4g}")
    y = serve(ex, b)
    print(f"served: {tuple(y.shape)}, 0.5 |y - target|^2 = {float(0.5 * (y.float() - target).square().sum()):.6g}")


if __name__ == "__main__":
    main()
