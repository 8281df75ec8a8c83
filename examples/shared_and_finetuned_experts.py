#!/usr/bin/env python3
"""The linear operators next to the fused layer, on its tiny workload.

* ``layer_with_shared_expert``: the fused MoE layer's output plus a shared
  expert held in fp8 with a scale per block of 128 (quantise, gate and up
  product, SwiGLU and quantise, down product).
* ``finetune_step``: one step on bf16 experts: the layer's own routing and
  bucketing give the rows and offsets, the grouped products run the experts
  forward and backward.

Run it on a GPU:  python examples/shared_and_finetuned_experts.py
"""

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_layer_sigmoid_amd as mx  # noqa: E402
import synth  # noqa: E402

BLOCK = 128


def to_fp8_blocks(w: torch.Tensor):
    """fp8 codes of w [N, K] and their scales [ceil(N/128), ceil(K/128)]."""
    N, K = w.shape
    nn, nk = -(-N // BLOCK), -(-K // BLOCK)
    v = torch.nn.functional.pad(w.float(), (0, nk * BLOCK - K, 0, nn * BLOCK - N)).view(nn, BLOCK, nk, BLOCK)
    s = (v.abs().amax((1, 3)) / 448.0).clamp_min(2.0 ** -126)
    q = (v / s[:, None, :, None]).view(nn * BLOCK, nk * BLOCK)[:N, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), s.contiguous()


class SharedExpert:
    """down(silu(gate(x)) * up(x)) in fp8 for up to ``rows`` rows of bf16; the
    result is a view of a buffer that the next call overwrites."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor, rows: int):
        H, F = down.shape
        dev = gate_up.device
        self.rows, self.H, self.F = rows, H, F
        self.w1, self.w1s = to_fp8_blocks(gate_up)   # [2F, H]
        self.w2, self.w2s = to_fp8_blocks(down)      # [H, F]
        n = lambda w: -(-w // BLOCK)  # noqa: E731
        self.xq = torch.empty(rows, H, dtype=torch.float8_e4m3fn, device=dev)
        self.xs = torch.empty(rows, n(H), device=dev)
        self.h = torch.empty(rows, 2 * F, dtype=torch.bfloat16, device=dev)
        self.aq = torch.empty(rows, F, dtype=torch.float8_e4m3fn, device=dev)
        self.asc = torch.empty(rows, n(F), device=dev)
        self.y = torch.empty(rows, H, dtype=torch.bfloat16, device=dev)
        # enough for any number of rows up to `rows`: fewer may need more
        need = max(mx.moe_linear_workspace_bytes(d) for r in range(1, rows + 1) for d in self._products(r))
        self.scratch = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)

    def _products(self, r: int):
        return mx.Linear(r, 2 * self.F, self.H, in_type="fp8"), mx.Linear(r, self.H, self.F, in_type="fp8")

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        r = x.shape[0]
        if r > self.rows:
            raise ValueError(f"{r} rows, made for at most {self.rows}")
        d1, d2 = self._products(r)
        xq, xs, h, aq, asc, y = (t[:r] for t in (self.xq, self.xs, self.h, self.aq, self.asc, self.y))
        mx.moe_fp8_quant(x, xq, xs)
        mx.moe_fp8_linear(d1, xq, xs, self.w1, self.w1s, h, self.scratch)
        mx.moe_fp8_swiglu_quant(h, aq, asc)
        mx.moe_fp8_linear(d2, aq, asc, self.w2, self.w2s, y, self.scratch)
        return y


class Buffers:
    """The tiny workload on the device."""

    def __init__(self, name: str = "tiny"):
        wl = synth.make(name)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.d = mx.Dims.of(wl.dims)
        self.x = t(wl.x.view(np.int16)).view(torch.bfloat16)
        self.logits, self.rep_count, self.rep_slots = t(wl.logits), t(wl.rep_count), t(wl.rep_slots)
        self.packed = mx.pack_weights(self.d, t(wl.w1), t(wl.w1s), t(wl.w2), t(wl.w2s))
        self.ws = mx.workspace(self.d)


def layer_with_shared_expert(b: Buffers, shared: SharedExpert) -> torch.Tensor:
    out = torch.empty_like(b.x)
    mx.moe_forward(b.d, b.x, b.logits, *b.packed, b.rep_count, b.rep_slots, out, b.ws)
    return out + shared(b.x)


def bucket(b: Buffers):
    """The layer's routing and bucketing: (tokens of the rows, their weights,
    offsets); rows past offsets[-1] belong to other GPUs' experts."""
    d, n = b.d, b.d.T * b.d.k
    z = lambda k, t: torch.zeros(k, dtype=t, device="cuda")  # noqa: E731
    ids, w, phys, hist = z(n, torch.int32), z(n, torch.float32), z(n, torch.int32), z(d.P_total, torch.int32)
    mx.moe_route(d, b.logits, ids, w)
    mx.moe_eplb_remap_record(d, ids, b.rep_count, b.rep_slots, phys, hist, b.ws)
    rows = d.T_max * d.k
    offsets, pair = z(d.P_local + 1, torch.int32), z(rows, torch.int32)
    mx.moe_quant_permute(d, b.x, phys, z(rows * d.H, torch.uint8), z(rows * (d.H // 128), torch.uint8),
                         z(d.P_local, torch.int32), offsets, z(n, torch.int32), pair, b.ws)
    pair = pair.long()
    return pair // d.k, w[pair], offsets


def finetune_step(x, w, tokens, offsets, w1, w2, dout):
    """y[t] = sum over t's rows of w * (silu(gate) up) w2^T with [gate | up] =
    x w1^T, and the gradients of <y, dout>: (y, dx, dw1, dw2).  w1 [G, 2F, H],
    w2 [G, H, F] in bf16; the weights' gradients are f32."""
    G, F2, H = w1.shape
    F, rows = F2 // 2, tokens.numel()
    d1, d2 = mx.Linear(rows, F2, H, groups=G), mx.Linear(rows, H, F, groups=G)
    g1 = mx.Linear(rows, F2, H, groups=G, out_type="f32")
    g2 = mx.Linear(rows, H, F, groups=G, out_type="f32")
    s = torch.empty(max(mx.moe_linear_workspace_bytes(d1), mx.moe_linear_workspace_bytes(d2), 256),
                    dtype=torch.uint8, device=x.device)
    e = lambda *n, t=torch.bfloat16: torch.zeros(*n, dtype=t, device=x.device)  # noqa: E731  rows in no group: 0

    xr = x[tokens]
    h, o = e(rows, F2), e(rows, H)
    mx.moe_grouped_linear(d1, xr, w1, h, s, offsets=offsets)
    gate, up = h.float().split(F, 1)
    sig = torch.sigmoid(gate)
    act = (gate * sig * up).bfloat16()
    mx.moe_grouped_linear(d2, act, w2, o, s, offsets=offsets)
    y = torch.zeros(x.shape, device=x.device).index_add_(0, tokens, o.float() * w[:, None])

    do = (dout[tokens].float() * w[:, None]).bfloat16()
    dact, dh, dxr = e(rows, F), e(rows, F2), e(rows, H)
    dw1, dw2 = torch.empty(G, F2, H, device=x.device), torch.empty(G, H, F, device=x.device)
    mx.moe_grouped_linear_dw(g2, do, act, dw2, s, offsets=offsets)
    mx.moe_grouped_linear_dx(d2, do, w2, dact, s, offsets=offsets)
    da = dact.float()
    dh[:, :F] = (da * up * sig * (1 + gate * (1 - sig))).bfloat16()
    dh[:, F:] = (da * gate * sig).bfloat16()
    mx.moe_grouped_linear_dw(g1, dh, xr, dw1, s, offsets=offsets)
    mx.moe_grouped_linear_dx(d1, dh, w1, dxr, s, offsets=offsets)
    dx = torch.zeros(x.shape, device=x.device).index_add_(0, tokens, dxr.float())
    return y, dx, dw1, dw2


def main() -> None:
    b = Buffers()
    H, F, G = b.d.H, b.d.F, b.d.P_local
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    r = lambda *n: (torch.randn(*n, generator=g, device="cuda") * 0.02).bfloat16()  # noqa: E731
    out = layer_with_shared_expert(b, SharedExpert(r(2 * F, H), r(H, F), b.d.T))
    print(f"layer with shared expert: {tuple(out.shape)}, norm {float(out.float().norm()):.4g}")

    tokens, w, offsets = bucket(b)
    w1, w2, target = r(G, 2 * F, H), r(G, H, F), torch.randn(b.d.T, H, generator=g, device="cuda")
    for step in range(3):   # plain gradient steps on 0.5 |y - target|^2
        y = finetune_step(b.x, w, tokens, offsets, w1, w2, torch.zeros_like(b.x))[0]
        err = y - target
        _, _, dw1, dw2 = finetune_step(b.x, w, tokens, offsets, w1, w2, err.bfloat16())
        print(f"step {step}: loss {float(0.5 * err.square().sum()):.6g}")
        w1 = (w1.float() - 0.01 * dw1).bfloat16()
        w2 = (w2.float() - 0.01 * dw2).bfloat16()


if __name__ == "__main__":
    main()
