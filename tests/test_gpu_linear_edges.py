"""GPU tests of the linear operators at the ends of their ranges: values near
f32's smallest, and the sizes and weights at which other code runs.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from oracle import linear as ol

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _say(*a):
    print(*a, flush=True)


def _np(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------------------
# SwiGLU of gates whose sigmoid is below f32's normal range
# ---------------------------------------------------------------------------

GATES = (-64.0, -79.5, -80.0, -80.5, -86.5, -87.5, -88.0, -88.5, -88.75, -89.0, -95.0, -104.0, -120.0, -150.0, -177.0,
         -200.0, -348.0, -1e4, -60000.0)


@pytest.mark.parametrize("dt,ups", [("f32", (1.0, -3e38, 1e30, 5e-5)), ("bf16", (1.0, -3e38, 1e30, 5e-5)),
                                    ("f16", (1.0, -60000.0, 256.0, 6e-5))])
def test_swiglu_quant_of_very_negative_gates(dt, ups):
    """silu(g) u is a value that a scale of at least 2^-126 carries long after
    silu(g) has left f32's normal range: each (gate, up) fills a block alone, and
    one block mixes them with ordinary gates."""
    g = torch.tensor(GATES, dtype=torch.float64)
    rows = [(torch.full((128,), float(v)), torch.full((128,), u)) for v in g for u in ups]
    mixed = g.repeat(7)[:128].clone()
    mixed[::3] = -86.0
    rows.append((mixed, torch.full((128,), ups[1])))
    gate, up = (torch.stack([r[i].double() for r in rows]) for i in (0, 1))
    x = torch.cat([gate, up], 1).to(T[dt]).cuda()
    q = torch.empty(len(rows), 128, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(len(rows), 1, device="cuda")
    mx.moe_fp8_swiglu_quant(x, q, s)
    with np.errstate(over="ignore"):
        h = ol.swiglu(_np(x))
    # the exponential's error four times over and five roundings, then the scale's own and 1 / s
    rel = 21 * 2.0 ** -24
    ref = np.maximum(np.abs(h).max(1, keepdims=True) / 448, 2.0 ** -126)
    got = _np(s)
    assert np.all(np.abs(got - ref) <= (rel + 2.0 ** -24) * ref), np.abs(got / ref - 1).max()
    err = np.abs(_np(q.float()) * got - h)
    bound = np.abs(h) * (2.0 ** -4 + 2 * rel) + got * 2.0 ** -10   # half a step of e4m3
    worst = int((err / bound).max(1).argmax())
    _say(f"   {dt}: worst {np.max(err / bound):.3g} of the bound at {GATES[min(worst // len(ups), len(GATES) - 1)]}")
    assert np.all(err <= bound)
    assert np.count_nonzero(h) and np.count_nonzero(_np(q.float())[np.abs(h) > 2.0 ** -126])
