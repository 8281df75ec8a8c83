"""The example that trains unquantised experts and serves them: each stage in
float64 from what it was given, within the oracle's bounds."""

import numpy as np
import pytest
import torch

from oracle import experts as oe
from oracle import linear as ol

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8   # half a step of bf16


def _np(t):
    return t.detach().double().cpu().numpy()


def _in(got, ref, tol, half=HALF):
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - ref) <= tol + half * (np.abs(ref) + tol) + 1e-38)


def test_a_step_and_the_layer_on_its_result():
    from examples import finetune_and_serve_experts as ex
    b = ex.Buffers()
    H, F, G = b.d.H, b.d.F, b.d.P_local
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    r = lambda *n: (torch.randn(*n, generator=g, device="cuda") * 0.05).bfloat16()  # noqa: E731
    tokens, w, offsets = ex.bucket(b)
    e = ex.Experts(r(G, 2 * F, H), r(G, H, F), tokens.numel())
    target = torch.randn(b.d.T, H, generator=g, device="cuda")
    w1, w2, off = _np(e.w1), _np(e.w2), offsets.cpu().numpy()
    n = int(off[-1])
    rows = b.x[tokens]

    o = e.forward(rows, offsets)
    x = _np(rows)
    y, ty, z, tz = oe.linear_act(x, w1, name="silu", gated=True, offsets=off)
    _in(_np(e.pre)[:n], z[:n], tz[:n])
    _in(_np(e.act)[:n], y[:n], ty[:n])
    _in(_np(o)[:n], *(v[:n] for v in ol.grouped(_np(e.act), w2, off)))
    do = (torch.randn(tokens.numel(), H, generator=g, device="cuda")).bfloat16()
    dx = e.backward(rows, do, offsets)
    _in(_np(e.dw2), *ol.grouped_dw(_np(do), _np(e.act), G, off), half=oe.U)
    _in(_np(e.dact)[:n], *(v[:n] for v in ol.grouped_dx(_np(do), w2, off)))
    dz, tdz, _, _ = oe.act_backward(_np(e.dact), _np(e.pre), G, "silu", True, off)
    _in(_np(e.dz)[:n], dz[:n], tdz[:n])
    _in(_np(e.dw1), *ol.grouped_dw(_np(e.dz), x, G, off), half=oe.U)
    _in(_np(dx)[:n], *(v[:n] for v in ol.grouped_dx(_np(e.dz), w1, off)))
    before = [_np(e.dw1), _np(e.dw2)]
    norm = float(e.clip(0.5))
    ref, c = oe.clip(before, 0.5)
    assert c < 1 and abs(norm - ref) <= 2 * oe.U * ref
    for got, was in zip((e.dw1, e.dw2), before):
        assert np.all(np.abs(_np(got) - was * c) <= 3 * oe.U * np.abs(was * c) + 2.0 ** -149)

    loss, _ = ex.step(e, b.x, tokens, w, offsets, target, 0.1, 1.0)
    assert torch.isfinite(loss)
    out = ex.serve(e, b)
    ids = torch.zeros(b.d.T * b.d.k, dtype=torch.int32, device="cuda")
    wt = torch.zeros(b.d.T * b.d.k, device="cuda")
    ex.mx.moe_route(b.d, b.logits, ids, wt)
    ids, wt = ids.view(b.d.T, b.d.k).cpu().numpy(), _np(wt.view(b.d.T, b.d.k))   # the tiny workload: slot = expert
    ref, tol = oe.layer(_np(b.x), _np(e.w1), _np(e.w2), ids, wt, b.d.p0, 2.0 ** -7)
    _in(_np(out), ref, tol)
    # and the same experts by the bucketed calls: what their intermediate roundings allow
    many = ex.mix(e.forward(rows, offsets)[:n], tokens[:n], w[:n], b.d.T)
    assert float((many - out.float()).norm() / many.norm()) <= 4 * HALF


def test_it_runs(capsys):
    from examples import finetune_and_serve_experts as ex
    ex.main()
    assert "served" in capsys.readouterr().out
