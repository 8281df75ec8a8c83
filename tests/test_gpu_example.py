"""The example that runs the linear operators next to the fused layer, against
the same formulas in float64."""

import numpy as np
import pytest
import torch

from oracle import linear as ol

pytestmark = pytest.mark.gpu


def _example():
    from examples import shared_and_finetuned_experts as ex
    return ex


def _norm_err(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def _weights(G, F, H, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    r = lambda *n: (torch.randn(*n, generator=g) * 0.05).bfloat16().cuda()  # noqa: E731
    return r(G, 2 * F, H), r(G, H, F)


def test_shared_expert_beside_the_fused_layer():
    """Stage by stage in float64 from the codes and scales that each stage was
    given, within the oracle's bounds, so that a stage wired to the wrong
    weights, scales or rows shows."""
    ex = _example()
    b = ex.Buffers()
    F, H = b.d.F, b.d.H
    w1, w2 = _weights(1, F, H, 1)
    shared = ex.SharedExpert(w1[0], w2[0], b.d.T)
    out = ex.layer_with_shared_expert(b, shared)
    alone = torch.empty_like(b.x)
    ex.mx.moe_forward(b.d, b.x, b.logits, *b.packed, b.rep_count, b.rep_slots, alone, b.ws)
    assert torch.equal(out, alone + shared.y)

    n = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    spread = lambda s, K: ol.spread(n(s), K, 1)  # noqa: E731
    # the codes of x: within half a step of e4m3 (2^-4 of the value, 2^-10 scales below its normals)
    x = n(b.x)
    sv = spread(shared.xs, H)
    assert np.all(np.abs(n(shared.xq.float()) * sv - x) <= np.abs(x) * 2.0 ** -4 + sv * 2.0 ** -10)
    for w, q, s in ((w1[0], shared.w1, shared.w1s), (w2[0], shared.w2, shared.w2s)):
        sv = ol.spread(ol.spread(n(s), w.shape[0], 0), w.shape[1], 1)
        assert np.all(np.abs(n(q.float()) * sv - n(w)) <= np.abs(n(w)) * (2.0 ** -4 + 2.0 ** -23) + sv * 2.0 ** -10)
    ref, tol = ol.fp8_linear(n(shared.xq.float()), n(shared.xs), n(shared.w1.float())[None], n(shared.w1s)[None])
    assert np.all(np.abs(n(shared.h) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))
    a = ol.swiglu(n(shared.h))
    sv = spread(shared.asc, F)
    assert np.all(np.abs(n(shared.aq.float()) * sv - a) <= np.abs(a) * (2.0 ** -4 + 2.0 ** -20) + sv * 2.0 ** -10)
    ref, tol = ol.fp8_linear(n(shared.aq.float()), n(shared.asc), n(shared.w2.float())[None], n(shared.w2s)[None])
    assert np.all(np.abs(n(shared.y) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))


def test_finetune_step_against_float64():
    """Every tensor passes at most four bf16 roundings (2^-8 each, of either
    sign): 2^-6 normwise."""
    ex = _example()
    b = ex.Buffers()
    G, F, H = b.d.P_local, b.d.F, b.d.H
    tokens, w, offsets = ex.bucket(b)
    w1, w2 = _weights(G, F, H, 2)
    g = torch.Generator()
    g.manual_seed(3)
    dout = torch.randn(b.d.T, H, generator=g).bfloat16().cuda()
    got = ex.finetune_step(b.x, w, tokens, offsets, w1, w2, dout)

    x, a1, a2 = (t.double().cpu().requires_grad_() for t in (b.x, w1, w2))
    o = offsets.tolist()
    assert o[0] == 0 and o[-1] == tokens.numel()
    tok, wc = tokens.cpu(), w.double().cpu()
    y = torch.zeros(b.d.T, H, dtype=torch.float64)
    for e in range(G):
        t = tok[o[e]:o[e + 1]]
        gate, up = (x[t] @ a1[e].t()).split(F, 1)
        y = y.index_add(0, t, (torch.nn.functional.silu(gate) * up @ a2[e].t()) * wc[o[e]:o[e + 1], None])
    (y * dout.double().cpu()).sum().backward()
    for name, v, ref in zip(("y", "dx", "dw1", "dw2"), got, (y.detach(), x.grad, a1.grad, a2.grad)):
        err = _norm_err(v.cpu(), ref)
        print(f"   {name}: {err:.2e}", flush=True)
        assert err < 2.0 ** -6, name
