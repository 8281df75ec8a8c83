"""GPU tests of how clipping rounds: the factor and the product in f64, then to f32,
and from there to a 16-bit type."""

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from oracle import experts as oe

pytestmark = pytest.mark.gpu

F64 = 2.0 ** -53


def _clip(grads, max_norm):
    outs = [torch.empty_like(g) for g in grads]
    h = mx.GradList(grads, outs)
    norm = torch.empty(1, device="cuda")
    mx.moe_grad_clip(h, max_norm, norm, mx.grad_workspace(h))
    torch.cuda.synchronize()
    return outs, float(norm)


def _check(grads, outs, max_norm):
    # max_norm is a C float: the call sees it rounded to f32
    ref, c = oe.clip([g.cpu().double().numpy() for g in grads], np.float64(np.float32(max_norm)))
    assert c < 1.0
    for g, o in zip(grads, outs):
        want, fi = g.cpu().double().numpy() * c, torch.finfo(o.dtype)
        # the oracle's and the kernel's own f64: sums of squares by pairs or in order (their order
        # counts by the root of the number of terms, for which 2^10 is plenty here), a root, a
        # division, a product
        tol = 2.0 ** 10 * F64 * np.abs(want)
        tol = tol + 2.0 ** -24 * (np.abs(want) + tol) + 2.0 ** -150          # to f32: half a step
        if o.dtype != torch.float32:
            tol = tol + fi.eps / 2 * (np.abs(want) + tol) + fi.smallest_normal * fi.eps / 2
        err = np.abs(o.cpu().double().numpy() - want)
        bad = err > tol
        assert not bad.any(), f"{o.dtype}: worst {np.max(err / tol):.4g} of the bound"


@pytest.mark.parametrize("max_norm", [0.1, 1.0, 0.7])
def test_f32_is_off_by_half_a_step(max_norm):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    grads = [torch.randn(n, generator=g, device="cuda").to(t) for n, t in
             ((40000, torch.float32), (3, torch.float32), (20000, torch.bfloat16), (16385, torch.float16), (777, torch.float32))]
    outs, _ = _clip(grads, max_norm)
    _check(grads, outs, max_norm)


@pytest.mark.parametrize("v,max_norm", [(1e20, 1e-38), (3e38, 1e-22), (1e38, 1e-30), (2e38, 3e-45)])
def test_factors_far_below_f32s_range(v, max_norm):
    """norm 1e20 to 1e40 and max_norm down to f32's smallest number: outputs that f32 holds."""
    g = torch.full((1000,), v, device="cuda")
    g[::3] *= 0.3
    g[1::7] = 1.0
    outs, _ = _clip([g], max_norm)
    _check([g], outs, max_norm)
