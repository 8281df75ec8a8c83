"""GPU tests of the global gradient norm and of clipping, against float64.

The norm's sum is f64, so that the norm is off by its own rounding alone (and the
square root's): 2^-24 of it, taken twice.  The factor is rounded to f32 once, the
product once, the output once.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from oracle import experts as oe

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _np(t):
    return t.detach().cpu().double().numpy()


def _say(*a):
    print(*a, flush=True)


def _tensors(sizes, seed, std=0.1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(T[t]) for n, t in sizes]


def _check(grads, outs, norm, max_norm, before=None):
    ref, c = oe.clip([_np(g) for g in (before or grads)], max_norm)
    got = float(norm)
    assert abs(got - ref) <= 2 * oe.U * ref, (got, ref)
    for g, o in zip(before or grads, outs):
        want, fi = _np(g) * c, torch.finfo(o.dtype)
        tol = 3 * oe.U * np.abs(want) + fi.eps / 2 * np.abs(want) * (1 + 3 * oe.U) + fi.smallest_normal * fi.eps / 2
        assert np.all(np.abs(_np(o) - want) <= tol)


SIZES = {
    "one": [(1, "f32")],
    "three": [(3, "bf16"), (0, "f16"), (7, "f32")],
    "chunks": [(8191, "bf16"), (8192, "f16"), (8193, "f32"), (16384, "bf16"), (24577, "f32")],
    "empty": [(0, "f32"), (0, "bf16")],
    "large": [(3_000_001, "f32"), (5, "bf16"), (20_000_003, "bf16"), (9_999_999, "f16")],
    "many": [(1 + 37 * i % 500, ("bf16", "f16", "f32")[i % 3]) for i in range(500)],
    "table": [(64, "f32")] * 168,
    "table_and_one": [(64, "f32")] * 169,
}


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("name", list(SIZES))
def test_norm_and_clip(name, max_norm):
    _say(f"[case] clip {name} max_norm={max_norm}")
    grads = _tensors(SIZES[name], 1)
    outs = [torch.full_like(g, 7.0) for g in grads]
    h = mx.GradList(grads, outs)
    ws, norm = mx.grad_workspace(h), torch.full((1,), -1.0, device="cuda")
    ws.fill_(0xFF)
    mx.moe_grad_clip(h, max_norm, norm, ws)
    torch.cuda.synchronize()
    _check(grads, outs, norm, max_norm)
    again = torch.full((1,), -1.0, device="cuda")
    ws.fill_(0xFF)
    mx.moe_grad_norm(mx.GradList(grads), again, ws)
    assert torch.equal(again, norm)
    # in place, without the norm
    before = [g.clone() for g in grads]
    mx.moe_grad_clip(mx.GradList(grads), max_norm, None, ws)
    torch.cuda.synchronize()
    for g, o, b in zip(grads, outs, before):
        assert torch.equal(g, o) and (max_norm < 1e9 or torch.equal(g, b))


def test_no_tensors():
    h = mx.GradList([])
    norm, ws = torch.full((1,), 5.0, device="cuda"), mx.grad_workspace(h)
    mx.moe_grad_clip(h, 1.0, norm, ws)
    assert float(norm) == 0.0
    norm.fill_(5.0)
    mx.moe_grad_norm(h, norm, ws)
    assert float(norm) == 0.0


def test_views_at_odd_addresses_and_neighbours():
    """Inputs and outputs that start at any element of a buffer; what lies between
    them keeps its values."""
    for t in T.values():
        flat, out = torch.randn(70000, device="cuda").to(t), torch.full((70000,), 7.0, device="cuda").to(t)
        spans = [(1, 2), (3, 20), (21, 8214), (8215, 16407), (16409, 50001)]
        grads, outs = [flat[a:b] for a, b in spans], [out[a + 1:b + 1] for a, b in spans]
        h = mx.GradList(grads, outs)
        norm = torch.empty(1, device="cuda")
        mx.moe_grad_clip(h, 1.0, norm, mx.grad_workspace(h))
        torch.cuda.synchronize()
        _check(grads, outs, norm, 1.0)
        keep = torch.ones(70000, dtype=torch.bool)
        for a, b in spans:
            keep[a + 1:b + 1] = False
        assert torch.all(out[keep.cuda()] == 7.0)


def test_range_of_the_norm():
    """Squares beyond f32's range on both sides, infinities and NaN."""
    for v in (1e25, 1e-30, 3e38):
        g = torch.full((1000,), v, device="cuda")
        o = torch.empty_like(g)
        h = mx.GradList([g], [o])
        norm, ws = torch.empty(1, device="cuda"), mx.grad_workspace(h)
        mx.moe_grad_clip(h, 1.0, norm, ws)
        ref, c = oe.clip([_np(g)], 1.0)
        assert np.isinf(float(norm)) if ref > 3.4e38 else abs(float(norm) - ref) <= 2 * oe.U * ref
        assert np.all(np.abs(_np(o) - _np(g) * c) <= 3 * oe.U * np.abs(_np(g) * c) + 2.0 ** -149)
    g = torch.ones(20000, device="cuda")
    g[12345] = float("inf")
    o = torch.empty_like(g)
    h = mx.GradList([g], [o])
    norm, ws = torch.empty(1, device="cuda"), mx.grad_workspace(h)
    mx.moe_grad_clip(h, 1.0, norm, ws)
    assert float(norm) == float("inf") and torch.isnan(o[12345]) and float(o.nansum()) == 0.0
    g[3] = float("nan")
    mx.moe_grad_clip(h, 1.0, norm, ws)
    assert torch.isnan(norm).all() and torch.isnan(o).all()


def test_a_tensor_past_two_to_the_31_elements():
    n = 2 ** 31 + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-7000:] = 2.0
    g[2 ** 31 - 3:2 ** 31 + 3] = 4.0
    h = mx.GradList([g])
    norm = torch.empty(1, device="cuda")
    mx.moe_grad_clip(h, 1.0, norm, mx.grad_workspace(h))
    ref = (4.0 * 7000 + 16.0 * 6) ** 0.5
    assert abs(float(norm) - ref) <= 2 * oe.U * ref
    for i, v in ((n - 1, 2.0), (n - 7000, 2.0), (2 ** 31 - 3, 4.0), (2 ** 31 + 2, 4.0)):
        assert abs(float(g[i]) - v / ref) <= 2.0 ** -8 * v / ref
    assert float(g[2 ** 31 + 3]) == 0.0 and float(g[n - 7001]) == 0.0


def test_overlaps_are_refused():
    f = torch.zeros(100, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        mx.GradList([f, f])
    with pytest.raises(ValueError, match="overlap"):
        mx.GradList([f[:60], f[50:]])
    with pytest.raises(ValueError, match="overlap"):
        mx.GradList([f[:50]], [f[20:70]])
    with pytest.raises(ValueError, match="overlap"):
        mx.GradList([f[:10], f[20:30]], [f[40:50], f[45:55]])
    with pytest.raises(ValueError):
        mx.GradList([f[::2]])
    with pytest.raises(TypeError):
        mx.GradList([f], [f.bfloat16()])
    o = torch.zeros(200, device="cuda")
    mx.GradList([f, f], [o[:100], o[100:]])   # read twice, written apart


def test_same_bits_streams_and_graph():
    grads = _tensors(SIZES["large"], 2)
    outs = [torch.empty_like(g) for g in grads]
    h = mx.GradList(grads, outs)
    ws, norm = mx.grad_workspace(h), torch.empty(1, device="cuda")
    mx.moe_grad_clip(h, 1.0, norm, ws)
    first = [norm.clone()] + [o.clone() for o in outs]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for o in outs:
        o.zero_()
    st.wait_stream(torch.cuda.current_stream())
    mx.moe_grad_clip(h, 1.0, norm, ws, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, [norm] + outs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.moe_grad_clip(h, 1.0, norm, ws)
    for i in range(3):
        for v in grads:
            v.mul_(0.75 + i)
        g.replay()
        torch.cuda.synchronize()
        got = [norm.clone()] + [o.clone() for o in outs]
        mx.moe_grad_clip(h, 1.0, norm, ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, [norm] + outs))
