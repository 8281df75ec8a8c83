"""The linear operators' host side: sizes, refusals before any launch (no GPU
needed), and the oracle against plain loops."""

import ctypes
import os

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from oracle import linear as ol

needs_lib = pytest.mark.skipif(not os.path.exists(mx.LIB_PATH), reason="libmoe.so not built")
P = ctypes.c_void_p
A = [0x10000 * (i + 1) for i in range(8)]   # aligned addresses that are never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def _fp8(d, xq=A[0], xs=A[1], w=A[2], ws=A[3], off=None, y=A[4], scratch=A[5], nbytes=None):
    n = mx.moe_linear_workspace_bytes(d) if nbytes is None else nbytes
    return mx.lib().moe_fp8_linear(ctypes.byref(d) if d else None, xq, xs, w, ws, off, y, scratch, n, None)


def _grouped(fn, d, a=A[0], b=A[1], off=None, out=A[2], scratch=A[3], nbytes=None):
    n = mx.moe_linear_workspace_bytes(d) if nbytes is None else nbytes
    return getattr(mx.lib(), fn)(ctypes.byref(d), a, b, off, out, scratch, n, None)


@needs_lib
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(groups=0), INVALID),
    (dict(K=100), INVALID), (dict(K=24), INVALID), (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(N=32769), UNSUPPORTED),
    (dict(K=32784), UNSUPPORTED), (dict(groups=1025), UNSUPPORTED), (dict(in_type="bf16"), INVALID),
    (dict(in_type="f32"), INVALID), (dict(out_type="fp8"), INVALID)])
def test_fp8_linear_refuses_sizes_and_types(kw, code):
    d = mx.Linear(**{**dict(rows=4, N=33, K=128, in_type="fp8", out_type="bf16"), **kw})
    assert _fp8(d, off=A[6]) == code
    if "in_type" not in kw:
        assert mx.moe_linear_workspace_bytes(d) == 0


@needs_lib
def test_fp8_linear_refuses_pointers():
    d = mx.Linear(4, 33, 128, in_type="fp8")
    assert _fp8(None, nbytes=0) == INVALID
    for name in ("xq", "xs", "w", "ws", "y"):
        assert _fp8(d, **{name: None}) == INVALID, name
        assert _fp8(d, **{name: A[0] + 8}) == INVALID, name
    assert _fp8(d, off=A[0] + 4) == INVALID
    assert _fp8(d, scratch=A[0] + 8) == INVALID
    assert _fp8(mx.Linear(4, 33, 128, groups=2, in_type="fp8")) == INVALID   # groups without offsets
    # no rows: nothing to launch, row tensors may be missing
    assert _fp8(mx.Linear(0, 33, 128, in_type="fp8"), xq=None, xs=None, y=None) == 0
    assert _fp8(mx.Linear(0, 33, 128, in_type="fp8"), w=None) == INVALID


@needs_lib
@pytest.mark.parametrize("fn", ["moe_grouped_linear", "moe_grouped_linear_dx", "moe_grouped_linear_dw"])
def test_grouped_refusals(fn):
    d = mx.Linear(4, 64, 64, in_type="bf16")
    for name in ("a", "b", "out"):
        assert _grouped(fn, d, **{name: None}) == INVALID, name
        assert _grouped(fn, d, **{name: A[0] + 4}) == INVALID, name
    assert _grouped(fn, mx.Linear(4, 64, 64, groups=3)) == INVALID
    assert _grouped(fn, mx.Linear(4, 64, 68)) == INVALID
    assert _grouped(fn, mx.Linear(4, 64, 64, in_type="fp8")) == INVALID
    assert _grouped(fn, mx.Linear(4, 64, 64, in_type="bf16", out_type="f16")) == INVALID
    assert _grouped(fn, mx.Linear(4, 32776, 64)) == UNSUPPORTED
    if fn != "moe_grouped_linear":   # the gradients read rows of N values in 16-byte pieces
        assert _grouped(fn, mx.Linear(4, 33, 64)) == INVALID
    if fn != "moe_grouped_linear_dw":
        d0 = mx.Linear(0, 64, 64)
        assert _grouped(fn, d0, a=None, out=None) == 0
        assert _grouped(fn, d0, b=None) == INVALID
    else:
        assert _grouped(fn, mx.Linear(0, 64, 64), out=None) == INVALID


@needs_lib
@pytest.mark.parametrize("fn,parts", [("moe_fp8_quant", 1), ("moe_fp8_swiglu_quant", 2)])
def test_quant_refusals(fn, parts):
    f = getattr(mx.lib(), fn)

    def call(rows=4, K=128, t=0, x=A[0], ldx=None, q=A[1], qs=A[2]):
        return f(rows, K, t, x, K * parts if ldx is None else ldx, q, qs, None)

    for kw in (dict(rows=-1), dict(K=0), dict(K=8), dict(K=120), dict(t=3), dict(t=-1), dict(ldx=128 * parts - 16),
               dict(ldx=128 * parts + 8), dict(x=None), dict(q=None), dict(qs=None), dict(x=A[0] + 8),
               dict(q=A[1] + 4), dict(qs=A[2] + 4)):
        assert call(**kw) == INVALID, kw
    assert call(rows=(1 << 20) + 1) == UNSUPPORTED
    assert call(K=32784) == UNSUPPORTED
    assert call(rows=0, x=None, q=None, qs=None) == 0


@needs_lib
def test_workspace_query():
    small = mx.moe_linear_workspace_bytes(mx.Linear(1, 64, 64))
    assert small == mx.moe_linear_workspace_bytes(mx.Linear(1, 64, 64, out_type="f32"))
    for d in (mx.Linear(8192, 4096, 7168, in_type="fp8"), mx.Linear(64, 64, 32768), mx.Linear(1 << 20, 64, 64)):
        n = mx.moe_linear_workspace_bytes(d)
        assert n < 1 << 31
        if n:
            assert mx.lib().moe_status_string(-3)
            fn = _fp8 if d.in_type == 3 else (lambda d, **kw: _grouped("moe_grouped_linear", d, **kw))
            assert fn(d, nbytes=n - 1) == WORKSPACE
            assert fn(d, scratch=None) == WORKSPACE


def test_linear_struct_arguments():
    assert mx.Linear(1, 2, 16, in_type="fp8").out_type == mx.TYPES["bf16"]
    assert mx.Linear(1, 2, 16, in_type="f16").out_type == mx.TYPES["f16"]
    with pytest.raises(ValueError):
        mx.Linear(1, 2, 16, in_type="int8")
    with pytest.raises(ValueError):
        mx.Linear(1, 2, 16, out_type="float")


def test_binding_refuses_host_tensors():
    d = mx.Linear(2, 16, 16)
    x, w, y = torch.zeros(2, 16).bfloat16(), torch.zeros(1, 16, 16).bfloat16(), torch.zeros(2, 16).bfloat16()
    with pytest.raises(ValueError):
        mx.moe_grouped_linear(d, x, w, y, None)
    with pytest.raises(TypeError):
        mx.moe_grouped_linear(d, x.float(), w, y, None)
    with pytest.raises(ValueError):
        mx.moe_fp8_quant(x, torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1))
    with pytest.raises(TypeError):
        mx.moe_fp8_quant(x[0], torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1))


# ---- the oracle against plain loops ----------------------------------------

def test_oracle_quant_and_fp8_product():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 160)).astype(np.float32)
    s = ol.quant_scales(x)
    assert s.shape == (3, 2)
    for r in range(3):
        assert s[r, 0] == np.float32(max(abs(float(v)) for v in x[r, :128])) / np.float32(448)
        assert s[r, 1] == np.float32(max(abs(float(v)) for v in x[r, 128:])) / np.float32(448)
    assert np.all(ol.quant_scales(np.zeros((2, 16))) == np.float32(2.0 ** -126))
    xq = rng.integers(-8, 9, (3, 160)).astype(float)
    w = rng.integers(-8, 9, (2, 130, 160)).astype(float)
    xs, ws = rng.random((3, 2)), rng.random((2, 2, 2))
    y, tol = ol.fp8_linear(xq, xs, w, ws, [0, 1, 3])
    for r in range(3):
        g = 0 if r < 1 else 1
        for n in (0, 127, 128, 129):
            ref = sum(xq[r, k] * w[g, n, k] * xs[r, k // 128] * ws[g, n // 128, k // 128] for k in range(160))
            assert abs(y[r, n] - ref) <= 1e-12 * np.abs(y).max() and 0 < tol[r, n] < np.abs(y).max()


def test_oracle_grouped_and_gradients():
    rng = np.random.default_rng(6)
    x, w, dy = rng.standard_normal((5, 8)), rng.standard_normal((3, 16, 8)), rng.standard_normal((5, 16))
    off = [0, 2, 2, 5]
    y, _ = ol.grouped(x, w, off)
    g_of = [0, 0, 2, 2, 2]
    for r in range(5):
        assert np.allclose(y[r], [sum(x[r, k] * w[g_of[r], n, k] for k in range(8)) for n in range(16)], atol=1e-12)
    dx, _ = ol.grouped_dx(dy, w, off)
    dw, _ = ol.grouped_dw(dy, x, 3, off)
    assert np.all(dw[1] == 0)
    # gradients of <y, dy>: central differences (the product is bilinear: exact up to rounding)
    f = lambda x_, w_: float((ol.grouped(x_, w_, off)[0] * dy).sum())  # noqa: E731
    for _ in range(6):
        r, k, g, n = rng.integers(5), rng.integers(8), rng.integers(3), rng.integers(16)
        e = np.zeros_like(x)
        e[r, k] = 0.5
        assert abs(f(x + e, w) - f(x - e, w) - dx[r, k]) < 1e-10
        e = np.zeros_like(w)
        e[g, n, k] = 0.5
        assert abs(f(x, w + e) - f(x, w - e) - dw[g, n, k]) < 1e-10


@needs_lib
def test_binding_refuses_what_is_no_tensor_or_descriptor():
    d = mx.Linear(2, 16, 16)
    t = torch.zeros(2, 16).bfloat16()
    for f in (mx.moe_grouped_linear, mx.moe_grouped_linear_dx, mx.moe_grouped_linear_dw):
        with pytest.raises(TypeError):
            f(d, t, t, None, None)
        with pytest.raises((TypeError, ValueError)):
            f(d, None, t, t, None)
    with pytest.raises(TypeError):
        mx.moe_fp8_linear(mx.Linear(2, 16, 16, in_type="fp8"), t, t, t, t, 5, None)
    for f in (mx.moe_fp8_quant, mx.moe_fp8_swiglu_quant):
        with pytest.raises(TypeError):
            f(None, t, t)
    bad = mx.Linear(2, 16, 16)
    bad.in_type = 9
    with pytest.raises((ValueError, IndexError)):
        mx.moe_grouped_linear(bad, t, t, t, None)
