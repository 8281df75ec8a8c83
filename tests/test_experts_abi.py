"""The operators for unquantised experts on the host: refusals before any launch
(no GPU needed), and the oracle against plain loops and differences."""

import ctypes
import math
import os

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from oracle import experts as oe

needs_lib = pytest.mark.skipif(not os.path.exists(mx.LIB_PATH), reason="libmoe.so not built")
A = [0x10000 * (i + 1) for i in range(16)]   # aligned addresses that are never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def _fwd(d, act=2, gated=0, x=A[0], w=A[1], bias=A[2], res=A[3], off=None, y=A[4], pre=A[5], scratch=A[6], nbytes=None):
    n = mx.moe_linear_act_workspace_bytes(d) if nbytes is None else nbytes
    return mx.lib().moe_grouped_linear_act(ctypes.byref(d), act, gated, x, w, bias, res, off, y, pre, scratch, n, None)


def _bwd(d, act=2, gated=0, dy=A[0], pre=A[1], off=None, dz=A[2], db=A[3], scratch=A[4], nbytes=None):
    n = mx.moe_linear_act_workspace_bytes(d) if nbytes is None else nbytes
    return mx.lib().moe_grouped_linear_act_backward(ctypes.byref(d), act, gated, dy, pre, off, dz, db, scratch, n, None)


@needs_lib
@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_refusals_of_sizes_types_and_activations(call):
    ok = dict(rows=4, N=64, K=64)
    for kw, code in ((dict(rows=-1), INVALID), (dict(N=0), INVALID), (dict(K=68), INVALID), (dict(groups=0), INVALID),
                     (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(N=32776), UNSUPPORTED),
                     (dict(groups=1025), UNSUPPORTED), (dict(in_type="fp8"), INVALID), (dict(in_type="f32"), INVALID),
                     (dict(in_type="bf16", out_type="f16"), INVALID), (dict(groups=2), INVALID)):
        d = mx.Linear(**{**ok, **kw})
        assert call(d) == code, kw
        if "groups" not in kw or kw["groups"] != 2:
            assert mx.moe_linear_act_workspace_bytes(d) == 0 or kw == dict(groups=2)
    for kw in (dict(act=-1), dict(act=5), dict(gated=2), dict(gated=-1)):
        assert call(mx.Linear(**ok), **kw) == INVALID, kw
    assert call(mx.Linear(4, 63, 64), gated=1) == INVALID
    if call is _bwd:
        assert call(mx.Linear(4, 60, 64)) == INVALID


@needs_lib
def test_refusals_of_pointers():
    d = mx.Linear(4, 64, 64)
    for name in ("x", "w", "y"):
        assert _fwd(d, **{name: None}) == INVALID, name
    for name in ("x", "w", "y", "bias", "res", "pre", "off", "scratch"):
        assert _fwd(d, **{name: A[0] + 8}) == INVALID, name
    for name in ("dy", "pre", "dz"):
        assert _bwd(d, **{name: None}) == INVALID, name
    for name in ("dy", "pre", "dz", "db", "off", "scratch"):
        assert _bwd(d, **{name: A[0] + 8}) == INVALID, name
    e = mx.Linear(0, 64, 64)
    assert _fwd(e, x=None, y=None, bias=None, res=None, pre=None) == 0
    assert _fwd(e, w=None) == INVALID
    assert _bwd(e, dy=None, pre=None, dz=None, db=None) == 0


@needs_lib
def test_workspaces_are_asked_for():
    d = mx.Linear(100, 64, 4096)
    n = mx.moe_linear_act_workspace_bytes(d)
    assert n >= mx.moe_linear_workspace_bytes(d) > 0
    assert _fwd(d, nbytes=mx.moe_linear_workspace_bytes(d) - 1) == WORKSPACE and _fwd(d, scratch=None) == WORKSPACE
    # up to 256 rows the gradient is one launch, which writes db itself
    more = mx.Linear(257, 64, 4096)
    assert _bwd(more, nbytes=0) == WORKSPACE and _bwd(more, scratch=None) == WORKSPACE
    big = mx.Linear(1 << 20, 32768, 64, groups=1024)
    assert mx.moe_linear_act_workspace_bytes(big) >= 1024 * 32768 * 4   # a partial sum for every group at least


def _tensors(*rows):
    a = (mx._Tensor * max(len(rows), 1))()
    for i, r in enumerate(rows):
        a[i] = mx._Tensor(*r, 0)
    return a


@needs_lib
def test_gradient_list_refusals():
    f, L = mx.lib().moe_grad_clip, mx.lib()
    ws = mx.moe_grad_workspace_bytes(4)
    assert ws > 0 and mx.moe_grad_workspace_bytes(-1) == 0 and mx.moe_grad_workspace_bytes(1 << 20) == 0

    def call(rows, count=None, max_norm=1.0, norm=A[8], scratch=A[9], nbytes=ws):
        a = _tensors(*rows)
        return f(ctypes.addressof(a), len(rows) if count is None else count, max_norm, norm, scratch, nbytes, None)

    ok = (A[0], A[1], 8, 0)
    for rows in ([(None, A[1], 8, 0)], [(A[0], None, 8, 0)], [(A[0], A[1], -1, 0)], [(A[0], A[1], 8, 3)], [(A[0], A[1], 8, -1)],
                 [(A[0] + 1, A[1], 8, 0)], [(A[0] + 2, A[1], 8, 2)], [(A[0], A[1] + 2, 8, 2)], [ok, (A[0], A[1], 8, 9)]):
        assert call(rows) == INVALID, rows
    assert call([(A[0], A[1], (1 << 36) + 1, 0)]) == UNSUPPORTED
    assert call([ok], count=-1) == INVALID and call([ok], count=65537, nbytes=1 << 30) == UNSUPPORTED
    assert call([ok], max_norm=-1.0) == INVALID and call([ok], max_norm=float("nan")) == INVALID
    assert call([ok], norm=A[8] + 2) == INVALID and call([ok], scratch=A[9] + 8) == INVALID
    assert call([ok], scratch=None) == WORKSPACE and call([ok], nbytes=64) == WORKSPACE
    a = _tensors(ok)
    assert L.moe_grad_norm(ctypes.addressof(a), 1, None, A[9], ws, None) == INVALID
    assert f(None, 1, 1.0, None, A[9], ws, None) == INVALID


def test_gradient_list_of_the_binding_refuses():
    host = torch.zeros(4)
    with pytest.raises(ValueError):
        mx.GradList([host])
    with pytest.raises(TypeError):
        mx.GradList([host.double()])
    with pytest.raises(TypeError):
        mx.GradList([None])
    with pytest.raises(ValueError):
        mx.GradList([host], [host, host])
    with pytest.raises(TypeError):
        mx.moe_grad_norm([host], host, host)


def test_binding_refuses_host_tensors_and_names():
    d = mx.Linear(2, 16, 16)
    t = torch.zeros(2, 16).bfloat16()
    with pytest.raises(ValueError):
        mx.moe_grouped_linear_act(d, t, t, t, None, act="swish")
    with pytest.raises(ValueError):
        mx.moe_grouped_linear_act(d, t, t, t, None)
    with pytest.raises(TypeError):
        mx.moe_grouped_linear_act(d, t, t, None, None)
    with pytest.raises(ValueError):
        mx.moe_grouped_linear_act_backward(d, t, t, t, None, act="silu")
    with pytest.raises(TypeError):
        mx.moe_forward_a16w16(_dims(), t.float(), t, t, t, t, t, t, t)


def _dims(**kw):
    return mx.Dims(**{**dict(T=4, T_max=4, H=128, F=128, E=8, k=2, P_total=8, p0=0, P_local=8, R_max=1), **kw})


@needs_lib
def test_layer_refusals():
    f = mx.lib().moe_forward_a16w16
    taps = mx.Taps()

    def call(d=None, t=0, nt=None, x=A[0], lg=A[1], w1=A[2], w2=A[3], rc=A[4], rs=A[5], hist=None, out=A[6], tp=None,
             ws=A[7], nbytes=None):
        d = d or _dims()
        n = mx.moe_a16w16_workspace_bytes(d) if nbytes is None else nbytes
        return f(ctypes.byref(d), t, nt, x, lg, w1, w2, rc, rs, hist, out, tp, ws, n, None)

    for name in ("x", "lg", "w1", "w2", "rc", "rs", "out"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: A[0] + 8}) == INVALID, name
    assert call(hist=A[0] + 4) == INVALID and call(nt=A[0] + 2) == INVALID and call(ws=A[0] + 16) == INVALID
    assert call(t=2) == INVALID and call(t=3) == INVALID and call(t=-1) == INVALID
    taps.topk_w = A[0] + 4
    assert call(tp=ctypes.byref(taps)) == INVALID
    assert call(ws=None) == WORKSPACE and call(nbytes=1) == WORKSPACE
    assert call(_dims(T=33, T_max=33)) == UNSUPPORTED
    assert call(_dims(H=100)) == INVALID and call(_dims(k=17, E=32, P_total=32)) == UNSUPPORTED
    assert call(_dims(T=0)) == 0
    # T_max past the limit is a capacity like any other
    assert mx.moe_a16w16_workspace_bytes(_dims(T_max=1024)) == mx.moe_a16w16_workspace_bytes(_dims(T_max=32))
    assert mx.moe_a16w16_workspace_bytes(_dims(H=100)) == 0


# ---- the oracle --------------------------------------------------------------

@pytest.mark.parametrize("name", oe.ACTS)
def test_oracle_activations(name):
    """By their closed forms with math's functions, and slopes by differences."""
    z = np.array([-30.0, -9.0, -3.0, -0.7, -1e-3, 0.5, 2.0, 8.0, 25.0])
    f = {"none": lambda v: v, "relu": lambda v: max(v, 0.0), "silu": lambda v: v / (1 + math.exp(-v)),
         "gelu": lambda v: 0.5 * v * math.erfc(-v / math.sqrt(2)),
         "gelu_tanh": lambda v: v / (1 + math.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
         if v > -9 else 0.0}[name]
    ref = np.array([f(v) for v in z])
    assert np.all(np.abs(oe.act(name, z) - ref) <= 1e-13 * np.abs(ref) + 1e-13)
    h = 1e-6
    diff = (oe.act(name, z + h) - oe.act(name, z - h)) / (2 * h)
    assert np.all(np.abs(oe.slope(name, z) - diff) <= 1e-8 * (1 + np.abs(z)))
    assert np.max(np.abs(oe.slope(name, np.linspace(-8, 8, 4001)))) <= oe.MAX_SLOPE[name]


@pytest.mark.parametrize("gated", [False, True])
def test_oracle_product_and_gradient(gated):
    rng = np.random.default_rng(3)
    x, w, b = rng.standard_normal((5, 8)), rng.standard_normal((3, 12, 8)), rng.standard_normal((3, 12))
    off, g_of = [0, 2, 2, 5], [0, 0, 2, 2, 2]
    n = 6 if gated else 12
    r, dy = rng.standard_normal((5, n)), rng.standard_normal((5, n))
    y, t, z, _ = oe.linear_act(x, w, b, r, "silu", gated, off)
    for i in range(5):
        v = [sum(x[i, k] * w[g_of[i], c, k] for k in range(8)) + b[g_of[i], c] for c in range(12)]
        silu = lambda u: u / (1 + math.exp(-u))  # noqa: E731
        ref = [silu(v[c]) * v[c + 6] + r[i, c] if gated else silu(v[c]) + r[i, c] for c in range(n)]
        assert np.allclose(y[i], ref, atol=1e-12) and np.allclose(z[i], v, atol=1e-12)
    assert np.all(t > 0) and np.all(t < 1e-3)
    dz, tz, db, tb = oe.act_backward(dy, z, 3, "silu", gated, off)
    loss = lambda b_: float((oe.linear_act(x, w, b_, r, "silu", gated, off)[0] * dy).sum())  # noqa: E731
    for g in range(3):
        for c in (0, 5, 7, 11):
            e = np.zeros_like(b)
            e[g, c] = 1e-6
            assert abs((loss(b + e) - loss(b - e)) / 2e-6 - db[g, c]) < 1e-7
    assert np.all(db[1] == 0) and np.allclose(db[0], dz[:2].sum(0)) and np.all(tb >= 0) and np.all(tz >= 0)


def test_oracle_clip_and_layer():
    norm, c = oe.clip([np.array([3.0]), np.array([0.0, 4.0])], 1.0)
    assert norm == 5.0 and c == 1.0 / (5.0 + 1e-6)
    assert oe.clip([np.zeros(3)], 1.0) == (0.0, 1.0)
    # one expert per token, x = w = constants: h = 2, act = silu(2) 2, out = 3 * F * that * weight
    x, w1, w2 = np.ones((2, 4)), np.full((2, 6, 4), 0.5), np.full((2, 4, 3), 3.0)
    out, tol = oe.layer(x, w1, w2, np.array([[5], [9]]), np.array([[0.25], [1.0]]), 4, 2.0 ** -7)
    v = 2.0 / (1 + math.exp(-2.0)) * 2.0
    assert np.allclose(out[0], 9 * v * 0.25) and np.all(out[1] == 0) and np.all(tol[1] == 0) and np.all(tol[0] > 0)
