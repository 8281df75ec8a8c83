"""GPU tests of the activations and their slopes where their formulas are hard: at
zero, far out, at infinity.  Against the float64 oracle, in f32 outputs.

Forward: x is zero and the bias is z, so that z is what the test says, to the bit, in
the kernel of few rows, in tiles and in joined splits.  Gradient: every row is a group of
its own, so that db holds the row's f32 values before they are rounded to dz.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from oracle import experts as oe
from tests.test_gpu_linear_act import Back

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().cpu().double().numpy()


def _pad(v, n):
    """v (a list) as n values: repeated from the front."""
    return torch.tensor([v[i % len(v)] for i in range(n)], dtype=torch.float32)


FORWARD = [(3, 64), (40, 64), (40, 4104)]   # rows, K: few rows, tiles, joined splits


def forward(act, z, u=None, rows=3, K=64):
    """act(z) [* u], f32; z and u 1-D, of values that bf16 holds."""
    b = (z if u is None else torch.cat([z, u])).bfloat16().cuda()[None].contiguous()
    N = b.shape[1]
    d = mx.Linear(rows, N, K, out_type="f32")
    x, w = torch.zeros(rows, K, device="cuda").bfloat16(), torch.zeros(1, N, K, device="cuda").bfloat16()
    y = torch.full((rows, len(z)), 7.0, device="cuda")
    mx.moe_grouped_linear_act(d, x, w, y, mx.linear_act_workspace(d), act=act, gated=u is not None, bias=b)
    assert torch.equal(y.nan_to_num(1.5), y[:1].nan_to_num(1.5).expand_as(y))
    return y[0].cpu()


def backward(act, z, dy, u=None, rows=2):
    """The f32 gradient of z [and of u] for dy, all 1-D f32 (dz's rounding left out)."""
    pre = (z if u is None else torch.cat([z, u])).cuda()[None].expand(rows, -1).contiguous()
    N = pre.shape[1]
    d = mx.Linear(rows, N, 64, groups=rows, out_type="f32")
    off = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    dz, db = torch.empty(rows, N, device="cuda").bfloat16(), torch.empty(rows, N, device="cuda")
    mx.moe_grouped_linear_act_backward(d, dy.cuda()[None].expand(rows, -1).contiguous(), pre, dz, mx.linear_act_workspace(d),
                                       act=act, gated=u is not None, db=db, offsets=off)
    assert torch.equal(db.nan_to_num(1.5), db[:1].nan_to_num(1.5).expand_as(db))
    assert torch.equal(dz.nan_to_num(1.5), db.bfloat16().nan_to_num(1.5))
    return db[0].cpu()


BACKWARD = [2, 300]   # rows: one launch, two


@pytest.mark.parametrize("rows", BACKWARD)
def test_slopes_at_zero(rows):
    """Half of one, but for none and relu: exactly."""
    z = _pad([0.0, -0.0], 16)
    for act, want in (("none", 1.0), ("relu", 0.0), ("silu", 0.5), ("gelu", 0.5), ("gelu_tanh", 0.5)):
        got = backward(act, z, torch.full((16,), 3.0), rows=rows)
        assert torch.all(got == 3.0 * want), (act, got)
        got = backward(act, z, torch.full((16,), 3.0), torch.full((16,), -2.0), rows=rows)
        assert torch.all(got[:16] == -6.0 * want) and torch.all(got[16:] == 0.0), (act, got)


@pytest.mark.parametrize("rows,K", FORWARD)
def test_gelu_of_small_values(rows, K):
    """z Phi(z) to the tail's 6 x 2^-24, the reciprocal's and the exponential's ulps (2 x
    2^-24 each, three of the exponential's) and the products' roundings (3)."""
    z = torch.cat([torch.logspace(-30, -1, 60), torch.linspace(0.1, 1.0, 68)]).bfloat16().float()
    z = torch.cat([z, -z])
    y = _np(forward("gelu", z, rows=rows, K=K))
    ref = oe.act("gelu", z.double().numpy())
    rel = np.abs(y / ref - 1)
    assert np.all(rel <= (6 + 2 + 3 * 2 + 3) * oe.U), rel.max() / oe.U


INF, NAN = float("inf"), float("nan")


def _same(got, want):
    want = torch.tensor(want)
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0.5, INF, -INF), want.nan_to_num(0.5, INF, -INF))


@pytest.mark.parametrize("rows,K", FORWARD)
def test_infinite_z_forward(rows, K):
    """What the formula gives: 0 times infinity is NaN."""
    z, u = _pad([INF, -INF, NAN, 1.0], 16), _pad([-2.0] * 16, 16)
    want = {"none": [INF, -INF], "relu": [INF, 0.0], "silu": [INF, NAN], "gelu": [INF, NAN], "gelu_tanh": [INF, NAN]}
    for act, v in want.items():
        assert _same(forward(act, z, rows=rows, K=K)[:3], v + [NAN]), act
        assert _same(forward(act, z, u, rows=rows, K=K)[:3], [-2.0 * a for a in v] + [NAN]), act


@pytest.mark.parametrize("rows", BACKWARD)
def test_infinite_z_in_the_gradient(rows):
    """Slopes hold z times phi(z), or z times 1 - sigmoid: NaN at both ends."""
    z, dy, u = _pad([INF, -INF, 1.0, 2.0], 16), _pad([3.0, 3.0, 0.5, 0.25], 16), _pad([-2.0] * 16, 16)
    slope = {"none": [1.0, 1.0], "relu": [1.0, 0.0], "silu": [NAN, NAN], "gelu": [NAN, NAN], "gelu_tanh": [NAN, NAN]}
    value = {"none": [INF, -INF], "relu": [INF, 0.0], "silu": [INF, NAN], "gelu": [INF, NAN], "gelu_tanh": [INF, NAN]}
    for act in slope:
        got = backward(act, z, dy, rows=rows)
        assert _same(got[:2], [3.0 * a for a in slope[act]]), (act, got)
        gated = backward(act, z, dy, u, rows=rows)
        assert _same(gated[:2], [-6.0 * a for a in slope[act]]), (act, gated)
        assert _same(gated[16:18], [3.0 * a for a in value[act]]), (act, gated)
        assert torch.isfinite(got[2:4]).all() and torch.isfinite(gated[2:4]).all()


# Both sides of where the exponentials leave f32's normal range (-80, -13, -9), as far as a
# factor of 1e30 brings the product back.
FAR = {"silu": np.linspace(-150.0, -70.0, 161), "gelu": np.linspace(-16.5, -10.0, 131), "gelu_tanh": np.linspace(-12.5, -7.0, 111)}


@pytest.mark.parametrize("rows,K", FORWARD)
@pytest.mark.parametrize("act", list(FAR))
def test_far_values(act, rows, K):
    z = torch.tensor(FAR[act]).bfloat16().float()
    u = torch.cat([torch.full_like(z, v) for v in (1.0, -1e15, 1e30)]).bfloat16().float()
    z = torch.cat([z, z, z])
    n = len(z)
    got = _np(forward(act, z, u, rows=rows, K=K))
    zd, ud = z.double().numpy(), u.double().numpy()
    ref = oe.act(act, zd) * ud
    tol = (oe.act_rel(act, zd) + oe.U) * np.abs(ref) + 2.0 ** -126
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (zd[bad][:4], ud[bad][:4], got[bad][:4], ref[bad][:4])
    assert np.sum(np.abs(ref) > 2.0 ** -120) > n // 3   # (not for want of normal values)
    alone = _np(forward(act, z, rows=rows, K=K))
    ref = oe.act(act, zd)
    assert np.all(np.abs(alone - ref) <= oe.act_rel(act, zd) * np.abs(ref) + 2.0 ** -126)


@pytest.mark.parametrize("rows", BACKWARD)
@pytest.mark.parametrize("act", list(FAR))
def test_far_gradients(act, rows):
    z = torch.tensor(FAR[act], dtype=torch.float32)
    z = torch.cat([z, z, z])
    n = len(z) // 24 * 8   # of each factor
    z = torch.cat([z[:n], z[:n], z[:n]])
    dy = torch.cat([torch.full((n,), v) for v in (1.0, -1e15, 1e30)])
    zd, dd = z.double().numpy(), dy.double().numpy()
    got = _np(backward(act, z, dy, rows=rows))
    ref = oe.slope(act, zd) * dd
    tol = np.abs(dd) * oe.slope_tol(act, zd) + 2 * oe.U * np.abs(ref) + 2.0 ** -126
    assert np.all(np.abs(got - ref) <= tol), (got, ref)
    assert np.sum(np.abs(ref) > 2.0 ** -120) > n
    # gated: the factor in up (the value's gradient then takes dy), or in dy
    for d, u in ((torch.full_like(dy, 0.75), dy), (dy, torch.full_like(dy, -1.25))):
        got = _np(backward(act, z, d, u, rows=rows))
        d, u = d.double().numpy(), u.double().numpy()
        gate, up = oe.slope(act, zd) * d * u, oe.act(act, zd) * d
        tol = np.abs(d * u) * (oe.slope_tol(act, zd) + 2 * oe.U * np.abs(oe.slope(act, zd))) + 2.0 ** -126
        assert np.all(np.abs(got[:len(z)] - gate) <= tol), (got[:len(z)], gate)
        tol = (oe.act_rel(act, zd) + 2 * oe.U) * np.abs(up) + 2.0 ** -126
        assert np.all(np.abs(got[len(z):] - up) <= tol), (got[len(z):], up)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,groups,N", [(4000, 3, 264), (9000, 1, 4112), (3000, 40, 72)])
def test_gradient_in_place_of_long_tiles(rows, groups, N, gated):
    """dz over pre where a thread has four rows in flight, the last of them read twice."""
    c = Back(rows, groups, N, "silu", gated)
    c.check()
    clean = c.db.clone()
    z = c.pre.clone()
    c.db.fill_(7.0)
    c.run(dz=z, pre=z)
    torch.cuda.synchronize()
    assert torch.equal(z, c.dz) and torch.equal(c.db, clean)
