"""GPU tests of the products with bias, activation and residual in their epilogue
and of the gradient through it, against the float64 oracle.

Tolerances are the oracle's bounds plus the output's rounding: half a step,
finfo.eps / 2 of the value, and half the smallest subnormal.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from oracle import experts as oe
from tests import linear_cases as lc

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _say(*a):
    print(*a, flush=True)


def _t(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _np(t):
    return t.detach().cpu().double().numpy()


def _offsets(rng, rows, groups, empty=()):
    live = [g for g in range(groups) if g not in empty]
    n = np.zeros(groups, int)
    n[live] = rng.multinomial(rows, rng.dirichlet(np.ones(len(live))))
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def _check(got, ref, tol, dtype, what):
    fi = torch.finfo(dtype)
    half = fi.eps / 2 * (np.abs(ref) + tol) + fi.smallest_normal * fi.eps / 2
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    bad = err > tol + half
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} beyond the bound, first at {np.argwhere(bad)[0]}, "
                           f"worst {np.max(err / (tol + half)):.3g} of it")
    _say(f"   {what} ok: worst error {np.max(err / (tol + half), initial=0.0):.3g} of the bound")


class Case:
    def __init__(self, rows, groups, N, K, act="silu", gated=False, dt="bf16", out=None, bias=True, res=True, pre=True,
                 off=None, empty=()):
        rng = np.random.default_rng((rows, groups, N, K, len(act), gated))
        self.out = out or dt
        self.rows, self.groups, self.N, self.act, self.gated = rows, groups, N, act, gated
        n = N // 2 if gated else N
        r = lambda *s: rng.standard_normal(s)  # noqa: E731
        self.x, self.w = _t(r(rows, K), T[dt]), _t(r(groups, N, K) * 1.5 / np.sqrt(K), T[dt])
        self.b = _t(r(groups, N) * 0.5, T[dt]) if bias else None
        self.r = _t(r(rows, n), T[self.out]) if res else None
        self.off = off if off is not None else None if groups == 1 else _offsets(rng, rows, groups, empty)
        self.dev_off = None if self.off is None else torch.tensor(self.off, dtype=torch.int32, device="cuda")
        self.d = mx.Linear(rows, N, K, groups=groups, in_type=dt, out_type=self.out)
        self.y = torch.full((rows, n), 7.0, dtype=T[self.out], device="cuda")
        self.pre = torch.full((rows, N), 7.0, dtype=T[self.out], device="cuda") if pre else None
        self.ws = mx.linear_act_workspace(self.d)
        self.ws.fill_(0xFF)

    def run(self, y=None, pre=None, res=None, stream=None):
        mx.moe_grouped_linear_act(self.d, self.x, self.w, self.y if y is None else y, self.ws, act=self.act, gated=self.gated,
                                  bias=self.b, residual=self.r if res is None else res,
                                  pre=self.pre if pre is None else pre, offsets=self.dev_off, stream=stream)

    def ref(self):
        o = lambda t: None if t is None else _np(t)  # noqa: E731
        return oe.linear_act(_np(self.x), _np(self.w), o(self.b), o(self.r), self.act, self.gated, self.off)

    def check(self):
        self.run()
        torch.cuda.synchronize()
        y, ty, z, tz = self.ref()
        lo, hi = (0, self.rows) if self.off is None else (int(self.off[0]), int(self.off[-1]))
        _check(_np(self.y)[lo:hi], y[lo:hi], ty[lo:hi], T[self.out], "y")
        for t in (self.y, self.pre):
            if t is not None:
                assert torch.all(t[:lo] == 7.0) and torch.all(t[hi:] == 7.0), "rows in no group"
        if self.pre is not None:
            _check(_np(self.pre)[lo:hi], z[lo:hi], tz[lo:hi], T[self.out], "pre")


SMALL = [(1, 1, 32, 64), (1, 1, 2, 8), (16, 1, 130, 136), (17, 1, 66, 72), (33, 3, 258, 200), (5, 4, 34, 1024),
         (250, 9, 264, 392), (300, 2, 640, 64), (10, 100, 68, 80), (16, 16, 48, 3000), (300, 130, 40, 72)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", oe.ACTS)
@pytest.mark.parametrize("rows,groups,N,K", SMALL)
def test_activations(rows, groups, N, K, act, gated):
    dt = "f16" if (rows + len(act)) % 2 else "bf16"
    _say(f"[case] act rows={rows} groups={groups} N={N} K={K} {act} gated={gated} {dt}")
    Case(rows, groups, N, K, act, gated, dt, empty=(1,) if groups > 2 else ()).check()


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("bias,res,pre", [(0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)])
@pytest.mark.parametrize("rows,N,K,gated", [(3, 77, 64, False), (40, 77, 4104, False), (40, 154, 4104, True),
                                            (200, 301, 128, False), (200, 302, 128, True)])
def test_parts(rows, N, K, gated, bias, res, pre, out):
    """Each part of the epilogue alone, in the kernel of few rows, joined splits and
    tiles; odd numbers of columns."""
    _say(f"[case] parts rows={rows} N={N} K={K} gated={gated} {bias}{res}{pre} out={out}")
    Case(rows, 1, N, K, "gelu", gated, "bf16", "bf16" if out == "same" else out, bool(bias), bool(res), bool(pre)).check()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("i", range(len(lc.SHAPES["fwd"]) + len(lc.STREAMED["fwd"])))
def test_every_block_shape(i, gated):
    """Every block shape, whole and split, plain and streaming loads, on integers that
    every sum holds exactly: z (in pre) has to be exact, and y what the formula
    gives of it."""
    shape, rows, groups, N, K = (lc.SHAPES["fwd"] + lc.STREAMED["fwd"])[i]
    N += N % 2 if gated else 0
    _say(f"[case] shape {shape} rows={rows} groups={groups} N={N} K={K} gated={gated}")
    g = torch.Generator(device="cuda")
    g.manual_seed(i)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    n = N // 2 if gated else N
    x, w, b, r = ints(rows, K), ints(groups, N, K), ints(groups, N), ints(rows, n)
    off = [0, rows] if groups == 1 else _offsets(np.random.default_rng(i), rows, groups).tolist()
    dev = torch.tensor(off, dtype=torch.int32, device="cuda")
    dt = torch.bfloat16 if i % 2 else torch.float16
    y, pre = torch.full((rows, n), 7.0, device="cuda"), torch.full((rows, N), 7.0, device="cuda")
    d = mx.Linear(rows, N, K, groups=groups, in_type="bf16" if i % 2 else "f16", out_type="f32")
    s = 1.0 / 64   # scales z into the activation's curve, exactly
    ws = mx.linear_act_workspace(d)
    mx.moe_grouped_linear_act(d, x.to(dt), (w.float() * s).to(dt), y, ws, act="silu", gated=gated,
                              bias=(b.float() * s).to(dt), residual=r.float(), pre=pre, offsets=dev)
    torch.cuda.synchronize()
    for k, (lo, hi) in enumerate(zip(off, off[1:])):
        if lo == hi:
            continue
        z = (x[lo:hi].float() @ w[k].float().t() + b[k].float()) * s
        assert torch.equal(pre[lo:hi], z), f"z of group {k}"
        z = z.double()
        f = z * torch.sigmoid(z)
        v = torch.sigmoid(z[:, :n]) * z[:, :n] * z[:, n:] if gated else f
        ref = v + r[lo:hi].double()
        tol = 26 * oe.U * v.abs() + 2 * oe.U * ref.abs() + 1e-37
        assert bool(((y[lo:hi].double() - ref).abs() <= tol).all()), f"y of group {k}"


def test_rows_in_no_group_and_groups_apart():
    off = np.array([3, 20, 20, 61, 80], np.int32)
    for rows, N, K, gated in ((90, 136, 200, True), (90, 50, 7024, False)):
        c = Case(rows, 4, N, K, "gelu_tanh", gated, off=off)
        c.check()
        clean = c.y.clone()
        c.x[20:61], c.x[:3], c.x[80:] = float("nan"), float("inf"), float("nan")
        c.b[1], c.w[2, 0] = float("inf"), float("nan")
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.y[:20], clean[:20]) and torch.equal(c.y[61:], clean[61:])
        assert torch.all(torch.isnan(c.y[20:61]))


def test_residual_in_place_streams_and_bits():
    for rows, N, K in ((7, 96, 128), (60, 72, 8200), (700, 392, 264)):
        for gated in (False, True):
            c = Case(rows, 1, N, K, "silu", gated)
            c.run()
            y = c.r.clone()
            c.run(y=y, res=y)
            assert torch.equal(y, c.y)
            st = torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            z = torch.empty_like(y)
            c.run(y=z, stream=st)
            st.synchronize()
            assert torch.equal(z, c.y)


def test_far_gates_and_nan():
    """Identity weights: z is x, one (gate, up) a row.  Gates below -80 keep their
    value through a large factor; NaN stays NaN, relu's too."""
    K = 64
    gate = torch.tensor([-100.0, -88.0, -87.0, 90.0, -1e4, 3e4, float("nan"), -300.0])
    up = torch.tensor([1e30, 1e20, 1.0, 1e-3, 1e38, 2.0, 1.0, 3e38])
    n = len(gate)
    x = torch.zeros(n, 2 * K)
    x[range(n), range(n)], x[range(n), range(K, K + n)] = gate, up
    x = x.bfloat16().cuda()
    w = torch.eye(2 * K, device="cuda").bfloat16()[None].contiguous()
    d = mx.Linear(n, 2 * K, 2 * K, out_type="f32")
    a, u = (_np(x)[range(n), range(c, c + n)] for c in (0, K))
    for act in oe.ACTS:
        y = torch.empty(n, K, device="cuda")
        mx.moe_grouped_linear_act(d, x, w, y, mx.linear_act_workspace(d), act=act, gated=True)
        got = _np(y)[range(n), range(n)]
        assert np.isnan(got[6])
        fin = ~np.isnan(a)
        with np.errstate(over="ignore"):
            ref = oe.act(act, a[fin]) * u[fin]
        # the exponent's rounding counts by its size; where it is far, f32's range ends first
        far = np.where(np.abs(a[fin]) > 80, 1e-4, 0.0)
        tol = np.maximum(oe.act_rel(act, np.clip(a[fin], -20, 20)), far) * np.abs(ref) + 2.0 ** -126
        over = np.abs(ref) > np.finfo(np.float32).max   # (act none: the product itself)
        assert np.array_equal(got[fin][over], np.copysign(np.inf, ref[over]))
        assert np.all(np.abs(got[fin] - ref)[~over] <= tol[~over]), (act, got, ref)


def test_gated_weights_of_two_gib():
    """N = K = 32768: byte offsets in a group's weights reach 2^31."""
    N = K = 32768
    w = torch.zeros(1, N, K, dtype=torch.bfloat16, device="cuda")
    rows = 20
    x = torch.ones(rows, K, dtype=torch.bfloat16, device="cuda")
    x *= torch.arange(1, rows + 1, device="cuda")[:, None]
    w[0, :, K - 1] = (torch.arange(N, device="cuda") % 61).bfloat16()
    d = mx.Linear(rows, N, K, out_type="f32")
    y, pre = torch.empty(rows, N // 2, device="cuda"), torch.empty(rows, N, device="cuda")
    mx.moe_grouped_linear_act(d, x, w, y, mx.linear_act_workspace(d), act="none", gated=True, pre=pre)
    z = torch.arange(1, rows + 1, device="cuda")[:, None] * (torch.arange(N, device="cuda") % 61).float()
    assert torch.equal(pre, z) and torch.equal(y, z[:, :N // 2] * z[:, N // 2:])


# ---- the gradient ------------------------------------------------------------

class Back:
    def __init__(self, rows, groups, N, act="silu", gated=False, dt="bf16", out=None, db=True, off=None, empty=()):
        rng = np.random.default_rng((rows, groups, N, len(act), gated, 1))
        self.out, self.dt = out or dt, dt
        self.rows, self.groups, self.N, self.act, self.gated = rows, groups, N, act, gated
        n = N // 2 if gated else N
        self.dy = _t(rng.standard_normal((rows, n)), T[self.out])
        self.pre = _t(rng.standard_normal((rows, N)) * 2.0, T[self.out])
        self.off = off if off is not None else None if groups == 1 else _offsets(rng, rows, groups, empty)
        self.dev_off = None if self.off is None else torch.tensor(self.off, dtype=torch.int32, device="cuda")
        self.d = mx.Linear(rows, N, 64, groups=groups, in_type=dt, out_type=self.out)
        self.dz = torch.full((rows, N), 7.0, dtype=T[dt], device="cuda")
        self.db = torch.full((groups, N), 7.0, device="cuda") if db else None
        self.ws = mx.linear_act_workspace(self.d)
        self.ws.fill_(0xFF)

    def run(self, dz=None, db=None, pre=None, stream=None):
        mx.moe_grouped_linear_act_backward(self.d, self.dy, self.pre if pre is None else pre, self.dz if dz is None else dz,
                                           self.ws, act=self.act, gated=self.gated, db=self.db if db is None else db,
                                           offsets=self.dev_off, stream=stream)

    def check(self):
        self.run()
        torch.cuda.synchronize()
        dz, t, db, tb = oe.act_backward(_np(self.dy), _np(self.pre), self.groups, self.act, self.gated, self.off)
        lo, hi = (0, self.rows) if self.off is None else (int(self.off[0]), int(self.off[-1]))
        _check(_np(self.dz)[lo:hi], dz[lo:hi], t[lo:hi], T[self.dt], "dz")
        assert torch.all(self.dz[:lo] == 7.0) and torch.all(self.dz[hi:] == 7.0), "rows in no group"
        if self.db is not None:
            _check(_np(self.db), db, tb, torch.float32, "db")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", oe.ACTS)
@pytest.mark.parametrize("rows,groups,N", [(1, 1, 8), (3, 1, 24), (64, 1, 264), (65, 1, 264), (64, 3, 40), (250, 9, 264),
                                           (129, 3, 4104), (1000, 5, 2056), (700, 70, 64), (30, 200, 16), (3000, 1000, 16)])
def test_backward(rows, groups, N, act, gated):
    dt = "f16" if (rows + len(act)) % 2 else "bf16"
    out = "f32" if (rows + len(act)) % 3 == 0 else None
    _say(f"[case] backward rows={rows} groups={groups} N={N} {act} gated={gated} {dt} out={out}")
    Back(rows, groups, N, act, gated, dt, out, empty=(0, groups - 1) if groups > 2 else ()).check()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,groups,N", [(256, 1, 264), (257, 1, 264), (256, 1, 16), (256, 40, 4104), (64, 96, 4104), (128, 96, 4104), (129, 96, 4104),
                                           (16, 1024, 2056), (17, 1024, 2056), (250, 7, 4096), (256, 3, 72)])
def test_backward_in_one_launch_and_in_two(rows, groups, N, gated):
    """On both sides of the sizes up to which a block takes all rows of a group, all rows in one group too."""
    _say(f"[case] backward rows={rows} groups={groups} N={N} gated={gated}")
    Back(rows, groups, N, "silu", gated).check()
    if groups > 1:
        off = np.where(np.arange(groups + 1) > groups // 2, rows, 0).astype(np.int32)
        Back(rows, groups, N, "gelu", gated, out="f32", off=off).check()


@pytest.mark.parametrize("gated", [False, True])
def test_backward_of_many_rows(gated):
    Back(20000, 1, 136, "silu", gated, out="f32").check()
    Back(20000, 3, 2064, "gelu", gated).check()


def test_backward_without_db_in_place_and_apart():
    off = np.array([5, 40, 40, 200], np.int32)
    for gated in (False, True):
        for rows in (60, 230):
            o = np.minimum(off, rows - 9)
            Back(rows, 3, 72, "silu", gated, db=False, off=o).check()
            c = Back(rows, 3, 72, "silu", gated, off=o)
            c.check()
            z = c.pre.clone()
            c.run(dz=z, pre=z)
            lo, hi = int(o[0]), int(o[-1])
            assert torch.equal(z[lo:hi], c.dz[lo:hi]) and torch.equal(z[:lo], c.pre[:lo]) and torch.equal(z[hi:], c.pre[hi:])
            clean = c.db.clone()
            c.dy[:5], c.dy[40:], c.pre[:5] = float("nan"), float("inf"), float("nan")
            c.run()
            assert torch.equal(c.db[:2], clean[:2])


def test_backward_of_no_rows_writes_zeros():
    for G in (1, 3):
        d = mx.Linear(0, 72, 64, groups=G)
        off = None if G == 1 else torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        e = torch.empty(0, 72, dtype=torch.bfloat16, device="cuda")
        db = torch.full((G, 72), 7.0, device="cuda")
        mx.moe_grouped_linear_act_backward(d, e, e, e, mx.linear_act_workspace(d), act="silu", db=db, offsets=off)
        assert torch.all(db == 0)
        y = torch.empty(0, 36, dtype=torch.bfloat16, device="cuda")
        mx.moe_grouped_linear_act(d, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                                  torch.zeros(G, 72, 64, dtype=torch.bfloat16, device="cuda"), y,
                                  mx.linear_act_workspace(d), act="silu", gated=True, offsets=off)


def test_offsets_outside_the_rows_touch_nothing_outside():
    """Offsets that break the contract are clamped (no value is promised)."""
    rows, G, N, K = 200, 3, 64, 64
    x, w = torch.ones(rows + 64, K, device="cuda").bfloat16(), torch.ones(G, N, K, device="cuda").bfloat16()
    b = torch.ones(G, N, device="cuda").bfloat16()
    d = mx.Linear(rows, N, K, groups=G, out_type="f32")
    ws = mx.linear_act_workspace(d)
    for o in ([-5, 10, 1000, 2000], [150, 10, 5, 400], [2 ** 31 - 1, 0, -2 ** 31, 40], [0, 200, 0, 200]):
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        y, pre = torch.full((rows + 64, N // 2), 7.0, device="cuda"), torch.full((rows + 64, N), 7.0, device="cuda")
        mx.moe_grouped_linear_act(d, x, w, y, ws, act="silu", gated=True, bias=b, pre=pre, offsets=off)
        dz, db = torch.full((rows + 64, N), 7.0, device="cuda").bfloat16(), torch.full((G + 1, N), 7.0, device="cuda")
        mx.moe_grouped_linear_act_backward(d, y, pre, dz, ws, act="silu", gated=True, db=db, offsets=off)
        torch.cuda.synchronize()
        for t in (y, pre, dz):
            assert torch.all(t[rows:] == 7.0)
        assert torch.all(db[G:] == 7.0)


def test_gradients_against_differences():
    """<y, dy> by central differences in bias and x, on f32 outputs: dz, db, and dx by
    the product's own gradient."""
    rows, G, N, K = 24, 2, 64, 64
    for act in ("silu", "gelu", "gelu_tanh"):
        c = Case(rows, G, N, K, act, True, out="f32", res=False)
        c.run()
        rng = np.random.default_rng(9)
        dy = _t(rng.standard_normal((rows, N // 2)), torch.float32)
        dz, db = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda"), torch.empty(G, N, device="cuda")
        mx.moe_grouped_linear_act_backward(c.d, dy, c.pre, dz, c.ws, act=act, gated=True, db=db, offsets=c.dev_off)
        db = _np(db)

        def loss(b):
            y, *_ = oe.linear_act(_np(c.x), _np(c.w), b, None, act, True, c.off)
            return float((y * _np(dy)).sum())

        b0 = _np(c.b)
        for g in range(G):
            for n in (0, 7, 31, 32, 40, 63):
                e = np.zeros_like(b0)
                e[g, n] = 1e-4
                diff = (loss(b0 + e) - loss(b0 - e)) / 2e-4
                # third derivatives of at most about 10 in size per row: 1e-8 / 6 each
                assert abs(diff - db[g, n]) <= 1e-4 * (1 + np.abs(db).max()), (act, g, n, diff, db[g, n])


def test_forward_and_backward_in_a_captured_graph():
    rows, G, N, K = 100, 4, 136, 208
    c = Case(rows, G, N, K, "silu", True, empty=(1,))
    b = Back(rows, G, N, "silu", True)
    b.dev_off = c.dev_off

    def step(y, pre, dz, db):
        c.run(y=y, pre=pre)
        mx.moe_grouped_linear_act_backward(c.d, y, pre, dz, b.ws, act="silu", gated=True, db=db, offsets=c.dev_off)

    step(c.y, c.pre, b.dz, b.db)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c.y, c.pre, b.dz, b.db)
    for i in range(3):
        c.x.copy_(_t(np.random.default_rng(i).standard_normal((rows, K)), torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        e = [torch.empty_like(t) for t in (c.y, c.pre, b.dz, b.db)]
        step(*e)
        torch.cuda.synchronize()
        for got, want in zip((c.y, c.pre, b.dz, b.db), e):
            assert torch.equal(got, want)
