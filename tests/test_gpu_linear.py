"""GPU tests of the linear operators against the float64 oracle: fp8
quantisation with a scale per 128 columns, the fp8 product with a scale per
block of 128, the 16-bit products grouped by expert and their gradients.

Tolerances are the oracle's bounds of the f32 sums plus the output's rounding:
half a step, finfo.eps / 2 of the value, and half the smallest subnormal.
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


def _rng(*key):
    return np.random.default_rng(key)


def _t(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _np(t):
    return t.detach().cpu().double().numpy()


def _offsets(rng, rows, groups, empty=()):
    """Ragged groups over all rows; the groups of `empty` get none."""
    live = [g for g in range(groups) if g not in empty]
    n = np.zeros(groups, int)
    n[live] = rng.multinomial(rows, rng.dirichlet(np.ones(len(live))))
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def _check(got, ref, tol, dtype):
    fi = torch.finfo(dtype)
    half = fi.eps / 2 * (np.abs(ref) + tol) + fi.smallest_normal * fi.eps / 2
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), "not finite"
    bad = err > tol + half
    assert not bad.any(), (f"{bad.sum()} of {bad.size} beyond the bound, first at {np.argwhere(bad)[0]}, "
                           f"worst {np.max(err / (tol + half)):.3g} of it")
    _say(f"   ok: worst error {np.max(err / (tol + half), initial=0.0):.3g} of the bound")


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

def _codes(x, s):
    """e4m3 codes of x * (1 / s), every operation one f32 rounding."""
    inv = np.float32(1) / ol.spread(s, x.shape[1], 1)
    return torch.from_numpy(x.astype(np.float32) * inv).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


QUANT = [(1, 7168), (1, 16), (3, 128), (5, 144), (17, 112), (64, 2048), (2, 32768), (130, 1008)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K", QUANT)
def test_quant_is_bit_exact(rows, K, dt):
    _say(f"[case] quant rows={rows} K={K} {dt}")
    rng = _rng(1, rows, K)
    x = _t(rng.standard_normal((rows, K)) * 10.0 ** rng.integers(-3, 3, (rows, 1)), T[dt])
    q = torch.full((rows, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, ol.blocks(K)), -1.0, device="cuda")
    mx.moe_fp8_quant(x, q, s)
    xf = x.float().cpu().numpy()
    rs = ol.quant_scales(xf)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), _codes(xf, rs))


def test_quant_of_zeros_tiny_and_huge_values():
    x = torch.zeros(6, 256, device="cuda")
    x[1, 3] = 1e-38
    x[2] = 1e-45
    x[3, 200] = 3e38
    x[4, 0] = float("inf")
    x[4, 1] = 1.0
    x[5, 130] = float("nan")
    q = torch.empty(6, 256, dtype=torch.uint8, device="cuda")
    s = torch.empty(6, 2, device="cuda")
    mx.moe_fp8_quant(x, q, s)
    s, q = s.cpu().numpy(), q.cpu()
    xf = x.cpu().numpy()
    rs = ol.quant_scales(xf[:4])
    assert np.array_equal(s[:4], rs) and s[0, 0] == np.float32(2.0 ** -126)
    assert np.array_equal(q[:4].numpy(), _codes(xf[:4], rs))
    v = q.view(torch.float8_e4m3fn).float().numpy()
    assert np.isinf(s[4, 0]) and np.isnan(v[4, 0]) and np.all(v[4, 1:] == 0) and s[4, 1] == np.float32(2.0 ** -126)
    assert np.isnan(s[5, 1]) and np.all(np.isnan(v[5, 128:])) and np.all(v[5, :128] == 0)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 2048), (33, 144), (9, 7168)])
def test_swiglu_quant(rows, K, dt):
    _say(f"[case] swiglu quant rows={rows} K={K} {dt}")
    x = _t(_rng(2, rows, K).standard_normal((rows, 2 * K)) * 2, T[dt])
    x[0, 0] = -95.0   # exp(95) overflows f32: silu is then -0
    q = torch.empty(rows, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(rows, ol.blocks(K), device="cuda")
    mx.moe_fp8_swiglu_quant(x, q, s)
    h = ol.swiglu(_np(x))
    # exp within two roundings, its sum, the quotient and the product: under 8 x 2^-24
    # of h in all; gates below -80 lose f32's range: 1e-30 covers them
    rel = 8 * 2.0 ** -24
    amax = np.stack([np.abs(h[:, c:c + 128]).max(1) for c in range(0, K, 128)], 1)
    assert np.all(np.abs(_np(s) - amax / 448) <= (rel + 2.0 ** -24) * amax / 448 + 2.0 ** -126)
    sv = ol.spread(_np(s), K, 1)
    err = np.abs(_np(q.float()) * sv - h)
    assert np.all(err <= np.abs(h) * (2.0 ** -4 + 2 * rel) + sv * 2.0 ** -10 + 1e-30)


def test_swiglu_of_infinities():
    """silu(inf) = inf, silu(-inf) = -inf * 0 = NaN, and inf * 0 = NaN: a block
    holding one has an infinite or NaN scale; the other blocks keep theirs."""
    x = torch.ones(4, 512, device="cuda")
    x[0, 3], x[1, 3], x[2, 3], x[2, 259] = float("inf"), -float("inf"), float("inf"), 0.0
    x[3, :256] = 120.0
    q = torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(4, 2, device="cuda")
    mx.moe_fp8_swiglu_quant(x, q, s)
    s = s.cpu()
    one = np.float32(1 / (1 + np.exp(-1.0)))
    assert torch.isinf(s[0, 0]) and torch.isnan(s[1, 0]) and torch.isnan(s[2, 0])
    assert torch.all((s[:3, 1] * 448 - one).abs() < 1e-6)
    assert torch.all(s[3] == 120.0 / 448) and torch.all(q[3].float() == 448)


def test_quant_rows_further_apart_and_other_stream():
    base = _t(_rng(3).standard_normal((7, 512)), torch.bfloat16)
    x = base[:, 64:64 + 144]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q = torch.empty(7, 144, dtype=torch.uint8, device="cuda")
    s = torch.empty(7, 2, device="cuda")
    mx.moe_fp8_quant(x, q, s, stream=st)
    st.synchronize()
    xf = x.float().cpu().numpy()
    assert np.array_equal(q.cpu().numpy(), _codes(xf, ol.quant_scales(xf)))
    with pytest.raises(mx.MoeError):
        mx.moe_fp8_quant(base[:, 4:4 + 144], q, s)   # rows that start 8 bytes into a 16-byte piece
    with pytest.raises(ValueError):
        mx.moe_fp8_quant(base.t(), q, s)
    with pytest.raises(ValueError):
        mx.moe_fp8_quant(base[:1].expand(7, 512), torch.empty(7, 512, dtype=torch.uint8, device="cuda"),
                         torch.empty(7, 4, device="cuda"))


# ---------------------------------------------------------------------------
# fp8 product
# ---------------------------------------------------------------------------

def _fp8_case(rng, rows, groups, N, K, empty=(), scale=1.0):
    def blocks8(a):   # [.., n, K] -> codes and block scales
        n = a.shape[-2]
        s = np.stack([np.stack([np.abs(a[..., i:i + 128, j:j + 128]).max((-1, -2)) for j in range(0, K, 128)], -1)
                      for i in range(0, n, 128)], -2).astype(np.float32) / np.float32(448)
        return s

    x = (rng.standard_normal((rows, K)) * scale).astype(np.float32)
    w = (rng.standard_normal((groups, N, K)) * 0.02).astype(np.float32)
    xs = ol.quant_scales(x)
    ws = blocks8(w)
    xq = torch.from_numpy(x / ol.spread(xs, K, 1)).to(torch.float8_e4m3fn)
    wq = torch.from_numpy(w / ol.spread(ol.spread(ws, N, 1), K, 2)).to(torch.float8_e4m3fn)
    off = _offsets(rng, rows, groups, empty) if groups > 1 else None
    return xq, xs, wq, ws, off


def _run_fp8(xq, xs, wq, ws, off, out="bf16", rows=None, stream=None):
    rows = xq.shape[0] if rows is None else rows
    G, N, K = wq.shape
    d = mx.Linear(rows, N, K, groups=G, in_type="fp8", out_type=out)
    y = torch.full((max(rows, 1), N), 7.0, dtype=T[out], device="cuda")
    mx.moe_fp8_linear(d, xq.cuda(), _t(xs), wq.cuda(), _t(ws), y, mx.linear_workspace(d),
                      offsets=None if off is None else torch.from_numpy(off).cuda(), stream=stream)
    torch.cuda.synchronize()
    return y[:rows]


FP8 = [  # rows, groups, N, K, empty groups
    (1, 1, 33, 64, ()), (1, 1, 512, 2048, ()), (2, 1, 129, 16, ()), (7, 1, 255, 400, ()), (16, 1, 96, 1152, ()),
    (17, 1, 130, 144, ()), (33, 1, 257, 272, ()), (64, 1, 64, 256, ()), (77, 1, 261, 528, ()), (130, 1, 200, 128, ()),
    (300, 1, 300, 384, ()), (1, 4, 48, 160, ()), (5, 9, 130, 256, (0, 8)), (40, 3, 257, 144, (1,)),
    (150, 5, 140, 272, (2, 3)), (400, 2, 260, 256, ()), (3, 70, 40, 128, ()),
    (100, 8, 50, 1200, (3,)), (16, 1, 17, 32768, ())]


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,groups,N,K,empty", FP8)
def test_fp8_linear(rows, groups, N, K, empty, out):
    _say(f"[case] fp8 rows={rows} groups={groups} N={N} K={K} empty={empty} out={out}")
    c = _fp8_case(_rng(4, rows, groups, N, K), rows, groups, N, K, empty)
    y = _run_fp8(*c, out=out)
    ref, tol = ol.fp8_linear(_np(c[0].float()), c[1].astype(float), _np(c[2].float()), c[3].astype(float), c[4])
    _check(_np(y), ref, tol, T[out])


def test_fp8_linear_exact_on_small_integers():
    """Codes that are small integers and scales that are powers of two: every
    sum is exact in f32, so the result is the integer product."""
    rng = _rng(5)
    for rows, N, K in [(1, 160, 384), (20, 200, 272), (300, 130, 1024)]:
        xq = torch.from_numpy(rng.integers(-4, 5, (rows, K)).astype(np.float32)).to(torch.float8_e4m3fn)
        wq = torch.from_numpy(rng.integers(-4, 5, (1, N, K)).astype(np.float32)).to(torch.float8_e4m3fn)
        xs = 2.0 ** rng.integers(-2, 3, (rows, ol.blocks(K)))
        ws = 2.0 ** rng.integers(-2, 3, (1, ol.blocks(N), ol.blocks(K)))
        y = _run_fp8(xq, xs, wq, ws, None, out="f32")
        ref, _ = ol.fp8_linear(_np(xq.float()), xs, _np(wq.float()), ws)
        assert np.array_equal(_np(y), ref), (rows, N, K)


# Sizes at which every output tile shape is the one chosen, with tiles that
# end inside the matrices.
LARGE = [(4500, 1, 4352, 144), (2100, 3, 4232, 272), (1100, 12, 2200, 208), (400, 12, 2200, 208), (150, 12, 2200, 336)]


def _int16(rng, *s):
    return torch.from_numpy(rng.integers(-3, 4, s).astype(np.float32)).cuda()


@pytest.mark.parametrize("rows,groups,N,K", LARGE)
def test_large_tiles_exact_on_small_integers(rows, groups, N, K):
    """Small integers: every sum is exact in f32, so every product is the
    integer one, for every type."""
    _say(f"[case] large rows={rows} groups={groups} N={N} K={K}")
    rng = _rng(16, rows, groups, N, K)
    x, w, dy = _int16(rng, rows, K), _int16(rng, groups, N, K), _int16(rng, rows, N)
    off = _offsets(rng, rows, groups) if groups > 1 else None
    do = _dev_off(off)
    ref = [torch.zeros(rows, N, device="cuda"), torch.zeros(rows, K, device="cuda"), torch.zeros(groups, N, K, device="cuda")]
    for g, (lo, hi) in enumerate(ol.spans(off, rows)):
        ref[0][lo:hi] = (x[lo:hi].double() @ w[g].double().t()).float()
        ref[1][lo:hi] = (dy[lo:hi].double() @ w[g].double()).float()
        ref[2][g] = (dy[lo:hi].double().t() @ x[lo:hi].double()).float()
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    d8 = mx.Linear(rows, N, K, groups=groups, in_type="fp8", out_type="f32")
    y = torch.full((rows, N), 0.5, device="cuda")
    mx.moe_fp8_linear(d8, x.to(torch.float8_e4m3fn), one(rows, ol.blocks(K)), w.to(torch.float8_e4m3fn),
                      one(groups, ol.blocks(N), ol.blocks(K)), y, mx.linear_workspace(d8), offsets=do)
    assert torch.equal(y, ref[0])
    for dt in ("bf16", "f16"):
        d = mx.Linear(rows, N, K, groups=groups, in_type=dt, out_type="f32")
        ws = mx.linear_workspace(d)
        o = [torch.full_like(r, 0.5) for r in ref]
        xt, wt, dyt = x.to(T[dt]), w.to(T[dt]), dy.to(T[dt])
        mx.moe_grouped_linear(d, xt, wt, o[0], ws, offsets=do)
        mx.moe_grouped_linear_dx(d, dyt, wt, o[1], ws, offsets=do)
        mx.moe_grouped_linear_dw(d, dyt, xt, o[2], ws, offsets=do)
        torch.cuda.synchronize()
        for got, r, name in zip(o, ref, ("y", "dx", "dw")):
            assert torch.equal(got, r), (dt, name)


# For each product, sizes at which each of the block shapes is the one chosen.
SHAPES = [
    (2779, 3, 4376, 80), (2658, 12, 1976, 80), (2694, 5, 1464, 80), (2367, 1, 824, 80), (4475, 2, 272, 272),
    (135, 1, 136, 80), (4727, 5, 1648, 80), (2382, 12, 120, 3952), (3326, 1, 104, 2016), (3779, 3, 120, 1040),
    (2299, 5, 112, 832), (2708, 2, 112, 3424), (103, 30, 224, 1072), (311, 1, 2000, 3856), (144, 30, 1248, 80),
    (106, 30, 552, 80), (5383, 12, 632, 144), (471, 30, 1096, 144), (948, 12, 4840, 80), (5716, 3, 192, 416),
    (5893, 1, 1440, 80), (2500, 1, 4104, 1040)]


@pytest.mark.parametrize("rows,groups,N,K", SHAPES)
def test_every_shape_exact_on_small_integers(rows, groups, N, K):
    test_large_tiles_exact_on_small_integers(rows, groups, N, K)


def test_fp8_linear_keeps_other_groups_and_rows_apart():
    """NaN codes and scales in one group's rows and weights reach that group's
    outputs alone; rows in no group are not written."""
    rng = _rng(6)
    rows, G, N, K = 90, 3, 130, 272
    xq, xs, wq, ws, _ = _fp8_case(rng, rows, G, N, K)
    off = np.array([3, 20, 61, 80], np.int32)
    clean = _run_fp8(xq, xs, wq, ws, off, out="f32")
    assert torch.all(clean[:3] == 7.0) and torch.all(clean[80:] == 7.0)
    xq8, wq8 = xq.view(torch.uint8).clone(), wq.view(torch.uint8).clone()
    xq8[20:61], wq8[1] = 0x7F, 0x7F
    xq8[80:], xq8[:3] = 0x7F, 0x7F
    xs2, ws2 = xs.copy(), ws.copy()
    xs2[20:61], ws2[1], xs2[80:] = np.nan, np.inf, np.nan
    y = _run_fp8(xq8.view(torch.float8_e4m3fn), xs2, wq8.view(torch.float8_e4m3fn), ws2, off, out="f32")
    assert torch.equal(y[:20], clean[:20]) and torch.equal(y[61:], clean[61:])
    assert torch.all(torch.isnan(y[20:61]))


@pytest.mark.parametrize("rows,N,K", [(512, 4096, 784), (100, 4096, 5136)])
def test_fp8_scales_of_the_next_row_stay_out(rows, N, K):
    """An odd number of blocks of 128 on sizes whose tiles take them two at a
    time: the scale that follows a row's last one belongs to the next row."""
    _say(f"[case] next row's scales rows={rows} N={N} K={K}")
    rng = _rng(19, rows, N, K)
    x, w = _int16(rng, rows, K), _int16(rng, N, K)
    xs, ws = torch.ones(rows, ol.blocks(K), device="cuda"), torch.ones(1, ol.blocks(N), ol.blocks(K), device="cuda")
    xs[1::2, 0], ws[0, 1::2, 0] = float("nan"), float("inf")
    d = mx.Linear(rows, N, K, in_type="fp8", out_type="f32")
    y = torch.full((rows, N), 0.5, device="cuda")
    mx.moe_fp8_linear(d, x.to(torch.float8_e4m3fn), xs, w.to(torch.float8_e4m3fn), ws, y, mx.linear_workspace(d))
    ref = (x.double() @ w.double().t()).float()
    even = torch.arange(N, device="cuda") // 128 % 2 == 0
    assert torch.equal(y[::2][:, even], ref[::2][:, even])
    assert torch.all(torch.isnan(y[1::2]))


# ---------------------------------------------------------------------------
# 16-bit products by group
# ---------------------------------------------------------------------------

GROUPED = [  # rows, groups, N, K, empty groups
    (1, 1, 64, 64, ()), (1, 1, 8, 8, ()), (1, 3, 72, 2056, (0, 2)), (9, 1, 264, 392, ()), (16, 1, 72, 1096, ()),
    (31, 2, 136, 200, ()), (66, 1, 520, 72, ()), (128, 8, 256, 256, ()), (250, 9, 264, 392, (4,)),
    (300, 1, 200, 328, ()), (520, 2, 72, 136, (0,)), (515, 3, 264, 264, ()), (3, 70, 24, 40, ()),
    (100, 8, 56, 1192, (3,))]


def _case16(rng, dt, rows, groups, N, K, empty):
    x = _t(rng.standard_normal((rows, K)), T[dt])
    w = _t(rng.standard_normal((groups, N, K)) * 0.05, T[dt])
    dy = _t(rng.standard_normal((rows, N)), T[dt])
    off = _offsets(rng, rows, groups, empty) if groups > 1 else None
    return x, w, dy, off


def _dev_off(off):
    return None if off is None else torch.from_numpy(off).cuda()


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("rows,groups,N,K,empty", GROUPED)
def test_grouped_linear_and_gradients(rows, groups, N, K, empty, dt, out):
    out = dt if out == "same" else out
    _say(f"[case] grouped rows={rows} groups={groups} N={N} K={K} empty={empty} {dt} -> {out}")
    x, w, dy, off = _case16(_rng(7, rows, groups, N, K), dt, rows, groups, N, K, empty)
    d = mx.Linear(rows, N, K, groups=groups, in_type=dt, out_type=out)
    ws = mx.linear_workspace(d)
    ws.fill_(0xFF)   # NaN bits: nothing of the workspace may be taken as cleared
    y = torch.full((rows, N), 7.0, dtype=T[out], device="cuda")
    dx = torch.full((rows, K), 7.0, dtype=T[out], device="cuda")
    dw = torch.full((groups, N, K), 7.0, dtype=T[out], device="cuda")
    do = _dev_off(off)
    mx.moe_grouped_linear(d, x, w, y, ws, offsets=do)
    mx.moe_grouped_linear_dx(d, dy, w, dx, ws, offsets=do)
    mx.moe_grouped_linear_dw(d, dy, x, dw, ws, offsets=do)
    torch.cuda.synchronize()
    _check(_np(y), *ol.grouped(_np(x), _np(w), off), T[out])
    _check(_np(dx), *ol.grouped_dx(_np(dy), _np(w), off), T[out])
    _check(_np(dw), *ol.grouped_dw(_np(dy), _np(x), groups, off), T[out])


def test_forward_takes_any_number_of_columns():
    for N in (1, 2, 33, 67, 129, 255):
        x, w, _, off = _case16(_rng(8, N), "bf16", 37, 2, N, 72, ())
        d = mx.Linear(37, N, 72, groups=2)
        y = torch.full((37, N), 7.0, dtype=torch.bfloat16, device="cuda")
        mx.moe_grouped_linear(d, x, w, y, mx.linear_workspace(d), offsets=_dev_off(off))
        _check(_np(y), *ol.grouped(_np(x), _np(w), off), torch.bfloat16)


def test_gradients_are_the_differences_of_the_forward():
    """On small integers every f32 sum is exact, so <y(x + e, w), dy> - <y(x -
    e, w), dy> is exactly 2 <e, dx>, and likewise for w."""
    rng = _rng(9)
    rows, G, N, K = 70, 3, 72, 80
    off = np.array([0, 33, 33, 70], np.int32)
    i = lambda *s: rng.integers(-3, 4, s).astype(np.float32)  # noqa: E731
    x, w, dy, ex, ew = i(rows, K), i(G, N, K), i(rows, N), i(rows, K), i(G, N, K)
    d = mx.Linear(rows, N, K, groups=G, out_type="f32")
    ws, do = mx.linear_workspace(d), _dev_off(off)

    def loss(x_, w_):
        y = torch.empty(rows, N, device="cuda")
        mx.moe_grouped_linear(d, _t(x_, torch.bfloat16), _t(w_, torch.bfloat16), y, ws, offsets=do)
        return float((_np(y) * dy).sum())

    dx, dw = torch.empty(rows, K, device="cuda"), torch.empty(G, N, K, device="cuda")
    b = [_t(v, torch.bfloat16) for v in (dy, w, x)]
    mx.moe_grouped_linear_dx(d, b[0], b[1], dx, ws, offsets=do)
    mx.moe_grouped_linear_dw(d, b[0], b[2], dw, ws, offsets=do)
    assert loss(x + ex, w) - loss(x - ex, w) == 2 * float((_np(dx) * ex).sum())
    assert loss(x, w + ew) - loss(x, w - ew) == 2 * float((_np(dw) * ew).sum())
    assert torch.all(dw[1] == 0)


def test_grouped_keeps_other_groups_and_rows_apart():
    """NaN rows and weights of one group stay in that group's results, in
    every product; rows in no group are neither read nor written."""
    rng = _rng(10)
    rows, G, N, K = 90, 3, 136, 200
    x, w, dy, _ = _case16(rng, "bf16", rows, G, N, K, ())
    off = torch.tensor([3, 20, 61, 80], dtype=torch.int32, device="cuda")
    d = mx.Linear(rows, N, K, groups=G, out_type="f32")
    ws = mx.linear_workspace(d)

    def run(x, w, dy):
        o = [torch.full(s, 7.0, device="cuda") for s in ((rows, N), (rows, K), (G, N, K))]
        mx.moe_grouped_linear(d, x, w, o[0], ws, offsets=off)
        mx.moe_grouped_linear_dx(d, dy, w, o[1], ws, offsets=off)
        mx.moe_grouped_linear_dw(d, dy, x, o[2], ws, offsets=off)
        torch.cuda.synchronize()
        return o

    clean = run(x, w, dy)
    for t in (x, dy):
        t[20:61], t[:3], t[80:] = float("nan"), float("inf"), float("nan")
    w[1] = float("nan")
    y, dx, dw = run(x, w, dy)
    for got, ref in ((y, clean[0]), (dx, clean[1])):
        assert torch.all(got[:3] == 7.0) and torch.all(got[80:] == 7.0)
        assert torch.equal(got[3:20], ref[3:20]) and torch.equal(got[61:], ref[61:])
        assert torch.all(torch.isnan(got[20:61]))
    assert torch.equal(dw[0], clean[2][0]) and torch.equal(dw[2], clean[2][2]) and torch.all(torch.isnan(dw[1]))


def test_no_rows():
    for G in (1, 3):
        off = None if G == 1 else torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        d = mx.Linear(0, 72, 80, groups=G, out_type="f32")
        e = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        w = torch.zeros(G, 72, 80, dtype=torch.bfloat16, device="cuda")
        ws = mx.linear_workspace(d)
        mx.moe_grouped_linear(d, e(80), w, torch.empty(0, 72, device="cuda"), ws, offsets=off)
        mx.moe_grouped_linear_dx(d, e(72), w, torch.empty(0, 80, device="cuda"), ws, offsets=off)
        dw = torch.full((G, 72, 80), 7.0, device="cuda")
        mx.moe_grouped_linear_dw(d, e(72), e(80), dw, ws, offsets=off)
        assert torch.all(dw == 0)
    q = torch.empty(0, 128, dtype=torch.uint8, device="cuda")
    mx.moe_fp8_quant(torch.empty(0, 128, device="cuda"), q, torch.empty(0, 1, device="cuda"))


# Few tiles and a long reduction: it is split over blocks, whose partial sums a
# second kernel joins.
SPLIT = [(40, 1, 131, 6160), (77, 2, 257, 3088), (33, 3, 50, 7024)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows,groups,N,K", SPLIT)
def test_split_fp8(rows, groups, N, K, out):
    _say(f"[case] split fp8 rows={rows} groups={groups} N={N} K={K} out={out}")
    c = _fp8_case(_rng(17, rows, groups, N, K), rows, groups, N, K)
    y = _run_fp8(*c, out=out)
    ref, tol = ol.fp8_linear(_np(c[0].float()), c[1].astype(float), _np(c[2].float()), c[3].astype(float), c[4])
    _check(_np(y), ref, tol, T[out])


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows,groups,N,K", [(40, 2, 136, 4104), (40, 2, 4104, 136), (6000, 1, 64, 72), (5000, 2, 72, 64),
                                             (60, 1, 72, 8200)])
def test_split_grouped(rows, groups, N, K, out):
    """Rows outside every group keep their values here too."""
    _say(f"[case] split grouped rows={rows} groups={groups} N={N} K={K} out={out}")
    rng = _rng(18, rows, groups, N, K)
    x, w, dy, _ = _case16(rng, "bf16", rows, groups, N, K, ())
    off = np.array([5, rows - 3] if groups == 1 else [5, rows // 3, rows - 3], np.int32)
    d = mx.Linear(rows, N, K, groups=groups, out_type=out)
    ws, do = mx.linear_workspace(d), _dev_off(off)
    ws.fill_(0xFF)
    y, dx = (torch.full((rows, n), 7.0, dtype=T[out], device="cuda") for n in (N, K))
    dw = torch.full((groups, N, K), 7.0, dtype=T[out], device="cuda")
    mx.moe_grouped_linear(d, x, w, y, ws, offsets=do)
    mx.moe_grouped_linear_dx(d, dy, w, dx, ws, offsets=do)
    mx.moe_grouped_linear_dw(d, dy, x, dw, ws, offsets=do)
    torch.cuda.synchronize()
    for got, (ref, tol) in ((y, ol.grouped(_np(x), _np(w), off)), (dx, ol.grouped_dx(_np(dy), _np(w), off))):
        assert torch.all(got[:5] == 7.0) and torch.all(got[-3:] == 7.0)
        _check(_np(got)[5:-3], ref[5:-3], tol[5:-3], T[out])
    _check(_np(dw), *ol.grouped_dw(_np(dy), _np(x), groups, off), T[out])


def test_offsets_outside_the_rows_touch_nothing_outside():
    """Offsets that break the contract are clamped: the launch stays inside
    the tensors (no value is promised), and rows past `rows` keep theirs."""
    rows, G, N, K = 40, 3, 64, 64
    x, w, dy, _ = _case16(_rng(11), "bf16", rows + 64, G, N, K, ())
    d = mx.Linear(rows, N, K, groups=G, out_type="f32")
    ws = mx.linear_workspace(d)
    for o in ([-5, 10, 1000, 2000], [30, 10, 5, 100], [2 ** 31 - 1, 0, -2 ** 31, 40]):
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        y = torch.full((rows + 64, N), 7.0, device="cuda")
        dx = torch.full((rows + 64, K), 7.0, device="cuda")
        dw = torch.full((G + 1, N, K), 7.0, device="cuda")
        mx.moe_grouped_linear(d, x, w, y, ws, offsets=off)
        mx.moe_grouped_linear_dx(d, dy, w, dx, ws, offsets=off)
        mx.moe_grouped_linear_dw(d, dy, x, dw, ws, offsets=off)
        torch.cuda.synchronize()
        assert torch.all(y[rows:] == 7.0) and torch.all(dx[rows:] == 7.0) and torch.all(dw[G:] == 7.0)


def test_same_bits_again_and_on_another_stream():
    rng = _rng(12)
    c = _fp8_case(rng, 150, 3, 260, 272)
    a = _run_fp8(*c, out="f32")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    assert torch.equal(a, _run_fp8(*c, out="f32")) and torch.equal(a, _run_fp8(*c, out="f32", stream=st))


def test_calls_in_a_captured_graph():
    """quantise + fp8 product and the 16-bit forward with both gradients in one
    graph, replayed on new inputs with eager work in between."""
    rng = _rng(13)
    rows, G, N, K = 100, 4, 136, 208
    off = torch.tensor([0, 30, 30, 77, 100], dtype=torch.int32, device="cuda")
    _, _, wq, wsc, _ = _fp8_case(rng, 4, G, N, K)
    wq, wsc = wq.cuda(), _t(wsc)
    x, w, dy, _ = _case16(rng, "bf16", rows, G, N, K, ())
    d8 = mx.Linear(rows, N, K, groups=G, in_type="fp8")
    d = mx.Linear(rows, N, K, groups=G)
    s8, s = mx.linear_workspace(d8), mx.linear_workspace(d)
    o = dict(q=torch.empty(rows, K, dtype=torch.float8_e4m3fn, device="cuda"), qs=torch.empty(rows, 2, device="cuda"),
             y8=torch.empty(rows, N, dtype=torch.bfloat16, device="cuda"), y=torch.empty_like(dy),
             dx=torch.empty_like(x), dw=torch.empty_like(w))

    def step(o):
        mx.moe_fp8_quant(x, o["q"], o["qs"])
        mx.moe_fp8_linear(d8, o["q"], o["qs"], wq, wsc, o["y8"], s8, offsets=off)
        mx.moe_grouped_linear(d, x, w, o["y"], s, offsets=off)
        mx.moe_grouped_linear_dx(d, dy, w, o["dx"], s, offsets=off)
        mx.moe_grouped_linear_dw(d, dy, x, o["dw"], s, offsets=off)

    step(o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(o)
    for i in range(3):
        x.copy_(_t(_rng(14, i).standard_normal((rows, K)), torch.bfloat16))
        dy.copy_(_t(_rng(15, i).standard_normal((rows, N)), torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        e = {k: torch.empty_like(v) for k, v in o.items()}
        step(e)
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k].view(torch.uint8), e[k].view(torch.uint8)), k
