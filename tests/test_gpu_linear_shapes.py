"""GPU tests of every block shape of the linear operators, long enough that a
pipeline's steady state runs, against exact references.

All values are integers of at most 3 times a power of two per row, and fp8 scales
are powers of two drawn for each block, so that every f32 sum is exact (at most
9 K, times the scales' 2^-2 to 2^2: under 2^24 steps) and the outputs are the exact
product, rounded once.  Odd rows are scaled down to the type's subnormal values.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from tests import linear_cases as lc

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
FILL = 0.5
# a power of two at which integers to 3 are subnormal (bf16 has f32's range: none that sums stay exact in)
TINY = {"fp8": 2.0 ** -9, "f16": 2.0 ** -24, "bf16": 2.0 ** -30}


def _ints(g, *shape):
    return torch.randint(-3, 4, shape, generator=g, device="cuda", dtype=torch.int8)


def _pow2(g, *shape):
    return torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float())


def _offsets(rows, groups, seed):
    """Ragged groups; where there are enough rows, two before the first and three after the last belong to none."""
    rng = np.random.default_rng((rows, groups, seed))
    lead, trail = (2, 3) if rows >= 20 else (0, 0)
    n = rng.multinomial(rows - lead - trail, rng.dirichlet(np.full(groups, 2.0)))
    return np.concatenate([[lead], lead + np.cumsum(n)]).astype(np.int32).tolist()


def _equal(got, ref, what):
    ref = ref.to(got.dtype)
    if not torch.equal(got, ref):
        bad = (got != ref).nonzero()
        raise AssertionError(f"{what}: {len(bad)} of {got.numel()} differ, first at {bad[0].tolist()}: "
                             f"{float(got[tuple(bad[0])])} for {float(ref[tuple(bad[0])])}")


def _spread(s, n, axis):
    return s.repeat_interleave(128, axis).narrow(axis, 0, n)


def check(kind, rows, groups, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * 7 + groups * 5 + N * 3 + K)
    off = [0, rows] if rows < 20 and groups == 1 else _offsets(rows, groups, N + K)
    dev = torch.tensor(off, dtype=torch.int32, device="cuda")
    spans = list(zip(off, off[1:]))
    w = _ints(g, groups, N, K) if kind != "dw" else None
    a = _ints(g, rows, N if kind == "dx" else K)
    b = _ints(g, rows, N) if kind == "dw" else None
    shape = {"fp8": (rows, N), "fwd": (rows, N), "dx": (rows, K), "dw": (groups, N, K)}[kind]
    nb = -(-K // 128)
    for t in ("fp8",) if kind == "fp8" else ("bf16", "f16"):
        tiny = torch.where(torch.arange(rows, device="cuda") % 2 == 1, TINY[t], 1.0)[:, None]
        x = a.float() if kind == "dw" else a.float() * tiny
        ref = torch.full(shape, FILL, dtype=torch.float64, device="cuda")
        if kind == "fp8":
            xs, ws = _pow2(g, rows, nb), _pow2(g, groups, -(-N // 128), nb)
        for i, (lo, hi) in enumerate(spans):
            xi = x[lo:hi].double()
            if kind == "dw":
                ref[i] = b[lo:hi].double().t() @ xi
                continue
            if hi == lo:
                continue
            wi = w[i].double()
            if kind == "fp8":
                xi *= _spread(xs[lo:hi], K, 1)
                wi *= _spread(_spread(ws[i], N, 0), K, 1)
            ref[lo:hi] = xi @ (wi if kind == "dx" else wi.t())
        for out in ("f32", "bf16" if t == "fp8" else t):
            d = mx.Linear(rows, N, K, groups=groups, in_type=t, out_type=out)
            y = torch.full(shape, FILL, dtype=T[out], device="cuda")
            scratch = mx.linear_workspace(d).fill_(0xFF)   # NaN bits: nothing of it may be taken as cleared
            xt = x.to(T[t])
            if kind == "fp8":
                mx.moe_fp8_linear(d, xt, xs, w.float().to(T[t]), ws, y, scratch, offsets=dev)
            elif kind == "fwd":
                mx.moe_grouped_linear(d, xt, w.to(T[t]), y, scratch, offsets=dev)
            elif kind == "dx":
                mx.moe_grouped_linear_dx(d, xt, w.to(T[t]), y, scratch, offsets=dev)
            else:
                mx.moe_grouped_linear_dw(d, b.to(T[t]), xt, y, scratch, offsets=dev)
            torch.cuda.synchronize()
            _equal(y, ref, f"{t} -> {out}")


@pytest.mark.parametrize("kind,case", [(k, c) for k in lc.SHAPES for c in lc.SHAPES[k]],
                         ids=lambda v: v if isinstance(v, str) else "-".join(map(str, v)))
def test_every_shape(kind, case):
    print(f"[case] {kind} shape {case[0]}: rows={case[1]} groups={case[2]} N={case[3]} K={case[4]}", flush=True)
    check(kind, *case[1:])


@pytest.mark.parametrize("kind,case", [(k, c) for k in lc.STREAMED for c in lc.STREAMED[k]],
                         ids=lambda v: v if isinstance(v, str) else "-".join(map(str, v)))
def test_every_shape_with_weights_that_stream(kind, case):
    """Over 100 MiB of weights: another instance of the main loop, with the
    streaming cache policy on the weights' loads."""
    print(f"[case] {kind} shape {case[0]}: rows={case[1]} groups={case[2]} N={case[3]} K={case[4]}", flush=True)
    check(kind, *case[1:])
