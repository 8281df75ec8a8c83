"""GPU tests of the layer on 16-bit experts for a few tokens, against the float64
oracle: routing, remap and record bit-exact, outputs within the oracle's bound
plus the output's rounding."""

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from oracle import experts as oe
from oracle import moe as om

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16}


def _say(*a):
    print(*a, flush=True)


def _np(t):
    return t.detach().cpu().double().numpy()


class Case:
    def __init__(self, n, H, F, E, k, p0=0, local=None, replicas=1, total=None, dt="bf16", base=0, seed=0, T_max=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 1000 + n * 7 + H + F + E + k)
        r = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
        P = E * replicas if total is None else total
        local = P - p0 if local is None else local
        self.d = mx.Dims(T=n, T_max=T_max or n, H=H, F=F, E=E, k=k, P_total=P, p0=p0, P_local=local, R_max=max(replicas, 1),
                         token_id_base=base)
        self.dt = T[dt]
        self.x, self.logits = r(n, H).to(self.dt), r(n, E)
        self.w1 = (r(local, 2 * F, H, std=1.5 / H ** 0.5)).to(self.dt)
        self.w2 = (r(local, H, F, std=1.0 / F ** 0.5)).to(self.dt)
        rng = np.random.default_rng(seed)
        self.rc = rng.integers(1, replicas + 1, E).astype(np.int32)
        slots = rng.permutation(P)[:E * replicas].reshape(E, replicas).astype(np.int32)
        self.rs = np.where(np.arange(replicas)[None] < self.rc[:, None], slots, -1).astype(np.int32)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.drc, self.drs = t(self.rc), t(self.rs)
        self.out = torch.full((n, H), 7.0, dtype=self.dt, device="cuda")
        self.hist = torch.full((P,), 3, dtype=torch.int32, device="cuda")
        z = lambda dt_: torch.full((max(n * k, 1),), -5, dtype=dt_, device="cuda")  # noqa: E731
        self.taps = dict(topk_ids=z(torch.int32), topk_w=z(torch.float32), phys_ids=z(torch.int32))
        self.ws = mx.a16w16_workspace(self.d)
        self.ws.fill_(0xFF)

    def run(self, out=None, hist=True, taps=True, **kw):
        mx.moe_forward_a16w16(self.d, self.x, self.logits, self.w1, self.w2, self.drc, self.drs,
                              self.out if out is None else out, self.ws, load_hist=self.hist if hist else None,
                              taps=self.taps if taps else None, **kw)

    def ref(self, n=None):
        n = self.d.T if n is None else n
        d = self.d
        lg = self.logits[:n].cpu().numpy()
        ids = np.argsort(-lg, axis=1, kind="stable")[:, :d.k]
        s = 1.0 / (1.0 + np.exp(-np.take_along_axis(lg, ids, 1).astype(np.float64)))
        w = s / s.sum(1, keepdims=True)
        phys = np.empty_like(ids)
        for t in range(n):
            h = int(om.fmix32(np.uint32((d.token_id_base + t) & 0xFFFFFFFF)))
            for j in range(d.k):
                e = ids[t, j]
                phys[t, j] = self.rs[e, h % int(self.rc[e])]
        out, tol = oe.layer(_np(self.x[:n]), _np(self.w1), _np(self.w2), phys, w, d.p0, torch.finfo(self.dt).eps)
        return ids, w, phys, out, tol

    def check(self, n=None):
        n = self.d.T if n is None else n
        k = self.d.k
        ids, w, phys, out, tol = self.ref(n)
        torch.cuda.synchronize()
        tap = {a: v.cpu().numpy()[:n * k].reshape(n, k) for a, v in self.taps.items()}
        assert np.array_equal(tap["topk_ids"], ids) and np.array_equal(tap["phys_ids"], phys)
        assert np.all(np.abs(tap["topk_w"] - w) <= 4e-6 * w)
        hist = 3 + np.bincount(phys.reshape(-1), minlength=self.d.P_total)
        assert np.array_equal(self.hist.cpu().numpy(), hist)
        got = _np(self.out)
        fi = torch.finfo(self.dt)
        bound = tol + fi.eps / 2 * (np.abs(out) + tol) + fi.smallest_normal * fi.eps / 2
        assert np.all(np.isfinite(got))
        worst = np.max(np.abs(got[:n] - out) / np.maximum(bound, 1e-300), initial=0.0) if n else 0.0
        assert np.all(np.abs(got[:n] - out) <= bound), f"worst {worst:.3g} of the bound"
        assert np.all(got[n:] == 0.0)
        _say(f"   ok: worst error {worst:.3g} of the bound")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 2, 4, 5, 15, 16, 17, 31, 32])
def test_token_counts(n, dt):
    _say(f"[case] layer T={n} {dt}")
    c = Case(n, 256, 128, 8, 2, dt=dt)
    c.run()
    c.check()


@pytest.mark.parametrize("H,F", [(128, 128), (128, 640), (384, 256), (1152, 384), (2176, 128), (512, 2048), (16384, 128),
                                 (128, 16384)])
@pytest.mark.parametrize("n", [1, 7, 20])
def test_widths(H, F, n):
    _say(f"[case] layer T={n} H={H} F={F}")
    c = Case(n, H, F, 6, 3)
    c.run()
    c.check()


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (16, 16), (64, 6), (65, 1), (128, 8), (129, 3), (384, 6), (385, 16), (1024, 4)])
@pytest.mark.parametrize("n", [3, 32])
def test_experts(E, k, n):
    _say(f"[case] layer T={n} E={E} k={k}")
    c = Case(n, 128, 128, E, k, seed=E)
    c.run()
    c.check()


@pytest.mark.parametrize("n", [1, 9, 32])
def test_share_with_replicas(n):
    """Half the slots on other GPUs, up to three replicas an expert, a token base."""
    c = Case(n, 256, 256, 24, 4, p0=20, local=30, replicas=3, base=0xFFFFFFF0, seed=4)
    c.run()
    c.check()


def test_no_local_pairs_and_no_tokens():
    c = Case(5, 256, 128, 16, 2, p0=8, local=8)
    c.logits[:, 8:] = -50.0
    c.run()
    c.check()
    assert torch.all(c.out == 0)
    d = mx.Dims(T=0, T_max=8, H=256, F=128, E=16, k=2, P_total=16, p0=8, P_local=8, R_max=1)
    before = c.out.fill_(7.0)
    mx.moe_forward_a16w16(d, c.x[:0], c.logits[:0], c.w1, c.w2, c.drc, c.drs, c.out[:0], mx.a16w16_workspace(d))
    torch.cuda.synchronize()
    assert torch.all(before == 7.0)


def test_all_tokens_on_one_expert():
    for n in (16, 17, 32):
        c = Case(n, 384, 256, 12, 2)
        c.logits[:, 5] += 20.0
        c.run()
        c.check()


def test_equal_logits_go_to_the_lower_expert():
    c = Case(6, 128, 128, 40, 5)
    c.logits.fill_(0.25)
    c.run()
    torch.cuda.synchronize()
    assert np.array_equal(c.taps["topk_ids"].cpu().numpy().reshape(6, 5), np.tile(np.arange(5), (6, 1)))


def test_routing_is_the_layer_s():
    c = Case(32, 128, 128, 384, 6)
    c.run()
    ids = torch.zeros(32 * 6, dtype=torch.int32, device="cuda")
    w = torch.zeros(32 * 6, device="cuda")
    mx.moe_route(c.d, c.logits, ids, w)
    assert torch.equal(ids, c.taps["topk_ids"]) and torch.equal(w, c.taps["topk_w"])


def test_same_bits_again_and_on_another_stream():
    c = Case(32, 512, 384, 12, 3, seed=3)
    c.run()
    whole = c.out.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.run(out=c.out.zero_(), stream=st)
    st.synchronize()
    assert torch.equal(c.out, whole)
    c.run(hist=False, taps=False)
    assert torch.equal(c.out, whole)


def test_one_graph_for_every_token_count():
    n = 32
    c = Case(n, 256, 128, 16, 4, T_max=64, seed=6)
    count = torch.full((1,), n, dtype=torch.int32, device="cuda")
    c.run(num_tokens=count)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(num_tokens=count)
    for m in (32, 1, 17, 0, 4, 5, -3, 100):
        count.fill_(m)
        c.x.copy_(torch.randn(n, 256, device="cuda"))
        c.logits.copy_(torch.randn(n, 16, device="cuda"))
        c.hist.fill_(3)
        c.out.fill_(7.0)
        g.replay()
        v = min(max(m, 0), n)
        c.check(v)
        assert torch.all(c.taps["phys_ids"].view(n, 4)[v:] == -1)


def test_nan_of_one_token_stays_with_it():
    c = Case(20, 256, 128, 8, 2, seed=8)
    c.run()
    clean = c.out.clone()
    c.x[7] = float("nan")
    c.run()
    torch.cuda.synchronize()
    assert torch.all(torch.isnan(c.out[7]))
    keep = [t for t in range(20) if t != 7]
    assert torch.equal(c.out[keep], clean[keep])


def test_far_gates_and_f16_overflow():
    """silu of very negative gates is zero, not NaN; an f16 act beyond 65504 is infinite."""
    c = Case(2, 128, 128, 2, 1, dt="f16")
    c.logits[:] = torch.tensor([1.0, 0.0])
    c.x.fill_(1.0)
    c.w1.zero_()
    c.w1[0, :128, 0], c.w1[0, 128:, 0] = -200.0, 1.0
    c.run()
    assert torch.all(c.out == 0)
    c.w1[0, :128, 0], c.w1[0, 128:, 0] = 1000.0, 1000.0
    c.w2.fill_(1.0)
    c.run()
    assert torch.all(torch.isinf(c.out))


@pytest.mark.parametrize("n,H,F", [(3, 128, 128), (3, 2176, 256), (20, 256, 512), (20, 2176, 2048), (16, 8320, 1024)])
def test_weights_of_an_expert_that_are_not_finite_stay_with_its_tokens(n, H, F):
    """A token's output is a sum over its own experts; 0 times another's infinity has no place in it."""
    c = Case(n, H, F, 6, 2, seed=9)
    c.run()
    ids = c.taps["topk_ids"].view(n, 2)
    bad = int(ids[0, 0])
    slot = int(c.rs[bad, 0])
    clean = c.out.clone()
    c.w2[slot, ::3] = float("inf")
    c.w2[slot, 1::3] = float("nan")
    c.run()
    torch.cuda.synchronize()
    hit = (ids == bad).any(dim=1)
    assert hit.any() and not hit.all()
    assert torch.equal(c.out[~hit], clean[~hit])
    assert not torch.isfinite(c.out[hit][:, 0]).any() and torch.isnan(c.out[hit][:, 1::3]).all()
