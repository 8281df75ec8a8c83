"""The calls of the operators for unquantised experts by the native checks and by
those in Python: the same bits, and refusals that name what is wrong."""

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx

pytestmark = pytest.mark.gpu


def _r(*s, t=torch.bfloat16):
    return torch.randn(*s, device="cuda").to(t)


class Calls:
    """Every operator with tensors that fit; outputs in the order of `run`."""

    def __init__(self):
        torch.manual_seed(0)
        rows, G, N, K = 21, 3, 48, 64
        self.d = mx.Linear(rows, N, K, groups=G)
        self.off = torch.tensor([0, 9, 9, 21], dtype=torch.int32, device="cuda")
        self.x, self.w, self.b, self.r, self.dy = _r(rows, K), _r(G, N, K), _r(G, N), _r(rows, N // 2), _r(rows, N // 2)
        self.ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        self.y, self.pre, self.dz = (torch.empty(rows, n, dtype=torch.bfloat16, device="cuda") for n in (N // 2, N, N))
        self.db = torch.empty(G, N, device="cuda")
        self.grads = [_r(100), _r(77, t=torch.float32)]
        self.outs = [torch.empty_like(g) for g in self.grads]
        self.norm, self.norm2 = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        E, k, T = 6, 2, 5
        self.dims = mx.Dims(T=T, T_max=T, H=128, F=128, E=E, k=k, P_total=E, p0=0, P_local=E, R_max=1)
        self.lx, self.lg, self.w1, self.w2 = _r(T, 128), _r(T, E, t=torch.float32), _r(E, 256, 128), _r(E, 128, 128)
        self.rc = torch.ones(E, dtype=torch.int32, device="cuda")
        self.rs = torch.arange(E, dtype=torch.int32, device="cuda")
        self.out, self.hist = torch.empty(T, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
        self.lws = mx.a16w16_workspace(self.dims)

    def fwd(self, **kw):
        a = {**dict(x=self.x, w=self.w, y=self.y, scratch=self.ws, act="silu", gated=True, bias=self.b, residual=self.r,
                    pre=self.pre, offsets=self.off), **kw}
        mx.moe_grouped_linear_act(self.d, **a)

    def bwd(self, **kw):
        a = {**dict(dy=self.dy, pre=self.pre, dz=self.dz, scratch=self.ws, act="silu", gated=True, db=self.db,
                    offsets=self.off), **kw}
        mx.moe_grouped_linear_act_backward(self.d, **a)

    def layer(self, **kw):
        a = {**dict(x=self.lx, logits=self.lg, w1=self.w1, w2=self.w2, rep_count=self.rc, rep_slots=self.rs, out=self.out,
                    ws=self.lws, load_hist=self.hist), **kw}
        mx.moe_forward_a16w16(self.dims, **a)

    def run(self):
        self.hist.zero_()
        self.fwd()
        self.bwd()
        h = mx.GradList(self.grads, self.outs)
        mx.moe_grad_clip(h, 1.0, self.norm, self.ws)
        mx.moe_grad_norm(h, self.norm2, self.ws)
        self.layer()
        torch.cuda.synchronize()
        return [t.clone() for t in (self.y, self.pre, self.dz, self.db, *self.outs, self.norm, self.norm2, self.out, self.hist)]


def test_native_and_python_checks_give_the_same(monkeypatch):
    c = Calls()
    assert mx._short() is not mx._PythonChecks
    a = c.run()
    monkeypatch.setattr(mx, "_bind_module", mx._PythonChecks)
    for x, y in zip(a, c.run()):
        assert torch.equal(x, y)


@pytest.mark.parametrize("python", [False, True])
def test_refusals_name_the_argument(python, monkeypatch):
    c = Calls()
    if python:
        monkeypatch.setattr(mx, "_bind_module", mx._PythonChecks)
    f = c.x.float()
    for kw, what in ((dict(x=f), "x: dtype"), (dict(w=c.w[:2]), "w: "), (dict(y=c.y[:3]), "y: "), (dict(bias=f), "bias: dtype"),
                     (dict(residual=c.r.t().contiguous().t()), "residual: must be contiguous"), (dict(pre=c.y), "pre: "),
                     (dict(offsets=c.off.long()), "offsets: dtype"), (dict(x=c.x.cpu()), "x: must be a device")):
        with pytest.raises((TypeError, ValueError), match=what):
            c.fwd(**kw)
    for kw, what in ((dict(dy=f), "dy: dtype"), (dict(pre=c.y), "pre: "), (dict(db=c.db.bfloat16()), "db: dtype"),
                     (dict(db=c.db[:1]), "db: "), (dict(dz=c.y), "dz: ")):
        with pytest.raises((TypeError, ValueError), match=what):
            c.bwd(**kw)
    for kw, what in ((dict(w1=c.w1[:3]), "w1: "), (dict(w2=c.w2.half()), "w2: dtype"), (dict(logits=c.lg[:2]), "logits: "),
                     (dict(out=c.out.float()), "out: dtype"), (dict(num_tokens=c.off.long()), "num_tokens: dtype"),
                     (dict(load_hist=c.hist[:2]), "load_hist: ")):
        with pytest.raises((TypeError, ValueError), match=what):
            c.layer(**kw)
    with pytest.raises(mx.MoeError):
        c.layer(ws=c.lws[:64])
    with pytest.raises(mx.MoeError):
        mx.moe_grad_clip(mx.GradList(c.grads), -1.0, c.norm, c.ws)
    with pytest.raises((ValueError, TypeError)):
        mx.moe_grad_clip(mx.GradList(c.grads), 1.0, c.norm.double(), c.ws)


def test_two_captured_graphs_with_their_own_workspaces():
    """Two graphs of the whole run, replayed in turn with eager calls in between."""
    a, b = Calls(), Calls()
    b.x.copy_(b.x * 0.5)
    b.lx.copy_(b.lx * 0.5)
    want = [a.run(), b.run()]
    lists = [mx.GradList(c.grads, c.outs) for c in (a, b)]

    def body(c, h):
        c.fwd()
        c.bwd()
        mx.moe_grad_clip(h, 1.0, c.norm, c.ws)
        mx.moe_grad_norm(h, c.norm2, c.ws)
        c.layer(load_hist=None)

    graphs = []
    for c, h in zip((a, b), lists):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            body(c, h)
        graphs.append(g)
    for i in range(4):
        for c, g, ref in ((a, graphs[0], want[0]), (b, graphs[1], want[1])):
            for t in (c.y, c.pre, c.dz, c.db, *c.outs, c.norm, c.norm2, c.out):
                t.fill_(7.0)
            g.replay()
            Calls().run()   # eager work of the same kind on other tensors
            torch.cuda.synchronize()
            got = [c.y, c.pre, c.dz, c.db, *c.outs, c.norm, c.norm2, c.out]
            assert all(torch.equal(x, y) for x, y in zip(got, ref)), i


def test_two_calls_at_once_on_two_streams():
    a, b = Calls(), Calls()
    want = [a.run(), b.run()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for c, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                c.fwd()
                c.bwd()
                mx.moe_grad_clip(mx.GradList(c.grads, c.outs), 1.0, c.norm, c.ws)
                c.layer(load_hist=None)
    torch.cuda.synchronize()
    for c, ref in zip((a, b), want):
        got = [c.y, c.pre, c.dz, c.db, *c.outs, c.norm, c.norm2, c.out]
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
    assert np.isfinite(float(a.norm))
