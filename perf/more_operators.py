"""Cases and plain forms of the library's operators for unquantised experts.

* the 16-bit products by expert with bias, activation (gated or not) and
  residual in their epilogue, and the gradient through that epilogue;
* the global gradient norm over many tensors, and clipping by it;
* the whole expert layer on 16-bit experts for a few tokens.

``run`` computes a case in its plain form (elementary torch operations in
32 bits, long sums in 64) or, where ``own`` is true, with the library's calls;
``exact`` computes it in 64 bits from the operators' definitions.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

W_STD = 0.02   # weight deviation of the library's synthetic workloads

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    """Widths 7168 / 2048 with 48 local of 384 experts, top-6, are the library's
    benchmark layer, 256 / 128 with 8 experts, top-2, its tiny workload."""
    return [
        # down projection of a dense layer for one decoded token, added to the residual stream
        dict(name="act_token", op="act", rows=1, groups=0, N=7168, K=2048, skew=0.0, act="none", gated=False, bias=True,
             residual=True, pre=False, dtype="bf16", out="bf16"),
        # a short ragged batch on widths that fill no tile, everything in the epilogue
        dict(name="act_ragged", op="act", rows=77, groups=3, N=2042, K=7152, skew=0.5, act="gelu", gated=True, bias=True,
             residual=True, pre=True, dtype="f16", out="f16"),
        # gate and up projection of 48 local experts in a decode step, SwiGLU
        dict(name="act_experts_decode", op="act", rows=384, groups=48, N=4096, K=7168, skew=0.0, act="silu", gated=True,
             bias=False, residual=False, pre=False, dtype="bf16", out="bf16"),
        # the same in a fine-tuning step with uneven loads; the values before SwiGLU are kept for the gradient
        dict(name="act_experts_train", op="act", rows=6144, groups=48, N=4096, K=7168, skew=0.5, act="silu", gated=True,
             bias=True, residual=False, pre=True, dtype="bf16", out="bf16"),
        # gradient through bias and activation: small odd sizes with an empty group
        dict(name="act_backward_odd", op="act_backward", rows=250, groups=9, N=264, skew=3.0, act="gelu_tanh",
             gated=False, bias=True, dtype="f16", out="f16"),
        # ... and through SwiGLU for the rows of 8192 tokens, six experts each
        dict(name="act_backward", op="act_backward", rows=49152, groups=48, N=4096, skew=0.5, act="silu", gated=True,
             bias=True, dtype="bf16", out="bf16"),
        # clipping the gradients of two tiny layers, tensor by tensor: launch latency
        dict(name="clip_tiny", op="clip", layers=2, experts=8, H=256, F=128, dtype="mixed", max_norm=1.0),
        # clipping f32 gradients of twelve experts
        dict(name="clip_experts", op="clip", layers=1, experts=12, H=7168, F=2048, dtype="f32", max_norm=1.0),
        # one token through the tiny layer: launch latency
        dict(name="layer_tiny", op="layer", T=1, H=256, F=128, E=8, k=2, p0=0, local=8, dtype="bf16"),
        # one token through a layer whose 48 experts are all on this GPU
        dict(name="layer_token", op="layer", T=1, H=7168, F=2048, E=48, k=6, p0=0, local=48, dtype="bf16"),
        # 32 tokens of a data-parallel decode step on this GPU's 48 of 384 experts
        dict(name="layer_share", op="layer", T=32, H=7168, F=2048, E=384, k=6, p0=48, local=48, dtype="bf16"),
        # 16 tokens with all 48 experts here: nearly every expert is read
        dict(name="layer_decode", op="layer", T=16, H=7168, F=2048, E=48, k=6, p0=0, local=48, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["act", "act", "act", "act_backward", "act_backward", "clip", "layer", "layer"])
    if op == "act":
        dtype = rng.choice(["bf16", "f16"])
        gated = rng.random() < 0.5
        n = _log_int(rng, 32, 4096)
        return dict(op="act", rows=_log_int(rng, 1, 6144), groups=rng.choice([0, rng.randint(1, 48)]),
                    N=n - n % 2 if gated else n, K=8 * _log_int(rng, 8, 896), skew=rng.choice([0.0, 0.5, 1.5]),
                    act=rng.choice(ACTS), gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    pre=rng.random() < 0.5, dtype=dtype, out=rng.choice([dtype, dtype, "f32"]))
    if op == "act_backward":
        dtype = rng.choice(["bf16", "f16"])
        return dict(op="act_backward", rows=_log_int(rng, 1, 49152), groups=rng.choice([0, rng.randint(1, 48)]),
                    N=8 * _log_int(rng, 8, 512), skew=rng.choice([0.0, 0.5, 1.5]), act=rng.choice(ACTS),
                    gated=rng.random() < 0.5, bias=rng.random() < 0.7, dtype=dtype, out=rng.choice([dtype, dtype, "f32"]))
    if op == "clip":
        return dict(op="clip", layers=rng.randint(1, 4), experts=rng.randint(1, 12), H=_log_int(rng, 33, 3500),
                    F=_log_int(rng, 17, 1000), dtype=rng.choice(["bf16", "f16", "f32", "mixed"]),
                    max_norm=rng.choice([0.1, 1.0, 1e6]))
    E = _log_int(rng, 4, 384)
    T, k, local = _log_int(rng, 1, 32), rng.randint(1, min(E, 8)), rng.randint(1, min(E, 48))
    if T * k * local < 4 * E:   # too few pairs expected here: all experts on this GPU
        E = local = max(local, k)
    return dict(op="layer", T=T, H=128 * _log_int(rng, 1, 56), F=128 * _log_int(rng, 1, 16), E=E, k=k,
                p0=rng.randint(0, E - local), local=local, dtype=rng.choice(["bf16", "f16"]))


def _sizes(case):
    """Rows of each group before shuffling: shares proportional to
    (i + 1)^-skew, rounded so that they add up."""
    g = max(case["groups"], 1)
    w = [(i + 1.0) ** -case["skew"] for i in range(g)]
    shares = [case["rows"] * v / sum(w) for v in w]
    n = [int(v) for v in shares]
    order = sorted(range(g), key=lambda i: (n[i] - shares[i], i))
    for i in order[:case["rows"] - sum(n)]:
        n[i] += 1
    return n


def _tensors(case):
    """(elements, type) of the gradients of a case of clipping: per layer a norm,
    a router gate, and each expert's two matrices and biases."""
    H, F, G = case["H"], case["F"], case["experts"]
    big, small = ("bf16", "f32") if case["dtype"] == "mixed" else (case["dtype"], case["dtype"])
    layer = [(H, small), (G * H, small)] + [(2 * F * H, big), (2 * F, small), (H * F, big), (H, small)] * G
    return layer * case["layers"]


def _half(case):
    """Columns of the result of a product's epilogue."""
    return case["N"] // 2 if case["gated"] else case["N"]


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)

    op, st = case["op"], dict(case=case)
    if op == "clip":
        st["grads"] = [normal(n, std=1e-2, dtype=TYPES[t]) for n, t in _tensors(case)]
        return st
    dt = TYPES[case["dtype"]]
    if op == "layer":
        T, H, F, E, L = (case[n] for n in ("T", "H", "F", "E", "local"))
        st["x"], st["logits"] = normal(T, H, dtype=dt), normal(T, E)
        st["w1"] = torch.empty(L, 2 * F, H, dtype=dt, device="cuda")
        st["w2"] = torch.empty(L, H, F, dtype=dt, device="cuda")
        for i in range(L):
            st["w1"][i] = normal(2 * F, H, std=W_STD, dtype=dt)
            st["w2"][i] = normal(H, F, std=W_STD, dtype=dt)
        return st
    rows, N, groups = case["rows"], case["N"], max(case["groups"], 1)
    if case["groups"]:
        hg = torch.Generator()
        hg.manual_seed(seed)
        n = _sizes(case)
        bounds = [0]
        for i in torch.randperm(groups, generator=hg).tolist():
            bounds.append(bounds[-1] + n[i])
        st["offsets"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    else:
        bounds = [0, rows]
        st["offsets"] = None
    st["bounds"] = bounds  # the host's copy, for the plain form's loop
    out = TYPES[case["out"]]
    if op == "act_backward":
        st["dy"], st["z"] = normal(rows, _half(case), dtype=out), normal(rows, N, std=1.5, dtype=out)
        return st
    K = case["K"]
    st["x"] = normal(rows, K, dtype=dt)
    st["w"] = torch.empty(groups, N, K, dtype=dt, device="cuda")
    for i in range(groups):
        st["w"][i] = normal(N, K, std=W_STD, dtype=dt)
    st["b"] = normal(groups, N, std=0.1, dtype=dt) if case["bias"] else None
    st["r"] = normal(rows, _half(case), dtype=out) if case["residual"] else None
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if not own:
        return st
    import moe_expert_layer_sigmoid_amd as mx

    st["mx"], op = mx, case["op"]
    if op == "clip":
        # the clipped gradients go into one flat buffer per type, as an optimiser keeps them
        names = sorted({t for _, t in _tensors(case)})
        total = {t: sum(n for n, u in _tensors(case) if u == t) for t in names}
        st["flat"] = {t: torch.empty(total[t], dtype=TYPES[t], device="cuda") for t in names}
        at, outs = dict.fromkeys(names, 0), []
        for n, t in _tensors(case):
            outs.append(st["flat"][t][at[t]:at[t] + n])
            at[t] += n
        st["list"] = mx.GradList(st["grads"], outs)
        st["norm"] = torch.empty(1, device="cuda")
        st["scratch"] = mx.grad_workspace(st["list"])
        return st
    if op == "layer":
        E = case["E"]
        st["d"] = mx.Dims(T=case["T"], T_max=case["T"], H=case["H"], F=case["F"], E=E, k=case["k"], P_total=E,
                          p0=case["p0"], P_local=case["local"], R_max=1)
        st["rep_count"] = torch.ones(E, dtype=torch.int32, device="cuda")
        st["rep_slots"] = torch.arange(E, dtype=torch.int32, device="cuda")
        st["out"] = torch.empty_like(st["x"])
        st["scratch"] = mx.a16w16_workspace(st["d"])
        return st
    rows, N, groups, out = case["rows"], case["N"], max(case["groups"], 1), TYPES[case["out"]]
    st["d"] = mx.Linear(rows, N, case.get("K", 64), groups=groups, in_type=case["dtype"], out_type=case["out"])
    if op == "act":
        st["y"] = torch.empty(rows, _half(case), dtype=out, device="cuda")
        st["pre"] = torch.empty(rows, N, dtype=out, device="cuda") if case["pre"] else None
    else:
        st["dz"] = torch.empty(rows, N, dtype=TYPES[case["dtype"]], device="cuda")
        st["db"] = torch.empty(groups, N, device="cuda") if case["bias"] else None
    st["scratch"] = mx.linear_act_workspace(st["d"])
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    mx, case = st["mx"], st["case"]
    op = case["op"]
    if op == "clip":
        mx.moe_grad_clip(st["list"], case["max_norm"], st["norm"], st["scratch"])
        return [st["norm"], st["flat"]]
    if op == "layer":
        mx.moe_forward_a16w16(st["d"], st["x"], st["logits"], st["w1"], st["w2"], st["rep_count"], st["rep_slots"],
                              st["out"], st["scratch"])
        return st["out"]
    if op == "act":
        mx.moe_grouped_linear_act(st["d"], st["x"], st["w"], st["y"], st["scratch"], act=case["act"],
                                  gated=case["gated"], bias=st["b"], residual=st["r"], pre=st["pre"],
                                  offsets=st["offsets"])
        return [st["y"], st["pre"]]
    mx.moe_grouped_linear_act_backward(st["d"], st["dy"], st["z"], st["dz"], st["scratch"], act=case["act"],
                                       gated=case["gated"], db=st["db"], offsets=st["offsets"])
    return [st["dz"], st["db"]]


C_TANH = math.sqrt(2.0 / math.pi)


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(C_TANH * (z + 0.044715 * z * z * z)))
    return z


def _slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        t = torch.tanh(C_TANH * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * C_TANH * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "clip":
        sums = torch.stack([v.float().square().sum(dtype=torch.float64) for v in st["grads"]])
        norm = sums.sum().sqrt().float().reshape(1)
        c = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        flat = {}
        for t in sorted({t for _, t in _tensors(case)}):
            flat[t] = torch.cat([(v.float() * c).to(v.dtype) for v, (_, u) in zip(st["grads"], _tensors(case)) if u == t])
        return [norm, flat]
    if op == "layer":
        F, k = case["F"], case["k"]
        x = st["x"].float()
        # equal logits to the lower expert id
        ids = torch.argsort(st["logits"], dim=1, descending=True, stable=True)[:, :k]
        s = 1.0 / (1.0 + torch.exp(-st["logits"].gather(1, ids)))
        share = s / s.sum(1, keepdim=True)
        out = torch.zeros_like(x)
        slot = ids - case["p0"]
        here = (slot >= 0) & (slot < case["local"])
        for e in torch.unique(slot[here]).tolist():
            t, j = torch.nonzero(slot == e, as_tuple=True)
            h = x[t] @ st["w1"][e].float().t()
            a = _act("silu", h[:, :F]) * h[:, F:]
            out[t] += share[t, j, None] * (a @ st["w2"][e].float().t())
        return out.to(st["x"].dtype)
    rows, N, b = case["rows"], case["N"], st["bounds"]
    out, half = TYPES[case["out"]], N // 2
    if op == "act":
        y = torch.empty(rows, _half(case), dtype=out, device="cuda")
        pre = torch.empty(rows, N, dtype=out, device="cuda") if case["pre"] else None
        for g in range(len(b) - 1):
            if b[g + 1] == b[g]:
                continue
            span = slice(b[g], b[g + 1])
            z = torch.mm(st["x"][span].float(), st["w"][g].float().t())
            if case["bias"]:
                z = z + st["b"][g].float()
            v = _act(case["act"], z[:, :half]) * z[:, half:] if case["gated"] else _act(case["act"], z)
            y[span] = (v + st["r"][span].float() if case["residual"] else v).to(out)
            if case["pre"]:
                pre[span] = z.to(out)
        return [y, pre]
    dy, z = st["dy"].float(), st["z"].float()
    if case["gated"]:
        gate, up = z[:, :half], z[:, half:]
        dz = torch.cat([dy * up * _slope(case["act"], gate), dy * _act(case["act"], gate)], 1)
    else:
        dz = dy * _slope(case["act"], z)
    db = None
    if case["bias"]:
        db = torch.stack([dz[lo:hi].sum(0, dtype=torch.float64) for lo, hi in zip(b, b[1:])]).float()
    return [dz.to(TYPES[case["dtype"]]), db]


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(m for m, _ in _tensors(case))
        return {"bytes": 2 * sum(m * SIZE[t] for m, t in _tensors(case)), "flops": 3 * n}
    if op == "layer":
        T, H, F, k = case["T"], case["H"], case["F"], case["k"]
        share = k / case["E"]   # of a token's choices on one expert
        touched = case["local"] * (1.0 - (1.0 - share) ** T) if T > 1 else case["local"] * share
        pairs = T * share * case["local"]
        return {"bytes": touched * 6 * F * H + T * (4 * H + 4 * case["E"]), "flops": pairs * 6 * F * H}
    rows, N, o, n = case["rows"], case["N"], SIZE[case["out"]], _sizes(case)
    touched = sum(1 for v in n if v)
    if op == "act_backward":
        return {"bytes": rows * (o * (_half(case) + N) + SIZE[case["dtype"]] * N) + (4 * len(n) * N if case["bias"] else 0),
                "flops": 12 * rows * N}
    K = case["K"]
    b = rows * (2 * K + o * _half(case)) + touched * 2 * N * K
    b += touched * 2 * N if case["bias"] else 0
    b += rows * o * _half(case) if case["residual"] else 0
    b += rows * o * N if case["pre"] else 0
    return {"bytes": b, "flops": 2 * rows * N * K}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def _phi(v):
    """Activations by name, as functions of a float64 tensor."""
    cdf = lambda u: torch.special.ndtr(u)  # noqa: E731
    inner = lambda u: 2.0 * C_TANH * u * (1.0 + 0.044715 * u.square())  # noqa: E731
    return {"none": lambda u: u, "relu": torch.relu, "silu": lambda u: u * torch.sigmoid(u), "gelu": lambda u: u * cdf(u),
            "gelu_tanh": lambda u: u * torch.sigmoid(inner(u))}[v]


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "clip":
        total = 0.0
        for v in st["grads"]:
            for part in v.split(1 << 26):
                total += float(torch.linalg.vector_norm(part.double())) ** 2
        norm = math.sqrt(total)
        c = min(1.0, case["max_norm"] / (norm + 1e-6))
        flat = {}
        for i, (n, t) in enumerate(_tensors(case)):
            flat.setdefault(t, []).append(st["grads"][i].double() * c)
        return [np.array([norm]), {t: torch.cat(v) for t, v in flat.items()}]
    if op == "layer":
        F, k = case["F"], case["k"]
        x, logits = st["x"].double(), st["logits"].double().cpu().numpy()
        out = torch.zeros_like(x)
        by_slot = {}
        for t in range(case["T"]):
            chosen = sorted(range(case["E"]), key=lambda e: (-logits[t, e], e))[:k]
            s = [1.0 / (1.0 + math.exp(-logits[t, e])) for e in chosen]
            for e, v in zip(chosen, s):
                if 0 <= e - case["p0"] < case["local"]:
                    by_slot.setdefault(e - case["p0"], []).append((t, v / math.fsum(s)))
        for e, pairs in by_slot.items():
            t = [p[0] for p in pairs]
            gate = x[t] @ st["w1"][e, :F].double().T
            up = x[t] @ st["w1"][e, F:].double().T
            y = (gate * torch.sigmoid(gate) * up) @ st["w2"][e].double().T
            out[t] += y * torch.tensor([[p[1]] for p in pairs], dtype=torch.float64, device="cuda")
        return out
    N, half = case["N"], case["N"] // 2
    offsets = [0, case["rows"]] if st["offsets"] is None else st["offsets"].tolist()
    spans = [slice(lo, hi) for lo, hi in zip(offsets, offsets[1:])]
    f = _phi(case["act"])
    if op == "act":
        z = torch.cat([st["x"][s].double() @ st["w"][g].double().T + (st["b"][g].double() if case["bias"] else 0.0)
                       for g, s in enumerate(spans)])
        y = f(z[:, :half]) * z[:, half:] if case["gated"] else f(z)
        if case["residual"]:
            y = y + st["r"].double()
        return [y, z if case["pre"] else None]
    # the gradient of sum(dy * y) by the chain rule, in pieces of rows
    dz = torch.empty(case["rows"], N, dtype=torch.float64, device="cuda")
    for lo in range(0, case["rows"], 8192):
        z = st["z"][lo:lo + 8192].double().requires_grad_()
        y = f(z[:, :half]) * z[:, half:] if case["gated"] else f(z)
        y.backward(st["dy"][lo:lo + 8192].double())
        dz[lo:lo + 8192] = z.grad
    return [dz, torch.stack([dz[s].sum(0) for s in spans]) if case["bias"] else None]
