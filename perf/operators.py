"""Cases and plain forms of the library's linear operators.

* fp8 quantisation with one scale per 128 columns, plain and behind SwiGLU;
* the fp8 product with a scale per block of 128, dense and grouped by expert;
* the 16-bit products grouped by expert, forward and both gradients.

``run`` computes a case in its plain form (elementary torch operations in
32 bits) or, where ``own`` is true, with the library's calls; ``exact``
computes it in 64 bits from the operators' definitions.
"""

from __future__ import annotations

import math

import torch

own = False

BLOCK = 128          # columns (and weight rows) that share one fp8 scale
FP8_MAX = 448.0      # largest e4m3 value
MIN_SCALE = 2.0 ** -126
W_STD = 0.02         # weight deviation of the library's synthetic workloads

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _ceil(a, b):
    return -(-a // b)


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    """Widths 7168 / 2048 with 48 local experts are the library's benchmark
    layer, 256 / 256 with 8 experts its tiny workload."""
    return [
        # one decoded token in front of an fp8 layer: launch latency
        dict(name="quant_token", op="quant", rows=1, K=7168),
        # the activations of a shared expert's hidden layer in a prefill step
        dict(name="swiglu_quant_prefill", op="swiglu_quant", rows=8192, K=2048),
        # gate and up projection of a shared expert for one token: the weight stream
        dict(name="fp8_token", op="fp8", rows=1, groups=0, N=4096, K=7168, skew=0.0),
        # a short ragged batch on widths that fill neither tiles nor scale blocks
        dict(name="fp8_ragged", op="fp8", rows=77, groups=0, N=2041, K=7152, skew=0.0),
        # the same projection in a decode step at the benchmark's batch
        dict(name="fp8_decode", op="fp8", rows=512, groups=0, N=4096, K=7168, skew=0.0),
        # ... and in a prefill step
        dict(name="fp8_prefill", op="fp8", rows=8192, groups=0, N=4096, K=7168, skew=0.0),
        # 48 local fp8 experts in a decode step, 8 rows each
        dict(name="fp8_experts_decode", op="fp8", rows=384, groups=48, N=4096, K=7168, skew=0.0),
        # their down projection in a prefill step with uneven expert loads
        dict(name="fp8_experts_prefill", op="fp8", rows=6144, groups=48, N=7168, K=2048, skew=0.5),
        # the tiny workload's experts: launch latency
        dict(name="grouped_tiny", op="grouped", rows=128, groups=8, N=256, K=256, skew=0.0, dtype="bf16", out="bf16"),
        # fine-tuning, forward: gate and up projection of 48 experts
        dict(name="grouped_prefill", op="grouped", rows=6144, groups=48, N=4096, K=7168, skew=0.5, dtype="bf16",
             out="bf16"),
        # fine-tuning, both gradients, small odd sizes in fp16 with an empty group
        dict(name="grouped_backward_odd", op="backward", rows=250, groups=9, N=264, K=392, skew=3.0, dtype="f16",
             out="f16"),
        # both gradients of four experts' down projection, weight gradients in f32
        dict(name="grouped_backward", op="backward", rows=4096, groups=4, N=7168, K=2048, skew=0.5, dtype="bf16",
             out="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, step):
    v = _log_int(rng, lo // step, hi // step) * step
    return v + step if v == 3072 else v


def draw(rng):
    """One more case of the same ranges; weights are kept under those of the
    largest listed case of the operator."""
    op = rng.choice(["quant", "swiglu_quant", "fp8", "fp8", "experts", "experts", "grouped", "grouped", "backward",
                     "backward"])
    if op in ("quant", "swiglu_quant"):
        return dict(op=op, rows=_log_int(rng, 1, 8192), K=_width(rng, 64, 2048 if op == "swiglu_quant" else 7168, 16))
    if op == "fp8":
        return dict(op="fp8", rows=_log_int(rng, 1, 8192), groups=0, N=_width(rng, 33, 4096, 1),
                    K=_width(rng, 64, 7168, 16), skew=0.0)
    if op == "experts":
        return dict(op="fp8", rows=_log_int(rng, 1, 6144), groups=rng.randint(1, 48), N=_width(rng, 33, 4096, 1),
                    K=_width(rng, 64, 7168, 16), skew=rng.choice([0.0, 0.5, 1.5]))
    dtype = rng.choice(["bf16", "f16"])
    c = dict(op=op, rows=_log_int(rng, 1, 6144 if op == "grouped" else 4096),
             groups=rng.randint(1, 48 if op == "grouped" else 12), N=_width(rng, 64, 4096, 8),
             K=_width(rng, 64, 7168, 8), skew=rng.choice([0.0, 0.5, 1.5]), dtype=dtype,
             out=rng.choice([dtype, "f32"]))
    if op == "backward":  # the weight gradients are outputs
        while c["groups"] > 1 and c["groups"] * c["N"] * c["K"] > 4 * 7168 * 2048:
            c["groups"] -= 1
    return c


def _sizes(case):
    """Rows of each group before shuffling: shares proportional to
    (i + 1)^-skew, rounded so that they add up."""
    g = max(case["groups"], 1)
    w = [(i + 1.0) ** -case["skew"] for i in range(g)]
    exact_shares = [case["rows"] * v / sum(w) for v in w]
    n = [int(v) for v in exact_shares]
    order = sorted(range(g), key=lambda i: (n[i] - exact_shares[i], i))
    for i in order[:case["rows"] - sum(n)]:
        n[i] += 1
    return n


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _block_scale(amax):
    return (amax / FP8_MAX).clamp_min(MIN_SCALE)


def _to_fp8_rows(x):
    """fp8 codes [rows, K] and scales [rows, ceil(K / 128)] of f32 rows."""
    rows, K = x.shape
    nb = _ceil(K, BLOCK)
    v = torch.nn.functional.pad(x, (0, nb * BLOCK - K)).view(rows, nb, BLOCK)
    s = _block_scale(v.abs().amax(-1))
    q = (v * (1.0 / s)[..., None]).view(rows, nb * BLOCK)[:, :K].to(torch.float8_e4m3fn)
    return q.contiguous(), s


def _to_fp8_blocks(w):
    """fp8 codes [N, K] and scales [ceil(N / 128), ceil(K / 128)] of an f32 matrix."""
    N, K = w.shape
    nr, nb = _ceil(N, BLOCK), _ceil(K, BLOCK)
    v = torch.nn.functional.pad(w, (0, nb * BLOCK - K, 0, nr * BLOCK - N)).view(nr, BLOCK, nb, BLOCK)
    s = _block_scale(v.abs().amax((1, 3)))
    q = (v * (1.0 / s)[:, None, :, None]).view(nr * BLOCK, nb * BLOCK)[:N, :K].to(torch.float8_e4m3fn)
    return q.contiguous(), s


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)

    op, rows, K = case["op"], case["rows"], case["K"]
    st = dict(case=case)
    if op in ("quant", "swiglu_quant"):
        st["x"] = normal(rows, K if op == "quant" else 2 * K, dtype=torch.bfloat16)
        return st
    N, groups = case["N"], max(case["groups"], 1)
    if case["groups"]:
        hg = torch.Generator()
        hg.manual_seed(seed)
        n = _sizes(case)
        counts = [n[i] for i in torch.randperm(groups, generator=hg).tolist()]
        bounds = [0]
        for c in counts:
            bounds.append(bounds[-1] + c)
        st["offsets"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    else:
        bounds = [0, rows]
        st["offsets"] = None
    st["bounds"] = bounds  # the host's copy, for the plain form's loop
    if op == "fp8":
        st["xq"], st["xs"] = _to_fp8_rows(normal(rows, K))
        st["w"] = torch.empty(groups, N, K, dtype=torch.float8_e4m3fn, device="cuda")
        st["ws"] = torch.empty(groups, _ceil(N, BLOCK), _ceil(K, BLOCK), device="cuda")
        for i in range(groups):
            st["w"][i], st["ws"][i] = _to_fp8_blocks(normal(N, K, std=W_STD))
        return st
    dt = TYPES[case["dtype"]]
    st["x"] = normal(rows, K, dtype=dt)
    st["w"] = torch.empty(groups, N, K, dtype=dt, device="cuda")
    for i in range(groups):
        st["w"][i] = normal(N, K, std=W_STD, dtype=dt)
    if op == "backward":
        st["dy"] = normal(rows, N, dtype=dt)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    op, rows, K = case["op"], case["rows"], case["K"]
    if not own:
        return st
    import moe_expert_layer_sigmoid_amd as mx

    st["mx"] = mx
    if op in ("quant", "swiglu_quant"):
        st["q"] = torch.empty(rows, K, dtype=torch.float8_e4m3fn, device="cuda")
        st["qs"] = torch.empty(rows, _ceil(K, BLOCK), device="cuda")
        return st
    N, groups = case["N"], max(case["groups"], 1)
    if op == "fp8":
        st["d"] = mx.Linear(rows, N, K, groups=groups, in_type="fp8", out_type="bf16")
        st["y"] = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    else:
        st["d"] = mx.Linear(rows, N, K, groups=groups, in_type=case["dtype"], out_type=case["out"])
        if op == "grouped":
            st["y"] = torch.empty(rows, N, dtype=TYPES[case["out"]], device="cuda")
        else:  # the rows' gradient in their own type, the weights' in the type the case asks for
            st["d_dx"] = mx.Linear(rows, N, K, groups=groups, in_type=case["dtype"], out_type=case["dtype"])
            st["dx"] = torch.empty(rows, K, dtype=TYPES[case["dtype"]], device="cuda")
            st["dw"] = torch.empty(groups, N, K, dtype=TYPES[case["out"]], device="cuda")
    st["scratch"] = mx.linear_workspace(st["d"])
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    mx, op = st["mx"], st["case"]["op"]
    if op == "quant":
        mx.moe_fp8_quant(st["x"], st["q"], st["qs"])
        return st["q"], st["qs"]
    if op == "swiglu_quant":
        mx.moe_fp8_swiglu_quant(st["x"], st["q"], st["qs"])
        return st["q"], st["qs"]
    if op == "fp8":
        mx.moe_fp8_linear(st["d"], st["xq"], st["xs"], st["w"], st["ws"], st["y"], st["scratch"],
                          offsets=st["offsets"])
        return st["y"]
    if op == "grouped":
        mx.moe_grouped_linear(st["d"], st["x"], st["w"], st["y"], st["scratch"], offsets=st["offsets"])
        return st["y"]
    mx.moe_grouped_linear_dx(st["d_dx"], st["dy"], st["w"], st["dx"], st["scratch"], offsets=st["offsets"])
    mx.moe_grouped_linear_dw(st["d"], st["dy"], st["x"], st["dw"], st["scratch"], offsets=st["offsets"])
    return st["dx"], st["dw"]


def _run_plain(st):
    case = st["case"]
    op, K = case["op"], case["K"]
    if op == "quant":
        return _to_fp8_rows(st["x"].float())
    if op == "swiglu_quant":
        h = st["x"].float()
        gate, up = h[:, :K], h[:, K:]
        return _to_fp8_rows(gate / (1.0 + torch.exp(-gate)) * up)
    N, rows, b = case["N"], case["rows"], st["bounds"]
    if op == "fp8":
        col = torch.arange(K, device="cuda") // BLOCK
        row = torch.arange(N, device="cuda") // BLOCK
        x = st["xq"].float() * st["xs"][:, col]
        y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        for g in range(len(b) - 1):
            if b[g + 1] > b[g]:
                w = st["w"][g].float() * st["ws"][g][row][:, col]
                y[b[g]:b[g + 1]] = torch.mm(x[b[g]:b[g + 1]], w.t()).to(torch.bfloat16)
        return y
    out = TYPES[case["out"]]
    if op == "grouped":
        y = torch.empty(rows, N, dtype=out, device="cuda")
        for g in range(len(b) - 1):
            if b[g + 1] > b[g]:
                y[b[g]:b[g + 1]] = torch.mm(st["x"][b[g]:b[g + 1]].float(), st["w"][g].float().t()).to(out)
        return y
    dx = torch.empty(rows, K, dtype=TYPES[case["dtype"]], device="cuda")
    dw = torch.zeros(len(b) - 1, N, K, dtype=out, device="cuda")
    for g in range(len(b) - 1):
        if b[g + 1] > b[g]:
            dy, x = st["dy"][b[g]:b[g + 1]].float(), st["x"][b[g]:b[g + 1]].float()
            dx[b[g]:b[g + 1]] = torch.mm(dy, st["w"][g].float()).to(dx.dtype)
            dw[g] = torch.mm(dy.t(), x).to(out)
    return dx, dw


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    op, rows, K = case["op"], case["rows"], case["K"]
    nb = _ceil(K, BLOCK)
    if op == "quant":
        return {"bytes": rows * (2 * K + K + 4 * nb), "flops": 3 * rows * K}
    if op == "swiglu_quant":
        return {"bytes": rows * (4 * K + K + 4 * nb), "flops": 8 * rows * K}
    N = case["N"]
    n = _sizes(case)
    touched = sum(1 for v in n if v)
    flops = 2 * rows * N * K
    if op == "fp8":
        return {"bytes": rows * (K + 4 * nb + 2 * N) + touched * (N * K + 4 * nb * _ceil(N, BLOCK)), "flops": flops}
    o = 4 if case["out"] == "f32" else 2
    if op == "grouped":
        return {"bytes": rows * (2 * K + o * N) + touched * 2 * N * K, "flops": flops}
    # dy and W in, dx out; dy and x in, every group's dW out
    return {"bytes": rows * (2 * N + 2 * K) + touched * 2 * N * K + rows * 2 * (N + K) + len(n) * o * N * K,
            "flops": 2 * flops}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    st = _inputs(case, seed)
    op, K, rows = case["op"], case["K"], case["rows"]
    if op in ("quant", "swiglu_quant"):
        v = st["x"].double()
        if op == "swiglu_quant":
            v = v[:, :K] * torch.sigmoid(v[:, :K]) * v[:, K:]
        q = torch.empty(rows, K, dtype=torch.float64, device="cuda")
        s = torch.empty(rows, _ceil(K, BLOCK), dtype=torch.float64, device="cuda")
        for i, c in enumerate(range(0, K, BLOCK)):
            part = v[:, c:c + BLOCK]
            s[:, i] = torch.clamp(part.abs().max(dim=1).values / FP8_MAX, min=MIN_SCALE)
            q[:, c:c + BLOCK] = part / s[:, i:i + 1]
        return q, s
    N = case["N"]
    offsets = [0, rows] if st["offsets"] is None else st["offsets"].tolist()
    spans = [slice(lo, hi) for lo, hi in zip(offsets, offsets[1:])]
    if op == "fp8":
        y = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        for g, span in enumerate(spans):
            # unit by unit: one product per 128 columns, then its two scales
            for i, c in enumerate(range(0, K, BLOCK)):
                part = st["xq"][span, c:c + BLOCK].double() @ st["w"][g, :, c:c + BLOCK].double().T
                ws = st["ws"][g, :, i].double().repeat_interleave(BLOCK)[:N]
                y[span] += part * st["xs"][span, i:i + 1].double() * ws
        return y
    if op == "grouped":
        return torch.cat([st["x"][s].double() @ st["w"][g].double().T for g, s in enumerate(spans)])
    dx = torch.cat([st["dy"][s].double() @ st["w"][g].double() for g, s in enumerate(spans)])
    dw = torch.stack([st["dy"][s].double().T @ st["x"][s].double() for s in spans])
    return dx, dw
