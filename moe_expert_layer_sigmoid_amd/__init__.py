"""Python binding of libmoe, the gfx950 HIP library of one GPU's share of a
fused MoE expert layer (sigmoid top-k, EPLB remap + record, fp8 x MXFP4).

This module only marshals arguments: it checks dtypes and sizes of torch
tensors, reads their device pointers and the current HIP stream, and calls
the C ABI declared in ``include/moe.h`` by the same names.  Every step of the
layer runs in the library's kernels.  There is no fallback: if ``libmoe.so``
is missing or cannot be loaded, every call raises.
"""

from __future__ import annotations

import ctypes
import os
import warnings
from typing import Dict, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported size", -3: "workspace", -4: "hip",
          -5: "dims need more than the fixed scratch of moe_forward_noalloc"}
NOALLOC_SCRATCH_BYTES = 128 << 20   # MOE_NOALLOC_SCRATCH_BYTES of include/moe.h
PATHS = {"auto": 0, "small_m": 1, "staged": 2, "large_m": 3}
PATH_NAMES = {v: k for k, v in PATHS.items()}

EXPORTS = ("moe_workspace_bytes", "moe_select_path", "moe_status_string", "moe_packed_bytes",
           "moe_pack_weights", "moe_route",
           "moe_eplb_remap_record", "moe_quant_permute", "moe_grouped_gemm1_swiglu",
           "moe_grouped_gemm2_combine", "moe_grouped_gemm1_swiglu_pairs", "moe_grouped_gemm2_combine_pairs",
           "moe_forward", "moe_eplb_rebalance", "moe_eplb_migrate",
           "moe_router_workspace_bytes", "moe_router_logits", "moe_forward_small_m",
           "moe_a16w4_workspace_bytes", "moe_forward_a16w4", "moe_forward_noalloc", "moe_replica_of",
           "moe_linear_workspace_bytes", "moe_fp8_quant", "moe_fp8_swiglu_quant", "moe_fp8_linear",
           "moe_grouped_linear", "moe_grouped_linear_dx", "moe_grouped_linear_dw",
           "moe_linear_act_workspace_bytes", "moe_grouped_linear_act", "moe_grouped_linear_act_backward",
           "moe_grad_workspace_bytes", "moe_grad_norm", "moe_grad_clip",
           "moe_a16w16_workspace_bytes", "moe_forward_a16w16")


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed with status {code} ({STATUS.get(code, 'unknown')})")
        self.code = code


class Dims(ctypes.Structure):
    """moe_dims_t"""
    _fields_ = [("T", ctypes.c_int32), ("T_max", ctypes.c_int32), ("H", ctypes.c_int32),
                ("F", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("P_total", ctypes.c_int32), ("p0", ctypes.c_int32), ("P_local", ctypes.c_int32),
                ("R_max", ctypes.c_int32), ("token_id_base", ctypes.c_uint32),
                ("small_m_max", ctypes.c_int32), ("large_m_min", ctypes.c_int32)]

    @classmethod
    def of(cls, d, **kw) -> "Dims":
        """From any object with the same attribute names (e.g. synth.Dims)."""
        vals = {f: getattr(d, f, 0) for f, _ in cls._fields_}
        vals.update(kw)
        return cls(**{k: int(v) for k, v in vals.items()})


TYPES = {"bf16": 0, "f16": 1, "f32": 2, "fp8": 3}   # moe_type_t
_TORCH_TYPES = (torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn)
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}   # moe_act_t
_QUANT_TYPES = {t: i for i, t in enumerate(_TORCH_TYPES[:3])}


class Linear(ctypes.Structure):
    """moe_linear_t"""
    _fields_ = [("rows", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("in_type", ctypes.c_int32), ("out_type", ctypes.c_int32)]

    def __init__(self, rows: int, N: int, K: int, groups: int = 1, in_type: str = "bf16",
                 out_type: Optional[str] = None):
        """``in_type`` / ``out_type``: "bf16", "f16", "f32", "fp8"; the output
        defaults to in_type (bf16 for fp8)."""
        if out_type is None:
            out_type = "bf16" if in_type == "fp8" else in_type
        for n, t in (("in_type", in_type), ("out_type", out_type)):
            if t not in TYPES:
                raise ValueError(f"{n}: {t!r} is none of {', '.join(TYPES)}")
        for n, v in (("rows", rows), ("N", N), ("K", K), ("groups", groups)):   # ctypes would keep the low 32 bits
            if not -2 ** 31 <= int(v) < 2 ** 31:
                raise ValueError(f"{n}: {v} is no 32-bit integer")
        super().__init__(int(rows), int(N), int(K), int(groups), TYPES[in_type], TYPES[out_type])


class Taps(ctypes.Structure):
    """moe_taps_t"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_ids", "topk_w", "phys_ids", "counts", "offsets",
                                                "row_of_pair", "pair_of_row", "xq", "xs", "aq", "as_",
                                                "xq_tok", "xs_tok", "aq_pair", "as_pair")]
    _fields_ += [("gemm1_events", ctypes.c_void_p * 2), ("gemm2_events", ctypes.c_void_p * 2)]


def _event_handle(ev) -> int:
    """The hipEvent_t behind a torch.cuda.Event (torch creates it at the first record)."""
    if ev.cuda_event == 0:
        ev.record()
    return ev.cuda_event


_lib_handle = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (raises if it was not built)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m moe_expert_layer_sigmoid_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        D = ctypes.POINTER(Dims)
        I = ctypes.c_int
        L.moe_workspace_bytes.argtypes = [D]
        L.moe_workspace_bytes.restype = ctypes.c_size_t
        L.moe_select_path.argtypes = [D]
        L.moe_select_path.restype = I
        L.moe_status_string.argtypes = [I]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_packed_bytes.argtypes = [D, I]
        L.moe_packed_bytes.restype = ctypes.c_size_t
        L.moe_pack_weights.argtypes = [D, P, P, P, P, P, P, P, P, P]
        L.moe_route.argtypes = [D, P, P, P, P]
        L.moe_eplb_remap_record.argtypes = [D, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_quant_permute.argtypes = [D, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_grouped_gemm1_swiglu.argtypes = [D, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_grouped_gemm2_combine.argtypes = [D, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_grouped_gemm1_swiglu_pairs.argtypes = [D, P, P, P, P, P, P, P, P, P]
        L.moe_grouped_gemm2_combine_pairs.argtypes = [D, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_forward.argtypes = [D, I, P, P, P, P, P, P, P, P, P, P, ctypes.POINTER(Taps),
                                  ctypes.POINTER(ctypes.c_int), P, ctypes.c_size_t, P]
        L.moe_forward_small_m.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, ctypes.POINTER(Taps), P,
                                          ctypes.c_size_t, P]
        L.moe_forward_small_m.restype = I
        L.moe_forward_noalloc.argtypes = [D, I, P, P, P, P, P, P, P, P, P, P, ctypes.POINTER(ctypes.c_int), P]
        L.moe_forward_noalloc.restype = I
        L.moe_a16w4_workspace_bytes.argtypes = [D]
        L.moe_a16w4_workspace_bytes.restype = ctypes.c_size_t
        L.moe_forward_a16w4.argtypes = [D, P, P, P, P, P, P, P, P, P, P, ctypes.POINTER(Taps), P, P,
                                        ctypes.c_size_t, P]
        L.moe_forward_a16w4.restype = I
        L.moe_router_workspace_bytes.argtypes = [D]
        L.moe_router_workspace_bytes.restype = ctypes.c_size_t
        L.moe_router_logits.argtypes = [D, P, P, P, P, ctypes.c_size_t, P]
        L.moe_router_logits.restype = I
        L.moe_replica_of.argtypes = [ctypes.c_uint32, ctypes.c_int32, ctypes.c_int32]
        L.moe_replica_of.restype = ctypes.c_int32
        L.moe_eplb_rebalance.argtypes = [I, I, I, I, P, P, P, P, P]
        L.moe_eplb_migrate.argtypes = [D, P, I, P, P, P, P, P, P, P, P, P]
        N = ctypes.POINTER(Linear)
        S = ctypes.c_size_t
        L.moe_linear_workspace_bytes.argtypes = [N]
        L.moe_linear_workspace_bytes.restype = S
        for n in ("moe_fp8_quant", "moe_fp8_swiglu_quant"):
            getattr(L, n).argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, ctypes.c_int64, P, P, P]
            getattr(L, n).restype = I
        L.moe_fp8_linear.argtypes = [N, P, P, P, P, P, P, P, S, P]
        L.moe_fp8_linear.restype = I
        for n in ("moe_grouped_linear", "moe_grouped_linear_dx", "moe_grouped_linear_dw"):
            getattr(L, n).argtypes = [N, P, P, P, P, P, S, P]
            getattr(L, n).restype = I
        C = ctypes.c_int32
        L.moe_linear_act_workspace_bytes.argtypes = [N]
        L.moe_linear_act_workspace_bytes.restype = S
        L.moe_grouped_linear_act.argtypes = [N, C, C, P, P, P, P, P, P, P, P, S, P]
        L.moe_grouped_linear_act_backward.argtypes = [N, C, C, P, P, P, P, P, P, S, P]
        L.moe_grad_workspace_bytes.argtypes = [C]
        L.moe_grad_workspace_bytes.restype = S
        L.moe_grad_norm.argtypes = [P, C, P, P, S, P]
        L.moe_grad_clip.argtypes = [P, C, ctypes.c_float, P, P, S, P]
        L.moe_a16w16_workspace_bytes.argtypes = [D]
        L.moe_a16w16_workspace_bytes.restype = S
        L.moe_forward_a16w16.argtypes = [D, C, P, P, P, P, P, P, P, P, P, ctypes.POINTER(Taps), P, S, P]
        for n in ("moe_grouped_linear_act", "moe_grouped_linear_act_backward", "moe_grad_norm", "moe_grad_clip",
                  "moe_forward_a16w16"):
            getattr(L, n).restype = I
        for n in ("moe_pack_weights", "moe_route", "moe_eplb_remap_record", "moe_quant_permute",
                  "moe_grouped_gemm1_swiglu", "moe_grouped_gemm2_combine", "moe_grouped_gemm1_swiglu_pairs",
                  "moe_grouped_gemm2_combine_pairs", "moe_forward", "moe_eplb_rebalance", "moe_eplb_migrate"):
            getattr(L, n).restype = I
        _lib_handle = L
    return _lib_handle


# ----------------------------------------------------------------------------
# marshalling helpers
# ----------------------------------------------------------------------------

def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, numel_min: int = 0):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.numel() < numel_min:
        raise ValueError(f"{name}: {t.numel()} elements, need at least {numel_min}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(fn: str, rc: int):
    if rc != MOE_OK:
        raise MoeError(fn, rc)


u8, i32, f32, i16 = torch.uint8, torch.int32, torch.float32, torch.int16


def _bf16(t: torch.Tensor) -> torch.dtype:
    return t.dtype if t.dtype in (torch.bfloat16, torch.int16, torch.uint16) else torch.bfloat16


def _sizes(d: Dims):
    TK, TMK = d.T * d.k, d.T_max * d.k
    return TK, TMK


# ----------------------------------------------------------------------------
# the C ABI, same names
# ----------------------------------------------------------------------------

def moe_workspace_bytes(d: Dims) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(d)))


def moe_select_path(d: Dims) -> str:
    return PATH_NAMES[int(lib().moe_select_path(ctypes.byref(d)))]


def moe_status_string(code: int) -> str:
    return lib().moe_status_string(int(code)).decode()


def moe_replica_of(token_id: int, rep_count: int, R_max: int) -> int:
    return int(lib().moe_replica_of(int(token_id) & 0xFFFFFFFF, int(rep_count), int(R_max)))


def moe_packed_bytes(d: Dims, which: int) -> int:
    return int(lib().moe_packed_bytes(ctypes.byref(d), int(which)))


def moe_pack_weights(d: Dims, w1, w1s, w2, w2s, pw1, pw1s, pw2, pw2s, stream=None):
    nw1, ns1 = d.P_local * 2 * d.F * d.H // 2, d.P_local * 2 * d.F * d.H // 32
    nw2, ns2 = d.P_local * d.H * d.F // 2, d.P_local * d.H * d.F // 32
    rc = lib().moe_pack_weights(
        ctypes.byref(d), _ptr(w1, "w1", u8, nw1), _ptr(w1s, "w1s", u8, ns1), _ptr(w2, "w2", u8, nw2),
        _ptr(w2s, "w2s", u8, ns2), _ptr(pw1, "pw1", u8, moe_packed_bytes(d, 0)),
        _ptr(pw1s, "pw1s", u8, moe_packed_bytes(d, 1)), _ptr(pw2, "pw2", u8, moe_packed_bytes(d, 2)),
        _ptr(pw2s, "pw2s", u8, moe_packed_bytes(d, 3)), _stream(stream))
    _check("moe_pack_weights", rc)


def pack_weights(d: Dims, w1, w1s, w2, w2s, stream=None):
    """Allocate and fill the packed weight buffers; returns (pw1, pw1s, pw2, pw2s)."""
    dev = w1.device
    out = tuple(torch.empty(moe_packed_bytes(d, i), dtype=u8, device=dev) for i in range(4))
    moe_pack_weights(d, w1, w1s, w2, w2s, *out, stream=stream)
    return out


def workspace(d: Dims, device="cuda") -> torch.Tensor:
    """A workspace of moe_workspace_bytes(d) bytes (torch-allocated, 256-B aligned)."""
    n = moe_workspace_bytes(d)
    return torch.empty(max(n, 256), dtype=u8, device=device)


def moe_route(d: Dims, logits, topk_ids, topk_w, stream=None):
    TK, _ = _sizes(d)
    rc = lib().moe_route(ctypes.byref(d), _ptr(logits, "logits", f32, d.T * d.E),
                         _ptr(topk_ids, "topk_ids", i32, TK), _ptr(topk_w, "topk_w", f32, TK), _stream(stream))
    _check("moe_route", rc)


def moe_eplb_remap_record(d: Dims, topk_ids, rep_count, rep_slots, phys_ids, load_hist, ws, stream=None):
    TK, _ = _sizes(d)
    rc = lib().moe_eplb_remap_record(
        ctypes.byref(d), _ptr(topk_ids, "topk_ids", i32, TK), _ptr(rep_count, "rep_count", i32, d.E),
        _ptr(rep_slots, "rep_slots", i32, d.E * d.R_max), _ptr(phys_ids, "phys_ids", i32, TK),
        _ptr(load_hist, "load_hist", i32, d.P_total), _ptr(ws, "workspace", u8), ws.numel(), _stream(stream))
    _check("moe_eplb_remap_record", rc)


def moe_quant_permute(d: Dims, x, phys_ids, xq, xs, counts, offsets, row_of_pair, pair_of_row, ws, stream=None):
    TK, TMK = _sizes(d)
    rc = lib().moe_quant_permute(
        ctypes.byref(d), _ptr(x, "x", _bf16(x), d.T * d.H), _ptr(phys_ids, "phys_ids", i32, TK),
        _ptr(xq, "xq", u8, TMK * d.H), _ptr(xs, "xs", u8, TMK * (d.H // 128)),
        _ptr(counts, "counts", i32, d.P_local), _ptr(offsets, "offsets", i32, d.P_local + 1),
        _ptr(row_of_pair, "row_of_pair", i32, TK), _ptr(pair_of_row, "pair_of_row", i32, TMK),
        _ptr(ws, "workspace", u8), ws.numel(), _stream(stream))
    _check("moe_quant_permute", rc)


def moe_grouped_gemm1_swiglu(d: Dims, xq, xs, offsets, pw1, pw1s, aq, as_, ws, stream=None):
    _, TMK = _sizes(d)
    rc = lib().moe_grouped_gemm1_swiglu(
        ctypes.byref(d), _ptr(xq, "xq", u8, TMK * d.H), _ptr(xs, "xs", u8, TMK * (d.H // 128)),
        _ptr(offsets, "offsets", i32, d.P_local + 1),
        _ptr(pw1, "pw1", u8, moe_packed_bytes(d, 0)), _ptr(pw1s, "pw1s", u8, moe_packed_bytes(d, 1)),
        _ptr(aq, "aq", u8, TMK * d.F), _ptr(as_, "as", u8, TMK * (d.F // 128)),
        _ptr(ws, "workspace", u8), ws.numel(), _stream(stream))
    _check("moe_grouped_gemm1_swiglu", rc)


def moe_grouped_gemm2_combine(d: Dims, aq, as_, offsets, pw2, pw2s, row_of_pair, topk_w, out, ws, stream=None):
    TK, TMK = _sizes(d)
    rc = lib().moe_grouped_gemm2_combine(
        ctypes.byref(d), _ptr(aq, "aq", u8, TMK * d.F), _ptr(as_, "as", u8, TMK * (d.F // 128)),
        _ptr(offsets, "offsets", i32, d.P_local + 1),
        _ptr(pw2, "pw2", u8, moe_packed_bytes(d, 2)), _ptr(pw2s, "pw2s", u8, moe_packed_bytes(d, 3)),
        _ptr(row_of_pair, "row_of_pair", i32, TK), _ptr(topk_w, "topk_w", f32, TK),
        _ptr(out, "out", _bf16(out), d.T * d.H), _ptr(ws, "workspace", u8), ws.numel(), _stream(stream))
    _check("moe_grouped_gemm2_combine", rc)


def moe_grouped_gemm1_swiglu_pairs(d: Dims, xq_tok, xs_tok, phys_ids, pw1, pw1s, aq_pair, as_pair, counts,
                                   stream=None):
    TK = d.T * d.k
    rc = lib().moe_grouped_gemm1_swiglu_pairs(
        ctypes.byref(d), _ptr(xq_tok, "xq_tok", u8, d.T * d.H), _ptr(xs_tok, "xs_tok", u8, d.T * (d.H // 128)),
        _ptr(phys_ids, "phys_ids", i32, TK),
        _ptr(pw1, "pw1", u8, moe_packed_bytes(d, 0)), _ptr(pw1s, "pw1s", u8, moe_packed_bytes(d, 1)),
        _ptr(aq_pair, "aq_pair", u8, TK * d.F), _ptr(as_pair, "as_pair", u8, TK * (d.F // 128)),
        _ptr(counts, "counts", i32, d.P_local), _stream(stream))
    _check("moe_grouped_gemm1_swiglu_pairs", rc)


def moe_grouped_gemm2_combine_pairs(d: Dims, aq_pair, as_pair, phys_ids, pw2, pw2s, topk_w, counts, offsets, out, ws,
                                    stream=None):
    TK = d.T * d.k
    rc = lib().moe_grouped_gemm2_combine_pairs(
        ctypes.byref(d), _ptr(aq_pair, "aq_pair", u8, TK * d.F), _ptr(as_pair, "as_pair", u8, TK * (d.F // 128)),
        _ptr(phys_ids, "phys_ids", i32, TK),
        _ptr(pw2, "pw2", u8, moe_packed_bytes(d, 2)), _ptr(pw2s, "pw2s", u8, moe_packed_bytes(d, 3)),
        _ptr(topk_w, "topk_w", f32, TK), _ptr(counts, "counts", i32, d.P_local),
        _ptr(offsets, "offsets", i32, d.P_local + 1), _ptr(out, "out", _bf16(out), d.T * d.H),
        _ptr(ws, "workspace", u8), ws.numel(), _stream(stream))
    _check("moe_grouped_gemm2_combine_pairs", rc)


def make_taps(d: Dims, device="cuda") -> Dict[str, torch.Tensor]:
    """Device buffers for every tap of moe_forward."""
    TK, TMK = _sizes(d)
    z = lambda n, dt: torch.zeros(max(n, 1), dtype=dt, device=device)  # noqa: E731
    return dict(topk_ids=z(TK, i32), topk_w=z(TK, f32), phys_ids=z(TK, i32), counts=z(d.P_local, i32),
                offsets=z(d.P_local + 1, i32), row_of_pair=z(TK, i32), pair_of_row=z(TMK, i32),
                xq=z(TMK * d.H, u8), xs=z(TMK * (d.H // 128), u8), aq=z(TMK * d.F, u8),
                as_=z(TMK * (d.F // 128), u8), xq_tok=z(d.T * d.H, u8), xs_tok=z(d.T * (d.H // 128), u8),
                aq_pair=z(TK * d.F, u8), as_pair=z(TK * (d.F // 128), u8))


def moe_forward(d: Dims, x, logits, pw1, pw1s, pw2, pw2s, rep_count, rep_slots, out, ws, load_hist=None,
                path: str = "auto", taps: Optional[Dict[str, torch.Tensor]] = None, stream=None,
                gemm_events=None) -> str:
    """Run the whole layer on packed weights; returns the path taken
    ("small_m", "staged", "large_m").  ``gemm_events`` (optional): four
    torch.cuda.Event recorded around the GEMM1 and the GEMM2 launch
    (begin1, end1, begin2, end2)."""
    TK, TMK = _sizes(d)
    tp = None
    if taps is not None:
        need = dict(topk_ids=(i32, TK), topk_w=(f32, TK), phys_ids=(i32, TK), counts=(i32, d.P_local),
                    offsets=(i32, d.P_local + 1), row_of_pair=(i32, TK), pair_of_row=(i32, TMK),
                    xq=(u8, TMK * d.H), xs=(u8, TMK * (d.H // 128)), aq=(u8, TMK * d.F),
                    as_=(u8, TMK * (d.F // 128)), xq_tok=(u8, d.T * d.H), xs_tok=(u8, d.T * (d.H // 128)),
                    aq_pair=(u8, TK * d.F), as_pair=(u8, TK * (d.F // 128)))
        tp = Taps(**{n: _ptr(taps.get(n), n, *need[n]) for n in need})
    if gemm_events is not None:
        tp = tp if tp is not None else Taps()
        h = [_event_handle(e) for e in gemm_events]
        tp.gemm1_events[0], tp.gemm1_events[1], tp.gemm2_events[0], tp.gemm2_events[1] = h
    chosen = ctypes.c_int(-1)
    rc = lib().moe_forward(
        ctypes.byref(d), PATHS[path], _ptr(x, "x", _bf16(x), d.T * d.H), _ptr(logits, "logits", f32, d.T * d.E),
        _ptr(pw1, "pw1", u8, moe_packed_bytes(d, 0)), _ptr(pw1s, "pw1s", u8, moe_packed_bytes(d, 1)),
        _ptr(pw2, "pw2", u8, moe_packed_bytes(d, 2)), _ptr(pw2s, "pw2s", u8, moe_packed_bytes(d, 3)),
        _ptr(rep_count, "rep_count", i32, d.E), _ptr(rep_slots, "rep_slots", i32, d.E * d.R_max),
        _ptr(load_hist, "load_hist", i32, d.P_total), _ptr(out, "out", _bf16(out), d.T * d.H),
        ctypes.byref(tp) if tp is not None else None, ctypes.byref(chosen),
        _ptr(ws, "workspace", u8), ws.numel(), _stream(stream))
    _check("moe_forward", rc)
    return PATH_NAMES[chosen.value]


def moe_forward_noalloc(d: Dims, x, logits, pw1, pw1s, pw2, pw2s, rep_count, rep_slots, out, load_hist=None,
                        path: str = "auto", stream=None) -> str:
    """moe_forward without a workspace: the library's fixed per-GPU scratch
    (NOALLOC_SCRATCH_BYTES) serves instead, so the call allocates nothing.
    Calls that overlap in time on one GPU share that scratch and race.
    Returns the path taken."""
    chosen = ctypes.c_int(-1)
    rc = lib().moe_forward_noalloc(
        ctypes.byref(d), PATHS[path], _ptr(x, "x", _bf16(x), d.T * d.H), _ptr(logits, "logits", f32, d.T * d.E),
        _ptr(pw1, "pw1", u8, moe_packed_bytes(d, 0)), _ptr(pw1s, "pw1s", u8, moe_packed_bytes(d, 1)),
        _ptr(pw2, "pw2", u8, moe_packed_bytes(d, 2)), _ptr(pw2s, "pw2s", u8, moe_packed_bytes(d, 3)),
        _ptr(rep_count, "rep_count", i32, d.E), _ptr(rep_slots, "rep_slots", i32, d.E * d.R_max),
        _ptr(load_hist, "load_hist", i32, d.P_total), _ptr(out, "out", _bf16(out), d.T * d.H),
        ctypes.byref(chosen), _stream(stream))
    _check("moe_forward_noalloc", rc)
    return PATH_NAMES[chosen.value]


def moe_forward_small_m(d: Dims, num_tokens, x, logits, pw1, pw1s, pw2, pw2s, rep_count, rep_slots, out, ws,
                        load_hist=None, taps: Optional[Dict[str, torch.Tensor]] = None, stream=None) -> None:
    """The small-input path with the valid token count read on the device
    from ``num_tokens`` (int32 device tensor, one element); d.T is the bucket
    capacity.  Allocates nothing: safe inside torch.cuda.graph capture."""
    TK, _ = _sizes(d)
    tp = None
    if taps is not None:
        need = dict(topk_ids=(i32, TK), topk_w=(f32, TK), phys_ids=(i32, TK), counts=(i32, d.P_local),
                    offsets=(i32, d.P_local + 1), xq_tok=(u8, d.T * d.H), xs_tok=(u8, d.T * (d.H // 128)),
                    aq_pair=(u8, TK * d.F), as_pair=(u8, TK * (d.F // 128)))
        tp = Taps(**{n: _ptr(taps.get(n), n, *need[n]) for n in need})
    rc = lib().moe_forward_small_m(
        ctypes.byref(d), _ptr(num_tokens, "num_tokens", i32, 1), _ptr(x, "x", _bf16(x), d.T * d.H),
        _ptr(logits, "logits", f32, d.T * d.E),
        _ptr(pw1, "pw1", u8, moe_packed_bytes(d, 0)), _ptr(pw1s, "pw1s", u8, moe_packed_bytes(d, 1)),
        _ptr(pw2, "pw2", u8, moe_packed_bytes(d, 2)), _ptr(pw2s, "pw2s", u8, moe_packed_bytes(d, 3)),
        _ptr(rep_count, "rep_count", i32, d.E), _ptr(rep_slots, "rep_slots", i32, d.E * d.R_max),
        _ptr(load_hist, "load_hist", i32, d.P_total), _ptr(out, "out", _bf16(out), d.T * d.H),
        ctypes.byref(tp) if tp is not None else None, _ptr(ws, "workspace", u8), ws.numel(), _stream(stream))
    _check("moe_forward_small_m", rc)


# ----------------------------------------------------------------------------
# EPLB rebalance (host) and weight migration (device)
# ----------------------------------------------------------------------------

def _host_i32(a, name: str, n: int):
    import numpy as np
    if isinstance(a, torch.Tensor):
        if a.device.type != "cpu":
            raise ValueError(f"{name}: must be a host array")
        a = a.numpy()
    a = np.ascontiguousarray(a, dtype=np.int32)
    if a.size != n:
        raise ValueError(f"{name}: {a.size} elements, expected {n}")
    return a


def moe_eplb_rebalance(E: int, P_total: int, n_ranks: int, R_max: int, load_hist, slot_expert_old):
    """New replica table from recorded slot loads (host arrays in and out).
    Returns numpy int32 (rep_count [E], rep_slots [E, R_max], slot_expert_new [P_total])."""
    import numpy as np
    h = _host_i32(load_hist, "load_hist", P_total)
    old = _host_i32(slot_expert_old, "slot_expert_old", P_total)
    rc = np.zeros(E, np.int32)
    rs = np.zeros((E, R_max), np.int32)
    new = np.zeros(P_total, np.int32)
    c = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    st = lib().moe_eplb_rebalance(int(E), int(P_total), int(n_ranks), int(R_max), c(h), c(old), c(rc), c(rs), c(new))
    _check("moe_eplb_rebalance", st)
    return rc, rs, new


def moe_eplb_migrate(d: Dims, src_expert, n_pool: int, pool, slots, stream=None):
    """Copy pool experts into local slots: ``pool`` and ``slots`` are packed
    weight tuples (pw1, pw1s, pw2, pw2s) over n_pool experts and d.P_local
    slots; src_expert i32 [P_local] on the device (-1 = keep)."""
    per = [moe_packed_bytes(d, i) // d.P_local for i in range(4)]
    names = ("pw1", "pw1s", "pw2", "pw2s")
    pp = [_ptr(t, "pool_" + n, u8, per[i] * n_pool) for i, (t, n) in enumerate(zip(pool, names))]
    sp = [_ptr(t, n, u8, per[i] * d.P_local) for i, (t, n) in enumerate(zip(slots, names))]
    rc = lib().moe_eplb_migrate(ctypes.byref(d), _ptr(src_expert, "src_expert", i32, d.P_local), int(n_pool),
                                *pp, *sp, _stream(stream))
    _check("moe_eplb_migrate", rc)


# ----------------------------------------------------------------------------
# Router projection
# ----------------------------------------------------------------------------

def moe_router_workspace_bytes(d: Dims) -> int:
    return int(lib().moe_router_workspace_bytes(ctypes.byref(d)))


def router_workspace(d: Dims, device="cuda") -> torch.Tensor:
    return torch.empty(max(moe_router_workspace_bytes(d), 256), dtype=u8, device=device)


def moe_router_logits(d: Dims, x, w_gate, logits, ws, stream=None):
    """logits f32 [T, E] = x bf16 [T, H] (int16 bits or bfloat16) times w_gate bf16 [E, H] transposed."""
    rc = lib().moe_router_logits(ctypes.byref(d), _ptr(x, "x", _bf16(x), d.T * d.H),
                                 _ptr(w_gate, "w_gate", _bf16(w_gate), d.E * d.H),
                                 _ptr(logits, "logits", f32, d.T * d.E), _ptr(ws, "workspace", u8), ws.numel(),
                                 _stream(stream))
    _check("moe_router_logits", rc)


# ----------------------------------------------------------------------------
# a16w4 variant
# ----------------------------------------------------------------------------

def moe_a16w4_workspace_bytes(d: Dims) -> int:
    return int(lib().moe_a16w4_workspace_bytes(ctypes.byref(d)))


def a16w4_workspace(d: Dims, device="cuda") -> torch.Tensor:
    return torch.empty(max(moe_a16w4_workspace_bytes(d), 256), dtype=u8, device=device)


def moe_forward_a16w4(d: Dims, x, logits, pw1, pw1s, pw2, pw2s, rep_count, rep_slots, out, ws, load_hist=None,
                      taps: Optional[Dict[str, torch.Tensor]] = None, act=None, stream=None) -> None:
    """The layer with bf16 activations on the packed MXFP4 experts.  ``act``
    (optional, bf16 [T_max*k, F] as int16 bits) receives the GEMM1 act rows."""
    TK, TMK = _sizes(d)
    tp = None
    if taps is not None:
        need = dict(topk_ids=(i32, TK), topk_w=(f32, TK), phys_ids=(i32, TK), counts=(i32, d.P_local),
                    offsets=(i32, d.P_local + 1), row_of_pair=(i32, TK), pair_of_row=(i32, TMK))
        tp = Taps(**{n: _ptr(taps.get(n), n, *need[n]) for n in need})
    rc = lib().moe_forward_a16w4(
        ctypes.byref(d), _ptr(x, "x", _bf16(x), d.T * d.H), _ptr(logits, "logits", f32, d.T * d.E),
        _ptr(pw1, "pw1", u8, moe_packed_bytes(d, 0)), _ptr(pw1s, "pw1s", u8, moe_packed_bytes(d, 1)),
        _ptr(pw2, "pw2", u8, moe_packed_bytes(d, 2)), _ptr(pw2s, "pw2s", u8, moe_packed_bytes(d, 3)),
        _ptr(rep_count, "rep_count", i32, d.E), _ptr(rep_slots, "rep_slots", i32, d.E * d.R_max),
        _ptr(load_hist, "load_hist", i32, d.P_total), _ptr(out, "out", _bf16(out), d.T * d.H),
        ctypes.byref(tp) if tp is not None else None,
        _ptr(act, "act", _bf16(act), TMK * d.F) if act is not None else None,
        _ptr(ws, "workspace", u8), ws.numel(), _stream(stream))
    _check("moe_forward_a16w4", rc)


# ----------------------------------------------------------------------------
# Linear operators: fp8 with a scale per block of 128, 16-bit by expert
# ----------------------------------------------------------------------------

def moe_linear_workspace_bytes(d: Linear) -> int:
    return int(lib().moe_linear_workspace_bytes(ctypes.byref(d)))


def linear_workspace(d: Linear, device="cuda") -> torch.Tensor:
    """A workspace for every linear call on ``d``'s sizes, the gradients included."""
    return torch.empty(max(moe_linear_workspace_bytes(d), 256), dtype=u8, device=device)


# The smallest linear calls take 2 to 5 us on the GPU, so their host side is
# kept short: _bind (csrc/bind.cpp) checks the tensors and launches on the
# current stream in one call.  Where it finds something else than it expects (an
# explicit stream, another device, a tensor that does not fit) it launches
# nothing and returns None; the checks below then run, and say what is wrong.
# (A call of the quantiser, one row: 5.6 us with the checks in Python, 3.3 here,
# of which the launch is 3.2.)

# Where _bind is missing or was built for another torch, every call takes the
# checks in Python: the same kernels, 2 us more a call.

_bind_module = None


class _PythonChecks:
    """In place of _bind: launches nothing."""
    quant = fp8 = grouped = linear_act = act_backward = grad_clip = layer = staticmethod(lambda *a: None)


def _short():
    global _bind_module
    if _bind_module is None:
        lib()
        try:
            from . import _bind
            built = getattr(_bind, "torch_version", "of unknown version")
            if built != str(torch.__version__):
                raise ImportError(f"it was built for torch {built}, this is {torch.__version__}")
            if not hasattr(_bind, "layer"):
                raise ImportError("it was built from older sources")
            _bind_module = _bind
        except ImportError as e:
            warnings.warn(f"linear calls take longer on the host, _bind cannot be used: {e}; build it with "
                          "`python -m moe_expert_layer_sigmoid_amd.build`", RuntimeWarning, stacklevel=3)
            _bind_module = _PythonChecks
    return _bind_module


def _device(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    return t.get_device()


def _addr(t: torch.Tensor, name: str, dtype, numel_min: int, dev: int) -> int:
    """The address of a tensor that fits; _refuse says why one does not."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()
            and t.numel() >= numel_min and dev >= 0):
        return t.data_ptr()
    return _refuse(t, name, dtype, numel_min, dev)


def _refuse(t, name, dtype, numel_min, dev) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if dtype is torch.float8_e4m3fn and t.dtype is u8:   # codes as bytes
        return _addr(t, name, u8, numel_min, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, the other tensors on cuda:{dev}" if dev >= 0 else
                         f"{name}: on {t.device}, another tensor on the host")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    raise ValueError(f"{name}: {t.numel()} elements, need at least {numel_min}")


def _launch(fn: str, dev: int, stream, *args) -> None:
    """Call ``fn`` on the tensors' device, on its current stream by default."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _launch(fn, dev, stream, *args)
    st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    rc = getattr(lib(), fn)(*args, st)
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _fp8_quant(fn: str, x, q, qs, parts: int, stream) -> None:
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x: expected a torch.Tensor of two dimensions")
    rows, K = x.shape[0], x.shape[1] // parts
    if not x.is_cuda:
        raise ValueError("x: must be a device tensor")
    t = _QUANT_TYPES.get(x.dtype)
    if t is None:
        raise TypeError(f"x: dtype {x.dtype}, expected bfloat16, float16 or float32")
    if x.shape[1] != parts * K or (x.stride(1) != 1 and x.numel()):
        raise ValueError("x: the columns must be contiguous" + (" and even in number" if parts == 2 else ""))
    ldx = x.stride(0) if rows > 1 else parts * K
    if ldx < parts * K:
        raise ValueError("x: the rows must not overlap")
    dev = x.get_device()
    _launch(fn, dev, stream, rows, K, t, x.data_ptr(), ldx,
            _addr(q, "q", torch.float8_e4m3fn, rows * K, dev), _addr(qs, "qs", f32, rows * _blocks(K), dev))


def moe_fp8_quant(x, q, qs, stream=None) -> None:
    """q (float8_e4m3fn or uint8 [rows, K]) and qs (float32 [rows,
    ceil(K/128)]) of x [rows, K] (bfloat16, float16 or float32; rows may be
    further apart than K elements)."""
    rc = _short().quant(False, x, q, qs, stream)
    if rc is None:
        _fp8_quant("moe_fp8_quant", x, q, qs, 1, stream)
    elif rc:
        raise MoeError("moe_fp8_quant", rc)


def moe_fp8_swiglu_quant(x, q, qs, stream=None) -> None:
    """The same of silu(gate) * up, x [rows, 2K] holding gate | up."""
    rc = _short().quant(True, x, q, qs, stream)
    if rc is None:
        _fp8_quant("moe_fp8_swiglu_quant", x, q, qs, 2, stream)
    elif rc:
        raise MoeError("moe_fp8_swiglu_quant", rc)


def _offsets(d: Linear, offsets, dev):
    return None if offsets is None else _addr(offsets, "offsets", i32, d.groups + 1, dev)


def _scratch(ws, dev):
    return (None, 0) if ws is None else (_addr(ws, "workspace", u8, 0, dev), ws.numel())


def moe_fp8_linear(d: Linear, xq, xs, w, ws, y, scratch, offsets=None, stream=None) -> None:
    """y [rows, N] of fp8 rows xq [rows, K] with scales xs [rows, ceil(K/128)]
    and fp8 weights w [groups, N, K] with scales ws [groups, ceil(N/128),
    ceil(K/128)]; ``offsets`` int32 [groups + 1] on the device (None: one
    group of all rows)."""
    rc = _short().fp8(d, xq, xs, w, ws, y, scratch, offsets, stream)
    if rc == MOE_OK:
        return
    if rc is not None:
        raise MoeError("moe_fp8_linear", rc)
    dev = _device(y, "y")
    _launch("moe_fp8_linear", dev, stream, ctypes.byref(d),
            _addr(xq, "xq", torch.float8_e4m3fn, d.rows * d.K, dev), _addr(xs, "xs", f32, d.rows * _blocks(d.K), dev),
            _addr(w, "w", torch.float8_e4m3fn, d.groups * d.N * d.K, dev),
            _addr(ws, "ws", f32, d.groups * _blocks(d.N) * _blocks(d.K), dev), _offsets(d, offsets, dev),
            _addr(y, "y", _TORCH_TYPES[d.out_type], d.rows * d.N, dev), *_scratch(scratch, dev))


def _grouped(op, d: Linear, a, an, a_name, b, bn, b_name, out, on, out_name, scratch, offsets, stream) -> None:
    fn = _GROUPED[op]
    dev = _device(out, out_name)
    t = _TORCH_TYPES[d.in_type]
    _launch(fn, dev, stream, ctypes.byref(d), _addr(a, a_name, t, an, dev), _addr(b, b_name, t, bn, dev),
            _offsets(d, offsets, dev), _addr(out, out_name, _TORCH_TYPES[d.out_type], on, dev),
            *_scratch(scratch, dev))


_GROUPED = ("moe_grouped_linear", "moe_grouped_linear_dx", "moe_grouped_linear_dw")


def moe_grouped_linear(d: Linear, x, w, y, scratch, offsets=None, stream=None) -> None:
    """y [rows, N] = x [rows, K] times each group's w [N, K] transposed."""
    rc = _short().grouped(0, d, x, w, y, scratch, offsets, stream)
    if rc is None:
        _grouped(0, d, x, d.rows * d.K, "x", w, d.groups * d.N * d.K, "w", y, d.rows * d.N, "y", scratch, offsets, stream)
    elif rc:
        raise MoeError("moe_grouped_linear", rc)


def moe_grouped_linear_dx(d: Linear, dy, w, dx, scratch, offsets=None, stream=None) -> None:
    """dx [rows, K] = dy [rows, N] times each group's w [N, K]."""
    rc = _short().grouped(1, d, dy, w, dx, scratch, offsets, stream)
    if rc is None:
        _grouped(1, d, dy, d.rows * d.N, "dy", w, d.groups * d.N * d.K, "w", dx, d.rows * d.K, "dx", scratch, offsets,
                 stream)
    elif rc:
        raise MoeError("moe_grouped_linear_dx", rc)


def moe_grouped_linear_dw(d: Linear, dy, x, dw, scratch, offsets=None, stream=None) -> None:
    """dw [groups, N, K]: per group, dy [rows, N] transposed times x [rows, K]; zeros for an empty group."""
    rc = _short().grouped(2, d, dy, x, dw, scratch, offsets, stream)
    if rc is None:
        _grouped(2, d, dy, d.rows * d.N, "dy", x, d.rows * d.K, "x", dw, d.groups * d.N * d.K, "dw", scratch, offsets,
                 stream)
    elif rc:
        raise MoeError("moe_grouped_linear_dw", rc)


# ----------------------------------------------------------------------------
# Products with an epilogue, the gradient through it, clipping
# ----------------------------------------------------------------------------

def moe_linear_act_workspace_bytes(d: Linear) -> int:
    return int(lib().moe_linear_act_workspace_bytes(ctypes.byref(d)))


def linear_act_workspace(d: Linear, device="cuda") -> torch.Tensor:
    """A workspace for moe_grouped_linear_act and its backward on ``d``'s sizes."""
    return torch.empty(max(moe_linear_act_workspace_bytes(d), 256), dtype=u8, device=device)


def _act(act: str) -> int:
    a = ACTS.get(act)
    if a is None:
        raise ValueError(f"act: {act!r} is none of {', '.join(ACTS)}")
    return a


def _opt(t, name, dtype, numel_min, dev):
    return None if t is None else _addr(t, name, dtype, numel_min, dev)


def moe_grouped_linear_act(d: Linear, x, w, y, scratch, act: str = "none", gated: bool = False, bias=None,
                           residual=None, pre=None, offsets=None, stream=None) -> None:
    """y = act(z) + residual with z = x [rows, K] times each group's w [N, K]
    transposed, plus its bias [N] (bias: [groups, N]); ``gated``: y [rows, N/2]
    = act(z[:, :N/2]) * z[:, N/2:] + residual.  ``act``: "none", "relu", "silu",
    "gelu", "gelu_tanh".  x, w and bias of d's in_type, y, residual and pre of
    its out_type.  ``residual`` may be y; ``pre`` [rows, N] receives z."""
    a = _act(act)
    rc = _short().linear_act(d, x, w, y, scratch, a, bool(gated), bias, residual, pre, offsets, stream)
    if rc == MOE_OK:
        return
    if rc is not None:
        raise MoeError("moe_grouped_linear_act", rc)
    dev = _device(y, "y")
    t, o = _TORCH_TYPES[d.in_type], _TORCH_TYPES[d.out_type]
    n = d.rows * (d.N // 2 if gated else d.N)
    _launch("moe_grouped_linear_act", dev, stream, ctypes.byref(d), a, int(bool(gated)),
            _addr(x, "x", t, d.rows * d.K, dev), _addr(w, "w", t, d.groups * d.N * d.K, dev),
            _opt(bias, "bias", t, d.groups * d.N, dev), _opt(residual, "residual", o, n, dev), _offsets(d, offsets, dev),
            _addr(y, "y", o, n, dev), _opt(pre, "pre", o, d.rows * d.N, dev), *_scratch(scratch, dev))


def moe_grouped_linear_act_backward(d: Linear, dy, pre, dz, scratch, act: str = "none", gated: bool = False, db=None,
                                    offsets=None, stream=None) -> None:
    """dz [rows, N] (d's in_type) of dy [rows, N] (gated: N/2) and pre [rows, N]
    (its out_type), through the activation; ``db`` float32 [groups, N] receives
    the bias's gradient (zeros for an empty group)."""
    a = _act(act)
    rc = _short().act_backward(d, dy, pre, dz, scratch, a, bool(gated), db, offsets, stream)
    if rc == MOE_OK:
        return
    if rc is not None:
        raise MoeError("moe_grouped_linear_act_backward", rc)
    dev = _device(dz, "dz")
    o = _TORCH_TYPES[d.out_type]
    _launch("moe_grouped_linear_act_backward", dev, stream, ctypes.byref(d), a, int(bool(gated)),
            _addr(dy, "dy", o, d.rows * (d.N // 2 if gated else d.N), dev), _addr(pre, "pre", o, d.rows * d.N, dev),
            _offsets(d, offsets, dev), _addr(dz, "dz", _TORCH_TYPES[d.in_type], d.rows * d.N, dev),
            _opt(db, "db", f32, d.groups * d.N, dev), *_scratch(scratch, dev))


class _Tensor(ctypes.Structure):
    """moe_tensor_t"""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("type", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class GradList:
    """Tensors (bfloat16, float16 or float32, contiguous, on one device) for
    moe_grad_norm and moe_grad_clip, and where the clipped ones go: ``outs`` of
    the same sizes and types, or None for in place.  It holds the tensors, so
    that their addresses stay theirs; make a new one when gradients move."""

    def __init__(self, grads, outs=None):
        self.grads = tuple(grads)
        self.outs = self.grads if outs is None else tuple(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError(f"outs: {len(self.outs)} tensors for {len(self.grads)}")
        self.device = -1
        self._array = (_Tensor * max(len(self.grads), 1))()
        self.address = ctypes.addressof(self._array)
        spans = []
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            name = f"grads[{i}]"
            if i == 0:
                self.device = _device(g, name)
            t = _QUANT_TYPES.get(g.dtype) if isinstance(g, torch.Tensor) else None
            if isinstance(g, torch.Tensor) and t is None:
                raise TypeError(f"{name}: dtype {g.dtype}, expected bfloat16, float16 or float32")
            a = _addr(g, name, getattr(g, "dtype", None), 0, self.device)
            b = a if o is g else _addr(o, f"outs[{i}]", g.dtype, 0, self.device)
            n = g.numel()
            if o.numel() != n:
                raise ValueError(f"outs[{i}]: {o.numel()} elements, expected {n}")
            self._array[i] = _Tensor(a, b, n, t, 0)
            if n:
                size = n * g.element_size()
                spans.append((b, b + size, i, True))
                if a != b:
                    spans.append((a, a + size, i, False))
        # an output is written by one entry and read by none but its own
        spans.sort()
        end, by, out = -1, -1, False
        for lo, hi, i, is_out in spans:
            if lo < end and (is_out or out):
                raise ValueError(f"tensors {by} and {i} overlap")
            if hi > end:
                end, by, out = hi, i, is_out

    def __len__(self):
        return len(self.grads)


def moe_grad_workspace_bytes(count: int) -> int:
    return int(lib().moe_grad_workspace_bytes(int(count)))


def grad_workspace(grads: GradList, device=None) -> torch.Tensor:
    """A workspace for moe_grad_norm and moe_grad_clip on this list."""
    device = torch.device("cuda", grads.device) if device is None and grads.device >= 0 else device or "cuda"
    return torch.empty(max(moe_grad_workspace_bytes(len(grads)), 256), dtype=u8, device=device)


def _grad(fn: str, grads: GradList, norm, scratch, stream, *args) -> None:
    if not isinstance(grads, GradList):
        raise TypeError("grads: expected a GradList")
    dev = grads.device if len(grads) else _device(scratch, "workspace")
    _launch(fn, dev, stream, grads.address, len(grads), *args, _opt(norm, "norm", f32, 1, dev),
            *_scratch(scratch, dev))


def moe_grad_norm(grads: GradList, norm, scratch, stream=None) -> None:
    """norm float32 [1] = sqrt(sum of squares over all of the list's tensors)."""
    _grad("moe_grad_norm", grads, norm, scratch, stream)


def moe_grad_clip(grads: GradList, max_norm: float, norm, scratch, stream=None) -> None:
    """The list's outs = its grads times min(1, max_norm / (norm + 1e-6)); ``norm``
    (float32 [1] or None) receives the norm before."""
    if isinstance(grads, GradList):
        rc = _short().grad_clip(grads.address, len(grads.grads), max_norm, norm, scratch, grads.device, stream)
        if rc == MOE_OK:
            return
        if rc is not None:
            raise MoeError("moe_grad_clip", rc)
    _grad("moe_grad_clip", grads, norm, scratch, stream, float(max_norm))


# ----------------------------------------------------------------------------
# a16w16: the layer on unquantised experts for a few tokens
# ----------------------------------------------------------------------------

def moe_a16w16_workspace_bytes(d: Dims) -> int:
    return int(lib().moe_a16w16_workspace_bytes(ctypes.byref(d)))


def a16w16_workspace(d: Dims, device="cuda") -> torch.Tensor:
    return torch.empty(max(moe_a16w16_workspace_bytes(d), 256), dtype=u8, device=device)


def moe_forward_a16w16(d: Dims, x, logits, w1, w2, rep_count, rep_slots, out, ws, num_tokens=None, load_hist=None,
                       taps: Optional[Dict[str, torch.Tensor]] = None, stream=None) -> None:
    """The layer on bfloat16 or float16 experts w1 [P_local, 2F, H] and w2
    [P_local, H, F] for at most 32 tokens; x and out [T, H] of their type.
    ``num_tokens`` (int32 device tensor, one element): the step's token count,
    read by the kernels, for captured graphs.  ``taps``: topk_ids, topk_w,
    phys_ids."""
    if taps is None:
        rc = _short().layer(d, x, logits, w1, w2, rep_count, rep_slots, out, ws, num_tokens, load_hist, stream)
        if rc == MOE_OK:
            return
        if rc is not None:
            raise MoeError("moe_forward_a16w16", rc)
    dev = _device(out, "out")
    if not isinstance(x, torch.Tensor) or x.dtype not in _TORCH_TYPES[:2]:
        raise TypeError("x: expected a bfloat16 or float16 torch.Tensor")
    TK, _ = _sizes(d)
    t = x.dtype
    tp = None
    if taps is not None:
        tp = Taps(**{n: _opt(taps.get(n), n, dt, TK, dev) for n, dt in (("topk_ids", i32), ("topk_w", f32), ("phys_ids", i32))})
    _launch("moe_forward_a16w16", dev, stream, ctypes.byref(d), _QUANT_TYPES[t], _opt(num_tokens, "num_tokens", i32, 1, dev),
            _addr(x, "x", t, d.T * d.H, dev), _addr(logits, "logits", f32, d.T * d.E, dev),
            _addr(w1, "w1", t, d.P_local * 2 * d.F * d.H, dev), _addr(w2, "w2", t, d.P_local * d.H * d.F, dev),
            _addr(rep_count, "rep_count", i32, d.E, dev), _addr(rep_slots, "rep_slots", i32, d.E * d.R_max, dev),
            _opt(load_hist, "load_hist", i32, d.P_total, dev), _addr(out, "out", t, d.T * d.H, dev),
            ctypes.byref(tp) if tp is not None else None, *_scratch(ws, dev))
