"""Host side of the linear operators: the descriptor's range, and calls where
the native binding cannot be used."""

import os
import sys
import types
import warnings

import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx


@pytest.mark.parametrize("name", ["rows", "N", "K", "groups"])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 3, -2 ** 31 - 1, 2 ** 64])
def test_descriptor_refuses_what_32_bits_do_not_hold(name, value):
    """2^32 + 3 rows would otherwise be 3 rows without a word."""
    with pytest.raises(ValueError, match=name):
        mx.Linear(**{**dict(rows=4, N=16, K=16, groups=1), name: value})


def test_descriptor_keeps_32_bit_values():
    d = mx.Linear(2 ** 31 - 1, -1, -2 ** 31, groups=7)
    assert (d.rows, d.N, d.K, d.groups) == (2 ** 31 - 1, -1, -2 ** 31, 7)


needs_lib = pytest.mark.skipif(not os.path.exists(mx.LIB_PATH), reason="libmoe.so not built")


def _refused_by_python(match):
    """Every operator's call reaches the checks in Python, which name the argument."""
    x, w, y = torch.zeros(2, 16).bfloat16(), torch.zeros(1, 16, 16).bfloat16(), torch.zeros(2, 16).bfloat16()
    q, s = torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1)
    with pytest.warns(RuntimeWarning, match=match):
        with pytest.raises(ValueError, match="x: must be a device tensor"):
            mx.moe_fp8_quant(x, q, s)
    with pytest.raises(ValueError, match="x: must be a device tensor"):
        mx.moe_fp8_swiglu_quant(torch.zeros(2, 32), q, s)
    with pytest.raises(ValueError, match="xq: must be a device tensor"):
        mx.moe_fp8_linear(mx.Linear(2, 16, 16, in_type="fp8"), q, s, torch.zeros(16, 16, dtype=torch.uint8),
                          torch.zeros(1), y, None)
    d = mx.Linear(2, 16, 16)
    for f, a, b, out in ((mx.moe_grouped_linear, x, w, y), (mx.moe_grouped_linear_dx, y, w, x),
                         (mx.moe_grouped_linear_dw, y, x, w)):
        with pytest.raises(ValueError, match="must be a device tensor"):
            f(d, a, b, out, None)


@needs_lib
def test_calls_without_the_native_binding(monkeypatch):
    monkeypatch.setattr(mx, "_bind_module", None)
    monkeypatch.delattr(mx, "_bind", raising=False)
    monkeypatch.setitem(sys.modules, mx.__name__ + "._bind", None)   # its import fails
    _refused_by_python("_bind")


@needs_lib
def test_calls_with_a_native_binding_for_another_torch(monkeypatch):
    other = types.ModuleType(mx.__name__ + "._bind")
    other.torch_version = "0.0"
    other.quant = other.fp8 = other.grouped = lambda *a: pytest.fail("used")
    monkeypatch.setattr(mx, "_bind_module", None)
    monkeypatch.setattr(mx, "_bind", other, raising=False)
    monkeypatch.setitem(sys.modules, other.__name__, other)
    _refused_by_python("built for torch 0.0")


@needs_lib
def test_native_binding_is_for_this_torch(monkeypatch):
    monkeypatch.setattr(mx, "_bind_module", None)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert mx._short().torch_version == torch.__version__
