"""The polynomial behind gelu (csrc/gelu_tail.hpp, no GPU needed): the errors that
its comment states."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
from scipy.special import erfcx

HERE = os.path.dirname(os.path.abspath(__file__))
CXX = shutil.which("g++") or shutil.which("c++") or shutil.which("hipcc", path="/opt/rocm/bin:" + os.environ["PATH"])

pytestmark = pytest.mark.skipif(CXX is None, reason="no C++ compiler")


@pytest.fixture(scope="module")
def tail(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("tail") / "tail.so")
    subprocess.run([CXX, "-O1", "-std=c++17", "-ffp-contract=off", "-Wall", "-Werror", "-shared", "-fPIC", "-o", so,
                    os.path.join(HERE, "probe", "gelu_tail.cpp")], check=True)
    lib = ctypes.CDLL(so)
    lib.gelu_tail_f32.argtypes, lib.gelu_tail_f32.restype = [ctypes.c_float], ctypes.c_float
    lib.gelu_tail_f64.argtypes, lib.gelu_tail_f64.restype = [ctypes.c_double], ctypes.c_double
    return lib


def test_half_at_zero(tail):
    assert tail.gelu_tail_f32(0.0) == 0.5
    assert abs(tail.gelu_tail_f64(0.0) - 0.5) <= 1e-15


def test_errors_over_the_range(tail):
    a = np.concatenate([np.linspace(0.0, 27.0, 20001), np.geomspace(1e-7, 2.0, 5001)]).astype(np.float32).astype(np.float64)
    ref = 0.5 * erfcx(a / np.sqrt(2.0))
    f64 = np.array([tail.gelu_tail_f64(v) for v in a])
    f32 = np.array([tail.gelu_tail_f32(v) for v in a])
    assert np.max(np.abs(f64 / ref - 1)) <= 5.25e-8
    assert np.max(np.abs(f32 / ref - 1)) <= 6 * 2.0 ** -24
