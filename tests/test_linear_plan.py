"""What the linear operators choose for the sizes of their GPU tests (no GPU
needed): csrc/linear_plan.hpp compiled by itself."""

import ctypes
import os
import shutil
import subprocess

import pytest

from tests import linear_cases as lc

HERE = os.path.dirname(os.path.abspath(__file__))
CXX = shutil.which("g++") or shutil.which("c++") or shutil.which("hipcc", path="/opt/rocm/bin:" + os.environ["PATH"])

pytestmark = pytest.mark.skipif(CXX is None, reason="no C++ compiler")

OP = {"fp8": (0, 3), "fwd": (0, 0), "dx": (1, 0), "dw": (2, 0)}   # product, input type


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run([CXX, "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-o", so,
                    os.path.join(HERE, "probe", "linear_plan.cpp")], check=True)
    lib = ctypes.CDLL(so)

    def f(kind, rows, groups, N, K):
        o = (ctypes.c_int * 6)()
        lib.linear_plan(*OP[kind], rows, N, K, groups, o)
        return dict(zip(("shape", "ta", "tb", "splits", "stages", "streams"), o))

    return f


@pytest.mark.parametrize("kind", list(OP))
def test_shapes_are_the_ones_named(plan, kind):
    seen = set()
    for shape, rows, groups, N, K in lc.SHAPES[kind]:
        p = plan(kind, rows, groups, N, K)
        assert p["shape"] == shape, (kind, rows, groups, N, K, p)
        assert p["stages"] >= lc.stages(kind, shape), (kind, rows, groups, N, K, p)
        seen.add((shape, p["splits"] > 1))
        if kind != "dw":   # tiles and stages that end inside the matrices
            assert (K if kind == "dx" else N) % p["ta"], (kind, N, K, p)
            assert (N if kind == "dx" else K) % (128 if kind == "fp8" else 64), (kind, N, K)
    shapes = set(lc.RING) - ({6} if kind == "dw" else set())   # 192 rows cannot be read transposed
    assert {s for s, _ in seen} == shapes
    assert {split for _, split in seen} == {False, True}


@pytest.mark.parametrize("kind", list(lc.STREAMED))
def test_streamed_sizes_take_the_streaming_policy(plan, kind):
    seen = set()
    for shape, rows, groups, N, K in lc.STREAMED[kind]:
        p = plan(kind, rows, groups, N, K)
        assert p["shape"] == shape and p["streams"], (kind, rows, groups, N, K, p)
        if shape >= 0:   # row tiles of the average group: within those for which weights are read once
            assert p["stages"] >= lc.stages(kind, shape), (kind, rows, groups, N, K, p)
            assert rows <= groups * p["tb"] * (8 if kind == "dx" else 1), (kind, rows, groups, N, K, p)
        seen.add((shape, p["splits"] > 1))
    assert {s for s, _ in seen} == set(lc.RING) | (set() if kind == "dx" else {-1})
    assert {split for s, split in seen if s >= 0} == {False, True}
