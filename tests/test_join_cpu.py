"""The join of partials' references (csrc/pa_join.h), compiled for the host: a piece
that met a bad page keeps its mark (+inf) whatever it is joined with, NaN included."""
import ctypes
import itertools
import math
import os
import shutil
import subprocess

import pytest

from paged_kv_attention_16_gb300 import build as pbuild

NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def join(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    out = tmp_path_factory.mktemp("join")
    src, lib = out / "join.cpp", out / "join.so"
    src.write_text('#include "pa_join.h"\n'
                   'extern "C" float join_top(float a, float b) { return pa::join_top(a, b); }\n')
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.abspath(pbuild.CSRC), str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).join_top
    f.argtypes, f.restype = [ctypes.c_float] * 2, ctypes.c_float
    return f


def wanted(parts):
    if INF in parts:
        return INF
    if any(x != x for x in parts):
        return NAN
    return max(parts)


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_every_order(join, n):
    for parts in itertools.product([NAN, INF, -INF, 0.0, 3.5, -100.0, 3.4e38], repeat=n):
        top = -INF  # as a row without partials begins
        for x in parts:
            top = join(top, x)
        want = wanted([ctypes.c_float(x).value for x in parts])
        assert top == want or (top != top and want != want), parts


def test_groups_that_meet(join):
    """Sums over pieces taken by several groups of lanes, joined in any order."""
    for parts in itertools.permutations([NAN, INF, 1.0, -INF, NAN, 2.0]):
        a, b = -INF, -INF
        for x in parts[:3]:
            a = join(a, x)
        for x in parts[3:]:
            b = join(b, x)
        assert join(a, b) == INF and join(b, a) == INF
