"""Which kernel a product takes: that of tests/_mx_plans.py for the sizes there, and for
drawn sizes one that fits a launch and the workspace that is asked for."""

import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest

from scaled_fp8_casting_amd import _lib
from scaled_fp8_casting_amd._lib import NcMxMatrix
from tests._mx_plans import CALLS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = {"e4m3": _lib.NC_E4M3, "e5m2": _lib.NC_E5M2, "e2m1": _lib.NC_E2M1}


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """Plans of (rows of a, of b, columns, format of a, of b, type of the result): (strips, units, splits) each."""
    exe = str(tmp_path_factory.mktemp("plan") / "mx_plan")
    cc = os.environ.get("CXX") or shutil.which("g++") or "c++"
    subprocess.run([cc, "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "scaled_fp8_casting_amd", "csrc"), os.path.join(ROOT, "tests", "mx_plan.cpp"), "-o", exe], check=True)

    def of(calls):
        lines = "\n".join(f"{m} {n} {k} {CODE[a]} {CODE[b]} {int(t == 'fp32')}" for m, n, k, a, b, t in calls)
        r = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True)
        got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(calls)
        return got
    return of


def test_cases(plans):
    """The tests on the GPU reach the kernels that they are written for."""
    got = plans([(m, n, k, a, b, t) for m, n, k, _, a, b, t in CALLS])
    assert [(c[:3], g) for c, g in zip(CALLS, got) if g != c[3]] == []
    assert {(g[:2], g[2] > 1) for g in got} == {((1, 0), False), ((2, 0), False), ((0, 2), False), ((0, 2), True), ((0, 4), False)}


def test_drawn(plans):
    """Launches of at most 2^32 - 1 threads; splits that the workspace asked for (for these rows and for more) holds,
    of four chunks and more, with no more than 512 tiles between them."""
    rng = random.Random(1)
    lib = _lib.load()

    def size(top):
        return int(math.exp(rng.uniform(0, math.log(top))))
    calls = []
    for _ in range(4000):
        m, n, k = size(1 << 31), size(1 << 31), size(1 << 31)
        if -(-m // 32) * -(-k // 256) < 1 << 24 and -(-n // 32) * -(-k // 256) < 1 << 24 and -(-m // 128) * -(-n // 128) < 1 << 24:
            calls.append((m, n, k, rng.choice(list(CODE)), rng.choice(list(CODE)), rng.choice(["bf16", "fp32"])))
    assert len(calls) > 500
    for (m, n, k, a, b, dtype), (t, w, splits) in zip(calls, plans(calls)):
        chunks = -(-k // 256)
        if t:
            assert t in (1, 2) and splits == 1
            assert -(-m // (32 * t)) * -(-n // (32 * t)) * 512 < 1 << 32
            continue
        tiles = -(-m // (64 * w)) * -(-n // (64 * w))
        assert w in (2, 4) and tiles * splits * 256 < 1 << 32
        assert not (w == 4 and dtype == "fp32" and (a, b) != ("e2m1", "e2m1"))
        if splits > 1:
            assert w == 2 and tiles * splits <= 512 and splits <= chunks // 4
            need = -(-m * n * 4 * splits // 256) * 256
            for rows in (m, m + 1, 3 * m):
                d = NcMxMatrix(0x10000, n, k, CODE[b], 0)
                assert lib.nc_mx_workspace_bytes(ctypes.byref(d), rows, -1) >= need
