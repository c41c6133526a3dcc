"""The division of the products with an epilogue into tiles and k ranges (host arithmetic, compiled for the CPU): every
plan covers K, fits the launch limits and uses a variant that exists."""
import ctypes
import os
import random
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
#include "act_plan.hpp"
extern "C" void plan(int grouped, long a, long b, long n, long k, int half, long* out) {
    const fp8k::ActPlan p = grouped ? fp8k::grouped_act_plan(a, b, n, k, half) : fp8k::act_plan(a, n, k, half);
    out[0] = p.tile, out[1] = p.stages, out[2] = p.splits, out[3] = p.split_k;
    out[4] = grouped ? 0 : (long)fp8k::act_plan_ws_bytes(p, a, n);
}
"""
MOST = (2**32 - 1) // 256 - 8


@pytest.fixture(scope="module")
def plan():
    d = tempfile.mkdtemp(prefix="actplan_")
    with open(os.path.join(d, "p.cpp"), "w") as f:
        f.write(CODE)
    lib = os.path.join(d, "p.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + os.path.join(ROOT, "fp8_w8a8_quantized_quantize_amd",
                                                                                   "csrc"), os.path.join(d, "p.cpp"), "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    L.plan.argtypes = [ctypes.c_int] + [ctypes.c_long] * 4 + [ctypes.c_int, ctypes.c_void_p]

    def call(grouped, a, b, n, k, half):
        out = (ctypes.c_long * 5)()
        L.plan(int(grouped), a, b, n, k, int(half), out)
        return list(out)

    return call


def ceil(a, b):
    return -(-a // b)


def sizes():
    rng = random.Random(5)
    some = [(17, 1, 16), (65, 1, 0), (64, 8192, 28672), (8192, 8192, 8192), (2**31 - 129, 100, 16), (100, 2**30, 16),
            (20, 300, 16384), (33, 64, 2**31 - 16), (1, 1, 16)]
    for _ in range(3000):
        m, n = (int(2 ** rng.uniform(0, 20)) for _ in range(2))
        some.append((m, n, 16 * int(2 ** rng.uniform(0, 14))))
    return some


def test_dense_plans(plan):
    splits = set()
    for M, N, K in sizes():
        if ceil(M, 128) * ceil(N, 128) > MOST:
            continue
        for half in (False, True):
            tile, stages, s, per, ws = plan(False, M, 0, N, K, half)
            kinds = {(64, 2), (64, 4), (128, 2)} | (set() if half else {(128, 4), (256, 2)})
            assert (tile, stages) in kinds, (M, N, K, half, tile, stages)
            assert ceil(M, tile) * ceil(N, tile) <= MOST
            kt = max(1, ceil(K, 128))
            splits.add(s)
            if s == 1:
                assert per >= K and ws == 0
            else:
                # every range begins inside K, all of them together end past it
                assert tile == 64 and per % 128 == 0 and (s - 1) * per < K <= s * per and 2 <= s <= 16
                assert ceil(M, tile) * ceil(N, tile) * s <= 512 and ws == s * M * N * 4 and per // 128 <= kt
    assert splits >= {1, 2, 4, 8}


def test_grouped_plans(plan):
    rng = random.Random(6)
    for _ in range(3000):
        R, E, N = int(2 ** rng.uniform(0, 24)), rng.randint(1, 1024), int(2 ** rng.uniform(0, 18))
        if (ceil(R, 128) + E) * ceil(N, 128) > MOST:
            continue
        for half in (False, True):
            tile, stages, s, _, _ = plan(True, R, E, N, 16 * rng.randint(1, 1000), half)
            assert (tile, stages) in {(64, 2), (64, 4), (128, 2)} | (set() if half else {(256, 2)})
            assert s == 1 and (ceil(R, tile) + E) * ceil(N, tile) <= MOST
