"""Which rows the attention of packed rows writes, whatever query_starts holds: a
row belongs to one sequence at most, and planner and scan agree on it."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("starts") / "libpacked_starts.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-fPIC", "-shared", "-I",
                    os.path.join(ROOT, "paged_kv_cache_274_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "native", "packed_starts.cpp")], check=True)
    return ctypes.CDLL(so)


def decide(rules, starts, N, T):
    starts = np.ascontiguousarray(starts, np.int32)
    B = len(starts) - 1
    served, owner = np.zeros(B, np.int32), np.zeros(N, np.int32)
    p = lambda a: ctypes.c_void_p(a.ctypes.data)
    rules.packed_starts(p(starts), B, N, T, p(served), p(owner))
    return served.astype(bool), owner


def check(rules, starts, N, T):
    served, owner = decide(rules, starts, N, T)
    times = np.zeros(N, int)
    for b in np.flatnonzero(served):
        times[starts[b]:starts[b + 1]] += 1
        assert (owner[starts[b]:starts[b + 1]] == b).all(), (starts, b)
    assert (times <= 1).all(), (starts, np.flatnonzero(times > 1))
    assert (owner[times == 0] == -1).all(), starts
    return served


def test_rising_starts_are_all_served(rules):
    rng = np.random.Generator(np.random.PCG64(1))
    for _ in range(500):
        B = int(rng.integers(1, 40))
        starts = np.sort(rng.integers(0, 100, B + 1))  # (with sequences that have no rows)
        assert check(rules, starts, 100, 100).all()


def test_starts_that_fall(rules):
    # rows 30 .. 39 lie in two sequences that each rise by themselves
    assert check(rules, np.array([0, 40, 30, 76]), 76, 76).tolist() == [True, False, False]
    assert check(rules, np.array([0, 40, 30, 35, 76]), 76, 76).tolist() == [True, False, False, False]
    assert check(rules, np.array([0, 10, 5, 40, 20, 30]), 76, 76).tolist() == [True, False, False, False, False]
    assert check(rules, np.array([5, 0, 76]), 76, 76).tolist() == [False, False]


def test_starts_out_of_range(rules):
    assert check(rules, np.array([-1, 40, 75, 76]), 76, 76).tolist() == [False, True, True]
    assert check(rules, np.array([0, 40, 75, 200]), 76, 76).tolist() == [True, True, False]
    assert check(rules, np.array([0, 40, 75, 76]), 76, 39).tolist() == [False, True, True]


def test_any_starts(rules):
    rng = np.random.Generator(np.random.PCG64(2))
    for _ in range(3000):
        B, N = int(rng.integers(1, 9)), int(rng.integers(1, 60))
        starts = np.sort(rng.integers(-5, N + 6, B + 1))
        for _ in range(int(rng.integers(0, 3))):
            starts[rng.integers(0, B + 1)] = rng.integers(-2 ** 31, 2 ** 31) if rng.random() < 0.3 else rng.integers(-3, N + 4)
        check(rules, starts, N, int(rng.integers(1, N + 2)))
