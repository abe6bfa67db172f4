"""The fractions of a turn that the rotary append keeps its frequencies as, in 64
bits, against exact ones: the position multiplies what they are off by."""
import ctypes
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from tests._turns import turns

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kept(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("turns") / "librope_turns.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I",
                    os.path.join(ROOT, "paged_kv_cache_274_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "native", "rope_turns.cpp")], check=True)
    lib = ctypes.CDLL(so)
    lib.rope_turns.restype, lib.rope_turns.argtypes = ctypes.c_uint64, [ctypes.c_double]
    return lib.rope_turns


def _off(kept, freq):
    """What the kept fraction is off by, in 2^-64 of a turn."""
    d = (Fraction(kept(float(freq)), 1 << 64) - turns(freq)) % 1
    return float(min(d, 1 - d) * (1 << 64))


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e6])
def test_usual_tables(kept, base):
    # two parts of the quotient, each to its unit
    for R in (16, 32, 64, 96, 128):
        for f in base ** (-2.0 * np.arange(R // 2) / R):
            assert _off(kept, f) <= 2.0, f


def test_frequencies_of_any_size(kept):
    rng = np.random.Generator(np.random.PCG64(4))
    some = np.concatenate([[0.0, -0.0, 1.0, -1.0, 2 * np.pi, -2 * np.pi, np.pi, 100.0, 1e9, 2.0 ** 40, 5e-324, -1e-300, -1e-19, 1e-20],
                           np.exp2(rng.uniform(-70, 40, 3000)) * rng.choice([-1.0, 1.0], 3000)])
    for f in some:
        assert _off(kept, f) <= 2.0, f


def test_an_angle_far_away(kept):
    # the header's bound on angles, 2^-26 of half a turn, leaves the frequency 2^-28 of one at any position
    for f in (1.0, 0.7, -3.0, 6.0, 100.0, 1e-3):
        for pos in (2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 131071):
            d = (Fraction((pos * kept(f)) % (1 << 64), 1 << 64) - turns(f, pos)) % 1
            assert float(min(d, 1 - d)) * 2 <= 2.0 ** -28, (f, pos)
