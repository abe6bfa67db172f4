"""The work shares of the attention of packed rows: one an SM, never more than the
workspace has room for."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("grid") / "libpacked_grid.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-fPIC", "-shared", "-I",
                    os.path.join(ROOT, "paged_kv_cache_274_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "native", "packed_grid.cpp")], check=True)
    lib = ctypes.CDLL(so)
    lib.used_shares.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return lib


@pytest.mark.parametrize("sms", [1, 2, 20, 76, 132, 148, 151, 152, 160, 304])
def test_one_share_an_sm(rules, sms):
    assert rules.launch_shares(sms) == min(sms, rules.workspace_shares())
    assert rules.used_shares(1 << 50, 1, sms) == min(sms, rules.workspace_shares())
    assert rules.used_shares(0, 1, sms) == 0 and rules.used_shares(1, 1, sms) == 1


def test_a_device_without_a_count(rules):
    assert rules.launch_shares(0) == 1
