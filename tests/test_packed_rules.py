"""The work shares of the attention of packed rows, run on the host as its
planner, its attention and its merge use them; and what the C ABI refuses."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import paged_kv_cache_274_gb300 as pkv
from paged_kv_cache_274_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rules") / "libpacked_rules.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-fPIC", "-shared", "-I",
                    os.path.join(ROOT, "paged_kv_cache_274_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "native", "packed_rules.cpp")], check=True)
    return ctypes.CDLL(so)


def shares(rules, ctx, m, Hkv, span, item_steps=3, min_steps=1, max_shares=152, alone=8):
    ctx, m = np.ascontiguousarray(ctx, np.int32), np.ascontiguousarray(m, np.int32)
    what = np.full(8, -1, np.int32)
    fault = rules.packed_shares_check(ctypes.c_void_p(ctx.ctypes.data), ctypes.c_void_p(m.ctypes.data), len(ctx), Hkv, span, span if alone == 8 else (span + 1) // 2, alone,
                                      item_steps, min_steps, max_shares, ctypes.c_void_p(what.ctypes.data))
    return fault, what.tolist()


@pytest.mark.parametrize("B,most_new,most_before,Hkv", [(1, 9000, 0, 8), (1, 5, 700, 8), (8, 600, 9000, 8), (64, 40, 4000, 2), (5, 3000, 3000, 1),
                                                        (300, 3, 500, 1), (3, 1, 130000, 2), (40, 1500, 0, 3)])
@pytest.mark.parametrize("idle", [0.0, 0.3])
def test_parts_are_read_where_they_were_written(rules, B, most_new, most_before, Hkv, idle):
    rng = np.random.Generator(np.random.PCG64(B + most_new + Hkv))
    joined = 0
    for i in range(120):
        m, before = rng.integers(1, most_new + 1, B), rng.integers(0, most_before + 1, B)
        ctx = m + before
        ctx[rng.random(B) < idle / 3] = 0                  # refused requests: rows, no cache
        m[rng.random(B) < idle / 3] = 0                    # nothing new
        short = rng.random(B) < idle / 3                   # fewer cached tokens than rows
        ctx[short] = rng.integers(0, ctx[short] + 1)
        span = int(rng.choice([1, 2, 16, 21, 32, 64, 128, 256]))
        if m.sum() / span * Hkv > 20000:
            span = 256
        item, least, most = int(rng.choice([3, 4, 6])), int(rng.choice([1, 1, 2, 8, 31])), int(rng.choice([152, 152, 76, 9, 1]))
        alone = int(rng.choice([8, 8, 6, 4, 1]))
        fault, what = shares(rules, ctx, m, Hkv, span, item, least, most, alone)
        assert fault == 0, (fault, what, ctx.tolist(), m.tolist(), span, item, least, most, alone)
        joined += what[1]
    assert joined > 0 or most_new + most_before < 640  # (items of four steps are not split)


def test_no_share_lies_within_a_step(rules):
    # shares of a little less than a step: two boundaries in the second step of (sequence 0, KV head 2)
    fault, what = shares(rules, [287, 251], [37, 250], 4, 64)
    assert fault == 0, what
    for n in range(129, 700):
        for hkv in (1, 3, 8):
            fault, what = shares(rules, [n], [min(n, 37)], hkv, 64, 4)
            assert fault == 0, (n, hkv, what)


def test_nothing_to_share(rules):
    assert shares(rules, [], [], 8, 64)[0] == 0
    fault, what = shares(rules, [0, 5, 0], [3, 0, 0], 8, 64)
    assert fault == 0 and what[0] == 0


def test_shares_of_a_long_prompt_are_equal(rules):
    # (items that cost nothing by themselves, so that a share's cost is its steps)
    fault, what = shares(rules, [8192], [8192], 8, 64, item_steps=0)
    assert fault == 0 and what[0] == 152 and what[7] <= 1.1 * what[6]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def _p(i):
    return ctypes.c_void_p(0x10000000 * i)


def _call(lib, desc=None, **kw):
    d = dict(num_slots=2, num_blocks=100, block_size=16, num_kv_heads=8, head_dim=128, dtype=0)
    d.update(desc or {})
    a = dict(q=_p(1), N=40, B=4, T=40, Hq=32, k=_p(2), v=_p(3), ks=None, vs=None, bt=_p(4), MB=20, ctx=_p(5), starts=_p(6), gp=[0, 1],
             L=2, layer=1, scale=0.1, out=_p(7), ws=_p(8), size=1 << 40, opts=None)
    a.update(kw)
    gp = (ctypes.c_int32 * len(a["gp"]))(*a["gp"]) if a["gp"] is not None else None
    opts = ctypes.byref(a["opts"]) if a["opts"] is not None else None
    return lib.pkv_paged_decode_packed(ctypes.byref(pkv.CacheDesc(**d)), a["q"], a["N"], a["B"], a["T"], a["Hq"], a["k"], a["v"], a["ks"],
                                       a["vs"], a["bt"], a["MB"], a["ctx"], a["starts"], gp, a["L"], a["layer"], a["scale"], a["out"],
                                       a["ws"], a["size"], opts, None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(N=-1)), (1, dict(B=-1)), (1, dict(T=0)), (1, dict(MB=0)), (1, dict(Hq=0)), (1, dict(Hq=30)), (2, dict(Hq=8 * 129)),
    (2, dict(N=1 << 20, Hq=32)), (2, dict(opts=pkv.decode_opts(math=pkv.MATH_MMA))), (1, dict(opts=pkv.decode_opts(partition_blocks=257))),
    (1, dict(gp=None)), (1, dict(layer=2)), (1, dict(layer=-1)), (1, dict(gp=[0, 2])), (1, dict(scale=float("nan"))), (1, dict(q=None)),
    (1, dict(k=None)), (1, dict(v=None)), (1, dict(bt=None)), (1, dict(ctx=None)), (1, dict(starts=None)), (1, dict(out=None)),
    (6, dict(ws=None)), (6, dict(size=1000)), (3, dict(q=ctypes.c_void_p(0x10000008))), (3, dict(ws=ctypes.c_void_p(0x80000008))),
    (3, dict(starts=ctypes.c_void_p(0x60000002))), (1, dict(out=_p(1))), (1, dict(out=_p(2))), (1, dict(out=_p(6))),
    (1, dict(desc=dict(dtype=1))), (3, dict(desc=dict(dtype=1), ks=ctypes.c_void_p(0x90000002), vs=_p(10))),
    (2, dict(desc=dict(block_size=8))), (2, dict(desc=dict(dtype=2, head_dim=64), Hq=8)),
])
def test_refused(lib, want, kw):
    assert _call(lib, **kw) == want, lib.pkv_last_error_message()


def test_nothing_to_attend(lib):
    assert _call(lib, N=0, q=None, out=None, ws=None, size=0) == 0
    assert _call(lib, B=0, ws=None, size=0) == 0


def test_workspace_bytes(lib):
    d = pkv.CacheDesc(1, 100, 16, 8, 128, 0)
    size = lambda N, B, T: lib.pkv_decode_packed_workspace_bytes(ctypes.byref(d), N, B, T, 32, 64, None)
    # partials: 152 shares x 2 places x 128 rows (a pair of tiles: 256) x (128 + 2) floats
    assert size(64, 64, 1) < 152 * 2 * 128 * 130 * 4 + 100000 < size(64, 64, 64)
    assert size(1000, 4, 0) == 0 and size(-1, 4, 5) == 0
