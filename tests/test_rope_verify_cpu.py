"""rope_append and verify_tree without a GPU: what the C ABI refuses before
anything is launched."""
import ctypes
import math

import pytest

import paged_kv_cache_274_gb300 as pkv
from paged_kv_cache_274_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def _p(i):
    return ctypes.c_void_p(0x10000000 * i)


def _rope(lib, desc=None, freqs=None, axes=None, **kw):
    d = dict(num_slots=2, num_blocks=100, block_size=16, num_kv_heads=8, head_dim=128, dtype=0)
    d.update(desc or {})
    R = kw.get("R", 128)
    freqs = [0.5] * 64 if freqs is None else freqs
    a = dict(slot=0, q=_p(1), qs=32 * 128, k=_p(2), ks=1024, v=_p(3), vs=1024, N=4, Hq=32, qw=None, kw=None, eps=1e-6, pos=_p(4),
             num_axes=1, R=R, inter=0, slots=_p(5), out=_p(6), os=32 * 128, kc=_p(7), vc=_p(8), ksc=None, vsc=None)
    a.update(kw)
    f = (ctypes.c_double * len(freqs))(*freqs) if freqs else None
    x = (ctypes.c_int32 * len(axes))(*axes) if axes else None
    return lib.pkv_rope_append(ctypes.byref(pkv.CacheDesc(**d)), a["slot"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["N"],
                               a["Hq"], a["qw"], a["kw"], a["eps"], a["pos"], a["num_axes"], f, x, a["R"], a["inter"], a["slots"],
                               a["out"], a["os"], a["kc"], a["vc"], a["ksc"], a["vsc"], None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(slot=2)), (1, dict(slot=-1)), (1, dict(N=-1)), (1, dict(Hq=0)), (2, dict(R=24)), (2, dict(R=144)), (2, dict(R=-16)),
    (1, dict(inter=2)), (1, dict(eps=-1.0)), (1, dict(eps=math.nan)), (1, dict(eps=math.inf)), (1, dict(k=None)), (1, dict(v=None)),
    (1, dict(qs=32 * 128 - 8)), (1, dict(ks=1016)), (1, dict(vs=1016)), (1, dict(os=0)), (3, dict(qs=32 * 128 + 4)), (3, dict(ks=1028)),
    (2, dict(qs=1 << 31)), (1, dict(num_axes=0)), (1, dict(num_axes=5)), (1, dict(freqs=[])), (1, dict(freqs=[0.5] * 63 + [math.nan])),
    (1, dict(freqs=[math.inf] * 64)), (1, dict(axes=[0] * 63 + [1])), (1, dict(axes=[-1] * 64)), (1, dict(q=None)), (1, dict(out=None)),
    (1, dict(pos=None)), (1, dict(slots=None)), (3, dict(q=ctypes.c_void_p(0x10000008))), (3, dict(qw=ctypes.c_void_p(0x90000008))),
    (3, dict(pos=ctypes.c_void_p(0x40000002))), (3, dict(slots=ctypes.c_void_p(0x50000004))), (1, dict(out=_p(2))), (1, dict(out=_p(5))),
    (1, dict(out=ctypes.c_void_p(0x10000000 + 4096))), (1, dict(out=_p(7))), (1, dict(os=32 * 128 + 8, out=_p(1))),
    (1, dict(desc=dict(dtype=1))), (1, dict(desc=dict(dtype=2), ksc=_p(9))), (3, dict(desc=dict(dtype=2), ksc=_p(9), vsc=ctypes.c_void_p(0xa0000004))),
    (2, dict(desc=dict(head_dim=96))), (2, dict(desc=dict(dtype=1, head_dim=64), R=64)), (2, dict(N=1 << 26)), (2, dict(N=(1 << 31) - 1)),
])
def test_rope_append_refuses(lib, want, kw):
    assert _rope(lib, **kw) == want, lib.pkv_last_error_message()


def test_rope_append_nothing_to_do(lib):
    assert _rope(lib, N=0, q=None, out=None) == 0


def _verify(lib, **kw):
    a = dict(tokens=_p(1), parents=_p(2), counts=None, p=_p(3), ps=1000, q=_p(4), qs=1000, B=4, T=8, V=1000, r=_p(5), u=_p(6), idx=_p(7),
             cnt=_p(8), A=8, nxt=_p(9))
    a.update(kw)
    return lib.pkv_verify_tree(a["tokens"], a["parents"], a["counts"], a["p"], a["ps"], a["q"], a["qs"], a["B"], a["T"], a["V"], a["r"],
                               a["u"], a["idx"], a["cnt"], a["A"], a["nxt"], None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(B=-1)), (1, dict(T=0)), (1, dict(T=513)), (1, dict(A=0)), (1, dict(A=513)), (1, dict(V=0)), (2, dict(V=(1 << 20) + 1, ps=1 << 21, qs=1 << 21)),
    (1, dict(ps=999)), (1, dict(qs=999)), (1, dict(ps=-1)), (2, dict(ps=1 << 41)), (2, dict(B=1 << 22)), (1, dict(tokens=None)), (1, dict(parents=None)),
    (1, dict(p=None)), (1, dict(r=None)), (1, dict(u=None)), (1, dict(idx=None)), (1, dict(cnt=None)), (1, dict(nxt=None)),
    (3, dict(p=ctypes.c_void_p(0x30000002))), (3, dict(counts=ctypes.c_void_p(0xb0000001))), (1, dict(idx=_p(1))), (1, dict(nxt=_p(8))),
    (1, dict(cnt=_p(3))), (1, dict(nxt=ctypes.c_void_p(0x70000000 + 4 * 31))),
])
def test_verify_tree_refuses(lib, want, kw):
    assert _verify(lib, **kw) == want, lib.pkv_last_error_message()


def test_verify_tree_nothing_to_do(lib):
    assert _verify(lib, B=0, tokens=None) == 0
