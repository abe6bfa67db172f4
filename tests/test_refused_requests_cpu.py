"""What pkv_compact_tokens_kept refuses before anything is launched."""
import ctypes

import pytest

import paged_kv_cache_274_gb300 as pkv
from paged_kv_cache_274_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def _p(i):
    return ctypes.c_void_p(0x100000 * i)


def _call(lib, **kw):
    d = pkv.CacheDesc(num_slots=1, num_blocks=100, block_size=16, num_kv_heads=8, head_dim=128, dtype=0)
    a = dict(idx=_p(1), cnt=_p(2), A=4, B=3, cl=_p(3), nodes=None, T=8, bt=_p(4), MB=8, k=_p(5), v=_p(6), ks=None, vs=None, new=_p(8),
             prev=_p(9), seq=_p(7))
    a.update(kw)
    return lib.pkv_compact_tokens_kept(ctypes.byref(d), *[a[n] for n in ("idx", "cnt", "A", "B", "cl", "nodes", "T", "bt", "MB", "k", "v",
                                                                         "ks", "vs", "new", "prev", "seq")], None)


@pytest.mark.parametrize("bad,status", [
    (dict(new=None), 1), (dict(prev=None), 1), (dict(new=ctypes.c_void_p(0x800002)), 3), (dict(prev=ctypes.c_void_p(0x900001)), 3),
    (dict(seq=_p(8)), 1), (dict(seq=ctypes.c_void_p(0x900004)), 1), (dict(seq=_p(3)), 1), (dict(A=0), 1), (dict(seq=None), 1)])
def test_refusals(lib, bad, status):
    assert _call(lib, **bad) == status


def test_an_empty_batch_launches_nothing(lib):
    assert _call(lib, B=0, new=None, prev=None) == 0
