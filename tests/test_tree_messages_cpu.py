"""What the library says about drafted-tree calls that it cannot run."""
import ctypes

import pytest

import paged_kv_cache_274_gb300 as pkv
from paged_kv_cache_274_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def _message(lib, tree, T, Hq, Hkv, math, head_dim=128):
    d = pkv.CacheDesc(num_slots=1, num_blocks=100, block_size=16, num_kv_heads=Hkv, head_dim=head_dim, dtype=0)
    fn = lib.pkv_decode_tree_describe if tree else lib.pkv_decode_multi_describe
    st = fn(ctypes.byref(d), 8, T, Hq, 64, ctypes.byref(pkv.decode_opts(math=math)), ctypes.byref(pkv.DecodePlan()))
    return st, lib.pkv_last_error_message().decode()


def test_tcgen05_limits(lib):
    # trees run with one node and with head_dim 64; linear drafts do not
    assert _message(lib, True, 1, 32, 8, pkv.MATH_TC)[0] == 0 and _message(lib, True, 4, 32, 8, pkv.MATH_TC, 64)[0] == 0
    st, text = _message(lib, True, 4, 129, 1, pkv.MATH_TC)
    assert st == 2 and "128" in text and "T >" not in text and "head_dim" not in text
    for T, D in ((1, 128), (4, 64)):
        st, text = _message(lib, False, T, 32, 8, pkv.MATH_TC, D)
        assert st == 2 and "T > 1" in text and "head_dim 128" in text


def test_trees_have_no_ffma_form(lib):
    st, text = _message(lib, True, 1, 32, 8, pkv.MATH_FFMA)
    assert st == 2 and "tree" in text
    st, text = _message(lib, False, 2, 32, 8, pkv.MATH_FFMA)
    assert st == 2 and "multi-token" in text
