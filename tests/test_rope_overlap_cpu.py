"""Where rope_append's queries may go: whichever rows they would overwrite before
another warp has read them is refused, in place as elsewhere.  (What may go ahead
fails later here, for want of a device, or runs on tests/test_gpu_rope_places.py.)"""
import ctypes

import pytest

from tests.test_rope_verify_cpu import _rope, lib  # noqa: F401  (a fixture)

Q, KV = 32 * 128, 8 * 128  # elements of a token's queries, keys
BASE = 0x10000000


def _at(elements):
    return ctypes.c_void_p(BASE + 2 * elements)


@pytest.mark.parametrize("kw", [
    dict(k=_at(0)),                                          # the keys are the queries' own first heads
    dict(v=_at(Q - 8)),                                      # by one 16-byte piece
    dict(k=_at(Q + 2 * KV - 8), qs=Q + 2 * KV, ks=Q + 2 * KV, os=Q + 2 * KV),  # the next token's queries
    dict(k=_at(Q), qs=Q + 2 * KV, os=Q + 2 * KV, ks=Q + KV),  # two strides
    dict(k=_at(Q + 2 * KV + 16), qs=Q + 2 * KV, ks=Q + 2 * KV, os=Q + 2 * KV),
    dict(v=_at(-KV + 8)), dict(N=1, k=_at(Q - 8)),
])
def test_in_place_over_keys_or_values(lib, kw):  # noqa: F811
    assert _rope(lib, **{**dict(out=_at(0), q=_at(0)), **kw}) == 1
    assert b"overlaps" in lib.pkv_last_error_message()


@pytest.mark.parametrize("kw", [
    dict(out=_at(0), os=Q + 8, N=2),                         # the queries themselves with another stride
    dict(out=_at(8)), dict(out=_at(Q - 8), qs=2 * Q, os=2 * Q),
])
def test_over_the_queries(lib, kw):  # noqa: F811
    assert _rope(lib, **{**dict(q=_at(0)), **kw}) == 1
    assert b"overlaps" in lib.pkv_last_error_message()
