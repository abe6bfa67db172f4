"""Attention of packed rows whose query_starts do not rise: a row is written by one
sequence at most, the sequences before the fall as if nothing followed, and no
other row at all."""
import numpy as np
import pytest

import paged_kv_cache_274_gb300 as pkv
from tests._gpu import bf16_dev_to_f64, to_dev
from tests._packed import PackedCase, packed_attention
from tests._tree import assert_tree_close
from tests.test_gpu_packed import attend

pytestmark = pytest.mark.gpu

MARK = 3.0


def check(pc, starts, kept, most=None):
    """`kept`: the sequences that are served; all others' rows keep the mark."""
    starts = np.asarray(starts, np.int32)
    got = bf16_dev_to_f64(attend(pc, starts, most, mark=MARK))
    assert pkv.read_device_error() == (pkv.DEVERR_QUERY if len(kept) < len(starts) - 1 else 0)
    ours = np.zeros(pc.N, bool)
    for b in kept:
        lo, hi = starts[b], starts[b + 1]
        ours[lo:hi] = True
        # the reference of this sequence alone
        only = np.full(len(starts), lo, np.int32)
        only[b + 1:] = hi
        out, wabs = packed_attention(pc.q, pc.c, only, pc.dc.k_host, pc.dc.v_host)
        assert_tree_close(got[lo:hi], out[lo:hi], wabs[lo:hi], f"sequence {b} of {starts.tolist()}")
    assert (got[~ours] == MARK).all(), starts.tolist()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("starts,kept,most", [
    ([0, 40, 30, 76], [0], None), ([0, 40, 30, 35], [0], None), ([30, 0, 40, 76], [], None), ([0, 40, 75, 60], [0, 1], None),
    ([-1, 40, 75, 76], [1, 2], None), ([0, 40, 75, 200], [0, 1], None), ([0, 40, 75, 76], [1, 2], 39), ([0, 2 ** 31 - 1, -2 ** 31, 5], [], None),
    ([0, 0, 40, 40], [0, 1, 2], None)])
def test_starts(dtype, starts, kept, most):
    pc = PackedCase(6440, [(40, 300), (35, 200), (1, 90)], 8, 2, 128, 16, dtype, poison=False)
    check(pc, starts, kept, most)


def test_the_rows_before_a_fall_see_their_own_values_alone():
    # sequence 2 names rows 30 .. 75, too: its new tokens' NaNs are none of sequence 0's
    pc = PackedCase(6441, [(40, 300), (35, 200), (46, 90)], 8, 2, 128, 16, poison=False)
    n, m = int(pc.c.context_lens[2]), 46
    pc.q, pc.N = pc.q[:76], 76
    for pos in (n - m + 1, n - m + 9):
        pc.dc.v[0, int(pc.c.block_tables[2, pos // 16]), :, pos % 16] = float("nan")
    check(pc, [0, 40, 30, 76], [0])


@pytest.mark.parametrize("B,fall", [(150, 149), (150, 3), (700, 650), (2500, 2300), (2500, 1)])
def test_a_fall_among_many(B, fall):
    pc = PackedCase(6442 + B, [(1, 20)] * B, 4, 1, 64, 16, poison=False)
    starts = np.arange(B + 1)
    starts[fall + 1:] = np.arange(B - fall)  # from this sequence on the rows of the first ones again
    check(pc, starts, list(range(fall)))
