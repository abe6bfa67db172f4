"""V rows that are not finite among a long run of new tokens: every later row of the
sequence is NaN in every column, in the row tiles behind the token's own too, and
no other row is changed."""
import numpy as np
import pytest

import paged_kv_cache_274_gb300 as pkv
from tests._gpu import bf16_dev_to_f64
from tests._packed import PackedCase
from tests._tree import assert_tree_close
from tests.test_gpu_packed import attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype,Hq,Hkv,seqs,bad", [
    (128, "bf16", 16, 2, [(7, 40), (400, 190), (1, 50), (90, 0)], [(1, 20), (3, 1)]),
    (128, "bf16", 8, 2, [(900, 0), (300, 1000)], [(0, 3), (1, 299)]),
    (64, "bf16", 8, 4, [(33, 7), (700, 130)], [(1, 1), (1, 350)]),
    (128, "fp8", 32, 4, [(177, 190), (5, 900), (260, 3)], [(0, 20), (2, 40)]),
    (128, "bf16", 32, 1, [(40, 300), (30, 0)], [(0, 2)]),       # four rows a tile
    (128, "fp8", 128, 1, [(9, 200), (6, 0)], [(0, 3), (1, 1)]),  # a row a tile
])
@pytest.mark.parametrize("share", [0, 24])
def test_values_of_early_new_tokens(D, dtype, Hq, Hkv, seqs, bad, share):
    pc = PackedCase(6470 + D + Hq + len(seqs), seqs, Hq, Hkv, D, 16, dtype, poison=False)
    opts = pkv.decode_opts(partition_blocks=share)
    clean, wabs = pc.reference()
    G = Hq // Hkv
    lost = np.zeros((pc.N, Hq), bool)
    for i, (b, u) in enumerate(bad):
        m, n = seqs[b][0], sum(seqs[b])
        pos, h = n - m + u, (i + 1) % Hkv
        at = (0, int(pc.c.block_tables[b, pos // 16]), h, pos % 16, (37 * i + 5) % D)  # one element
        pc.dc.v[at] = 0x7f if dtype == "fp8" else float("inf" if i else "nan")
        lost[pc.starts[b] + u:pc.starts[b + 1], h * G:(h + 1) * G] = True
    got = bf16_dev_to_f64(attend(pc, opts=opts))
    assert pkv.read_device_error() == 0
    assert np.isnan(got[lost]).all(), f"{(~np.isnan(got[lost]).all(-1)).sum()} of {lost.sum()} rows are not NaN in every column"
    assert_tree_close(np.where(lost[..., None], clean, got), clean, wabs, "the other rows")
