"""extend_tables where an ended request's row holds ids that are no blocks."""
import numpy as np
import pytest
import torch

import paged_kv_cache_274_gb300 as pkv
from tests._gpu import to_dev
from tests._tree import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,rows", [(6, 40), (6, 3000), (700, 2500)])  # one CTA, and many
@pytest.mark.parametrize("bad", [-1, "NB", 1 << 30])
def test_a_request_with_ids_that_are_no_blocks_gives_none_back(B, rows, bad, in_place):
    # nothing of it changes, the ring holds only blocks, the other requests are served as without it
    bs, MB = 16, 90
    rng = np.random.Generator(np.random.PCG64(B + rows))
    seq = rng.integers(0, 200, B)
    seq[:4] = [1200, 33, 700, 16 * MB]
    held = (-(-seq // bs)).astype(np.int32)
    NB = int(held.sum()) + 400
    ids = rng.permutation(NB).astype(np.int32)
    tables = np.full((B, MB), -7, np.int32)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    pool = Pool(NB, bs, MB, ids[at:].tolist(), head=NB - 5)
    new = np.ones(B, np.int64)
    new[[0, 1, 2, 3]] = -1
    new[4] = rows - (B - 4) - 7
    new[B // 2:][rng.random(B - B // 2) < 0.3] = -1
    new[4] = max(1, min(int(new[4]), 16 * MB - int(seq[4])))
    borrowed = np.zeros(B, np.int32)
    borrowed[1] = 2
    wrong = NB if bad == "NB" else bad
    tables[0, 70] = wrong      # one of 75
    tables[1, 0] = wrong       # borrowed, so not its to give back: its third block is
    tables[3, MB - 1] = wrong  # the row's last
    d = [to_dev(x) for x in (tables.copy(), held.copy(), pool.ring.copy(), np.array([pool.head, pool.free, 0, 0], np.int32))]
    kw = {} if in_place else dict(new_block_counts=torch.full_like(d[1], -3), new_free_state=torch.full_like(d[3], -3))
    got = pkv.extend_tables(to_dev(seq.astype(np.int32)), to_dev(new.astype(np.int32)), *d, bs, rows, borrowed_counts=to_dev(borrowed), **kw)
    assert pkv.read_device_error() & ~pkv.DEVERR_NO_BLOCKS == pkv.DEVERR_BLOCK_ID
    # the reference: those requests end without a block of theirs in the pool, and keep their counts
    counts = held.copy()
    keep_all = borrowed.copy()
    keep_all[[0, 3]] = MB
    want = pool.extend(seq, new, tables, counts, rows, keep_all)
    counts[[0, 3]] = held[[0, 3]]
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    cnt, state = (d[1], d[3]) if in_place else (kw["new_block_counts"], kw["new_free_state"])
    assert np.array_equal(cnt.cpu().numpy(), counts) and state.tolist() == [pool.head, pool.free, 0, 0]
    assert np.array_equal(d[0].cpu().numpy(), tables) and np.array_equal(d[2].cpu().numpy(), pool.ring)
    free = d[2].cpu().numpy()[(pool.head + np.arange(pool.free)) % NB]
    assert ((free >= 0) & (free < NB)).all() and len(set(free.tolist())) == len(free)
