"""Rules that the kernels keep in headers without CUDA, run on the host: every
order in which the staging warps may run, and the work shares of the
drafted-tree attention as its planner, its attention and its merge use them."""
import ctypes

import numpy as np
import pytest

from tests import _host_rules

WARPS = 4


@pytest.fixture(scope="module")
def rules():
    return _host_rules.build()


def _programs(units):
    """What each warp of the output staging does, in order, as (op, argument):
    the kernel's loops over a unit's chunks.  A unit is "direct" (two chunks)
    or "split" (four; a buffer is restaged once it has been read).  "meet"
    stands for the next unit's steps, which need every warp's P."""
    progs = [[] for _ in range(WARPS)]
    chunk = reads = 0
    for unit in units:
        first = chunk
        for k in range(2 if unit == "direct" else 4):
            for w in range(WARPS):
                if unit == "split" and k >= 2:
                    progs[w].append(("read", reads + k - 2))
                progs[w].append(("write", chunk))
                progs[w].append(("arrive", chunk))
            progs[0].append(("store", chunk))
            if unit == "split" and k in (1, 2):
                progs[0].append(("release", first + k - 1))
            chunk += 1
        reads += 2 if unit == "split" else 0
        for w in range(WARPS):
            progs[w].append(("meet", None))
    return progs


def _early_store(units, bar, parity, nbars):
    """Runs every interleaving; returns the first chunk that is stored before
    every warp has written it (None: there is none), and whether some order
    gets stuck."""
    progs = _programs(units)
    start = (tuple([0] * WARPS), tuple([(0, 0)] * nbars), 0, tuple([0] * WARPS))
    seen, todo, stuck = {start}, [start], False
    while todo:
        pc, bars, reads, written = todo.pop()  # bars: (phases completed, arrivals); reads: stores that have read
        at = [progs[w][pc[w]] if pc[w] < len(progs[w]) else None for w in range(WARPS)]
        moves = []
        if all(a == ("meet", None) for a in at):
            moves.append((tuple(p + 1 for p in pc), bars, reads, written))
        for w, a in enumerate(at):
            if a is None or a[0] == "meet":
                continue
            op, n = a
            b2, r2, w2 = bars, reads, written
            if op == "write":
                w2 = written[:w] + (n + 1,) + written[w + 1:]
            elif op == "arrive":
                done, count = bars[bar(n)]
                count += 1
                done, count = (done + 1, 0) if count == WARPS else (done, count)
                b2 = bars[:bar(n)] + ((done, count),) + bars[bar(n) + 1:]
            elif op == "store":
                if bars[bar(n)][0] % 2 == parity(n):  # the phase is open (a parity wait sees no more)
                    continue
                if any(x <= n for x in written):
                    return n, stuck
            elif op == "release":
                r2 = reads + 1
            elif op == "read" and reads % 2 == n % 2:
                continue
            moves.append((pc[:w] + (pc[w] + 1,) + pc[w + 1:], b2, r2, w2))
        if not moves and any(a is not None for a in at):
            stuck = True
        for m in moves:
            if m not in seen:
                seen.add(m)
                todo.append(m)
    return None, stuck


@pytest.mark.parametrize("units", [["direct"], ["split"], ["direct", "direct", "direct"], ["split", "direct", "split"],
                                   ["direct", "split", "direct"]])
def test_no_chunk_is_stored_before_every_warp_has_staged_it(rules, units):
    assert _early_store(units, rules.stage_bar_of, rules.stage_parity_of, rules.stage_bars_count()) == (None, False)


def test_one_barrier_for_neighbouring_chunks_stores_too_early():
    # why there are two: with one, a fast warp's second arrival stands in for a slow warp's first
    assert _early_store(["direct"], lambda n: 0, lambda n: n & 1, 1)[0] == 0
    assert _early_store(["split"], lambda n: 0, lambda n: n & 1, 1)[0] == 0


def _shares(rules, lens, Hkv, item_steps=4, min_steps=1, max_shares=152):
    """(fault, shares, joined items, where) of these lengths."""
    ctx = np.ascontiguousarray(lens, np.int32)
    what = np.full(5, -1, np.int32)
    fault = rules.tree_shares_check(ctypes.c_void_p(ctx.ctypes.data), len(ctx), Hkv, item_steps, min_steps, max_shares,
                                    ctypes.c_void_p(what.ctypes.data))
    return fault, int(what[0]), int(what[1]), what[2:].tolist()


# a boundary that moves past a sequence's last item, an inactive sequence behind
# it, and a split item after that
@pytest.mark.parametrize("lens,Hkv,min_steps", [([30295, 0, 31051, 30690], 8, 1), ([257, 0, 650], 2, 8)])
def test_shares_beside_an_inactive_sequence(rules, lens, Hkv, min_steps):
    fault, shares, joined, where = _shares(rules, lens, Hkv, min_steps=min_steps)
    assert fault == 0, (fault, where)
    assert shares > 1 and joined > 0


@pytest.mark.parametrize("B,lo,hi,Hkv", [(32, 2000, 8000, 2), (8, 4000, 16000, 8), (4, 8000, 32000, 8), (64, 1, 700, 3), (300, 0, 900, 1),
                                         (5, 1, 2000, 128), (2, 1, 130000, 1)])
@pytest.mark.parametrize("inactive", [0.0, 0.1, 0.6])
def test_parts_are_read_where_they_were_written(rules, B, lo, hi, Hkv, inactive):
    rng = np.random.Generator(np.random.PCG64(B + Hkv))
    joined = 0
    for i in range(300):
        lens = rng.integers(lo, hi + 1, B)
        lens[rng.random(B) < inactive] = 0
        item, least, most = int(rng.choice([3, 4, 6])), int(rng.choice([1, 1, 2, 8, 31])), int(rng.choice([152, 152, 76, 9, 1]))
        fault, _, n, where = _shares(rules, lens, Hkv, item, least, most)
        assert fault == 0, (fault, where, lens.tolist(), item, least, most)
        joined += n
    assert joined > 0


def test_shares_of_nothing(rules):
    assert _shares(rules, [0, 0, 0], 8)[:3] == (0, 0, 0)
    assert _shares(rules, [], 8)[:3] == (0, 0, 0)
