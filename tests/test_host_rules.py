"""Rules that the kernels keep in headers without CUDA, run on the host: every
order in which the staging warps may run."""
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
    assert _early_store(units, rules.stage_bar, rules.stage_parity, rules.stage_bars()) == (None, False)


def test_one_barrier_for_neighbouring_chunks_stores_too_early():
    # why there are two: with one, a fast warp's second arrival stands in for a slow warp's first
    assert _early_store(["direct"], lambda n: 0, lambda n: n & 1, 1)[0] == 0
    assert _early_store(["split"], lambda n: 0, lambda n: n & 1, 1)[0] == 0
