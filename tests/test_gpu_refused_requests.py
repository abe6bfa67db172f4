"""Requests that extend_tables refuses keep their tokens through the step:
compaction with the step's new_lens and prev_seq_lens, alone and in a loop
whose pool runs out."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_274_gb300 as pkv
from workloads import normal_bf16_bits, random_case
from tests._gpu import DEV, DeviceCase, bf16_dev_to_f64, to_dev, to_dev_bf16
from tests._tree import Pool, assert_tree_close, compact, pack, random_parents, tree_attention, visible

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S", [1, 3])
def test_inactive_sequences_keep_what_they_had(in_place, S):
    # served; refused, its counts of any value; ended; refused with nothing cached; served without nodes
    T, lens = 10, [30, 0, 0, 0, 25]
    c = random_case(9700 + S, 5, 4, 2, 128, 16, lens, S=S, MB=4)
    dc = DeviceCase(c)
    nodes = np.array([10, 99, 7, -4, 0], np.int32)
    idx = np.array([[1, 3, 7], [5, 5, 5], [0, 1, 2], [-9, 0, 0], [0, 0, 0]], np.int32)
    count = np.array([3, 77, 3, -1, 0], np.int32)
    new, prev = np.array([10, 12, -1, 50, 5], np.int32), np.array([20, 41, 33, 0, 20], np.int32)
    wk = compact(dc.k_host, idx[:1], count[:1], lens, nodes, c.block_tables)
    wv = compact(dc.v_host, idx[:1], count[:1], lens, nodes, c.block_tables)
    d_prev = to_dev(prev.copy())
    seq = pkv.compact_tokens(to_dev(idx), to_dev(count), dc.cl, dc.bt, dc.k, dc.v, T, node_counts=to_dev(nodes),
                             seq_lens=d_prev if in_place else None, new_lens=to_dev(new), prev_seq_lens=d_prev)
    assert pkv.read_device_error() == 0
    assert seq.tolist() == [23, 41, 0, 0, 25]
    assert d_prev.tolist() == (seq.tolist() if in_place else prev.tolist())
    assert np.array_equal(_bits(dc.k), wk) and np.array_equal(_bits(dc.v), wv)


def test_one_without_the_other_and_other_overlaps_are_refused():
    c = random_case(9710, 2, 4, 2, 128, 16, [30, 20])
    dc = DeviceCase(c)
    a = torch.zeros(5, dtype=torch.int32, device=DEV)
    args = (torch.zeros((2, 1), dtype=torch.int32, device=DEV), a[:2].clone(), dc.cl, dc.bt, dc.k, dc.v, 4)
    for kw in (dict(new_lens=a[:2]), dict(prev_seq_lens=a[:2]), dict(new_lens=a[:3], prev_seq_lens=a[:2]),
               dict(new_lens=a[:2], prev_seq_lens=a[2:4], seq_lens=a[1:3]), dict(new_lens=a[:2], prev_seq_lens=a[2:4], seq_lens=a[:2])):
        with pytest.raises(pkv.PkvError):
            pkv.compact_tokens(*args, **kw)


@pytest.mark.parametrize("graph", [False, True])
def test_a_loop_whose_pool_runs_out(graph):
    """Requests grow until one gets no blocks; it waits, with its prompt, while
    others go on and end, and is served from their blocks later.  The lengths
    stay on the GPU, updated in place by the compaction."""
    B, T, Hq, Hkv, D, bs, MB, NB, N = 3, 12, 16, 4, 128, 16, 12, 12, 130
    rng = np.random.Generator(np.random.PCG64(9720))
    k_host = normal_bf16_bits(9721, (1, NB, Hkv, bs, D))
    v_host = normal_bf16_bits(9722, (1, NB, Hkv, bs, D))
    k, v = to_dev_bf16(k_host), to_dev_bf16(v_host)
    pool = Pool(NB, bs, MB, rng.permutation(NB).tolist())
    ring, state = pkv.new_free_ring(pool.ring, NB)
    tables, counts = np.full((B, MB), -1, np.int32), np.zeros(B, np.int32)
    bt, cnt = to_dev(tables.copy()), to_dev(counts.copy())

    def ints(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=DEV)

    buf = dict(seq=ints(B), new=ints(B), parents=ints(B, T), nodes=ints(B), idx=ints(B, 4), acc=ints(B),
               q=torch.zeros((B, T, Hq, D), dtype=torch.bfloat16, device=DEV),
               kn=torch.zeros((N, Hkv, D), dtype=torch.bfloat16, device=DEV), vn=torch.zeros((N, Hkv, D), dtype=torch.bfloat16, device=DEV))
    out = torch.zeros((B, T, Hq, D), dtype=torch.bfloat16, device=DEV)
    ws = torch.full((pkv.decode_workspace_bytes(k, B, Hq, MB, None, T, tree=True),), 0xFF, dtype=torch.uint8, device=DEV)

    def step():
        ctx, _, slots, _ = pkv.extend_tables(buf["seq"], buf["new"], bt, cnt, ring, state, bs, N)
        pkv.kv_append(buf["kn"], buf["vn"], slots, k, v)
        mask, _ = pkv.tree_masks(buf["parents"], ctx, buf["nodes"])
        pkv.paged_decode_tree(buf["q"], k, v, bt, ctx, mask, buf["nodes"], out=out, workspace=ws)
        pkv.compact_tokens(buf["idx"], buf["acc"], ctx, bt, k, v, T, node_counts=buf["nodes"], seq_lens=buf["seq"],
                           new_lens=buf["new"], prev_seq_lens=buf["seq"])

    runner, seq = step, np.zeros(B, np.int32)
    refused_at, served_again = {}, set()
    for i in range(9):
        new = np.array([60, 40, 20]) if i == 0 else np.full(B, T)
        if i == 5:
            new[0] = -1
        if i == 6:
            new[0] = 5  # a new request in its place
        nodes = np.where((new == T) & (i > 0), T, 0).astype(np.int32)
        parents = random_parents(rng, B, T, 4)
        see, _ = visible(parents, nodes)
        idx, acc = np.zeros((B, 4), np.int32), np.zeros(B, np.int32)
        for b in range(B):
            t, path = int(nodes[b]) - 1, []
            while t >= 0:
                path.append(t)
                t = parents[b, t]
            path = path[::-1][:4]
            acc[b], idx[b, :len(path)] = len(path), path
        if i == 5:
            acc[0] = 3  # what a sampler leaves in the row of a request that has ended
        q, kn, vn = normal_bf16_bits(9730 + i, (B, T, Hq, D)), normal_bf16_bits(9740 + i, (N, Hkv, D)), normal_bf16_bits(9750 + i, (N, Hkv, D))
        if i == 0:
            buf["seq"].zero_()
        assert buf["seq"].tolist() == seq.tolist()
        for name, x in (("new", new), ("parents", parents), ("nodes", nodes), ("idx", idx), ("acc", acc)):
            buf[name].copy_(torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)))
        for name, x in (("q", q), ("kn", kn), ("vn", vn)):
            buf[name].copy_(to_dev_bf16(x))
        if graph and i == 1:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            runner = g.replay
        runner()
        torch.cuda.synchronize()
        ctx, _, slots, _, err = pool.extend(seq, new, tables, counts, N)
        assert pkv.read_device_error() == err and err in (0, pkv.DEVERR_NO_BLOCKS)
        assert np.array_equal(bt.cpu().numpy(), tables) and np.array_equal(cnt.cpu().numpy(), counts)
        assert oracle.kv_append(kn, vn, slots, k_host, v_host) == 0
        ref = tree_attention(q, k_host, v_host, tables, ctx, see, nodes, D ** -0.5)
        assert_tree_close(bf16_dev_to_f64(out), *ref, f"step {i}")
        active = ctx > 0
        k_host = compact(k_host, idx, np.where(active, acc, 0), ctx, nodes, tables)
        v_host = compact(v_host, idx, np.where(active, acc, 0), ctx, nodes, tables)
        assert np.array_equal(_bits(k), k_host) and np.array_equal(_bits(v), v_host), f"step {i}"
        for b in range(B):
            if not active[b] and new[b] != -1:
                refused_at.setdefault(b, i)
            elif b in refused_at and active[b] and seq[b] > 0:
                served_again.add(b)
        seq = np.where(new == -1, 0, np.where(active, ctx - nodes + acc, seq)).astype(np.int32)
    assert refused_at and served_again, (refused_at, served_again)
    assert buf["seq"].tolist() == seq.tolist()
