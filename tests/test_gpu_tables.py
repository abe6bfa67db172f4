"""Block tables on the GPU, compaction of accepted paths, and the whole loop
of drafted-tree steps, against plain references."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_274_gb300 as pkv
from workloads import normal_bf16_bits, random_case
from tests._gpu import DEV, DeviceCase, bf16_dev_to_f64, to_dev, to_dev_bf16
from tests._tree import Pool, assert_tree_close, compact, pack, random_parents, tree_attention, visible

pytestmark = pytest.mark.gpu


class Tables:
    """Device arrays of extend_tables beside the reference pool."""

    def __init__(self, seed, B, MB, bs, seq, spare, head):
        rng = np.random.Generator(np.random.PCG64(seed))
        held = -(-np.asarray(seq, np.int64) // bs)
        NB = int(held.sum()) + spare
        ids = rng.permutation(NB)
        self.bs, self.MB, self.NB, self.B = bs, MB, NB, B
        self.tables = np.full((B, MB), -7, np.int32)
        at = 0
        for b in range(B):
            self.tables[b, :held[b]] = ids[at:at + held[b]]
            at += held[b]
        self.counts = held.astype(np.int32)
        self.pool = Pool(NB, bs, MB, ids[at:], head % NB)
        self.d_tables, self.d_counts = to_dev(self.tables.copy()), to_dev(self.counts.copy())
        self.d_ring = to_dev(self.pool.ring.copy())
        self.d_state = to_dev(np.array([self.pool.head, self.pool.free, 0, 0], np.int32))

    def step(self, seq, new, N, borrowed=None, in_place=True):
        seq, new = np.asarray(seq, np.int32), np.asarray(new, np.int32)
        kw = {}
        if not in_place:
            kw = dict(new_block_counts=torch.full_like(self.d_counts, -3), new_free_state=torch.full_like(self.d_state, -3))
            before = (self.d_counts.clone(), self.d_state.clone())
        got = pkv.extend_tables(to_dev(seq), to_dev(new), self.d_tables, self.d_counts, self.d_ring, self.d_state, self.bs, N,
                                borrowed_counts=None if borrowed is None else to_dev(np.asarray(borrowed, np.int32)), **kw)
        err = pkv.read_device_error()
        if not in_place:
            assert torch.equal(before[0], self.d_counts) and torch.equal(before[1], self.d_state)
            self.d_counts, self.d_state = kw["new_block_counts"], kw["new_free_state"]
        want = self.pool.extend(seq, new, self.tables, self.counts, N, borrowed)
        names = ("context_lens", "query_starts", "slot_mapping", "positions")
        for name, g, w in zip(names, got, want):
            assert np.array_equal(g.cpu().numpy(), w), (name, np.argwhere(g.cpu().numpy() != w)[:5])
        assert err == want[4]
        assert np.array_equal(self.d_tables.cpu().numpy(), self.tables)
        assert np.array_equal(self.d_counts.cpu().numpy(), self.counts)
        assert np.array_equal(self.d_ring.cpu().numpy(), self.pool.ring)
        assert self.d_state.cpu().tolist() == [self.pool.head, self.pool.free, 0, 0]
        return want[0], err


@pytest.mark.parametrize("B,bs,hi,new_hi,done", [(1, 16, 0, 1, 0.0), (1, 16, 100, 4000, 0.0), (7, 32, 300, 40, 0.3), (100, 16, 1000, 9, 0.2),
                                                  (513, 16, 200, 33, 0.1), (1500, 32, 90, 3, 0.5), (40, 16, 50, 3000, 0.1),
                                                  (60, 16, 50, 4001, 0.0)])  # more rows than threads: runs of rows
@pytest.mark.parametrize("in_place", [True, False])
def test_steps_of_many_requests(B, bs, hi, new_hi, done, in_place):
    # several steps in a row: requests grow, end, and others start in their rows
    rng = np.random.Generator(np.random.PCG64(B + new_hi))
    MB = -(-(hi + 6 * new_hi) // bs) + 1
    seq = rng.integers(0, hi + 1, B)
    t = Tables(B, B, MB, bs, seq, spare=int(B * (new_hi / bs + 1) * 2) + 3, head=int(rng.integers(0, 1000)))
    for _ in range(5):
        new = rng.integers(0, new_hi + 1, B)
        new[rng.random(B) < done] = -1
        ctx, err = t.step(seq, new, int(np.maximum(new, 0).sum()) + int(rng.integers(0, 5)), in_place=in_place)
        assert err in (0, pkv.DEVERR_NO_BLOCKS)
        # ended requests start anew; refused ones stay; the others keep some of what they added
        kept = seq + rng.integers(0, np.maximum(new, 0) + 1)
        seq = np.where(new == -1, 0, np.where((ctx == 0) & (new >= 0) & (seq + new > 0), seq, kept))


def test_pool_runs_out():
    t = Tables(3, 4, 8, 16, [16, 5, 40, 0], spare=5, head=17)
    # needs 1, 2, 3, 0 blocks of 5: the third does not fit, the fourth needs none
    ctx, err = t.step([16, 5, 40, 0], [1, 30, 47, 0], 100)
    assert err == pkv.DEVERR_NO_BLOCKS and ctx.tolist() == [17, 35, 0, 0]
    # 2 are left: a large need at the front holds back the one behind it, but not one without need
    ctx, err = t.step([17, 35, 40, 0], [60, 13, 8, 1], 100)
    assert err == pkv.DEVERR_NO_BLOCKS and ctx.tolist() == [0, 48, 48, 0]
    # an ended request's blocks are free from the next call on
    ctx, err = t.step([17, 48, 48, 0], [-1, 0, 0, 60], 100)
    assert err == pkv.DEVERR_NO_BLOCKS and ctx.tolist() == [0, 48, 48, 0]
    ctx, err = t.step([0, 48, 48, 0], [0, 0, 0, 60], 100)
    assert err == 0 and ctx.tolist() == [0, 48, 48, 60]


def test_bad_numbers_refuse_only_their_request():
    seq = [10, 10, 10, -1, 10, 10, 10, 33, 10, 5]
    t = Tables(4, 10, 4, 16, [10] * 10, spare=50, head=0)
    for in_place in (True, False):
        # below -1; too long; a huge number; negative length; fine; ended; more tokens than blocks
        ctx, err = t.step(seq, [3, -2, 60, 1, 4, -1, 2, 5, 2**31 - 1, 6], 200, in_place=in_place)
        # (the rows of the huge number leave no room for the last request's)
        assert err == pkv.DEVERR_CONTEXT_LEN | pkv.DEVERR_SLOT
        assert ctx.tolist() == [13, 0, 0, 0, 14, 0, 12, 0, 0, 0]
        t.counts[5] = 1  # the ended one again
        t.d_counts[5] = 1


def test_token_rows_that_do_not_fit():
    t = Tables(5, 4, 16, 16, [0, 20, 3, 7], spare=40, head=3)
    ctx, err = t.step([0, 20, 3, 7], [10, 10, 10, 0], 25)
    assert err == pkv.DEVERR_SLOT and ctx.tolist() == [10, 30, 0, 7]
    ctx, err = t.step([10, 30, 3, 7], [1, 1, 1, 1], 0)
    assert err == pkv.DEVERR_SLOT and ctx.tolist() == [0, 0, 0, 0]


def test_borrowed_blocks_are_not_given_back():
    t = Tables(6, 4, 8, 16, [64, 40, 20, 100], spare=3, head=1)
    free = t.pool.free
    t.step([64, 40, 20, 100], [-1, -1, 4, -1], 10, borrowed=[2, 0, 1, 99])
    assert t.pool.free == free + 2 + 3


def test_no_requests_and_no_rows():
    t = Tables(7, 0, 3, 16, [], spare=4, head=2)
    t.step([], [], 5)
    t = Tables(8, 3, 3, 16, [5, 20, 16], spare=4, head=2)
    t.step([5, 20, 16], [-1, 0, -1], 0)


def test_largest_batch():
    B = 16384
    rng = np.random.Generator(np.random.PCG64(9))
    seq = rng.integers(0, 60, B)
    t = Tables(9, B, 6, 16, seq, spare=30000, head=12345)
    new = rng.integers(-1, 3, B)
    t.step(seq, new, int(np.maximum(new, 0).sum()))
    with pytest.raises(pkv.PkvError):
        z = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
        pkv.extend_tables(z, z, torch.zeros((B + 1, 2), dtype=torch.int32, device=DEV), z.clone(), t.d_ring, t.d_state, 16, 0)


# (of 40 blocks; the ended request gives 2 back, so 39 free ones are too many: 38 + 2 would just fit)
@pytest.mark.parametrize("state", [[-1, 3], [40, 3], [0, -2], [0, 41], [3, 39]])
def test_invalid_ring_state_refuses_all(state):
    t = Tables(10, 3, 4, 16, [10, 20, 30], spare=35, head=0)  # 40 blocks
    assert t.NB == 40
    st = to_dev(np.array(state + [0, 0], np.int32))
    before = [x.clone() for x in (t.d_tables, t.d_counts, t.d_ring)]
    ctx, starts, slots, pos = pkv.extend_tables(to_dev(np.array([10, 20, 30], np.int32)), to_dev(np.array([20, 3, -1], np.int32)), t.d_tables,
                                                t.d_counts, t.d_ring, st, 16, 23)
    assert pkv.read_device_error() == pkv.DEVERR_BLOCK_ID
    assert ctx.tolist() == [0, 0, 0] and (slots == -1).all() and (pos == 0).all() and starts.tolist() == [0, 20, 23, 23]
    for a, b in zip(before, (t.d_tables, t.d_counts, t.d_ring)):
        assert torch.equal(a, b)
    assert st.tolist() == state + [0, 0]


def test_bad_ids_in_the_ring_and_the_table():
    t = Tables(11, 2, 4, 16, [10, 16], spare=6, head=0)
    t.d_ring[1] = t.NB + 3
    t.d_tables[0, 0] = -9
    ctx, _, slots, _ = pkv.extend_tables(to_dev(np.array([10, 16], np.int32)), to_dev(np.array([10, 3], np.int32)), t.d_tables, t.d_counts,
                                         t.d_ring, t.d_state, 16, 13)
    assert pkv.read_device_error() == pkv.DEVERR_BLOCK_ID
    s = slots.cpu().numpy()
    assert (s[:6] == -1).all() and (s[6:10] >= 0).all() and (s[10:] == -1).all()
    assert ctx.tolist() == [20, 19]


# ---------------------------------------------------------------------------
# compaction
# ---------------------------------------------------------------------------
def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


COMPACT = [  # (D, bs, Hkv, S, dtype, T, contexts, accepted)
    (128, 16, 8, 1, "bf16", 8, [8, 30, 100], [[0, 1, 2], [0, 3, 7], [5]]),
    (64, 16, 2, 3, "bf16", 40, [40, 71, 55, 300], [list(range(0, 40, 2)), list(range(40)), [39], []]),
    (64, 32, 1, 2, "bf16", 70, [70, 100], [list(range(30, 70)), list(range(1, 70))]),   # long overlapping runs
    (128, 32, 4, 2, "fp8", 33, [33, 64, 200], [[1, 2, 3, 32], [0, 17, 31], list(range(16, 33))]),
    (128, 16, 8, 2, "int8a", 20, [20, 47, 64], [[2, 4, 19], list(range(3, 20)), [0, 1, 19]]),
    (128, 16, 2, 1, "int8", 20, [33, 47], [[2, 4, 19], [0]]),
]


@pytest.mark.parametrize("D,bs,Hkv,S,dtype,T,lens,paths", COMPACT)
def test_compact(D, bs, Hkv, S, dtype, T, lens, paths):
    c = random_case(9000 + T + D, len(lens), 2 * Hkv, Hkv, D, bs, lens, kv_dtype=dtype, S=S)
    if dtype != "bf16":  # some pages share their parameters
        c.k_scale[:, ::2] = c.k_scale[:, :1]
    dc = DeviceCase(c)
    A = max(1, max(map(len, paths)))
    idx = np.full((len(lens), A), -5, np.int32)
    for b, p in enumerate(paths):
        idx[b, :len(p)] = p
    count = np.array([len(p) for p in paths], np.int32)
    nodes = np.full(len(lens), T, np.int32)
    kind = {"bf16": "bf16", "fp8": "fp8"}.get(dtype, "int8")
    wk = compact(dc.k_host, idx, count, lens, nodes, c.block_tables, c.k_scale if kind != "bf16" else None, kind)
    wv = compact(dc.v_host, idx, count, lens, nodes, c.block_tables, c.v_scale if kind != "bf16" else None, kind)
    seq = pkv.compact_tokens(to_dev(idx), to_dev(count), dc.cl, dc.bt, dc.k, dc.v, T, k_scale=dc.ks, v_scale=dc.vs)
    assert pkv.read_device_error() == 0
    assert seq.tolist() == (np.array(lens) - T + count).tolist()
    assert np.array_equal(_bits(dc.k), wk) and np.array_equal(_bits(dc.v), wv)


def test_compact_node_counts_and_inactive_rows():
    T, lens = 10, [30, 0, 12, 7]
    nodes = np.array([4, 10, 10, 3], np.int32)
    c = random_case(9100, 4, 4, 2, 128, 16, lens)
    dc = DeviceCase(c)
    idx = np.array([[1, 3], [0, 0], [2, 9], [0, 2]], np.int32)
    count = np.array([2, 0, 2, 2], np.int32)
    wk = compact(dc.k_host, idx, count, lens, nodes, c.block_tables)
    seq = pkv.compact_tokens(to_dev(idx), to_dev(count), dc.cl, dc.bt, dc.k, dc.v, T, node_counts=to_dev(nodes))
    assert pkv.read_device_error() == 0
    assert seq.tolist() == [28, 0, 4, 6]  # an inactive row (0 tokens, nothing accepted) is no error
    assert np.array_equal(_bits(dc.k), wk)


@pytest.mark.parametrize("what,flag,seq1", [("order", 32, 20), ("range", 32, 20), ("negative", 32, 20), ("count", 32, 20), ("nodes", 32, 0),
                                             ("context", 4, 0), ("long", 4, 0), ("before", 32, 0), ("block", 1, 20)])
def test_compact_refusals_leave_the_sequence(what, flag, seq1):
    T, lens = 10, [30, 30, 30]
    c = random_case(9200, 3, 4, 2, 128, 16, lens, MB=4)
    dc = DeviceCase(c)
    idx = np.array([[1, 3, 7], [1, 3, 7], [2, 8, 9]], np.int32)
    count, nodes, cl, bt = np.array([3, 3, 3], np.int32), np.full(3, T, np.int32), c.context_lens.copy(), c.block_tables.copy()
    if what == "order":
        idx[1] = [1, 7, 7]
    elif what == "range":
        idx[1] = [1, 3, 10]
    elif what == "negative":
        idx[1] = [-1, 3, 7]
    elif what == "count":
        count[1] = 4
    elif what == "nodes":
        nodes[1] = 11
    elif what == "context":
        cl[1] = -1
    elif what == "long":
        cl[1] = 65
    elif what == "before":
        cl[1] = 9
    else:
        bt[1, 1] = c.NB
    good = count.copy()
    good[1] = 0
    wk = compact(dc.k_host, idx, good, lens, nodes, c.block_tables)
    seq = pkv.compact_tokens(to_dev(idx), to_dev(count), to_dev(cl), to_dev(bt), dc.k, dc.v, T, node_counts=to_dev(nodes))
    assert pkv.read_device_error() == flag
    assert seq.tolist() == [23, seq1, 23]
    assert np.array_equal(_bits(dc.k), wk)


# ---------------------------------------------------------------------------
# the loop
# ---------------------------------------------------------------------------
def _loop_state(dtype, seed):
    B, Hq, Hkv, D, bs, MB, S = 3, 16, 4, 128, 16, 20, 2
    NB = 50
    rng = np.random.Generator(np.random.PCG64(seed))
    if dtype == "bf16":
        k = normal_bf16_bits(seed, (S, NB, Hkv, bs, D))
        par = None
    else:
        k = np.zeros((S, NB, Hkv, bs, D), np.uint8)
        par = rng.uniform(0.005, 0.012, (S, NB, Hkv)).astype(np.float32)
    return dict(B=B, Hq=Hq, Hkv=Hkv, D=D, bs=bs, MB=MB, S=S, NB=NB, k=k, v=k.copy(), ks=par, vs=None if par is None else par[:, ::-1].copy())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_a_serving_loop(dtype, graph):
    """Prompts, then several verification steps: tables, append in every cache
    slot, masks, attention per slot, compaction; each step's outputs, caches
    and lengths against the references.  graph: the whole step captured once
    and replayed (its buffers stay in place)."""
    s = _loop_state(dtype, 9300)
    B, T, bs, MB = s["B"], 12, s["bs"], s["MB"]
    rng = np.random.Generator(np.random.PCG64(9301))
    kind = dtype
    k_host, v_host = s["k"], s["v"]
    dev = to_dev_bf16 if dtype == "bf16" else to_dev
    k, v = dev(k_host), dev(v_host)
    ks, vs = (None, None) if s["ks"] is None else (to_dev(s["ks"]), to_dev(s["vs"]))
    pool = Pool(s["NB"], bs, MB, rng.permutation(s["NB"]).tolist())
    ring, state = pkv.new_free_ring(pool.ring, s["NB"])
    tables, counts = np.full((B, MB), -1, np.int32), np.zeros(B, np.int32)
    bt, cnt = to_dev(tables.copy()), to_dev(counts.copy())
    N = 100
    buf = dict(seq=torch.zeros(B, dtype=torch.int32, device=DEV), new=torch.zeros(B, dtype=torch.int32, device=DEV),
               parents=torch.zeros((B, T), dtype=torch.int32, device=DEV), nodes=torch.zeros(B, dtype=torch.int32, device=DEV),
               idx=torch.zeros((B, 4), dtype=torch.int32, device=DEV), acc=torch.zeros(B, dtype=torch.int32, device=DEV),
               q=torch.zeros((s["S"], B, T, s["Hq"], s["D"]), dtype=torch.bfloat16, device=DEV),
               kn=torch.zeros((s["S"], N, s["Hkv"], s["D"]), dtype=torch.bfloat16, device=DEV),
               vn=torch.zeros((s["S"], N, s["Hkv"], s["D"]), dtype=torch.bfloat16, device=DEV))
    outs = [torch.zeros((B, T, s["Hq"], s["D"]), dtype=torch.bfloat16, device=DEV) for _ in range(s["S"])]
    ws = torch.empty(pkv.decode_workspace_bytes(k, B, s["Hq"], MB, None, T, tree=True), dtype=torch.uint8, device=DEV)
    keep = {}

    def step():
        ctx, starts, slots, pos = pkv.extend_tables(buf["seq"], buf["new"], bt, cnt, ring, state, bs, N)
        for l in range(s["S"]):
            pkv.kv_append(buf["kn"][l], buf["vn"][l], slots, k, v, ks, vs, slot=l)
        mask, npos = pkv.tree_masks(buf["parents"], ctx, buf["nodes"])
        for l in range(s["S"]):
            pkv.paged_decode_tree(buf["q"][l], k, v, bt, ctx, mask, buf["nodes"], list(range(s["S"])), l, out=outs[l],
                                  workspace=ws, k_scale=ks, v_scale=vs)
        seq = pkv.compact_tokens(buf["idx"], buf["acc"], ctx, bt, k, v, T, node_counts=buf["nodes"], k_scale=ks, v_scale=vs)
        keep.update(ctx=ctx, slots=slots, npos=npos, seq=seq)

    runner = step
    seq = np.zeros(B, np.int32)
    for i in range(6):
        prompt = i == 0
        new = np.array([40, 3, 21]) if prompt else rng.integers(1, T + 1, B)
        if i == 3:
            new[1] = -1  # the second request ends, and starts again as a new one in the next step
        nodes = np.zeros(B, np.int32) if prompt else np.maximum(new, 0).astype(np.int32)
        parents = random_parents(rng, B, T, 4)
        see, depth = visible(parents, nodes)
        idx, acc = np.zeros((B, 4), np.int32), np.zeros(B, np.int32)
        for b in range(B):
            t, path = int(nodes[b]) - 1, []
            while t >= 0:
                path.append(t)
                t = parents[b, t]
            path = path[::-1][:4]
            acc[b] = len(path)
            idx[b, :len(path)] = path
        q = normal_bf16_bits(9400 + i, (s["S"], B, T, s["Hq"], s["D"]))
        kn, vn = normal_bf16_bits(9500 + i, (s["S"], N, s["Hkv"], s["D"])), normal_bf16_bits(9600 + i, (s["S"], N, s["Hkv"], s["D"]))
        for name, x in (("seq", seq), ("new", new), ("parents", parents), ("nodes", nodes), ("idx", idx), ("acc", acc)):
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
        assert pkv.read_device_error() == 0
        # references
        ctx, _, slots, _, err = pool.extend(seq, new, tables, counts, N)
        assert err == 0 and np.array_equal(keep["slots"].cpu().numpy(), slots)
        assert np.array_equal(bt.cpu().numpy(), tables) and np.array_equal(keep["ctx"].cpu().numpy(), ctx)
        for l in range(s["S"]):
            assert oracle.kv_append(kn[l], vn[l], slots, k_host, v_host, s["ks"], s["vs"], slot=l) == 0
        want = np.where(depth >= 0, (ctx - nodes)[:, None] + depth, 0)
        assert np.array_equal(keep["npos"].cpu().numpy(), want)
        for l in range(s["S"]):
            ref = tree_attention(q[l], k_host, v_host, tables, ctx, see, nodes, s["D"] ** -0.5, s["ks"], s["vs"], slot=l)
            assert_tree_close(bf16_dev_to_f64(outs[l]), *ref, f"step {i} slot {l}")
        k_host = compact(k_host, idx, acc, ctx, nodes, tables, s["ks"], kind)
        v_host = compact(v_host, idx, acc, ctx, nodes, tables, s["vs"], kind)
        assert np.array_equal(_bits(k), k_host) and np.array_equal(_bits(v), v_host), f"step {i}"
        seq = (ctx - nodes + acc).astype(np.int32)
        assert np.array_equal(keep["seq"].cpu().numpy(), seq)


def test_prepared_calls_match_plain_ones():
    t = Tables(12, 3, 8, 16, [10, 20, 30], spare=20, head=4)
    seq, new = to_dev(np.array([10, 20, 30], np.int32)), to_dev(np.array([5, 16, -1], np.int32))
    c2, s2 = torch.empty_like(t.d_counts), torch.empty_like(t.d_state)
    call = pkv.PreparedCall(pkv.extend_tables, seq, new, t.d_tables, t.d_counts, t.d_ring, t.d_state, 16, 24, new_block_counts=c2,
                            new_free_state=s2)
    a = [x.clone() for x in call()]
    b = [x.clone() for x in call()]  # not in place: the same again
    want = t.pool.extend([10, 20, 30], [5, 16, -1], t.tables, t.counts, 24)
    for x, y, w in zip(a, b, want):
        assert torch.equal(x, y) and np.array_equal(x.cpu().numpy(), w)
    assert np.array_equal(c2.cpu().numpy(), t.counts) and s2.tolist() == [t.pool.head, t.pool.free, 0, 0]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    parents = to_dev(random_parents(np.random.Generator(np.random.PCG64(1)), 4, 9))
    m = pkv.PreparedCall(pkv.tree_masks, parents, stream=s)
    mask, pos = m()
    torch.cuda.synchronize()
    ref = pkv.tree_masks(parents)
    assert torch.equal(mask, ref[0]) and torch.equal(pos, ref[1])
    with pytest.raises(pkv.PkvError):
        pkv.PreparedCall(pkv.kv_append)
