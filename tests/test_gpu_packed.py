"""Attention of packed rows on the GPU against a float64 reference: types, head
layouts, sequences of one row to long prompts in one call, split items,
sequences without rows, cache or room, values that are not finite in places that
a row does not see, rows behind the last sequence, refused starts, cache
offsets past 32 bits, other streams, CUDA graphs."""
import numpy as np
import pytest
import torch

import paged_kv_cache_274_gb300 as pkv
from workloads import normal_bf16_bits
from workloads.gen import BF16_NAN
from tests._gpu import DEV, DeviceCase, bf16_dev_to_f64, to_dev, to_dev_bf16
from tests._packed import PackedCase, packed_attention
from tests._tree import assert_tree_close

pytestmark = pytest.mark.gpu


def attend(pc, starts=None, most=None, pad=0, mark=None, **kw):
    c, dc = pc.c, pc.dc
    q = to_dev_bf16(np.concatenate([pc.q, normal_bf16_bits(5, (pad,) + pc.q.shape[1:])])) if pad else to_dev_bf16(pc.q)
    out = torch.full_like(q, mark) if mark is not None else None
    got = pkv.paged_decode_packed(q, dc.k, dc.v, dc.bt, dc.cl, to_dev(pc.starts if starts is None else starts),
                                  most, c.kv_group_ptr.tolist(), 0, c.scale, out=out, k_scale=dc.ks, v_scale=dc.vs, **kw)
    torch.cuda.synchronize()
    return got


SWEEP = [  # (D, bs, Hq, Hkv, dtype, (new, before) of the sequences)
    (128, 16, 32, 8, "bf16", [(1, 0)]),
    (128, 16, 32, 8, "bf16", [(1, 299), (1, 15), (1, 16), (1, 0), (1, 1000)]),        # a decode step
    (128, 16, 32, 8, "bf16", [(5, 700)]),
    (128, 16, 32, 8, "bf16", [(32, 0), (33, 100), (1, 500), (64, 63), (7, 0)]),       # tile ends
    (128, 32, 32, 8, "bf16", [(65, 0), (200, 333), (1, 2000), (129, 1)]),             # several pairs
    (128, 16, 64, 8, "bf16", [(300, 0), (17, 127), (16, 128)]),
    (128, 16, 16, 1, "bf16", [(40, 300), (8, 0), (9, 5)]),                            # 16 heads on one KV head
    (128, 16, 32, 1, "bf16", [(3, 60), (9, 0), (4, 129)]),
    (128, 16, 128, 1, "bf16", [(3, 260), (1, 1)]),                                    # a row is a tile
    (128, 16, 12, 4, "bf16", [(50, 77), (43, 0)]),                                    # 3 heads a KV head
    (128, 16, 4, 4, "bf16", [(513, 0), (128, 128), (257, 20)]),                       # no shared heads
    (64, 16, 8, 8, "bf16", [(20, 20), (300, 5), (1, 700)]),
    (64, 32, 16, 4, "bf16", [(45, 0), (100, 260), (1, 1)]),
    (64, 16, 16, 16, "bf16", [(1, 90), (1, 3000)]),
    (128, 16, 32, 8, "fp8", [(2, 17), (1, 300), (31, 0)]),
    (128, 16, 32, 8, "fp8", [(70, 500), (1, 1000), (40, 0), (64, 64)]),
    (128, 32, 32, 8, "fp8", [(300, 0), (33, 700)]),
    (128, 32, 32, 8, "int8a", [(4, 70), (1, 300), (30, 0)]),
    (128, 16, 32, 8, "int8a", [(90, 600), (1, 77), (65, 0)]),
    (128, 16, 16, 4, "int8", [(37, 250), (250, 1)]),
]


@pytest.mark.parametrize("D,bs,Hq,Hkv,dtype,seqs", SWEEP)
@pytest.mark.parametrize("share", [0, 16, 250])
def test_sweep(D, bs, Hq, Hkv, dtype, seqs, share):
    pc = PackedCase(6000 + D + bs + Hq + 3 * Hkv + len(seqs), seqs, Hq, Hkv, D, bs, dtype)
    want = pc.reference()
    opts = pkv.decode_opts(partition_blocks=share)
    for most in (int(pc.new.max()), None):  # a tight bound, and any
        out = attend(pc, most=most, opts=opts)
        assert pkv.read_device_error() == 0
        assert_tree_close(bf16_dev_to_f64(out), *want, f"{dtype} share {share} most {most}")
    again = attend(pc, opts=opts)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("D,dtype,seqs", [
    (128, "bf16", [(700, 4000), (1, 9000), (1, 100), (130, 0), (1, 5000), (64, 2000)]),
    (64, "bf16", [(1500, 0), (1, 7000), (33, 900)]),
    (128, "fp8", [(400, 3000), (1, 6000), (2, 129), (90, 0)]),
    (128, "int8a", [(300, 2000), (1, 6000), (31, 128)]),
    (128, "bf16", [(1, 20000), (1, 3)]), (128, "fp8", [(1, 12000)])])
@pytest.mark.parametrize("share", [0, 24])
def test_split_items(D, dtype, seqs, share):
    pc = PackedCase(6200 + D + len(seqs), seqs, 12, 3, D, 16, dtype)
    out = attend(pc, most=int(pc.new.max()), opts=pkv.decode_opts(partition_blocks=share))
    assert pkv.read_device_error() == 0
    assert_tree_close(bf16_dev_to_f64(out), *pc.reference(), f"{dtype} share {share}")


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp8", 128), ("int8", 128), ("bf16", 64)])
def test_sequences_without_rows_cache_or_room(dtype, D):
    # no new rows; rows without cache (a refused request); more rows than cached tokens; rows behind the last sequence
    new, ctx = [3, 0, 40, 100, 0, 70, 1, 150], [90, 50, 0, 33, 0, 70, 1, 149]
    pc = PackedCase(6300 + D, list(zip(new, [0] * 8)), 8, 2, D, 16, dtype, lens=ctx)
    out, wabs = pc.reference()
    got = bf16_dev_to_f64(attend(pc, pad=11, mark=7.0, opts=pkv.decode_opts(partition_blocks=8)))
    assert pkv.read_device_error() == 0
    assert_tree_close(got[:pc.N], out, wabs)
    assert (got[pc.N:] == 7.0).all()
    assert (got[3:43] == 0).all() and (got[43:43 + 67] == 0).all() and (got[43 + 67] != 0).any()


def test_one_sequence_after_many_without_rows():
    new, ctx = [0] * 300 + [33] + [0] * 300 + [1], [17] * 300 + [200] + [0] * 300 + [60]
    pc = PackedCase(6310, list(zip(new, [0] * 602)), 8, 2, 128, 16, lens=ctx)
    assert_tree_close(bf16_dev_to_f64(attend(pc)), *pc.reference())


def test_many_sequences():
    # more than the planner searches in shared memory
    rng = np.random.Generator(np.random.PCG64(6320))
    seqs = [(int(rng.integers(1, 4)), int(rng.integers(0, 60))) for _ in range(1300)]
    pc = PackedCase(6321, seqs, 4, 1, 64, 16)
    assert_tree_close(bf16_dev_to_f64(attend(pc)), *pc.reference())
    assert pkv.read_device_error() == 0


@pytest.mark.parametrize("dtype,m", [("bf16", 90), ("bf16", 20), ("fp8", 90), ("fp8", 20)])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(dtype, m):
    # K and V of new tokens that early rows do not see
    pc = PackedCase(6400 + m, [(m, 100), (m, 0), (1, 50)], 8, 2, 128, 16, dtype, poison=False)
    c, dc = pc.c, pc.dc
    want = bf16_dev_to_f64(attend(pc))
    first = {}
    for b, u in ((0, m // 2), (1, m - 3)):
        pos = int(c.context_lens[b]) - m + u
        blk, off = int(c.block_tables[b, pos // 16]), pos % 16
        for t in (dc.k, dc.v):
            if dtype == "bf16":
                t[0, blk, 1, off, 5] = float("nan") if b == 0 else float("inf")
            else:
                t[0, blk, 1, off, 5] = 0x7f
        first[b] = int(pc.starts[b]) + u
    got = bf16_dev_to_f64(attend(pc))
    sees = np.zeros(got.shape, bool)
    for b, row in first.items():
        sees[row:pc.starts[b + 1], 4:] = True  # the heads of KV head 1
    assert np.array_equal(got[~sees], want[~sees])
    assert np.isnan(got[sees]).all()


def test_a_poisoned_query_stays_in_its_row():
    pc = PackedCase(6410, [(40, 100), (30, 0)], 8, 2, 128, 16)
    want = bf16_dev_to_f64(attend(pc))
    pc.q[17, 3, 9] = BF16_NAN
    pc.q[45, 7, 0] = 0x7f80  # infinity
    got = bf16_dev_to_f64(attend(pc))
    same = np.ones(got.shape[:2], bool)
    same[17, 3] = same[45, 7] = False
    assert np.array_equal(got[same], want[same]) and np.isnan(got[17, 3]).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(scale):
    pc = PackedCase(6420, [(40, 300), (1, 77), (70, 0)], 8, 2, 128, 16)
    pc.c.scale = scale
    assert_tree_close(bf16_dev_to_f64(attend(pc)), *pc.reference(), f"scale {scale}")


def test_bad_pages_and_lengths():
    pc = PackedCase(6430, [(40, 300), (35, 200), (1, 90)], 8, 2, 128, 16)
    c = pc.c
    c.block_tables[1, 5] = c.NB + 3
    pc.dc.bt = to_dev(c.block_tables)
    good = bf16_dev_to_f64(attend(pc))
    assert pkv.read_device_error() == pkv.DEVERR_BLOCK_ID
    # the page contributes nothing: as if its tokens were not there
    c.block_tables[1, 5] = 0
    out, wabs = pc.reference()
    keep = np.ones(pc.N, bool)
    keep[40:75] = False
    assert_tree_close(good[keep], out[keep], wabs[keep])
    assert np.isfinite(good).all()
    pc.dc.cl = to_dev(np.array([340, -5, 10 ** 6], np.int32))
    bad = bf16_dev_to_f64(attend(pc))
    assert pkv.read_device_error() & pkv.DEVERR_CONTEXT_LEN
    assert_tree_close(bad[:40], out[:40], wabs[:40])
    assert (bad[40:] == 0).all()


@pytest.mark.parametrize("starts,most,lost", [
    ([0, 40, 30, 76], None, [1]), ([-1, 40, 75, 76], None, [0]), ([0, 40, 75, 200], None, [2]), ([0, 40, 75, 76], 39, [0])])
def test_refused_starts(starts, most, lost):
    pc = PackedCase(6440, [(40, 300), (35, 200), (1, 90)], 8, 2, 128, 16)
    out, wabs = pc.reference()
    got = bf16_dev_to_f64(attend(pc, np.array(starts, np.int32), most, mark=3.0))
    assert pkv.read_device_error() == pkv.DEVERR_QUERY
    for b in range(3):
        lo, hi = pc.starts[b], pc.starts[b + 1]
        if b in lost:
            rows = slice(lo, hi if b != 1 else 30)
            assert (got[rows] == 3.0).all() or starts[1] == 40 and starts[2] == 30
        elif starts[b] == lo and starts[b + 1] == hi:
            assert_tree_close(got[lo:hi], out[lo:hi], wabs[lo:hi])


def test_slots_and_offsets_past_32_bits():
    # two cache slots of 4.4 GiB each: the second's pages lie past 2^31 elements
    Hq, Hkv, bs, D = 8, 8, 32, 128
    NB = 72000
    pc = PackedCase(6500, [(40, 500), (1, 300), (70, 0)], Hq, Hkv, D, bs, poison=False)
    c, small = pc.c, pc.dc
    k, v = (torch.zeros((2, NB, Hkv, bs, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    move = torch.randperm(NB, generator=torch.Generator().manual_seed(1))[:c.NB]
    move[0] = NB - 1
    k[1, move.to(DEV)], v[1, move.to(DEV)] = small.k[0], small.v[0]
    bt = torch.where(small.bt >= 0, move.to(DEV)[small.bt.clamp(0, c.NB - 1).long()].int(), small.bt)
    out = pkv.paged_decode_packed(to_dev_bf16(pc.q), k, v, bt, small.cl, to_dev(pc.starts), None, [0, 1], 1, c.scale)
    assert pkv.read_device_error() == 0
    assert torch.equal(out.view(torch.int16), attend(pc).view(torch.int16))


def test_matches_the_padded_call():
    # equal counts: the causal multi-token call's bounds hold against this call's output
    T, lens = 40, [45, 300, 1000]
    pc = PackedCase(6510, [(T, n - T) for n in lens], 32, 8, 128, 16)
    c = pc.c
    multi = pkv.paged_decode_multi(to_dev_bf16(pc.q.reshape(3, T, 32, 128)), pc.dc.k, pc.dc.v, pc.dc.bt, pc.dc.cl, [0], 0, c.scale)
    out, wabs = pc.reference()
    assert_tree_close(bf16_dev_to_f64(multi).reshape(out.shape), out, wabs)
    assert_tree_close(bf16_dev_to_f64(attend(pc)), out, wabs)


def test_streams_graphs_and_prepared():
    pc = PackedCase(6600, [(50, 400), (1, 900), (90, 0)], 32, 8, 128, 16, "fp8")
    c, dc = pc.c, pc.dc
    want = attend(pc, most=90)
    q, starts = to_dev_bf16(pc.q), to_dev(pc.starts)
    prep = [pkv.PreparedDecode(q, dc.k, dc.v, dc.bt, dc.cl, scale=c.scale, k_scale=dc.ks, v_scale=dc.vs, query_starts=starts,
                               max_query_tokens=90) for _ in range(2)]
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):  # two calls at the same time, each with its workspace
        outs = [p(stream=s) for p, s in zip(prep, sides)]
    torch.cuda.synchronize()
    assert all(torch.equal(o.view(torch.int16), want.view(torch.int16)) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prep[0]()
    # other lengths under the same graph
    dc.cl.copy_(torch.tensor([430, 700, 88], dtype=torch.int32))
    starts.copy_(torch.tensor([0, 30, 31, 119], dtype=torch.int32))
    pc.c.context_lens = np.array([430, 700, 88], np.int32)
    g.replay()
    torch.cuda.synchronize()
    out, wabs = packed_attention(pc.q, pc.c, np.array([0, 30, 31, 119]), dc.k_host, dc.v_host)
    assert_tree_close(bf16_dev_to_f64(prep[0].out)[:119], out[:119], wabs[:119])
    assert pkv.read_device_error() == 0


def test_binding_refuses():
    pc = PackedCase(6700, [(4, 30), (1, 9)], 8, 2, 128, 16)
    c, dc = pc.c, pc.dc
    q, starts = to_dev_bf16(pc.q), to_dev(pc.starts)
    call = lambda **kw: pkv.paged_decode_packed(**{**dict(q=q, k_cache=dc.k, v_cache=dc.v, block_tables=dc.bt, context_lens=dc.cl,
                                                          query_starts=starts), **kw})
    call()
    for kw in (dict(q=q[None]), dict(q=q[..., :64].contiguous()), dict(q=q.float()), dict(q=q.cpu()), dict(query_starts=starts[:2]),
               dict(query_starts=starts.long()), dict(context_lens=dc.cl[:1]), dict(v_cache=dc.v[:, 1:]), dict(max_query_tokens=0),
               dict(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)), dict(out=q), dict(opts=pkv.decode_opts(math=pkv.MATH_MMA)),
               dict(layer=1), dict(kv_group_ptr=[3])):
        with pytest.raises(pkv.PkvError):
            call(**kw)
    for kw in (dict(max_query_tokens=4), dict(query_starts=starts, node_counts=dc.cl)):
        with pytest.raises(pkv.PkvError):
            pkv.PreparedDecode(q, dc.k, dc.v, dc.bt, dc.cl, **kw)
    empty = call(q=q[:0], query_starts=torch.zeros_like(starts))
    assert empty.shape == (0, 8, 128)
