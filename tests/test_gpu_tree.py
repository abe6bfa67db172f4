"""Drafted-tree attention and masks on the GPU against float64 references:
types, head layouts, tree sizes, ragged counts, split-K, masks that leave a
row empty, non-finite values in places that a row does not attend to, shared
trees, cache offsets past 32 bits, other streams, CUDA graphs; a chain of
nodes gives the bits of the causal multi-token call."""
import numpy as np
import pytest
import torch

import paged_kv_cache_274_gb300 as pkv
from workloads import normal_bf16_bits, random_case
from workloads.gen import BF16_NAN
from tests._gpu import DEV, DeviceCase, bf16_dev_to_f64, to_dev, to_dev_bf16
from tests._tree import assert_tree_close, pack, random_parents, tree_attention, visible

pytestmark = pytest.mark.gpu


def _trees(seed, B, T, nodes=None, dense=False):
    rng = np.random.Generator(np.random.PCG64(seed))
    nodes = np.full(B, T, np.int32) if nodes is None else np.asarray(nodes, np.int32)
    see, _ = visible(random_parents(rng, B, T), nodes)
    if dense:  # any bits, rows without their own among them
        see = rng.random((B, T, T)) < 0.4
    return see, nodes


def _attend(dc, q, see, nodes=None, **kw):
    c = dc.c
    out = pkv.paged_decode_tree(to_dev_bf16(q), dc.k, dc.v, dc.bt, dc.cl, to_dev(pack(see)),
                                None if nodes is None else to_dev(nodes), c.kv_group_ptr.tolist(), 0, c.scale,
                                k_scale=dc.ks, v_scale=dc.vs, **kw)
    torch.cuda.synchronize()
    return out


def _reference(dc, q, see, nodes):
    c = dc.c
    return tree_attention(q, dc.k_host, dc.v_host, c.block_tables, c.context_lens, see, nodes, c.scale, c.k_scale, c.v_scale)


SWEEP = [  # (D, bs, Hq, Hkv, T, dtype, contexts)
    (128, 16, 32, 8, 1, "bf16", [1, 16, 17, 300]),
    (128, 16, 32, 8, 3, "bf16", [3, 4, 33, 257]),            # 12 rows: one mma.sync tile
    (128, 32, 32, 8, 5, "bf16", [5, 31, 64, 700]),           # 20 rows: tcgen05, rotated rows
    (128, 16, 32, 8, 32, "bf16", [32, 33, 80, 1000]),        # a full 128-row tile
    (128, 16, 32, 8, 50, "bf16", [50, 64, 65, 130, 900]),    # two tiles: the pair kernel
    (128, 32, 64, 8, 70, "bf16", [70, 129, 500]),            # five tiles, an odd last one
    (128, 16, 16, 1, 33, "bf16", [33, 40, 260]),             # one KV head, 16 heads on it
    (128, 16, 32, 1, 1, "bf16", [1, 50, 130]),               # 32 heads on one KV head, one node
    (128, 16, 12, 4, 40, "bf16", [40, 77]),                  # 3 heads a KV head
    (128, 16, 8, 8, 200, "bf16", [200, 333]),                # no shared heads, many nodes
    (64, 16, 8, 8, 20, "bf16", [20, 21, 40, 333]),
    (64, 32, 16, 4, 45, "bf16", [45, 100, 260]),
    (128, 16, 32, 8, 2, "fp8", [2, 19, 300]),
    (128, 16, 32, 8, 21, "fp8", [21, 70, 500]),
    (128, 32, 32, 8, 40, "fp8", [40, 300, 700]),             # two tiles on a one-byte cache
    (128, 32, 32, 8, 4, "int8a", [4, 70, 300]),
    (128, 16, 32, 8, 32, "int8a", [32, 70, 600]),
    (128, 16, 16, 4, 37, "int8", [37, 250]),
]


@pytest.mark.parametrize("D,bs,Hq,Hkv,T,dtype,lens", SWEEP)
@pytest.mark.parametrize("ppu", [0, 2])
def test_tree_sweep(D, bs, Hq, Hkv, T, dtype, lens, ppu):
    seed = 7000 + D + 3 * bs + 7 * Hq + 11 * Hkv + 13 * T + len(lens)
    c = random_case(seed, len(lens), Hq, Hkv, D, bs, lens, kv_dtype=dtype, poison=dtype == "bf16")
    dc = DeviceCase(c)
    q = normal_bf16_bits(seed + 1, (c.B, T, Hq, D))
    see, nodes = _trees(seed + 2, c.B, T)
    out = _attend(dc, q, see, opts=pkv.decode_opts(partition_blocks=ppu))
    assert pkv.read_device_error() == 0
    assert_tree_close(bf16_dev_to_f64(out), *_reference(dc, q, see, nodes), f"T={T} {dtype} ppu={ppu}")


@pytest.mark.parametrize("D,Hq,Hkv,T,dtype,math", [
    (128, 32, 8, 24, "bf16", pkv.MATH_MMA), (128, 32, 8, 24, "bf16", pkv.MATH_TC), (128, 32, 8, 70, "bf16", pkv.MATH_TC),
    (64, 8, 4, 24, "bf16", pkv.MATH_AUTO), (128, 32, 8, 24, "fp8", pkv.MATH_TC), (128, 32, 8, 24, "int8a", pkv.MATH_TC),
    (128, 32, 8, 24, "int8a", pkv.MATH_MMA)])
def test_ragged_counts_and_any_bits(D, Hq, Hkv, T, dtype, math):
    # counts from none to T, any mask bits, rows that see nothing before or in the tree, an inactive sequence
    nodes = np.array([T, 0, 1, T - 1, 7, T, 0], np.int32)
    lens = [T, 40, 1, 300, 7, 200, 0]
    seed = 7500 + T + D + math
    c = random_case(seed, len(lens), Hq, Hkv, D, 16, lens, kv_dtype=dtype, poison=dtype == "bf16")
    dc = DeviceCase(c)
    q = normal_bf16_bits(seed + 1, (c.B, T, Hq, D))
    see, _ = _trees(seed + 2, c.B, T, nodes, dense=True)
    see[0, 3] = False  # no token before this tree: the row sees nothing
    see[4, :3] = False
    for ppu in (0, 3):
        out = bf16_dev_to_f64(_attend(dc, q, see, nodes, opts=pkv.decode_opts(partition_blocks=ppu, math=math)))
        assert pkv.read_device_error() == 0
        assert_tree_close(out, *_reference(dc, q, see, nodes), f"ppu={ppu}")
        assert (out[0, 3] == 0).all() and (out[4, :3] == 0).all() and (out[1] == 0).all() and (out[6] == 0).all()
        assert (out[3, T - 1:] == 0).all() and (out[4, 7:] == 0).all()


@pytest.mark.parametrize("T,dtype,D,lens", [
    (24, "bf16", 128, [5000, 1, 24, 130, 0, 3000, 700]), (24, "fp8", 128, [129, 6000, 24, 2000]), (30, "int8a", 128, [6000, 31, 128, 999]),
    (70, "bf16", 128, [4100, 70, 90, 1500]), (24, "bf16", 64, [24, 25, 7000, 128, 129]), (70, "fp8", 128, [2100, 70, 300]),
    (60, "int8", 128, [60, 1900, 300]), (24, "bf16", 128, [16000])])
@pytest.mark.parametrize("share", [0, 24, 250])
def test_shares_of_uneven_lengths(T, dtype, D, lens, share):
    # shares start and end anywhere in the items, short items among long ones;
    # share: fewest blocks of a share (0: one step; 250: few CTAs, whole items)
    c = random_case(7400 + T + D + len(lens), len(lens), 12, 3, D, 16, lens, kv_dtype=dtype)
    dc = DeviceCase(c)
    nodes = np.minimum(np.array(lens), T).astype(np.int32)
    q = normal_bf16_bits(7401, (c.B, T, 12, D))
    see, _ = _trees(7402, c.B, T, nodes)
    opts = pkv.decode_opts(partition_blocks=share, math=pkv.MATH_TC)
    out = _attend(dc, q, see, nodes, opts=opts)
    assert pkv.read_device_error() == 0
    assert_tree_close(bf16_dev_to_f64(out), *_reference(dc, q, see, nodes), f"share {share}")
    again = _attend(dc, q, see, nodes, opts=opts)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("dtype", ["fp8", "int8a"])
@pytest.mark.parametrize("order", ["up", "down", "mixed", "zero first"])
def test_page_scales_over_three_decades(dtype, order):
    # V page scales that grow, fall or jump along the sequence, and pages of zeros before the first others
    T, lens = 24, [900, 333]
    c = random_case(7450, 2, 16, 4, 128, 16, lens, kv_dtype=dtype)
    rng = np.random.Generator(np.random.PCG64(7451))
    for b, n in enumerate(lens):
        pages = c.block_tables[b, :-(-n // 16)]
        f = 10.0 ** rng.uniform(-3, 0, len(pages))
        f = np.sort(f) if order == "up" else np.sort(f)[::-1] if order == "down" else f
        f = np.where(np.arange(len(pages)) < 9, 0.0, f) if order == "zero first" else f
        scale = c.v_scale[0, pages] if dtype == "fp8" else c.v_scale[0, pages][..., 0]
        new = (scale * f[:, None]).astype(np.float32)
        if dtype == "fp8":
            c.v_scale[0, pages] = new
        else:
            c.v_scale[0, pages, :, 0] = new
    stored = [c.k_scale.copy(), c.v_scale.copy()]
    c.v_scale = np.where(c.v_scale == 0, np.float32(1), c.v_scale) if dtype == "fp8" else c.v_scale
    if dtype == "int8a":
        c.v_scale[..., 0] = np.where(c.v_scale[..., 0] == 0, np.float32(1), c.v_scale[..., 0])
    dc = DeviceCase(c)
    c.v_scale = stored[1]
    dc.vs = to_dev(c.v_scale)
    q = normal_bf16_bits(7452, (2, T, 16, 128))
    see, nodes = _trees(7453, 2, T)
    for share in (0, 1000):
        out = _attend(dc, q, see, nodes, opts=pkv.decode_opts(partition_blocks=min(share, 256), math=pkv.MATH_TC))
        assert_tree_close(bf16_dev_to_f64(out), *_reference(dc, q, see, nodes), f"{order} {share}")


@pytest.mark.parametrize("dtype", ["fp8", "int8a"])
@pytest.mark.parametrize("T", [24, 60])
@pytest.mark.parametrize("turn", [1, -1])
def test_page_scales_of_any_sign(dtype, T, turn):
    # negative K scales, negative and zero V scales, a negative softmax scale; some steps have only plain ones
    lens = [T, 700, 130, 1500]
    c = random_case(7460 + T, 4, 16, 4, 128, 16, lens, kv_dtype=dtype)
    dc = DeviceCase(c)
    rng = np.random.Generator(np.random.PCG64(7461))
    for s, signs in ((c.k_scale, [1, 1, -1]), (c.v_scale, [1, 1, -1, 0, 0.25])):
        f = rng.choice(signs, s.shape[1:3]).astype(np.float32)
        f[c.block_tables[3, :40]] = 1  # the long sequence's first five steps
        if dtype == "fp8":
            s *= f
        else:
            s[..., 0] *= f
    dc.ks, dc.vs = to_dev(c.k_scale), to_dev(c.v_scale)
    c.scale *= turn
    q = normal_bf16_bits(7462, (4, T, 16, 128))
    see, nodes = _trees(7463, 4, T)
    for share in (0, 256):
        out = _attend(dc, q, see, nodes, opts=pkv.decode_opts(partition_blocks=share, math=pkv.MATH_TC))
        assert_tree_close(bf16_dev_to_f64(out), *_reference(dc, q, see, nodes), f"share {share}")


@pytest.mark.parametrize("dtype,D,T", [("bf16", 128, 24), ("bf16", 128, 60), ("bf16", 64, 24), ("fp8", 128, 24), ("fp8", 128, 60),
                                       ("int8a", 128, 24)])
def test_non_finite_queries_stay_in_their_rows(dtype, D, T):
    c = random_case(7470 + T, 2, 16, 4, D, 16, [T + 3, 400], kv_dtype=dtype)
    dc = DeviceCase(c)
    q = normal_bf16_bits(7471, (2, T, 16, D))
    see, nodes = _trees(7472, 2, T)
    want = _reference(dc, q, see, nodes)
    bad = [(0, 0, 3, 5, 0x7F80), (0, T - 1, 15, D - 1, 0xFF80), (1, 7, 0, 0, BF16_NAN)]
    for b, t, h, d, bits in bad:
        q[b, t, h, d] = bits
    got = bf16_dev_to_f64(_attend(dc, q, see, nodes, opts=pkv.decode_opts(math=pkv.MATH_TC)))
    for b, t, h, _, _ in bad:
        assert np.isnan(got[b, t, h]).all()
        got[b, t, h] = want[0][b, t, h]
    assert_tree_close(got, *want, dtype)


@pytest.mark.parametrize("B", [192, 193, 1100, 2100])
def test_batches_of_many_short_sequences(B):
    # some without tokens; more sequences than the planner has threads, or room in shared memory
    T, rng = 3, np.random.Generator(np.random.PCG64(B))
    lens = rng.integers(0, 50, B)
    lens[rng.random(B) < 0.2] = 0
    lens[B // 2] = 900
    c = random_case(7480 + B, B, 8, 2, 64, 16, lens.tolist())
    dc = DeviceCase(c)
    nodes = np.minimum(lens, rng.integers(0, T + 1, B)).astype(np.int32)
    q = normal_bf16_bits(7481, (B, T, 8, 64))
    see, _ = _trees(7482, B, T, nodes)
    out = _attend(dc, q, see, nodes)
    assert pkv.decode_plan(dc.k, B, 8, c.MB, None, T, tree=True)["math"] == pkv.MATH_TC
    assert pkv.read_device_error() == 0
    assert_tree_close(bf16_dev_to_f64(out), *_reference(dc, q, see, nodes), f"B={B}")


@pytest.mark.parametrize("dtype,T,math", [("bf16", 6, pkv.MATH_MMA), ("bf16", 20, pkv.MATH_TC), ("bf16", 60, pkv.MATH_TC), ("fp8", 20, pkv.MATH_TC)])
def test_fewer_tokens_than_nodes(dtype, T, math):
    # nodes before position 0 do not exist; the others are attended to as the mask says
    lens = [T - 3, 2, T + 1]
    c = random_case(7600 + T, 3, 32, 8, 128, 16, lens, kv_dtype=dtype)
    dc = DeviceCase(c)
    q = normal_bf16_bits(7601, (3, T, 32, 128))
    see, nodes = _trees(7602, 3, T, dense=True)
    out = bf16_dev_to_f64(_attend(dc, q, see, opts=pkv.decode_opts(math=math)))
    assert_tree_close(out, *_reference(dc, q, see, nodes), "short contexts")
    assert pkv.read_device_error() == 0


@pytest.mark.parametrize("D,Hq,Hkv,T,dtype,math", [
    (128, 32, 8, 4, "bf16", pkv.MATH_AUTO), (128, 32, 8, 24, "bf16", pkv.MATH_TC), (128, 32, 8, 70, "bf16", pkv.MATH_TC),
    (64, 8, 8, 20, "bf16", pkv.MATH_MMA), (128, 32, 8, 24, "fp8", pkv.MATH_TC), (128, 32, 8, 3, "fp8", pkv.MATH_MMA),
    (128, 32, 8, 24, "int8a", pkv.MATH_TC)])
@pytest.mark.parametrize("ppu", [0, 3])
def test_chain_gives_the_causal_result(D, Hq, Hkv, T, dtype, math, ppu):
    lens = [T, T + 5, 300, 1000]
    c = random_case(7700 + T + D, 4, Hq, Hkv, D, 16, lens, kv_dtype=dtype)
    dc = DeviceCase(c)
    q = normal_bf16_bits(7701, (4, T, Hq, D))
    see = np.broadcast_to(np.tril(np.ones((T, T), bool)), (4, T, T))
    opts = pkv.decode_opts(partition_blocks=ppu, math=math)
    tree = _attend(dc, q, see, opts=opts)
    multi = pkv.paged_decode_multi(to_dev_bf16(q), dc.k, dc.v, dc.bt, dc.cl, c.kv_group_ptr.tolist(), 0, c.scale,
                                   k_scale=dc.ks, v_scale=dc.vs, opts=opts)
    torch.cuda.synchronize()
    if pkv.decode_plan(dc.k, 4, Hq, c.MB, opts, T, tree=True)["math"] == pkv.MATH_MMA:  # the same tiles and partitions
        assert torch.equal(tree.view(torch.int16), multi.view(torch.int16))
    ref = _reference(dc, q, see, np.full(4, T))
    assert_tree_close(bf16_dev_to_f64(tree), *ref, "tree")
    assert_tree_close(bf16_dev_to_f64(multi), *ref, "causal")


@pytest.mark.parametrize("T", [3, 20, 60])
def test_one_tree_for_all(T):
    c = random_case(7800 + T, 4, 32, 8, 128, 16, [T, 90, 300, 41 + T])
    dc = DeviceCase(c)
    q = normal_bf16_bits(7801, (4, T, 32, 128))
    see, _ = _trees(7802, 1, T)
    nodes = np.array([T, max(1, T - 2), T, 1], np.int32)
    one = _attend(dc, q, see, nodes)
    each = _attend(dc, q, np.repeat(see, 4, 0), nodes)
    assert torch.equal(one.view(torch.int16), each.view(torch.int16))


@pytest.mark.parametrize("dtype,D,T,math", [("bf16", 128, 4, pkv.MATH_MMA), ("bf16", 64, 20, pkv.MATH_MMA), ("bf16", 128, 24, pkv.MATH_TC),
                                            ("bf16", 128, 60, pkv.MATH_TC), ("fp8", 128, 24, pkv.MATH_TC), ("fp8", 128, 4, pkv.MATH_MMA)])
@pytest.mark.parametrize("ppu", [0, 1])
def test_non_finite_values_stay_where_they_are_seen(dtype, D, T, math, ppu):
    # K and V of some nodes hold NaN or infinity, in every element or in one:
    # rows that do not attend to them are as without, the others are NaN
    Hq, Hkv = (32, 8) if D == 128 else (8, 8)
    nodes = np.array([T, T - 1, T], np.int32)
    lens = [T + 37, 150, T]
    c = random_case(7900 + T + D, 3, Hq, Hkv, D, 16, lens, kv_dtype=dtype)
    dc = DeviceCase(c)
    q = normal_bf16_bits(7901, (3, T, Hq, D))
    q[1, T - 1] = BF16_NAN  # a row past the count: zeros all the same
    see, _ = _trees(7902, 3, T, nodes)
    clean, wabs = _reference(dc, q, see, nodes)
    bad = {0: T - 2, 1: 1, 2: T - 1}  # node of each sequence
    k, v = dc.k_host.copy(), dc.v_host.copy()
    nan = BF16_NAN if dtype == "bf16" else np.uint8(0x7F)
    inf = np.uint16(0xFF80) if dtype == "bf16" else np.uint8(0xFF)
    for b, u in bad.items():
        pos = lens[b] - nodes[b] + u
        blk, off = c.block_tables[b, pos // 16], pos % 16
        if b == 0:
            k[0, blk, :, off] = nan
            v[0, blk, :, off] = nan
        elif b == 1:
            v[0, blk, :, off, D - 1] = inf
        else:
            v[0, blk, Hkv - 1, off, 0] = nan  # one KV head only
    dc.k, dc.v = (to_dev_bf16(k), to_dev_bf16(v)) if dtype == "bf16" else (to_dev(k), to_dev(v))
    out = bf16_dev_to_f64(_attend(dc, q, see, nodes, opts=pkv.decode_opts(partition_blocks=ppu, math=math)))
    touched = np.zeros((3, T, Hq), bool)
    for b, u in bad.items():
        heads = slice(None) if b != 2 else slice(Hq - Hq // Hkv, None)
        touched[b, see[b, :, u], heads] = True
    assert touched.any() and not touched.all()
    assert np.isnan(out[touched]).all()
    assert_tree_close(np.where(touched[..., None], clean, out), clean, wabs, "rows that do not attend to them")
    assert (out[1, T - 1] == 0).all()
    assert pkv.read_device_error() == 0


def test_rows_past_the_count_are_zero_beside_a_nan_before_the_tree():
    for T, math in ((4, pkv.MATH_MMA), (24, pkv.MATH_TC), (60, pkv.MATH_TC)):
        c = random_case(8000 + T, 1, 32, 8, 128, 16, [100])
        dc = DeviceCase(c)
        v = dc.v_host.copy()
        v[0, c.block_tables[0, 0], :, 3] = BF16_NAN  # every node attends to it
        dc.v = to_dev_bf16(v)
        see, nodes = _trees(8001, 1, T, [T - 2])
        for ppu in (0, 1):
            out = bf16_dev_to_f64(_attend(dc, normal_bf16_bits(8002, (1, T, 32, 128)), see, nodes,
                                          opts=pkv.decode_opts(partition_blocks=ppu, math=math)))
            assert np.isnan(out[0, :T - 2]).all() and (out[0, T - 2:] == 0).all(), (T, ppu)


@pytest.mark.parametrize("T,math", [(4, pkv.MATH_MMA), (24, pkv.MATH_TC), (60, pkv.MATH_TC)])
def test_bad_counts_lengths_and_blocks(T, math):
    lens = [T + 20, 90, 130, 64]
    c = random_case(8100 + T, 4, 32, 8, 128, 16, lens)
    dc = DeviceCase(c)
    q = normal_bf16_bits(8101, (4, T, 32, 128))
    see, nodes = _trees(8102, 4, T)
    opts = pkv.decode_opts(math=math)
    good = bf16_dev_to_f64(_attend(dc, q, see, nodes, opts=opts))
    for wrong in (T + 1, -1, 1 << 30):
        n2 = nodes.copy()
        n2[1] = wrong
        out = bf16_dev_to_f64(_attend(dc, q, see, n2, opts=opts))
        assert pkv.read_device_error() == pkv.DEVERR_TREE
        assert (out[1] == 0).all() and np.array_equal(out[[0, 2, 3]], good[[0, 2, 3]])
    for wrong in (-1, c.MB * 16 + 1):
        cl = c.context_lens.copy()
        cl[2] = wrong
        dc.cl = to_dev(cl)
        out = bf16_dev_to_f64(_attend(dc, q, see, nodes, opts=opts))
        assert pkv.read_device_error() == pkv.DEVERR_CONTEXT_LEN
        assert (out[2] == 0).all() and np.array_equal(out[[0, 1, 3]], good[[0, 1, 3]])
    dc.cl = to_dev(c.context_lens)
    bt = c.block_tables.copy()
    bt[3, 1] = c.NB  # its 16 tokens take no part
    dc.bt = to_dev(bt)
    out = bf16_dev_to_f64(_attend(dc, q, see, nodes, opts=opts))
    assert pkv.read_device_error() == pkv.DEVERR_BLOCK_ID
    assert np.isfinite(out).all() and np.array_equal(out[:3], good[:3])


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
def test_other_scales(scale):
    for T in (3, 24, 60):
        c = random_case(8200 + T, 2, 32, 8, 128, 16, [T + 9, 200])
        dc = DeviceCase(c)
        q = normal_bf16_bits(8201, (2, T, 32, 128))
        see, nodes = _trees(8202, 2, T)
        out = pkv.paged_decode_tree(to_dev_bf16(q), dc.k, dc.v, dc.bt, dc.cl, to_dev(pack(see)), scale=scale)
        want, wabs = tree_attention(q, dc.k_host, dc.v_host, c.block_tables, c.context_lens, see, nodes, scale)
        # scores 20 times the usual ones at scale 1.7: off by 20 times 2^-12 each
        err = np.abs(bf16_dev_to_f64(out) - want)
        assert (err <= (2.0 ** -8 + 2.0 ** -7) * wabs + 2.0 ** -8 * np.abs(want) + 1e-30).all(), (T, (err / wabs).max())


def test_cache_offsets_past_32_bits():
    # a pool of more than 2^31 elements (and 2^32 bytes); the sequences' blocks are its last ones
    Hkv, D, bs, T = 8, 128, 16, 24
    NB = (1 << 31) // (Hkv * bs * D) + 64
    c = random_case(8300, 2, 32, Hkv, D, bs, [90, 300])
    dc = DeviceCase(c)
    shift = NB - c.NB
    k = torch.empty((1, NB, Hkv, bs, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty((1, NB, Hkv, bs, D), dtype=torch.bfloat16, device=DEV)
    k[:, shift:], v[:, shift:] = dc.k, dc.v
    bt = to_dev(np.where(c.block_tables >= 0, c.block_tables + shift, -1).astype(np.int32))
    see, _ = _trees(8301, 2, T)
    mask = to_dev(pack(see))
    for rows in (2, T):
        q = to_dev_bf16(normal_bf16_bits(8302, (2, T, 32, D)))[:, :rows].contiguous()
        m = mask[:, :rows].contiguous()
        small = pkv.paged_decode_tree(q, dc.k, dc.v, dc.bt, dc.cl, m)
        large = pkv.paged_decode_tree(q, k, v, bt, dc.cl, m)
        assert torch.equal(small.view(torch.int16), large.view(torch.int16))
    # rows moved there: node 3 of the second sequence onto its node 1, in the small and the large pool
    idx, count = to_dev(np.array([[0, 0], [0, 3]], np.int32)), to_dev(np.array([1, 2], np.int32))
    pkv.compact_tokens(idx, count, dc.cl, dc.bt, dc.k, dc.v, T)
    pkv.compact_tokens(idx, count, dc.cl, bt, k, v, T)
    assert torch.equal(k[:, shift:].view(torch.int16), dc.k.view(torch.int16))
    assert torch.equal(v[:, shift:].view(torch.int16), dc.v.view(torch.int16))
    assert pkv.read_device_error() == 0


def test_other_stream_and_prepared():
    T = 24
    c = random_case(8400, 3, 32, 8, 128, 16, [90, 700, 41])
    dc = DeviceCase(c)
    q = to_dev_bf16(normal_bf16_bits(8401, (3, T, 32, 128)))
    see, nodes = _trees(8402, 3, T, [T, 3, 11])
    mask, counts = to_dev(pack(see)), to_dev(nodes)
    ref = pkv.paged_decode_tree(q, dc.k, dc.v, dc.bt, dc.cl, mask, counts)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [pkv.paged_decode_tree(q, dc.k, dc.v, dc.bt, dc.cl, mask, counts, stream=s) for _ in range(4)]
    n = pkv.decode_workspace_bytes(dc.k, 3, 32, c.MB, None, T, tree=True)
    call = pkv.PreparedDecode(q, dc.k, dc.v, dc.bt, dc.cl, tree_mask=mask, node_counts=counts, stream=s,
                              workspace=torch.full((n,), 0xEE, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    outs.append(call())
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), ref.view(torch.int16))
    assert pkv.read_device_error() == 0


@pytest.mark.parametrize("dtype,T", [("bf16", 24), ("int8a", 24), ("fp8", 60)])
def test_calls_at_the_same_time(dtype, T):
    # two streams, a workspace each: persistent kernels that fill the GPU take turns, and change nothing of each other's
    calls, refs = [], []
    for i, lens in enumerate(([T, 900, 2500], [1400, T + 1, 60])):
        c = random_case(8500 + i, 3, 16, 4, 128, 16, lens, kv_dtype=dtype)
        dc = DeviceCase(c)
        q = to_dev_bf16(normal_bf16_bits(8501 + i, (3, T, 16, 128)))
        see, _ = _trees(8502 + i, 3, T)
        mask = to_dev(pack(see))
        refs.append(pkv.paged_decode_tree(q, dc.k, dc.v, dc.bt, dc.cl, mask, k_scale=dc.ks, v_scale=dc.vs))
        n = pkv.decode_workspace_bytes(dc.k, 3, 16, c.MB, None, T, tree=True)
        calls.append(pkv.PreparedDecode(q, dc.k, dc.v, dc.bt, dc.cl, k_scale=dc.ks, v_scale=dc.vs, tree_mask=mask,
                                        stream=torch.cuda.Stream(), workspace=torch.empty(n, dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(10):
        for call in calls:
            call.out.fill_(float("nan"))
        torch.cuda.synchronize()
        outs = [[call() for call in calls] for _ in range(5)][-1]
        torch.cuda.synchronize()
        for o, ref in zip(outs, refs):
            assert torch.equal(o.view(torch.int16), ref.view(torch.int16))
    assert pkv.read_device_error() == 0


def test_two_graphs_with_one_workspace():
    # replayed one after the other, each gives its own results
    cases, graphs = [], []
    T = 40
    n = 0
    for i, lens in enumerate(([60, 900, 333], [2000, 41, 700])):
        c = random_case(8500 + i, 3, 32, 8, 128, 16, lens)
        dc = DeviceCase(c)
        q = to_dev_bf16(normal_bf16_bits(8510 + i, (3, T, 32, 128)))
        see, nodes = _trees(8520 + i, 3, T, [T, T - 3, 5])
        ref = pkv.paged_decode_tree(q, dc.k, dc.v, dc.bt, dc.cl, to_dev(pack(see)), to_dev(nodes))
        cases.append((dc, q, to_dev(pack(see)), to_dev(nodes), torch.empty_like(q), ref))
        n = max(n, pkv.decode_workspace_bytes(dc.k, 3, 32, c.MB, None, T, tree=True))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for dc, q, mask, nodes, out, _ in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_decode_tree(q, dc.k, dc.v, dc.bt, dc.cl, mask, nodes, out=out, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for (_, _, _, _, out, _), g in zip(cases, graphs):
            out.zero_()
            g.replay()
        for (_, _, _, _, out, ref), g in zip(cases, graphs):
            assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    assert pkv.read_device_error() == 0


# ---------------------------------------------------------------------------
# masks
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,T", [(1, 1), (3, 2), (5, 31), (4, 32), (4, 33), (7, 64), (2, 100), (3, 257), (2, 512), (300, 17)])
@pytest.mark.parametrize("kind", ["tree", "chain", "star", "ragged"])
def test_masks(B, T, kind):
    rng = np.random.Generator(np.random.PCG64(B * 1000 + T))
    parents = random_parents(rng, B, T, 9)
    if kind == "chain":
        parents = np.broadcast_to(np.arange(-1, T - 1, dtype=np.int32), (B, T)).copy()
    if kind == "star":
        parents = np.zeros((B, T), np.int32) - (np.arange(T) == 0)
    nodes = rng.integers(0, T + 1, B).astype(np.int32) if kind == "ragged" else np.full(B, T, np.int32)
    see, depth = visible(parents, nodes)
    ctx = nodes + rng.integers(0, 5000, B).astype(np.int32)
    mask, pos = pkv.tree_masks(to_dev(parents.astype(np.int32)), to_dev(ctx), to_dev(nodes) if kind == "ragged" else None)
    torch.cuda.synchronize()
    assert np.array_equal(mask.cpu().numpy(), pack(see))
    assert np.array_equal(pos.cpu().numpy(), np.where(depth >= 0, (ctx - nodes)[:, None] + depth, 0))
    _, pos = pkv.tree_masks(to_dev(parents.astype(np.int32)), None, to_dev(nodes))
    assert np.array_equal(pos.cpu().numpy(), np.maximum(depth, 0))
    assert pkv.read_device_error() == 0


def test_masks_bad_parents_and_counts():
    parents = np.array([[-1, 0, 1, 2], [-1, 5, 1, 3], [-2, 0, 0, -7], [-1, 0, 0, 2]], np.int32)
    nodes = np.array([4, 4, 4, 9], np.int32)
    fixed = np.array([[-1, 0, 1, 2], [-1, -1, 1, -1], [-1, 0, 0, -1], [-1, 0, 0, 2]], np.int32)
    ctx = np.array([10, 2, 4, 9], np.int32)  # the second: fewer tokens than nodes, positions stop at 0
    mask, pos = pkv.tree_masks(to_dev(parents), to_dev(ctx), to_dev(nodes))
    torch.cuda.synchronize()
    assert pkv.read_device_error() == pkv.DEVERR_TREE
    see, depth = visible(fixed, [4, 4, 4, 0])
    assert np.array_equal(mask.cpu().numpy(), pack(see))
    want = np.where(depth >= 0, np.maximum((ctx - 4)[:, None] + depth, 0), 0)
    assert np.array_equal(pos.cpu().numpy(), want)
