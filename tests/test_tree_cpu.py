"""Drafted-tree operators without a GPU: the plans, and what the C ABI and the
binding refuse before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_274_gb300 as pkv
from paged_kv_cache_274_gb300 import _build
from tests._tree import Pool, pack, random_parents, visible


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pkv.load()


def _desc(**kw):
    d = dict(num_slots=1, num_blocks=100, block_size=16, num_kv_heads=8, head_dim=128, dtype=0)
    d.update(kw)
    return pkv.CacheDesc(**d)


def _p(i):
    return ctypes.c_void_p(0x100000 * i)


def _plan(lib, d, B, T, Hq, MB, opts=None):
    plan = pkv.DecodePlan()
    st = lib.pkv_decode_tree_describe(ctypes.byref(d), B, T, Hq, MB, ctypes.byref(opts) if opts is not None else None,
                                      ctypes.byref(plan))
    return st, plan


def test_tree_plans(lib):
    # rows (nodes x heads of a KV head) up to which mma.sync is chosen
    for dtype, D, rows in ((0, 128, 0), (0, 64, 8), (1, 128, 16), (2, 128, 16)):
        for T in (1, 2, 3, 4, 5, 32):
            st, plan = _plan(lib, _desc(dtype=dtype, head_dim=D), 8, T, 32, 64)
            assert st == 0 and plan.math == (pkv.MATH_MMA if 4 * T <= rows else pkv.MATH_TC)
    st, plan = _plan(lib, _desc(dtype=1, num_kv_heads=1), 8, 1, 32, 64)   # 32 heads on one KV head, one node
    assert st == 0 and plan.math == pkv.MATH_TC
    assert _plan(lib, _desc(), 8, 4, 32, 64, pkv.decode_opts(math=pkv.MATH_FFMA))[0] == 2
    assert _plan(lib, _desc(), 8, 1, 32, 64, pkv.decode_opts(math=pkv.MATH_FFMA))[0] == 2
    assert _plan(lib, _desc(), 8, 0, 32, 64)[0] == 1
    assert _plan(lib, _desc(), 8, pkv.MAX_QUERY_TOKENS + 1, 32, 64)[0] == 1
    # mma.sync: the workspace adds a word of 32 nodes per (sequence, KV head)
    d = _desc()
    mma = pkv.decode_opts(math=pkv.MATH_MMA)
    multi = lib.pkv_decode_multi_workspace_bytes(ctypes.byref(d), 64, 33, 32, 64, ctypes.byref(mma))
    tree = lib.pkv_decode_tree_workspace_bytes(ctypes.byref(d), 64, 33, 32, 64, ctypes.byref(mma))
    assert tree == multi + 64 * 8 * 2 * 4
    assert lib.pkv_decode_tree_workspace_bytes(ctypes.byref(d), 64, 0, 32, 64, None) == 0


@pytest.mark.parametrize("dtype,D", [(0, 128), (0, 64), (1, 128), (2, 128)])
@pytest.mark.parametrize("T", [9, 32, 33, 512])
def test_tcgen05_tree_plans(lib, dtype, D, T):
    st, plan = _plan(lib, _desc(dtype=dtype, head_dim=D), 8, T, 32, 64)
    assert st == 0 and plan.math == pkv.MATH_TC and plan.kernels_per_call == (3 if T <= 512 else 2)
    assert plan.smem_bytes_per_cta <= 227 * 1024 and plan.warps_per_cta == (20 if dtype == 0 else 28)
    assert plan.row_tiles == -(-T // min(T, 32))
    # partials: at most two per CTA, whatever the lengths
    rows = 128 if plan.row_tiles == 1 else 256
    assert plan.workspace_bytes < 152 * 2 * rows * (D + 2) * 4 + (1 << 20)
    st, longer = _plan(lib, _desc(dtype=dtype, head_dim=D, num_blocks=100000), 8, T, 32, 8192)
    assert st == 0 and longer.workspace_bytes == plan.workspace_bytes


def _attend(lib, **kw):
    a = dict(q=_p(1), B=2, T=4, Hq=32, k=_p(2), v=_p(3), bt=_p(4), MB=4, cl=_p(5), mask=_p(6), TB=2, nodes=None, out=_p(7), ws=_p(8),
             wsb=1 << 30, scale=0.1, desc=_desc(), layer=0)
    a.update(kw)
    gp = (ctypes.c_int32 * 1)(0)
    return lib.pkv_paged_decode_tree(ctypes.byref(a["desc"]), a["q"], a["B"], a["T"], a["Hq"], a["k"], a["v"], None, None, a["bt"],
                                     a["MB"], a["cl"], a["mask"], a["TB"], a["nodes"], gp, 1, a["layer"], a["scale"], a["out"], a["ws"],
                                     a["wsb"], None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(mask=None), 1), (dict(TB=3), 1), (dict(TB=0), 1), (dict(T=0), 1), (dict(T=513), 1), (dict(Hq=12), 1), (dict(q=None), 1),
    (dict(mask=ctypes.c_void_p(0x600002)), 3), (dict(nodes=ctypes.c_void_p(0x600001)), 3), (dict(out=_p(1)), 1), (dict(ws=None), 6),
    (dict(wsb=64), 6), (dict(scale=float("inf")), 1), (dict(layer=1), 1), (dict(desc=_desc(head_dim=64, dtype=1)), 2),
    (dict(desc=_desc(num_kv_heads=1), Hq=129), 2),       # 129 heads on one KV head
    (dict(desc=_desc(dtype=1)), 1)])                     # E4M3 without scales
def test_attention_refusals(lib, bad, status):
    assert _attend(lib, **bad) == status


def test_empty_batches_launch_nothing(lib):
    assert _attend(lib, B=0, TB=1) == 0
    assert lib.pkv_tree_masks(None, None, None, 0, 5, None, None, None) == 0
    d = _desc()
    assert lib.pkv_compact_tokens(ctypes.byref(d), None, None, 1, 0, None, None, 4, None, 4, None, None, None, None, None, None) == 0


@pytest.mark.parametrize("args,status", [
    ((None, None, None, 2, 4, _p(2), None), 1), ((_p(1), None, None, 2, 4, None, None), 1), ((_p(1), None, None, -1, 4, _p(2), None), 1),
    ((_p(1), None, None, 2, 0, _p(2), None), 1), ((_p(1), None, None, 2, 513, _p(2), None), 1),
    ((_p(1), None, ctypes.c_void_p(0x300002), 2, 4, _p(2), None), 3), ((_p(1), None, None, 2, 4, _p(1), None), 1),
    ((_p(1), None, None, 2, 4, _p(2), ctypes.c_void_p(0x200008)), 1), ((_p(1), _p(2), None, 2, 4, _p(2), None), 1)])
def test_mask_refusals(lib, args, status):
    assert lib.pkv_tree_masks(*args, None) == status


def _extend(lib, **kw):
    a = dict(B=4, bs=16, MB=8, NB=64, seq=_p(1), new=_p(2), bor=None, bt=_p(3), cnt=_p(4), cnt2=_p(4), ring=_p(5), st=_p(6), st2=_p(6),
             ctx=_p(7), qs=_p(8), slots=_p(9), pos=_p(10), N=32)
    a.update(kw)
    return lib.pkv_extend_tables(*[a[k] for k in ("B", "bs", "MB", "NB", "seq", "new", "bor", "bt", "cnt", "cnt2", "ring", "st", "st2", "ctx",
                                                  "qs", "slots", "pos", "N")], None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), 1), (dict(B=16385), 1), (dict(bs=8), 2), (dict(MB=0), 1), (dict(NB=0), 1), (dict(N=-1), 1), (dict(NB=1 << 30), 2),
    (dict(B=16384, MB=1 << 17), 2), (dict(MB=1 << 27), 2), (dict(seq=None), 1), (dict(new=None), 1), (dict(bt=None), 1), (dict(cnt=None), 1),
    (dict(cnt2=None), 1), (dict(ring=None), 1), (dict(st=None), 1), (dict(st2=None), 1), (dict(ctx=None), 1), (dict(qs=None), 1),
    (dict(slots=None), 1), (dict(seq=ctypes.c_void_p(0x100002)), 3), (dict(slots=ctypes.c_void_p(0x900004)), 3),
    (dict(ctx=_p(1)), 1), (dict(qs=ctypes.c_void_p(0x700008)), 1), (dict(pos=ctypes.c_void_p(0x900010)), 1), (dict(cnt2=_p(1)), 1),
    (dict(st2=_p(5)), 1), (dict(bor=_p(7)), 1), (dict(cnt2=ctypes.c_void_p(0x400004)), 1)])
def test_extend_refusals(lib, bad, status):
    assert _extend(lib, **bad) == status


def _compact(lib, **kw):
    a = dict(desc=_desc(), idx=_p(1), cnt=_p(2), A=4, B=3, cl=_p(3), nodes=None, T=8, bt=_p(4), MB=8, k=_p(5), v=_p(6), ks=None, vs=None,
             seq=_p(7))
    a.update(kw)
    return lib.pkv_compact_tokens(ctypes.byref(a["desc"]), *[a[k] for k in ("idx", "cnt", "A", "B", "cl", "nodes", "T", "bt", "MB", "k", "v",
                                                                            "ks", "vs", "seq")], None)


@pytest.mark.parametrize("bad,status", [
    (dict(desc=_desc(block_size=8)), 2), (dict(A=0), 1), (dict(A=513), 1), (dict(T=0), 1), (dict(T=513), 1), (dict(B=-1), 1), (dict(MB=0), 1),
    (dict(MB=1 << 27), 2), (dict(idx=None), 1), (dict(seq=None), 1), (dict(k=None), 1), (dict(desc=_desc(dtype=2)), 1),
    (dict(desc=_desc(dtype=2), ks=ctypes.c_void_p(0x800004), vs=_p(9)), 3), (dict(k=ctypes.c_void_p(0x500008)), 3),
    (dict(cl=ctypes.c_void_p(0x300002)), 3), (dict(seq=_p(3)), 1), (dict(seq=ctypes.c_void_p(0x100010)), 1)])
def test_compact_refusals(lib, bad, status):
    assert _compact(lib, **bad) == status


def test_binding_refuses_host_tensors():
    k = torch.zeros((1, 4, 2, 16, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    q = torch.zeros((2, 4, 4, 64), dtype=torch.bfloat16)
    for call in (lambda: pkv.paged_decode_tree(q, k, k, t, i, torch.zeros((2, 4, 1), dtype=torch.int32)),
                 lambda: pkv.PreparedDecode(q, k, k, t, i, tree_mask=torch.zeros((2, 4, 1), dtype=torch.int32)),
                 lambda: pkv.tree_masks(t), lambda: pkv.extend_tables(i, i, t, i, i, i, 16, 4),
                 lambda: pkv.compact_tokens(t, i, i, t, k, k, 4)):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.status == 1 and "CUDA tensor" in str(e.value)
    with pytest.raises(pkv.PkvError):
        pkv.new_free_ring(range(5), 4, "cpu")
    ring, state = pkv.new_free_ring([3, 1], 4, "cpu")
    assert ring.tolist() == [3, 1, -1, -1] and state.tolist() == [0, 2, 0, 0]


def test_references():
    # the references of the GPU tests on a case worked out by hand
    parents = np.array([[-1, 0, 0, 1, 3, 2]], np.int32)
    see, depth = visible(parents, [6])
    assert [np.flatnonzero(r).tolist() for r in see[0]] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [0, 2, 5]]
    assert depth.tolist() == [[0, 1, 1, 2, 3, 2]] and pack(see)[0, :, 0].tolist() == [1, 3, 5, 11, 27, 37]
    pool = Pool(6, 16, 4, [4, 2, 5], head=5)
    tables, counts = np.array([[0, -1, -1, -1], [1, 3, -1, -1]], np.int32), np.array([1, 2], np.int32)
    ctx, starts, slots, pos, err = pool.extend([15, 20], [3, -1], tables, counts, 5)
    assert ctx.tolist() == [18, 0] and starts.tolist() == [0, 3, 3] and slots.tolist() == [15, 64, 65, -1, -1] and err == 0
    assert pos.tolist() == [15, 16, 17, 0, 0] and counts.tolist() == [2, 0] and tables[0].tolist() == [0, 4, -1, -1]
    assert (pool.head, pool.free) == (0, 4) and [pool.ring[k % 6] for k in range(4)] == [2, 5, 1, 3]
    assert random_parents(np.random.Generator(np.random.PCG64(0)), 2, 5)[:, 0].tolist() == [-1, -1]
