"""Drafted-tree attention over keys, values and page scales that are not finite:
rows that attend to them are NaN, the others are as without."""
import numpy as np
import pytest

import paged_kv_cache_274_gb300 as pkv
from workloads import normal_bf16_bits, random_case
from workloads.gen import BF16_NAN
from tests._gpu import DeviceCase, bf16_dev_to_f64, to_dev, to_dev_bf16
from tests._tree import assert_tree_close, pack, random_parents, tree_attention, visible

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("fp8", 128)])
@pytest.mark.parametrize("T,math", [(3, pkv.MATH_MMA), (40, pkv.MATH_MMA), (24, pkv.MATH_TC), (60, pkv.MATH_TC)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_rows_that_attend_to_nans_alone(dtype, D, T, math, what):
    # nothing before the tree, every node sees only itself, some hold NaNs: in
    # partitions of their own, too, such a row has no finite score at all
    c = random_case(7480 + T, 2, 16, 4, D, 16, [T, T + 40], kv_dtype=dtype)
    dc = DeviceCase(c)
    q = normal_bf16_bits(7481, (2, T, 16, D))
    see, nodes = np.broadcast_to(np.eye(T, dtype=bool), (2, T, T)).copy(), np.full(2, T, np.int32)
    clean, wabs = tree_attention(q, dc.k_host, dc.v_host, c.block_tables, c.context_lens, see, nodes, c.scale, c.k_scale, c.v_scale)
    host = (dc.k_host if what == "k" else dc.v_host).copy()
    bad = np.zeros((2, T), bool)
    bad[:, 1] = bad[:, T - 1] = True
    for b, t in np.argwhere(bad):
        pos = int(c.context_lens[b]) - T + t
        host[0, c.block_tables[b, pos // 16], :, pos % 16] = BF16_NAN if dtype == "bf16" else 0x7F
    put = to_dev_bf16(host) if dtype == "bf16" else to_dev(host)
    dc.k, dc.v = (put, dc.v) if what == "k" else (dc.k, put)
    for share in (0, 1, 2):
        out = pkv.paged_decode_tree(to_dev_bf16(q), dc.k, dc.v, dc.bt, dc.cl, to_dev(pack(see)), scale=c.scale, k_scale=dc.ks,
                                    v_scale=dc.vs, opts=pkv.decode_opts(partition_blocks=share, math=math))
        got = bf16_dev_to_f64(out)
        assert pkv.read_device_error() == 0
        assert np.isnan(got[bad]).all(), f"share {share}"
        assert_tree_close(np.where(bad[..., None, None], clean, got), clean, wabs, f"share {share}")


@pytest.mark.parametrize("dtype", ["fp8", "int8a"])
@pytest.mark.parametrize("T,math", [(4, pkv.MATH_MMA), (24, pkv.MATH_MMA), (24, pkv.MATH_TC), (60, pkv.MATH_TC)])
@pytest.mark.parametrize("which,bad", [("v", np.nan), ("v", np.inf), ("v", -np.inf), ("k", np.nan), ("v and k", np.nan)])
def test_scales_that_are_not_finite(dtype, T, math, which, bad):
    # the pages of the last nodes: in the same step as every other page, in a
    # later step, and in a sequence that is nothing but nodes
    Hq, Hkv, late = 16, 4, T - 2 if T < 16 else 16
    lens = [32 - late % 16 + T, 608 - late % 16 + T, T]
    c = random_case(7490 + T, 3, Hq, Hkv, 128, 16, lens, kv_dtype=dtype)
    dc = DeviceCase(c)
    q = normal_bf16_bits(7491, (3, T, Hq, 128))
    nodes = np.full(3, T, np.int32)
    see, _ = visible(random_parents(np.random.Generator(np.random.PCG64(7492)), 3, T, 40), nodes)
    clean, wabs = tree_attention(q, dc.k_host, dc.v_host, c.block_tables, c.context_lens, see, nodes, c.scale, c.k_scale, c.v_scale)
    touched = np.zeros((3, T), bool)
    for b, n in enumerate(lens):
        page = (n - 1) // 16
        first = max(0, page * 16 - (n - T))  # its first node
        if n - T > page * 16 or (n == T and T < 16):  # (holds tokens that every row attends to, or is the only page)
            continue
        touched[b] = see[b, :, first:].any(1)
        for s in ([c.v_scale] if which == "v" else [c.k_scale] if which == "k" else [c.v_scale, c.k_scale]):
            if dtype == "fp8":
                s[0, c.block_tables[b, page]] = bad
            else:
                s[0, c.block_tables[b, page], :, 0] = bad
    assert touched.any() and not touched.all()
    dc.ks, dc.vs = to_dev(c.k_scale), to_dev(c.v_scale)
    for share in (0, 1, 256 if math == pkv.MATH_TC else 64):
        out = pkv.paged_decode_tree(to_dev_bf16(q), dc.k, dc.v, dc.bt, dc.cl, to_dev(pack(see)), scale=c.scale, k_scale=dc.ks,
                                    v_scale=dc.vs, opts=pkv.decode_opts(partition_blocks=share, math=math))
        got = bf16_dev_to_f64(out)
        assert pkv.read_device_error() == 0
        assert np.isnan(got[touched]).all(), f"share {share}"
        assert_tree_close(np.where(touched[..., None, None], clean, got), clean, wabs, f"share {share}")
