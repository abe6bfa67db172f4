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
