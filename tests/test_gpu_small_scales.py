"""One-byte caches with pages whose v scale is positive and next to nothing beside
the others' (the least a page of zeros may be clamped to): its tokens' weights
count in a row's sum all the same, although its values do not.

Beside what tests._tree.tree_bound counts, a weight is an f16 value times the
page's scale over the largest: half a step of the least is 2^-25, so a column is
off by up to 2^-25 n max |v code| max vs whatever its own sum is."""
import numpy as np
import pytest

import paged_kv_cache_274_gb300 as pkv
from workloads import normal_bf16_bits, random_case
from tests._gpu import DeviceCase, bf16_dev_to_f64, to_dev, to_dev_bf16
from tests._packed import PackedCase
from tests._tree import pack, random_parents, tree_attention, tree_bound, visible
from tests.test_gpu_packed import attend

pytestmark = pytest.mark.gpu

TINY = [2.0 ** -149, 2.0 ** -126, 2.0 ** -90, 2.0 ** -60]


def shrink(c, value, where):
    """v scales of some pages of every sequence: of every third, of the first twelve, or of all but one."""
    for b, n in enumerate(c.context_lens):
        pages = np.asarray(c.block_tables[b][:-(-int(n) // c.k_src.shape[3])])
        at = pages[1::3] if where == "third" else pages[:12] if where == "first" else np.delete(pages, len(pages) // 2)
        if c.kv_dtype == "fp8":
            c.v_scale[:, at] = value
        else:
            c.v_scale[:, at, :, 0] = value


def check(got, out, wabs, c, what):
    scale = np.max(c.v_scale if c.kv_dtype == "fp8" else c.v_scale[..., 0]).astype(np.float64)
    code = 448.0 if c.kv_dtype == "fp8" else 255.0
    bound = tree_bound(out, wabs) + 2.0 ** -25 * int(max(c.context_lens)) * code * scale
    assert np.isfinite(got).all(), f"{what}: {(~np.isfinite(got)).sum()} not finite"
    err = np.abs(got - out)
    assert (err <= bound).all(), f"{what}: worst {(err / bound).max():.2f} x the bound"


@pytest.mark.parametrize("dtype", ["fp8", "int8a"])
@pytest.mark.parametrize("seqs", [[(90, 1900), (250, 0), (1, 700)], [(20, 1200), (1, 3000)]])
@pytest.mark.parametrize("value", TINY)
@pytest.mark.parametrize("where", ["third", "first", "all but one"])
def test_packed_rows(dtype, seqs, value, where):
    pc = PackedCase(6900 + len(seqs), seqs, 16, 4, 128, 16, dtype, poison=False)
    shrink(pc.c, value, where)
    pc.dc.vs = to_dev(pc.c.v_scale)
    want = pc.reference()
    for share in (0, 24):
        got = bf16_dev_to_f64(attend(pc, opts=pkv.decode_opts(partition_blocks=share)))
        check(got, *want, pc.c, f"{dtype} {value} {where} share {share}")
    assert pkv.read_device_error() == 0


@pytest.mark.parametrize("dtype", ["fp8", "int8a"])
@pytest.mark.parametrize("T,math", [(4, pkv.MATH_MMA), (24, pkv.MATH_TC), (60, pkv.MATH_TC)])
@pytest.mark.parametrize("value", TINY)
def test_drafted_trees(dtype, T, math, value):
    c = random_case(6950 + T, 3, 16, 4, 128, 16, [900 + T, 300, 2000], kv_dtype=dtype)
    dc = DeviceCase(c)
    q = normal_bf16_bits(6951, (3, T, 16, 128))
    nodes = np.full(3, T, np.int32)
    see, _ = visible(random_parents(np.random.Generator(np.random.PCG64(6952)), 3, T), nodes)
    for where in ("third", "first"):
        shrink(c, value, where)
        dc.vs = to_dev(c.v_scale)
        want = tree_attention(q, dc.k_host, dc.v_host, c.block_tables, c.context_lens, see, nodes, c.scale, c.k_scale, c.v_scale)
        for share in (0, 24):
            out = pkv.paged_decode_tree(to_dev_bf16(q), dc.k, dc.v, dc.bt, dc.cl, to_dev(pack(see)), scale=c.scale, k_scale=dc.ks,
                                        v_scale=dc.vs, opts=pkv.decode_opts(partition_blocks=share, math=math))
            check(bf16_dev_to_f64(out), *want, c, f"{dtype} {T} {value} {where} share {share}")
    assert pkv.read_device_error() == 0
