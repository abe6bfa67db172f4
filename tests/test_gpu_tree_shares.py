"""Drafted-tree attention on tcgen05 where shares begin or end beside inactive
sequences (no tokens, or no nodes), with a workspace full of NaNs: a partial
that no unit of the call wrote shows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_274_gb300 as pkv
from workloads import normal_bf16_bits, random_case
from tests._gpu import DEV, DeviceCase, bf16_dev_to_f64, to_dev, to_dev_bf16
from tests._tree import assert_tree_close, pack, random_parents, tree_attention, visible

pytestmark = pytest.mark.gpu


def _check(seed, dtype, D, T, Hq, Hkv, share_blocks, lens, nodes=None):
    lens = [int(n) for n in lens]
    nodes = np.minimum(np.array(lens), T).astype(np.int32) if nodes is None else np.array(nodes, np.int32)
    c = random_case(seed, len(lens), Hq, Hkv, D, 16, lens, kv_dtype=dtype)
    dc = DeviceCase(c)
    q = normal_bf16_bits(seed + 1, (c.B, T, Hq, D))
    see, _ = visible(random_parents(np.random.Generator(np.random.PCG64(seed + 2)), c.B, T), nodes)
    opts = pkv.decode_opts(partition_blocks=share_blocks, math=pkv.MATH_TC)
    n = pkv.decode_workspace_bytes(dc.k, c.B, Hq, c.MB, opts, T, tree=True)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    out = pkv.paged_decode_tree(to_dev_bf16(q), dc.k, dc.v, dc.bt, dc.cl, to_dev(pack(see)), to_dev(nodes), scale=c.scale,
                                workspace=ws, k_scale=dc.ks, v_scale=dc.vs, opts=opts)
    torch.cuda.synchronize()
    assert pkv.read_device_error() == 0
    ref = tree_attention(q, dc.k_host, dc.v_host, c.block_tables, c.context_lens, see, nodes, c.scale, c.k_scale, c.v_scale)
    assert_tree_close(bf16_dev_to_f64(out), *ref, f"{dtype} D={D} T={T} lens={lens} nodes={nodes.tolist()}")


# (lengths at which a boundary moves off the first sequence's last item and the
# third sequence is split right behind it, by what an item's start costs there)
@pytest.mark.parametrize("dtype,D,T,Hq,Hkv,share_blocks,lens", [
    ("bf16", 128, 24, 8, 2, 64, [267, 0, 661]), ("bf16", 128, 24, 8, 2, 64, [257, 0, 650]), ("bf16", 64, 24, 8, 2, 64, [267, 0, 661]),
    ("fp8", 128, 24, 8, 2, 128, [911, 0, 1543]), ("int8a", 128, 24, 8, 2, 128, [911, 0, 1548]),
    ("bf16", 128, 60, 4, 1, 64, [262, 0, 898]), ("fp8", 128, 60, 4, 1, 64, [261, 0, 905]), ("int8", 128, 60, 4, 1, 64, [258, 0, 913]),
    ("bf16", 64, 60, 4, 1, 64, [262, 0, 898])])
def test_inactive_sequence_between_others(dtype, D, T, Hq, Hkv, share_blocks, lens):
    _check(8900 + T + D, dtype, D, T, Hq, Hkv, share_blocks, lens)
    # no nodes instead of no tokens, and several inactive ones
    _check(8901 + T + D, dtype, D, T, Hq, Hkv, share_blocks, [lens[0], 40, lens[2]], [T, 0, T])
    _check(8902 + T + D, dtype, D, T, Hq, Hkv, share_blocks, [0, lens[0], 0, 17, 0, lens[2], 0], [0, T, T, 0, 0, T, 3])


def test_inactive_sequence_with_default_options():
    _check(8910, "bf16", 128, 24, 8, 8, 0, [30295, 0, 31051, 30690])


@pytest.mark.parametrize("dtype,D,T", [("bf16", 128, 24), ("bf16", 64, 24), ("bf16", 128, 60), ("fp8", 128, 24), ("int8a", 128, 40)])
def test_mixes_with_inactive_sequences(dtype, D, T):
    rng = np.random.Generator(np.random.PCG64(8920 + T + D))
    for i in range(6):
        lens = rng.integers(T, 2500, 9)
        lens[rng.random(9) < 0.35] = 0
        lens[rng.integers(0, 9)] = 3000
        nodes = np.where(lens > 0, rng.integers(0, T + 1, 9), 0) if i % 2 else None
        _check(8930 + i, dtype, D, T, 8, 2, int(rng.choice([0, 64, 128, 200])), lens, nodes)
