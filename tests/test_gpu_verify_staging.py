"""The one-tile tcgen05 verify kernel's staged output: many short units, so
that a call is mostly output, over and over; every call the same bits, and
within the tolerance of the oracle."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_274_gb300 as pkv
from workloads import normal_bf16_bits, random_case
from tests._gpu import DeviceCase, assert_close, bf16_dev_to_f64, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,dtype,lens,ppu", [
    (32, "bf16", (32, 97), 0),      # full tiles, whole sequences: the bf16 output is staged
    (32, "bf16", (200, 400), 4),    # partitions of 64 tokens: fp32 partials are staged
    (8, "bf16", (16, 200), 0),      # 32 rows, rotated; some sequences in partitions
    (32, "fp8", (32, 97), 0),
    (32, "int8a", (32, 97), 4),
])
def test_repeated_calls_give_the_same_rows(T, dtype, lens, ppu):
    B, Hq, Hkv = 192, 32, 8
    rng = np.random.Generator(np.random.PCG64(8800 + T + ppu))
    c = random_case(8801 + T + ppu, B, Hq, Hkv, 128, 16, rng.integers(lens[0], lens[1], B).tolist(), kv_dtype=dtype)
    dc = DeviceCase(c)
    qbits = normal_bf16_bits(8802, (B, T, Hq, 128))
    q, opts = to_dev_bf16(qbits), pkv.decode_opts(partition_blocks=ppu, math=pkv.MATH_TC)
    plan = pkv.decode_plan(dc.k, B, Hq, c.MB, opts, T)
    assert plan["math"] == pkv.MATH_TC and plan["row_tiles"] == 1
    n = pkv.decode_workspace_bytes(dc.k, B, Hq, c.MB, opts, T)
    ws = torch.zeros(n, dtype=torch.uint8, device=q.device)
    outs = torch.empty((100,) + tuple(q.shape), dtype=torch.bfloat16, device=q.device)
    for out in outs:
        pkv.paged_decode_multi(q, dc.k, dc.v, dc.bt, dc.cl, [0], 0, c.scale, out=out, workspace=ws, k_scale=dc.ks, v_scale=dc.vs,
                               opts=opts)
    torch.cuda.synchronize()
    assert pkv.read_device_error() == 0
    want = oracle.paged_decode_multi(qbits, dc.k_host, dc.v_host, c.block_tables, c.context_lens, c.kv_group_ptr, 0, c.scale,
                                     k_scale=c.k_scale, v_scale=c.v_scale)
    assert_close(bf16_dev_to_f64(outs[0]), want, f"T={T} {dtype}")
    bits = outs.view(torch.int16)
    wrong = (bits != bits[:1]).flatten(1).any(1)
    where = [tuple(torch.nonzero(bits[i] != bits[0])[0].tolist()) for i in torch.nonzero(wrong).flatten().tolist()[:5]]
    assert not wrong.any(), f"{int(wrong.sum())} of 100 calls differ, first at {where}"
