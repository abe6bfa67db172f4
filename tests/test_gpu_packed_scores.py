"""Attention of packed rows whose scores rise, fall or jump along the sequence, so
that a row's running maximum moves in any of its steps, and one-byte caches whose
pages' scales lie far apart.

Queries are +-1, so that the products are exact in every type.  A score is a sum of
D of them in fp32: with each addition off by at most 2^-23 (rounded towards zero)
of sum |q k| scale < 16 x 12, 128 additions leave less than 2^-8 of a score, thus of
its weight, and as much of the sum of weights: 2^-7 of the weights together, beside
what tests._tree.tree_bound counts.

One-byte caches' weights are f16 values, w_j vs_j / max vs with w = 1 or more for a
row's largest: half a step of the least is 2^-25, so what a column is off by for its
weights below 2^-14 is up to 2^-25 sum |code_j| max vs <= 2^-25 n max |v code| max vs
whatever the column's own sum of weights is (a token with weight 1 and a value of 0
leaves 1e-11 there)."""
import numpy as np
import pytest

import paged_kv_cache_274_gb300 as pkv
from workloads import bf16_bits_from_f32, bf16_bits_to_f32
from tests._gpu import DeviceCase, bf16_dev_to_f64, to_dev
from tests._packed import PackedCase
from tests._tree import tree_bound
from tests.test_gpu_packed import attend

pytestmark = pytest.mark.gpu

RAMPS = {
    "rise": lambda n: np.linspace(0.25, 16, n),
    "fall": lambda n: np.linspace(16, 0.25, n),
    "jump": lambda n: np.where(np.arange(n) == n // 2, 16.0, 0.5),
    "saw": lambda n: 1.0 + 9.0 * (np.arange(n) % 11 == 10) + np.arange(n) % 7,
    "tiny": lambda n: np.where(np.arange(n) % 2 == 0, 1e-30, 1e-3),
}


def assert_scores_close(got, pc, out, wabs, what):
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err, bound = np.abs(got - out), tree_bound(out, wabs) + 2.0 ** -7 * wabs
    if pc.c.kv_dtype != "bf16":
        fp8 = pc.c.kv_dtype == "fp8"
        scale = np.max(pc.c.v_scale if fp8 else pc.c.v_scale[..., 0])
        code = 448.0 if fp8 else 255.0
        bound = bound + 2.0 ** -25 * int(max(pc.c.context_lens)) * code * scale
    assert (err <= bound).all(), f"{what}: worst {(err / bound).max():.2f} x the bound at {np.argwhere(err > bound)[:4].tolist()}"


@pytest.mark.parametrize("ramp", sorted(RAMPS))
@pytest.mark.parametrize("dtype,D,Hq,Hkv,seqs", [
    ("bf16", 128, 16, 4, [(90, 1900), (250, 0), (1, 700)]), ("bf16", 64, 16, 4, [(90, 1900), (250, 0), (1, 700)]),
    ("bf16", 128, 16, 4, [(20, 1200), (1, 3000)]), ("bf16", 64, 16, 4, [(20, 1200), (1, 3000)]),
    ("fp8", 128, 16, 4, [(90, 1900), (250, 0), (1, 700)]), ("fp8", 128, 16, 4, [(20, 1200), (1, 3000)]),
    ("int8a", 128, 16, 4, [(90, 1900), (250, 0), (1, 700)]), ("int8", 128, 16, 4, [(20, 1200), (1, 3000)])])
def test_scores_along_the_sequence(dtype, D, Hq, Hkv, seqs, ramp):
    pc = PackedCase(6800 + D, seqs, Hq, Hkv, D, 16, dtype, poison=False)
    c, rng = pc.c, np.random.Generator(np.random.PCG64(len(ramp) + D))
    pc.q = bf16_bits_from_f32(rng.choice(np.array([-1.0, 1.0], np.float32), pc.q.shape))
    for b, n in enumerate(c.context_lens):
        pages = np.asarray(c.block_tables[b][:-(-int(n) // 16)])
        f = RAMPS[ramp](len(pages)).astype(np.float32)
        if dtype == "bf16":
            c.k_src[:, pages] = bf16_bits_from_f32(bf16_bits_to_f32(c.k_src[:, pages]) * f[None, :, None, None, None])
        elif dtype == "fp8":
            c.k_scale[:, pages] *= f[None, :, None]
        else:
            c.k_scale[:, pages] *= np.stack([f, np.ones_like(f)], -1)[None, :, None]
    if dtype == "bf16":
        pc.dc = DeviceCase(c)
    else:  # (the codes stay those of the pages' own scales)
        pc.dc.ks = to_dev(c.k_scale)
    want = pc.reference()
    for share in (0, 24):
        got = bf16_dev_to_f64(attend(pc, opts=pkv.decode_opts(partition_blocks=share)))
        assert_scores_close(got, pc, *want, f"{dtype} {ramp} share {share}")
    assert pkv.read_device_error() == 0


@pytest.mark.parametrize("dtype", ["fp8", "int8a"])
@pytest.mark.parametrize("seqs", [[(90, 1900), (250, 0), (1, 700)], [(20, 1200), (1, 3000)]])
def test_page_scales_far_apart(dtype, seqs):
    # v scales over 2^12, k scales over 2^3 (sum |q k| scale < 4 x 12)
    pc = PackedCase(6850, seqs, 16, 4, 128, 16, dtype, poison=False)
    c, rng = pc.c, np.random.Generator(np.random.PCG64(6851))
    pc.q = bf16_bits_from_f32(rng.choice(np.array([-1.0, 1.0], np.float32), pc.q.shape))
    ks, vs = (c.k_scale, c.v_scale) if dtype == "fp8" else (c.k_scale[..., 0], c.v_scale[..., 0])
    ks *= np.exp2(rng.uniform(-1, 2, ks.shape)).astype(np.float32)
    vs *= np.exp2(rng.uniform(-6, 6, vs.shape)).astype(np.float32)
    pc.dc.ks, pc.dc.vs = to_dev(c.k_scale), to_dev(c.v_scale)
    assert_scores_close(bf16_dev_to_f64(attend(pc)), pc, *pc.reference(), dtype)
    assert pkv.read_device_error() == 0
