"""rope_append where an angle is a great many turns: far positions and frequencies
far above a turn, against angles in exact arithmetic."""
import numpy as np
import pytest

import paged_kv_cache_274_gb300 as pkv
from tests._gpu import bf16_dev_to_f64
from tests._turns import cos_sin
from tests.test_gpu_rope_append import Case, _freq

pytestmark = pytest.mark.gpu

FAR = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 2 ** 29 - 7, 131071, 2 ** 31 - 1000, -123456789, 1]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("what", ["usual", "fast"])
def test_far_angles(what, interleaved):
    D, N = 128, len(FAR)
    c = Case(9700, N, 8, 2, D, 16)
    c.pos[0] = FAR
    f = _freq(D, 500000.0) if what == "usual" else np.concatenate([np.linspace(50.0, 40000.0, 32), -np.linspace(7.0, 9e6, 32)])
    got = bf16_dev_to_f64(c.call(f, False, interleaved=interleaved))
    x = bf16_dev_to_f64(c.q)
    co, si = (t[:, None] for t in cos_sin(np.repeat(c.pos[0][:, None].astype(np.int64), D // 2, 1), f))
    i = np.arange(D // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + D // 2)
    want, size = np.zeros_like(x), np.zeros_like(x)
    want[..., a], want[..., b] = x[..., a] * co - x[..., b] * si, x[..., b] * co + x[..., a] * si
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    # the angle to 2^-26 of half a turn, cos and sin and the sum by some four fp32 roundings, one to bf16
    bound = 2.0 ** -8 * np.abs(want) + (np.pi * 2.0 ** -26 + 6 * 2.0 ** -24) * size
    err = np.abs(got - want)
    assert (err <= bound).all(), f"{(err > bound).sum()} of {err.size}, worst {(err / bound).max():.1f} x the bound"
    assert pkv.read_device_error() == 0
