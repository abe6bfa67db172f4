"""rope_append whose queries go between the rows of one projection: in place, and to
columns of their own behind q, k and v."""
import numpy as np
import pytest
import torch

import paged_kv_cache_274_gb300 as pkv
from tests._gpu import DEV, to_dev
from tests.test_gpu_rope_append import Case, _freq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 2, 45])
def test_columns_of_one_buffer(N):
    Hq, Hkv, D = 12, 4, 128
    c = Case(9800, N, Hq, Hkv, D, 16, fused=True)
    want, kc, vc = c.call(_freq(D), True).clone(), c.kc.clone(), c.vc.clone()
    rows = torch.full((N, 2 * Hq + 2 * Hkv, D), 5.0, dtype=torch.bfloat16, device=DEV)
    rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:Hq + 2 * Hkv] = c.q, c.k, c.v
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:Hq + 2 * Hkv]
    call = lambda out: pkv.rope_append(q, k, v, to_dev(c.pos), _freq(D), to_dev(c.slots), c.kc, c.vc, q_weight=c.qw, k_weight=c.kw, out=out)
    same = lambda x, y: torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))
    for out in (rows[:, Hq + 2 * Hkv:], q):  # behind them, then in place
        c.kc.zero_(), c.vc.zero_()
        call(out)
        at = to_dev(c.slots)
        b, o = at // 16, at % 16
        assert same(out, want) and same(c.kc[0, b, :, o], kc[0, b, :, o]) and same(c.vc[0, b, :, o], vc[0, b, :, o])
        assert same(k, c.k) and same(v, c.v)
    # over the keys: not even with the queries' own stride
    with pytest.raises(pkv.PkvError):
        pkv.rope_append(q, rows[:, 2:2 + Hkv], v, to_dev(c.pos), _freq(D), to_dev(c.slots), c.kc, c.vc, out=q)
    assert pkv.read_device_error() == 0
