"""rope_append on the GPU against a float64 reference: norms, rotations of both
pairings over parts of the head and several position axes, far positions,
cache types, strided rows, padding, in place, cache offsets past 32 bits, other
streams, CUDA graphs."""
import numpy as np
import pytest
import torch

import paged_kv_cache_274_gb300 as pkv
from workloads import bf16_bits_to_f32, normal_bf16_bits
from tests._gpu import DEV, bf16_dev_to_f64, to_dev, to_dev_bf16
from tests._rope import fp32_error, rotate

pytestmark = pytest.mark.gpu


def _freq(R, base=10000.0):
    return base ** (-2.0 * np.arange(R // 2) / max(R, 1))


class Case:
    def __init__(self, seed, N, Hq, Hkv, D, bs, kind="bf16", axes=1, far=5000, S=1, fused=False, spare=5):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.N, self.Hq, self.Hkv, self.D, self.bs, self.kind = N, Hq, Hkv, D, bs, kind
        rows = to_dev_bf16(normal_bf16_bits(seed, (N, Hq + 2 * Hkv, D)))
        if fused:
            self.q, self.k, self.v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = (t.contiguous() for t in rows.split([Hq, Hkv, Hkv], 1))
        NB = -(-N // bs) + spare
        shape = (S, NB, Hkv, bs, D)
        self.slots = rng.permutation(NB * bs)[:N].astype(np.int64)
        self.pos = rng.integers(0, far, (axes, N)).astype(np.int32)
        self.ks = self.vs = None
        if kind == "bf16":
            self.kc, self.vc = (to_dev_bf16(normal_bf16_bits(seed + i, shape)) for i in (1, 2))
        else:
            codes = rng.integers(0, 120, (2,) + shape)
            t = np.uint8 if kind == "fp8" else np.int8
            self.kc, self.vc = to_dev(codes[0].astype(t)), to_dev(codes[1].astype(t))
            scale = (rng.uniform(0.5, 2.0, (2,) + shape[:3]) * (4 / (448 if kind == "fp8" else 127))).astype(np.float32)
            if kind != "fp8":
                zero = rng.integers(-20, 20, scale.shape) * rng.integers(0, 2, scale.shape)  # some symmetric pages
                scale = np.stack([scale, zero.astype(np.float32)], -1)
            self.ks, self.vs = to_dev(scale[0]), to_dev(scale[1])
        self.qw = (1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(seed))).bfloat16().to(DEV)
        self.kw = (1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(seed + 1))).bfloat16().to(DEV)

    def call(self, inv_freq, norm, eps=1e-6, freq_axes=None, interleaved=False, slots=None, slot=0, out=None, stream=None):
        return pkv.rope_append(self.q, self.k, self.v, to_dev(self.pos), inv_freq, to_dev(self.slots if slots is None else slots),
                               self.kc, self.vc, k_scale=self.ks, v_scale=self.vs, slot=slot, q_weight=self.qw if norm else None,
                               k_weight=self.kw if norm else None, eps=eps, freq_axes=freq_axes, interleaved=interleaved, out=out,
                               stream=stream)


def _close_bf16(got, want, err, what):
    # one rounding to bf16: half a step is 2^-9 of the power of two above the value, at most 2^-8 of the value
    bad = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + err + 1e-37
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bounds, first at {np.argwhere(bad)[:3].tolist()}"


def check(c, inv_freq, norm, eps=1e-6, freq_axes=None, interleaved=False, slots=None, slot=0):
    slots = c.slots if slots is None else slots
    axes = np.zeros(len(inv_freq), int) if freq_axes is None else np.asarray(freq_axes)
    k0, v0 = c.kc.clone(), c.vc.clone()
    args = (eps, c.pos, inv_freq, axes, interleaved)
    q, qs = rotate(bf16_dev_to_f64(c.q), bf16_dev_to_f64(c.qw) if norm else None, *args)
    k, ks = rotate(bf16_dev_to_f64(c.k), bf16_dev_to_f64(c.kw) if norm else None, *args)
    mark = torch.full((c.N, c.Hq, c.D), 77.0, dtype=torch.bfloat16, device=DEV)
    out = c.call(inv_freq, norm, eps, freq_axes, interleaved, slots, slot, out=mark)
    torch.cuda.synchronize()
    err = lambda s: fp32_error(s, c.pos, inv_freq)
    live = slots >= 0
    got = bf16_dev_to_f64(out)
    _close_bf16(got[live], q[live], err(qs)[live], "queries")
    assert (got[~live] == 77.0).all()
    # the values and every untouched place: as kv_append leaves them
    kv = (c.k.contiguous(), c.v.contiguous())
    pkv.kv_append(kv[0], kv[1], to_dev(slots), k0, v0, c.ks, c.vs, slot)
    assert torch.equal(c.vc.view(torch.uint8), v0.view(torch.uint8))
    blk, off = slots[live] // c.bs, slots[live] % c.bs
    rows = c.kc[slot].cpu()[blk, :, off]  # [n][Hkv][D]
    rest, rest0 = c.kc.clone(), k0
    b, o = torch.from_numpy(blk).to(DEV), torch.from_numpy(off).to(DEV)
    rest[slot, b, :, o] = 0
    rest0[slot, b, :, o] = 0
    assert torch.equal(rest.view(torch.uint8), rest0.view(torch.uint8))
    k, ek = k[live], err(ks)[live]
    if c.kind == "bf16":
        _close_bf16(rows.float().numpy().astype(np.float64), k, ek, "keys")
        return out
    par = c.ks.cpu().numpy().astype(np.float64)[slot][blk]
    if c.kind == "fp8":
        s = par[..., None]
        x, code = k / s, rows.view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
        # half a step: 2^-4 of the value, 2^-10 below the smallest normal; the division rounds once more
        bound = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) * (1 + 2.0 ** -20) + ek / s + 2.0 ** -23 * np.abs(x)
        assert (np.abs(code - np.clip(x, -448, 448)) <= bound).all()
    else:
        s, z = par[..., 0, None], par[..., 1, None]
        lo = np.where(z == 0, -127, -128)
        x = np.clip(k / s + z, lo, 127)
        assert (np.abs(rows.numpy().astype(np.float64) - x) <= 0.5 + ek / s + 2.0 ** -23 * np.abs(k / s)).all()
    return out


SWEEP = [  # (N, Hq, Hkv, D, bs, kind, R, axes, interleaved, norm, fused)
    (1, 32, 8, 128, 16, "bf16", 128, 1, False, True, False),
    (7, 32, 8, 128, 16, "bf16", 128, 1, False, False, True),
    (64, 8, 8, 64, 16, "bf16", 64, 1, False, True, True),
    (33, 6, 2, 64, 32, "bf16", 32, 1, True, True, False),
    (5, 3, 1, 128, 16, "bf16", 16, 2, False, True, True),      # one KV head: half a warp without a row
    (130, 16, 4, 128, 32, "bf16", 96, 3, False, False, False),  # a rotated part that is no power of two
    (19, 12, 3, 64, 16, "bf16", 16, 4, True, True, True),
    (50, 5, 5, 128, 16, "bf16", 0, 1, False, True, True),       # norms alone
    (900, 32, 8, 128, 16, "fp8", 128, 1, False, True, True),
    (77, 64, 8, 128, 32, "fp8", 64, 3, True, False, False),
    (41, 7, 1, 128, 16, "fp8", 128, 1, True, True, False),
    (61, 16, 8, 128, 16, "int8", 128, 1, False, True, True),
    (30, 9, 3, 128, 32, "int8", 32, 2, True, False, False),
    (4000, 4, 2, 128, 16, "bf16", 128, 1, False, True, True),
]


@pytest.mark.parametrize("N,Hq,Hkv,D,bs,kind,R,axes,interleaved,norm,fused", SWEEP)
def test_sweep(N, Hq, Hkv, D, bs, kind, R, axes, interleaved, norm, fused):
    c = Case(9000 + N + R, N, Hq, Hkv, D, bs, kind, axes, fused=fused, S=2)
    which = [i % axes for i in range(R // 2)] if axes > 1 else None
    check(c, _freq(R), norm, freq_axes=which, interleaved=interleaved, slot=1)
    assert pkv.read_device_error() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    c = Case(9100, 24, 4, 2, 128, 16)
    c.pos[0] = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 2 ** 30 + 7, 131071] * 3
    check(c, _freq(128, 500000.0), False, interleaved=interleaved)


def test_frequencies_of_any_size():
    # above a turn per position, negative, zero
    c = Case(9110, 40, 4, 2, 64, 16, far=3000)
    f = np.array([0.0, 7.5, -0.3, 1e-9] * 4)
    check(c, f, True)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int8"])
def test_padding_and_bad_slots(kind):
    c = Case(9200, 40, 8, 2, 128, 16, kind)
    slots = c.slots.copy()
    slots[[0, 7, 39]] = -1
    check(c, _freq(128), True, slots=slots)
    assert pkv.read_device_error() == 0
    k0, v0 = c.kc.clone(), c.vc.clone()
    bad = np.full_like(slots, -1)
    bad[3], bad[4] = c.kc.shape[1] * c.bs, -2
    mark = torch.full((40, 8, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    c.call(_freq(128), True, slots=bad, out=mark)
    assert pkv.read_device_error() == pkv.DEVERR_SLOT
    assert torch.equal(c.kc.view(torch.uint8), k0.view(torch.uint8)) and torch.equal(c.vc.view(torch.uint8), v0.view(torch.uint8))
    assert (mark == 5.0).all()


@pytest.mark.parametrize("fused", [False, True])
def test_in_place(fused):
    a, b = (Case(9300, 37, 12, 4, 128, 16, fused=fused) for _ in range(2))
    want = a.call(_freq(128), True)
    got = b.call(_freq(128), True, out=b.q)
    assert got.data_ptr() == b.q.data_ptr()
    assert torch.equal(got.contiguous().view(torch.int16), want.view(torch.int16))
    assert torch.equal(a.kc.view(torch.int16), b.kc.view(torch.int16)) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_queries_alone():
    # a layer that reads another layer's cache: no keys, with and without padding
    c = Case(9310, 21, 8, 2, 128, 16)
    want = c.call(_freq(128), True)
    k0 = c.kc.clone()
    one = pkv.rope_append(c.q, None, None, to_dev(c.pos[0]), _freq(128), None, c.kc, c.vc, q_weight=c.qw)
    assert torch.equal(one.view(torch.int16), want.view(torch.int16))
    slots = np.where(np.arange(21) % 3 == 0, -1, 0).astype(np.int64)
    mark = torch.full_like(want, 3.0)
    pkv.rope_append(c.q, None, None, to_dev(c.pos[0]), _freq(128), to_dev(slots), c.kc, c.vc, q_weight=c.qw, out=mark)
    assert (mark[::3] == 3.0).all() and torch.equal(mark[1::3].view(torch.int16), want[1::3].view(torch.int16))
    assert torch.equal(c.kc.view(torch.int16), k0.view(torch.int16)) and pkv.read_device_error() == 0


def test_non_finite_values_stay_in_their_row():
    c = Case(9320, 8, 4, 2, 128, 16)
    want = c.call(_freq(64), False).clone()
    c.q[2, 1, 100] = float("inf")  # past the rotated part
    c.q[3, 0, 5] = float("nan")
    c.q[4, 3, 7] = float("-inf")
    got = c.call(_freq(64), False)
    same = torch.ones_like(got, dtype=torch.bool)
    same[2, 1, 100] = False
    same[3, 0, [5, 37]] = False
    same[4, 3, [7, 39]] = False
    assert torch.equal(got[same], want[same])
    assert got[2, 1, 100] == float("inf") and not torch.isfinite(got[~same]).any()
    # with norms the row itself is lost, and only that row
    want = Case(9320, 8, 4, 2, 128, 16).call(_freq(64), True)
    got = c.call(_freq(64), True)
    rows = torch.ones((8, 4), dtype=torch.bool)
    rows[2, 1] = rows[3, 0] = rows[4, 3] = False
    assert torch.equal(got[rows], want[rows]) and torch.isnan(got[3, 0]).all()


def test_cache_offsets_past_32_bits():
    # 5 GiB a cache: the last blocks lie past 4 GiB, in elements past 2^31
    Hkv, bs, D = 8, 32, 128
    NB = (5 << 30) // (Hkv * bs * D * 2)
    c = Case(9400, 6, 8, Hkv, D, bs)
    c.kc, c.vc = (torch.zeros((1, NB, Hkv, bs, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c.slots = np.array([NB * bs - 1, NB * bs - 40, 3, (NB - 2) * bs, NB * bs // 2, 0], np.int64)
    c.call(_freq(128), True)
    k, _ = rotate(bf16_dev_to_f64(c.k), bf16_dev_to_f64(c.kw), 1e-6, c.pos, _freq(128), np.zeros(64, int), False)
    for i, s in enumerate(c.slots):
        got = bf16_dev_to_f64(c.kc[0, s // bs, :, s % bs])
        assert (np.abs(got - k[i]) <= 2.0 ** -8 * np.abs(k[i]) + 1e-5).all()
        assert torch.equal(c.vc[0, s // bs, :, s % bs], c.v[i])


def test_stream_graph_and_prepared():
    a, b = (Case(9500, 50, 16, 4, 128, 16, "fp8", fused=True) for _ in range(2))
    want = a.call(_freq(128), True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    prep = pkv.PreparedCall(pkv.rope_append, b.q, b.k, b.v, to_dev(b.pos), _freq(128), to_dev(b.slots), b.kc, b.vc, k_scale=b.ks,
                            v_scale=b.vs, q_weight=b.qw, k_weight=b.kw)
    torch.cuda.synchronize()
    out = prep(stream=side)
    side.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(a.kc, b.kc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prep()
    b.q.mul_(-1)
    b.kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)
    blk, off = torch.from_numpy(b.slots // 16).to(DEV), torch.from_numpy(b.slots % 16).to(DEV)
    assert torch.equal(b.kc[0, blk, :, off], a.kc[0, blk, :, off])


def test_values_keep_their_bits():
    c = Case(9610, 64, 4, 4, 128, 16)
    c.v.view(torch.int16).copy_(torch.arange(-32768, 32768, 2, device=DEV).to(torch.int16).view(64, 4, 128))  # NaNs with payloads
    c.call(_freq(128), True)
    blk, off = torch.from_numpy(c.slots // 16).to(DEV), torch.from_numpy(c.slots % 16).to(DEV)
    assert torch.equal(c.vc[0, blk, :, off].view(torch.int16), c.v.view(torch.int16))


def test_empty_and_zero_rows():
    c = Case(9600, 4, 4, 2, 64, 16)
    empty = pkv.rope_append(c.q[:0], c.k[:0], c.v[:0], to_dev(c.pos[0, :0]), _freq(64), to_dev(c.slots[:0]), c.kc, c.vc)
    assert empty.shape == (0, 4, 64)
    c.q.zero_()
    assert (c.call(_freq(64), True) == 0).all()  # eps keeps 0 / 0 away
    assert pkv.read_device_error() == 0
