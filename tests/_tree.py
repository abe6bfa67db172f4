"""Plain float64 / Python references of the drafted-tree operators."""
import numpy as np

import oracle
from workloads import bf16_bits_to_f32


def pack(see):
    """Boolean [B][T][T] (row t sees node u) -> mask words int32 [B][T][ceil(T/32)]."""
    B, T, _ = see.shape
    W = -(-T // 32)
    bits = np.zeros((B, T, W * 32), np.uint64)
    bits[:, :, :T] = see
    words = (bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)


def visible(parents, nodes):
    """Ancestors of every node by walking: boolean [B][T][T], depths [B][T] (-1 past the count)."""
    B, T = parents.shape
    see = np.zeros((B, T, T), bool)
    depth = np.full((B, T), -1, np.int64)
    for b in range(B):
        for t in range(nodes[b]):
            u = t
            while u >= 0:
                see[b, t, u] = True
                depth[b, t] += 1
                u = parents[b, u]
    return see, depth


def random_parents(rng, B, T, reach=6):
    p = np.full((B, T), -1, np.int32)
    for t in range(1, T):
        p[:, t] = rng.integers(max(-1, t - reach), t, size=B)
    return p


def tree_attention(q_bits, k_cache, v_cache, block_tables, context_lens, see, nodes, scale, k_scale=None, v_scale=None,
                   slot=0):
    """float64 attention of tree nodes.  Returns (out, wabs) [B][T][Hq][D]:
    the result and sum_j p_j |v_j|, the scale of what rounding P costs."""
    q = bf16_bits_to_f32(q_bits).astype(np.float64)
    B, T, Hq, D = q.shape
    Hkv, bs = k_cache.shape[2], k_cache.shape[3]
    G = Hq // Hkv
    out, wabs = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq, D))
    for b in range(B):
        n, m = int(context_lens[b]), int(nodes[b])
        if n == 0 or m == 0:
            continue
        ids = np.asarray(block_tables[b][:-(-n // bs)])
        k = oracle._cache_values(k_cache, k_scale, slot, ids).astype(np.float64)  # [blocks][Hkv][bs][D]
        v = oracle._cache_values(v_cache, v_scale, slot, ids).astype(np.float64)
        k = np.moveaxis(k, 1, 0).reshape(Hkv, -1, D)[:, :n]
        v = np.moveaxis(v, 1, 0).reshape(Hkv, -1, D)[:, :n]
        base = n - m
        rows = np.zeros((T, n), bool)
        if base > 0:
            rows[:m, :base] = True
        lo = max(0, -base)  # nodes before position 0 do not exist
        rows[:m, base + lo:] = see[b, :m, lo:m]
        for h in range(Hq):
            s = (q[b, :, h] @ k[h // G].T) * scale
            s = np.where(rows, s, -np.inf)
            top = s.max(1, keepdims=True)
            p = np.where(rows, np.exp(s - np.where(np.isfinite(top), top, 0)), 0.0)
            l = p.sum(1, keepdims=True)
            p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
            vv = np.where(rows.any(0)[:, None], v[h // G], 0.0)
            out[b, :, h] = p @ vv
            wabs[b, :, h] = p @ np.abs(vv)
    return out, wabs


def tree_bound(out, wabs):
    """Largest error of the kernels' output.  P is rounded to bf16 at worst
    (half a step: 2^-8 of each weight), the output once to bf16 (2^-8 of it);
    scores, sums and exponentials in fp32 (an N(0, 1) score of up to 256
    products of sum |q k| scale < 16 is off by less than 2^-12, its weight and
    the sum of weights by 2^-12 each; sums of up to 4096 fp32 terms by 2^-12;
    E4M3: the query's two parts leave 2^-17 of its largest element, 2^-12 of
    a score) take less than 2^-10 of the weights together."""
    return (2.0 ** -8 + 2.0 ** -10) * wabs + 2.0 ** -8 * np.abs(out) + 1e-30


def assert_tree_close(got, out, wabs, what=""):
    assert got.shape == out.shape
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err, bound = np.abs(got - out), tree_bound(out, wabs)
    bad = err > bound
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} elements out of bounds, worst "
                           f"{(err / bound).max():.2f} x the bound, first at {np.argwhere(bad)[:4].tolist()}")


class Pool:
    """The block pool as extend_tables defines it, request by request."""

    def __init__(self, NB, bs, MB, free_ids, head=0):
        self.NB, self.bs, self.MB = NB, bs, MB
        self.ring = np.full(NB, -1, np.int32)
        for k, i in enumerate(free_ids):
            self.ring[(head + k) % NB] = i
        self.head, self.free = head, len(free_ids)

    def extend(self, seq, new, tables, counts, N, borrowed=None):
        """Returns (context_lens, query_starts, slots, positions, error bits); tables, counts and the pool change."""
        B = len(seq)
        ctx = np.zeros(B, np.int32)
        starts = np.zeros(B + 1, np.int32)
        slots, pos = np.full(N, -1, np.int64), np.zeros(N, np.int32)
        err, at, short = 0, 0, False
        given_back, old_free = [], self.free
        for b in range(B):
            starts[b] = min(at, N)
            s, a, held = int(seq[b]), int(new[b]), int(counts[b])
            first = at
            at += max(a, 0)
            if not 0 <= held <= self.MB or a < -1 or (a >= 0 and (s < 0 or s + a > self.MB * self.bs or s > held * self.bs)):
                err |= 4
                continue
            if a == -1:
                keep = 0 if borrowed is None else min(max(int(borrowed[b]), 0), held)
                given_back += [int(i) for i in tables[b, keep:held]]
                counts[b] = 0
                continue
            need = max(0, -(-(s + a) // self.bs) - held)
            # the blocks needed so far, served or not, come off the same list
            if min(at, N) - min(first, N) != a:
                err |= 2
                short = short or need > 0
                continue
            if need > 0 and (short or need > self.free):
                err |= 16
                short = True
                continue
            for j in range(need):
                tables[b, held + j] = self.ring[(self.head + j) % self.NB]
            self.head, self.free = (self.head + need) % self.NB, self.free - need
            counts[b] = held + need
            ctx[b] = s + a
            for i in range(a):
                p = s + i
                slots[first + i] = int(tables[b, p // self.bs]) * self.bs + p % self.bs
                pos[first + i] = p
        starts[B] = min(at, N)
        for i in given_back:
            self.ring[(self.head + self.free) % self.NB] = i
            self.free += 1
        return ctx, starts, slots, pos, err


def compact(k_cache, accept, counts, ctx, nodes, tables, params=None, kind="bf16"):
    """Move accepted rows in a host cache array [S][NB][Hkv][bs][D], in order; returns the new array."""
    out = k_cache.copy()
    bs = k_cache.shape[3]
    for b in range(len(counts)):
        base = int(ctx[b]) - int(nodes[b])
        for i in range(int(counts[b])):
            u = int(accept[b][i])
            if u == i:
                continue
            ps, pd = base + u, base + i
            sb, db = int(tables[b][ps // bs]), int(tables[b][pd // bs])
            row = out[:, sb, :, ps % bs].copy()  # [S][Hkv][D]
            if params is not None:
                row = requantise(row, params[:, sb], params[:, db], kind)
            out[:, db, :, pd % bs] = row
    return out


def requantise(codes, src, dst, kind):
    """Codes [S][Hkv][D] of one page's parameters in another's, in IEEE binary32."""
    import torch
    if kind == "fp8":
        x = torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).float().numpy()
        y = (x * src[..., None]).astype(np.float32) / dst[..., None]
        y = torch.from_numpy(np.clip(y.astype(np.float32), -448, 448))
        new = y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        return np.where((src == dst)[..., None], codes, new)
    s, z = src[..., 0, None], src[..., 1, None]
    d, w = dst[..., 0, None], dst[..., 1, None]
    x = ((codes.astype(np.float32) - z) * s).astype(np.float32)
    y = np.rint((x / d).astype(np.float32)) + w
    y = np.clip(y, np.where(w == 0, -127, -128), 127).astype(np.int8)
    return np.where((s == d) & (z == w), codes, y)
