"""Plain float64 reference of paged_decode_packed."""
import numpy as np

import oracle
from workloads import bf16_bits_to_f32, normal_bf16_bits, random_case
from tests._gpu import DeviceCase


def packed_attention(q_bits, c, starts, k_host, v_host, slot=0, what=None):
    """Returns (out, wabs) [N][Hq][D] as tests._tree.tree_attention does."""
    q = bf16_bits_to_f32(q_bits).astype(np.float64)
    N, Hq, D = q.shape
    Hkv, bs = k_host.shape[2], k_host.shape[3]
    G = Hq // Hkv
    out, wabs = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    for b in range(len(starts) - 1):
        lo, m, n = int(starts[b]), int(starts[b + 1] - starts[b]), int(c.context_lens[b])
        if m == 0 or n == 0:
            continue
        ids = np.asarray(c.block_tables[b][:-(-n // bs)])
        k = np.moveaxis(oracle._cache_values(k_host, c.k_scale, slot, ids).astype(np.float64), 1, 0).reshape(Hkv, -1, D)[:, :n]
        v = np.moveaxis(oracle._cache_values(v_host, c.v_scale, slot, ids).astype(np.float64), 1, 0).reshape(Hkv, -1, D)[:, :n]
        see = np.arange(n)[None] <= (n - m + np.arange(m))[:, None]
        for h in range(Hq):
            s = np.where(see, (q[lo:lo + m, h] @ k[h // G].T) * c.scale, -np.inf)
            top = s.max(1, keepdims=True)
            p = np.where(see, np.exp(s - np.where(np.isfinite(top), top, 0)), 0.0)
            l = p.sum(1, keepdims=True)
            p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
            out[lo:lo + m, h], wabs[lo:lo + m, h] = p @ v[h // G], p @ np.abs(v[h // G])
    return out, wabs


class PackedCase:
    """Sequences of these (new tokens, cached tokens before them)."""

    def __init__(self, seed, seqs, Hq, Hkv, D, bs, dtype="bf16", lens=None, poison=None):
        self.new = np.array([m for m, _ in seqs], np.int32)
        lens = [m + n for m, n in seqs] if lens is None else lens
        c = random_case(seed, len(lens), Hq, Hkv, D, bs, lens, kv_dtype=dtype, poison=dtype == "bf16" if poison is None else poison)
        self.c, self.dc = c, DeviceCase(c)
        self.starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.N = int(self.starts[-1])
        self.q = normal_bf16_bits(seed + 1, (max(self.N, 1), Hq, D))[:self.N]

    def reference(self):
        return packed_attention(self.q, self.c, self.starts, self.dc.k_host, self.dc.v_host)
