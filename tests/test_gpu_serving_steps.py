"""Whole steps of a serving loop over the calls of the library: prompts in
chunks beside requests that decode, and a speculative step with drafted trees,
each against a float64 reference that keeps the requests' keys and values
without pages."""
import numpy as np
import pytest
import torch

import paged_kv_cache_274_gb300 as pkv
from workloads import normal_bf16_bits
from tests._gpu import DEV, bf16_dev_to_f64, to_dev, to_dev_bf16
from tests._rope import rotate
from tests._tree import assert_tree_close, random_parents, visible
from tests._verify import walk

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, R = 8, 2, 128, 16, 128
FREQ = 10000.0 ** (-2.0 * np.arange(R // 2) / R)


class Loop:
    """Requests over one pool of blocks, one layer."""

    def __init__(self, B, MB, NB, seed):
        self.B, self.MB, self.NB = B, MB, NB
        shape = (1, NB, HKV, BS, D)
        self.kc, self.vc = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.tables = torch.full((B, MB), -1, dtype=torch.int32, device=DEV)
        self.counts = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.ring, self.state = pkv.new_free_ring(np.random.Generator(np.random.PCG64(seed)).permutation(NB), NB)
        self.seq = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.kept = [[np.zeros((0, HKV, D)), np.zeros((0, HKV, D))] for _ in range(B)]  # keys, values of each request
        g = torch.Generator().manual_seed(seed)
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=g)).bfloat16().to(DEV) for _ in range(2))

    def tables_for(self, new, N):
        self.new = to_dev(np.asarray(new, np.int32))
        return pkv.extend_tables(self.seq, self.new, self.tables, self.counts, self.ring, self.state, BS, N)

    def project(self, seed, N, positions, slots):
        """The step's rows: queries as the attention takes them; keys and values into the cache."""
        rows = to_dev_bf16(normal_bf16_bits(seed, (N, HQ + 2 * HKV, D)))
        q, k, v = rows[:, :HQ], rows[:, HQ:HQ + HKV], rows[:, HQ + HKV:]
        k_ref, _ = rotate(bf16_dev_to_f64(k), bf16_dev_to_f64(self.kw), 1e-6, positions.cpu().numpy()[None], FREQ, np.zeros(R // 2, int), False)
        q_ref, _ = rotate(bf16_dev_to_f64(q), bf16_dev_to_f64(self.qw), 1e-6, positions.cpu().numpy()[None], FREQ, np.zeros(R // 2, int), False)
        out = pkv.rope_append(q, k, v, positions, FREQ, slots, self.kc, self.vc, q_weight=self.qw, k_weight=self.kw, out=q)
        got = bf16_dev_to_f64(out)
        live = slots.cpu().numpy() >= 0
        assert (np.abs(got - q_ref)[live] <= 2.0 ** -8 * np.abs(q_ref[live]) + 1e-4).all()
        return out.contiguous(), got, k_ref, bf16_dev_to_f64(v)


def attention(q, k, v, see):
    """q [m][HQ][D], k, v [n][HKV][D] float64, see [m][n]: (result, sum of weights x |v|)."""
    out, wabs = np.zeros_like(q), np.zeros_like(q)
    for h in range(HQ):
        s = np.where(see, (q[:, h] @ k[:, h // (HQ // HKV)].T) * D ** -0.5, -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[:, h], wabs[:, h] = p @ v[:, h // (HQ // HKV)], p @ np.abs(v[:, h // (HQ // HKV)])
    return out, wabs


def test_chunks_of_prompts_beside_requests_that_decode():
    # prompts of these lengths arrive at these steps, in chunks of at most 48 tokens, then decode; one ends, another takes its blocks
    B, N = 5, 160
    loop = Loop(B, 20, 60, 31)
    prompts, arrive = [130, 7, 49, 90, 33], [0, 0, 1, 2, 3]
    left = list(prompts)
    for step in range(8):
        new = []
        for b in range(B):
            if step < arrive[b]:
                new.append(0)
            elif b == 1 and step >= 5:
                new.append(-1 if step == 5 else 0)
            else:
                new.append(min(48, left[b]) if left[b] else 1)
        ctx, starts, slots, pos = loop.tables_for(new, N)
        assert pkv.read_device_error() == 0
        q, q64, k64, v64 = loop.project(900 + step, N, pos, slots)
        # the cache's own keys from here on: rounding is rope_append's test's
        mark = torch.full((N, HQ, D), 9.0, dtype=torch.bfloat16, device=DEV)
        out = pkv.paged_decode_packed(q, loop.kc, loop.vc, loop.tables, ctx, starts, 48, out=mark)
        assert pkv.read_device_error() == 0
        got, rows = bf16_dev_to_f64(out), starts.cpu().numpy()
        assert (got[rows[-1]:] == 9.0).all()
        table, slot = loop.tables.cpu().numpy(), slots.cpu().numpy()
        kc, vc = bf16_dev_to_f64(loop.kc[0]), bf16_dev_to_f64(loop.vc[0])
        for b in range(B):
            lo, m = rows[b], max(new[b], 0)
            if new[b] == -1:
                loop.kept[b] = [np.zeros((0, HKV, D)), np.zeros((0, HKV, D))]
                continue
            if m == 0:
                continue
            ks = kc[slot[lo:lo + m] // BS, :, slot[lo:lo + m] % BS]
            assert (np.abs(ks - k64[lo:lo + m]) <= 2.0 ** -8 * np.abs(k64[lo:lo + m]) + 1e-4).all()
            loop.kept[b] = [np.concatenate([loop.kept[b][0], ks]), np.concatenate([loop.kept[b][1], v64[lo:lo + m]])]
            n = len(loop.kept[b][0])
            assert n == ctx[b].item()
            see = np.arange(n)[None] <= (n - m + np.arange(m))[:, None]
            assert_tree_close(got[lo:lo + m], *attention(q64[lo:lo + m], *loop.kept[b], see), f"step {step} request {b}")
            left[b] = max(0, left[b] - m)
        loop.seq = torch.where(loop.new == -1, 0, torch.where(ctx > 0, ctx, loop.seq)).to(torch.int32)


@pytest.mark.parametrize("draft", [True, False])
def test_speculative_steps(draft):
    # prompt by the packed call, then steps of: tables, rows into the cache, masks, attention of the nodes, verification,
    # compaction; the walk and the lengths against the reference, the attention of the step after against what was kept
    B, T, V = 4, 9, 64
    rng = np.random.Generator(np.random.PCG64(77))
    loop = Loop(B, 16, 64, 41)
    prompt = [37, 5, 16, 61]
    ctx, starts, slots, pos = loop.tables_for(prompt, sum(prompt))
    q, q64, k64, v64 = loop.project(1900, sum(prompt), pos, slots)
    pkv.paged_decode_packed(q, loop.kc, loop.vc, loop.tables, ctx, starts, max(prompt))
    loop.seq = ctx.clone()
    kc, slot = bf16_dev_to_f64(loop.kc[0]), slots.cpu().numpy()
    for b, lo in enumerate(starts.cpu().numpy()[:-1]):
        at = slot[lo:lo + prompt[b]]
        loop.kept[b] = [kc[at // BS, :, at % BS], v64[lo:lo + prompt[b]]]
    for step in range(4):
        parents = random_parents(rng, B, T, reach=4)
        parents[:, 1:] = np.maximum(parents[:, 1:], 0)  # one root
        nodes = rng.integers(3, T + 1, B).astype(np.int32)
        before = loop.seq.clone()
        ctx, starts, slots, _ = loop.tables_for(nodes, int(nodes.sum()))
        mask, place = pkv.tree_masks(to_dev(parents), ctx, to_dev(nodes))
        # the packed rows of the step: the nodes of each request, at their depth's position
        packed = torch.cat([place[b, :nodes[b]] for b in range(B)])
        q, q64, _, v64 = loop.project(2000 + step, int(nodes.sum()), packed, slots)
        wide = torch.zeros((B, T, HQ, D), dtype=torch.bfloat16, device=DEV)
        row = np.concatenate([[0], np.cumsum(nodes)])
        for b in range(B):
            wide[b, :nodes[b]] = q[row[b]:row[b + 1]]
        out = bf16_dev_to_f64(pkv.paged_decode_tree(wide, loop.kc, loop.vc, loop.tables, ctx, mask, to_dev(nodes)))
        assert pkv.read_device_error() == 0
        kc, slot = bf16_dev_to_f64(loop.kc[0]), slots.cpu().numpy()
        see, _ = visible(parents, nodes)
        fresh = []
        for b in range(B):
            at = slot[row[b]:row[b + 1]]
            fresh.append((kc[at // BS, :, at % BS], v64[row[b]:row[b + 1]]))
            k, v = (np.concatenate([old, new]) for old, new in zip(loop.kept[b], fresh[b]))
            m = nodes[b]
            vis = np.concatenate([np.ones((m, len(k) - m), bool), see[b, :m, :m]], 1)
            assert_tree_close(out[b, :m], *attention(q64[row[b]:row[b + 1]], k, v, vis), f"step {step} request {b}")
        # logits of the nodes from their attention's first column, for the sake of a target distribution
        z = rng.standard_normal((B, T, V)) + out[:, :, 0, :1]
        p = (np.exp(z) / np.exp(z).sum(-1, keepdims=True)).astype(np.float32)
        dq = np.full((B, T, V), 1.0 / V, np.float32)
        tokens = np.argsort(rng.random((B, V)), 1)[:, :T].astype(np.int32) if draft else np.argsort(-p[:, 0], 1)[:, :T].astype(np.int32)
        r, u = rng.random((B, T), np.float32), rng.random(B, np.float32)
        idx, count, nxt = pkv.verify_tree(to_dev(tokens), to_dev(parents), to_dev(p), to_dev(r), to_dev(u),
                                          draft_probs=to_dev(dq) if draft else None, node_counts=to_dev(nodes))
        lens = pkv.compact_tokens(idx, count, ctx, loop.tables, loop.kc, loop.vc, T, to_dev(nodes), new_lens=loop.new, prev_seq_lens=before)
        assert pkv.read_device_error() == 0
        for b in range(B):
            path, token = walk(tokens[b], parents[b], int(nodes[b]), p[b], dq[b] if draft else None, r[b], u[b], T)
            assert idx[b, :count[b]].tolist() == path and nxt[b].item() == token
            loop.kept[b] = [np.concatenate([old, new[path]]) for old, new in zip(loop.kept[b], fresh[b])]
            assert lens[b].item() == len(loop.kept[b][0])
        loop.seq = lens
