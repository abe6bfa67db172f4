"""verify_tree on the GPU against a float64 walk: vocabularies and row strides,
trees of one to 512 nodes, drafts with and without probabilities, rows that
leave nothing, values that are no probabilities, refused nodes, the
distribution of what comes out, other streams, CUDA graphs."""
import numpy as np
import pytest
import torch

import paged_kv_cache_274_gb300 as pkv
from tests._gpu import DEV, to_dev
from tests._verify import verify

pytestmark = pytest.mark.gpu


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Case:
    def __init__(self, seed, B, T, V, draft=True, reach=6, sharp=2.0, noise=0.7, nodes=None):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.B, self.T, self.V = B, T, V
        logits = rng.standard_normal((B, T, V)) * sharp
        self.p = _softmax(logits)
        dl = logits + noise * rng.standard_normal((B, T, V))
        self.q = _softmax(dl) if draft else None
        self.parents = np.full((B, T), -1, np.int32)
        for t in range(1, T):
            self.parents[:, t] = rng.integers(max(0, t - reach), t, size=B)
        # children of a node: a draw without replacement from its draft row (with draft), else the best
        order = np.argsort(-(dl - (np.log(rng.exponential(size=dl.shape)) if draft else 0)), -1, kind="stable") if V > 1 else np.zeros((B, T, 1), int)
        self.tokens = np.zeros((B, T), np.int32)
        for b in range(B):
            seen = np.zeros(T, int)
            for t in range(1, T):
                u = self.parents[b, t]
                self.tokens[b, t] = order[b, u, seen[u] % V]
                seen[u] += 1
        self.r, self.u = rng.random((B, T), np.float32), rng.random(B, np.float32)
        self.nodes = np.full(B, T, np.int32) if nodes is None else np.asarray(nodes, np.int32)

    def rows(self, x, pad):
        if x is None:
            return None
        wide = np.full((self.B, self.T, self.V + pad), np.nan, np.float32)
        wide[..., :self.V] = x
        return to_dev(wide)[..., :self.V]

    def call(self, pad=0, most=None, counts=True, **kw):
        return pkv.verify_tree(to_dev(self.tokens), to_dev(self.parents), self.rows(self.p, pad), to_dev(self.r), to_dev(self.u),
                               draft_probs=self.rows(self.q, pad), node_counts=to_dev(self.nodes) if counts else None, max_accept=most, **kw)

    def check(self, pad=0, most=None, error=0):
        got = [t.cpu().numpy() for t in self.call(pad, most)]
        assert pkv.read_device_error() == error
        want = verify(self.tokens, self.parents, self.nodes, self.p, self.q, self.r, self.u, most or self.T)
        for g, w, name in zip(got, want, ("nodes", "counts", "next")):
            assert np.array_equal(g, w), f"{name}: {np.argwhere(g != w)[:5].tolist()}, got {g[g != w][:5]}, want {w[g != w][:5]}"
        return want


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,T,V,pad", [
    (3, 1, 1, 0), (4, 5, 2, 0), (6, 8, 5, 3), (8, 16, 31, 0), (5, 32, 512, 0), (5, 20, 513, 0), (4, 33, 1000, 24), (3, 12, 4099, 0),
    (2, 9, 32000, 0), (2, 7, 32003, 1), (1, 6, 128256, 0), (1, 4, 300001, 0), (40, 12, 700, 0), (90, 6, 9000, 0), (400, 4, 600, 0)])
def test_sweep(B, T, V, pad, draft):
    Case(8000 + B + T + V, B, T, V, draft).check(pad)


@pytest.mark.parametrize("draft", [True, False])
def test_many_rounds_and_wide_trees(draft):
    # every node a child of the root: up to 30 rejections at one node; 512 nodes; short paths by max_accept
    Case(8100, 12, 31, 2000, draft, reach=40).check()
    c = Case(8101, 6, 40, 900, draft)
    c.parents[:, 1:] = 0
    c.check()
    Case(8102, 2, 512, 300, draft, reach=3).check()
    for most in (1, 2, 3):
        Case(8103, 10, 24, 400, draft, reach=2, noise=0.1).check(most=most)


def test_counts():
    c = Case(8200, 6, 10, 333, nodes=[10, 0, 1, 5, 9, 2])
    idx, count, nxt = c.check()
    assert count[1] == 0 and nxt[1] == -1 and count[2] == 1
    full = Case(8201, 5, 10, 333)
    a, b = full.call(counts=True), full.call(counts=False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_equal_rows_accept_everything():
    # draft and target alike: r q < p for every r < 1
    c = Case(8300, 8, 12, 250, noise=0.0)
    c.q = c.p.copy()
    c.parents[:, 1:] = np.arange(11)
    _, count, _ = c.check()
    assert (count == 12).all()


def test_nothing_left_after_a_rejection():
    # the draft has at least the target's weight everywhere: the target's own row is sampled
    c = Case(8310, 6, 3, 64)
    c.q = np.float32(2) * c.p
    c.parents[:, 1:] = 0
    c.r[:] = 0.99
    _, count, nxt = c.check()
    assert (count == 1).all() and (nxt >= 0).all()


def test_drafts_that_the_draft_row_denies_and_repeated_tokens():
    c = Case(8320, 10, 9, 50)
    c.parents[:, 1:] = 0
    c.tokens[:, 2] = c.tokens[:, 1]  # a sibling's token again
    c.q[np.arange(10), 0, c.tokens[:, 3]] = 0.0  # never proposed by that row
    c.check()
    c.q[:] = 0.0
    c.check()
    d = Case(8321, 10, 9, 50, draft=False)
    d.parents[:, 1:] = 0
    d.tokens[:, 2:5] = d.tokens[:, 1:2]
    d.check()


def test_all_weight_on_rejected_tokens():
    # one-hot target rows: the child is taken whatever r, or what is left is exactly the target's token
    c = Case(8330, 16, 4, 77, draft=False)
    hot = np.random.Generator(np.random.PCG64(1)).integers(0, 77, (16, 4))
    c.p = np.zeros_like(c.p)
    np.put_along_axis(c.p, hot[..., None], 1.0, -1)
    c.tokens[::2, 1] = hot[::2, 0]
    c.check()


def test_uniforms_at_their_ends():
    c = Case(8340, 6, 3, 1000)
    c.u[:] = [0.0, np.nextafter(np.float32(1), np.float32(0)), 0.0, 0.5, 1.0, 2.0]
    c.p[2, :, :10] = 0.0   # the first weight is not at the first index
    c.p[1, :, -7:] = 0.0
    c.p[4, :, -600:] = 0.0
    c.r[0], c.r[1] = 0.0, np.nextafter(np.float32(1), np.float32(0))
    c.check()


def test_tiny_weights_and_long_sums():
    # a likely token and 100,000 of 1e-9 each behind it: sums in 32 bits would lose them
    V = 100001
    c = Case(8350, 4, 2, V, draft=False)
    c.p[:] = 1e-9
    c.p[:, :, 0] = 1.0
    c.tokens[:, 1] = 0
    c.r[:] = 1.0  # never below p
    c.u[:] = [0.1, 0.25, 0.6, 0.999]
    c.check()
    d = Case(8351, 4, 1, V, draft=False)
    d.p[:] = 1e-9
    d.p[:, :, 0] = 1.0
    d.u[:] = [0.99999, 0.99995, 0.99991, 0.99994]
    d.check()


def test_values_that_are_no_probabilities():
    c = Case(8360, 6, 5, 600)
    c.p[0, 0, 3], c.p[1, 0, 4], c.p[2, 0, 5], c.p[3, 0, :] = -0.5, np.nan, np.inf, np.nan
    c.q[4, 0, 6], c.q[4, 0, 7] = 0.0, 0.0
    c.nodes[:] = 1  # (no comparison with what is no number: the sampled row alone)
    _, _, nxt = c.check(error=pkv.DEVERR_TREE)
    assert nxt[3] == -1
    c = Case(8361, 3, 5, 600, draft=False)
    c.p[0, 0] = 0.0
    c.nodes[:] = 1
    _, _, nxt = c.check(error=pkv.DEVERR_TREE)
    assert nxt[0] == -1


@pytest.mark.parametrize("what", ["count", "count below", "root", "later", "orphan", "token", "token below"])
def test_refused_nodes(what):
    c = Case(8400, 5, 8, 90)
    want = [t.cpu().numpy() for t in c.call()]
    if what == "count":
        c.nodes[2] = 9
    elif what == "count below":
        c.nodes[2] = -1
    elif what == "root":
        c.parents[2, 0] = 0
    elif what == "later":
        c.parents[2, 3] = 3
    elif what == "orphan":
        c.parents[2, 3] = -1
    else:
        c.tokens[2, 5] = 90 if what == "token" else -1
    got = [t.cpu().numpy() for t in c.call()]
    assert pkv.read_device_error() == pkv.DEVERR_TREE
    assert got[1][2] == 0 and got[2][2] == -1 and (got[0][2] == -1).all()
    keep = [0, 1, 3, 4]
    assert all(np.array_equal(g[keep], w[keep]) for g, w in zip(got, want))


@pytest.mark.parametrize("draft", [True, False])
def test_tokens_follow_the_target(draft):
    # 60,000 requests with the same rows of 6 tokens and three children of the root: the token that follows the
    # root (the first accepted child's, or the sampled one) has the target's distribution
    B, T, V = 60000, 4, 6
    rng = np.random.Generator(np.random.PCG64(8500))
    p, q = _softmax(rng.standard_normal((T, V))), _softmax(rng.standard_normal((T, V)))
    parents = np.zeros((B, T), np.int32)
    parents[:, 0] = -1
    keys = np.log(q[0].astype(np.float64)) - (np.log(rng.exponential(size=(B, V))) if draft else 0)
    tokens = np.zeros((B, T), np.int32)
    tokens[:, 1:] = np.argsort(-keys, -1)[..., :T - 1]
    rows = lambda x: to_dev(np.broadcast_to(x, (B, T, V)).astype(np.float32))
    idx, count, nxt = pkv.verify_tree(to_dev(tokens), to_dev(parents), rows(p), to_dev(rng.random((B, T), np.float32)),
                                      to_dev(rng.random(B, np.float32)), draft_probs=rows(q) if draft else None)
    idx, count, nxt = idx.cpu().numpy(), count.cpu().numpy(), nxt.cpu().numpy()
    after = np.where(count > 1, tokens[np.arange(B), idx[:, 1].clip(0)], nxt)
    share, want = np.bincount(after, minlength=V) / B, p[0].astype(np.float64)
    assert (np.abs(share - want) <= 5 * np.sqrt(want * (1 - want) / B)).all(), (share, want)


def test_row_offsets_past_32_bits():
    # target rows whose last lie past 2^32 elements
    B, T, V, stride = 3, 2, 1000, 1 << 30
    c = Case(8600, B, T, V, draft=False)
    big = torch.zeros((B * T - 1) * stride + V, dtype=torch.float32, device=DEV)
    rows = torch.as_strided(big, (B, T, V), (T * stride, stride, 1))
    rows.copy_(to_dev(c.p))
    got = pkv.verify_tree(to_dev(c.tokens), to_dev(c.parents), rows, to_dev(c.r), to_dev(c.u))
    want = verify(c.tokens, c.parents, c.nodes, c.p, None, c.r, c.u, T)
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want))


def test_stream_graph_and_prepared():
    c = Case(8700, 20, 12, 3000)
    want = c.call()
    p, q, u = c.rows(c.p, 0), c.rows(c.q, 0), to_dev(c.u)
    prep = pkv.PreparedCall(pkv.verify_tree, to_dev(c.tokens), to_dev(c.parents), p, to_dev(c.r), u, draft_probs=q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = prep(stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prep()
    u.copy_(torch.rand(20, generator=torch.Generator().manual_seed(3)).to(DEV))
    c.u = u.cpu().numpy()
    g.replay()
    torch.cuda.synchronize()
    want = verify(c.tokens, c.parents, c.nodes, c.p, c.q, c.r, c.u, c.T)
    assert all(np.array_equal(x.cpu().numpy(), w) for x, w in zip(got, want))


def test_binding_refuses():
    c = Case(8800, 4, 6, 40)
    t = lambda x: to_dev(x)
    good = (t(c.tokens), t(c.parents), t(c.p), t(c.r), t(c.u))
    for i, bad in ((0, t(c.tokens[:3])), (1, t(c.parents.astype(np.int64))), (2, t(c.p[:, :5])), (2, t(c.p).half()), (2, t(c.p).cpu()),
                   (2, t(c.p).transpose(1, 2).contiguous().transpose(1, 2)), (3, t(c.r[:, :5])), (4, t(c.u[:3]))):
        with pytest.raises(pkv.PkvError):
            pkv.verify_tree(*[bad if j == i else x for j, x in enumerate(good)])
    for kw in (dict(max_accept=0), dict(max_accept=513), dict(draft_probs=t(c.p[:, :, :39])), dict(node_counts=t(c.nodes[:3]))):
        with pytest.raises(pkv.PkvError):
            pkv.verify_tree(*good, **kw)


def test_draft_values_that_are_no_probabilities():
    # in rows that lose children: each counts as 0, at the children's own tokens too
    rng = np.random.Generator(np.random.PCG64(8370))
    c = Case(8370, 24, 7, 700, noise=2.0, reach=3)
    c.r[:] = np.float32(0.999)
    for value in (-0.25, -np.inf, np.inf, np.nan):
        for b in range(c.B):
            c.q[b, :, rng.choice(c.V, 20, replace=False)] = value
    at = c.tokens[:12, 1]
    c.q[np.arange(12), c.parents[:12, 1], at] = np.array([np.nan, np.inf, -np.inf, -1.0] * 3, np.float32)
    _, count, _ = c.check()
    assert (count == 1).any() and (count > 1).any()


@pytest.mark.parametrize("pad", [0, 1])
def test_draft_rows_of_nodes_without_children_are_not_read(pad):
    c = Case(8380, 20, 9, 1500, noise=0.3)
    for b in range(c.B):
        leaf = ~np.isin(np.arange(c.T), c.parents[b])
        c.q[b, leaf] = np.nan
    c.r[:10] = 0.0  # (the walk ends at a leaf)
    want, count, _ = c.check(pad)
    assert all(want[b, count[b] - 1] not in c.parents[b] for b in range(10))


@pytest.mark.parametrize("draft", [True, False])
def test_the_largest_vocabulary(draft):
    V = 1 << 20
    c = Case(8390, 6, 3, V, draft, sharp=0.3)
    c.tokens[3:, 1:] = V - 1  # (unlikely children: rejected)
    c.r[3:] = np.float32(0.999)
    c.u[:] = [0.0, 0.3, 0.9999, 0.01, 0.51, 0.99]
    c.check()
    c.check(pad=1)
