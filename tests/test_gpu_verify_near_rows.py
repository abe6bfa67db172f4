"""verify_tree where little or nothing is left of the target row behind a second
rejection, because it is next to a multiple of what is left of the draft row."""
import numpy as np
import pytest

import paged_kv_cache_274_gb300 as pkv
from tests.test_gpu_verify_tree import Case

pytestmark = pytest.mark.gpu


def one_node(seed, p, q, tokens, r, u):
    """B requests whose tree is the root and its children."""
    B, T, V = len(r), len(tokens) + 1, len(p)
    c = Case(seed, B, T, V)
    c.parents[:, 1:] = 0
    c.tokens[:, 1:] = tokens
    c.p[:], c.q[:] = np.asarray(p, np.float32), np.asarray(q, np.float32)
    c.r[:, 1:], c.u[:] = r, u
    return c


def test_a_weight_whose_high_part_is_negative():
    # 2^-29 of what is subtracted is left at token 0: the difference's rounded part
    # outweighs it, with the other sign
    f = float.fromhex
    p = [f("0x1.9947bap-2"), f("0x1.335aa4p-1"), f("0x1.729adap-17"), f("0x1.8e0304p-22")]
    q = [f("0x1.6cd71ap-3"), f("0x1.a4c8f4p-1"), f("0x1.3500cep-17"), f("0x1.fcfaf6p-22")]
    r = np.tile(np.float32([f("0x1.974db6p-1"), f("0x1.0bba5p-4"), f("0x1.0d2bb2p-1")]), (8, 1))
    c = one_node(8960, p, q, [1, 1, 2], r, np.linspace(0.02, 0.98, 8))
    _, _, nxt = c.check()
    assert (nxt == 0).all()


@pytest.mark.parametrize("V", [2, 900])
def test_a_repeated_token_leaves_nothing_of_a_multiple(V):
    # all of the draft row that is left is on one token, and all of the target row, too:
    # a second rejection of the first child's token takes all of it, by the definition
    # exactly, and the target's own row is drawn from
    B = 64
    rng = np.random.Generator(np.random.PCG64(8961))
    c = Case(8961, B, 4, V)
    c.parents[:, 1:] = 0
    a, b = rng.integers(0, V // 2, B), rng.integers(V // 2, V, B)
    c.tokens[:, 1:] = a[:, None]
    at = np.arange(B)
    c.p[:], c.q[:] = 0.0, 0.0
    c.p[at, 0, a] = rng.uniform(0.3, 0.9, B)
    c.p[at, 0, b] = np.float32(1) - c.p[at, 0, a]
    c.q[at, 0, a] = np.float32(1) - np.float32(rng.uniform(0.01, 0.5, B)) * c.p[at, 0, b]
    c.q[at, 0, b] = np.float32(1) - c.q[at, 0, a]
    c.r[:] = np.float32(0.9999)
    c.u[:] = rng.uniform(0.01, 0.25, B)
    # q(a) - p(a) >= p(b) / 2 >= 0.05, so r q(a) > p(a): rejected, and again with Q(a) = 0.  Then P(b) = Z and
    # Q(b) = Y, so P - (Z / Y) Q = 0: the target's row, p(a) >= 0.3 > u.  (In 64 bits (Z / Y) Y may miss Z.)
    _, count, nxt = [t.cpu().numpy() for t in c.call()]
    assert pkv.read_device_error() == 0
    assert (count == 1).all() and np.array_equal(nxt, a)
