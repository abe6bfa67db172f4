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
