"""verify_tree with draft rows whose weight is almost all on one token: once that
token is rejected, what is left of the row is far below fp32's normal range (a
softmax of logits 90 apart), and the ratio of the target's rest to it above its
largest number."""
import numpy as np
import pytest

import paged_kv_cache_274_gb300 as pkv
from tests._verify import clean
from tests.test_gpu_verify_tree import Case

pytestmark = pytest.mark.gpu


def peaked(seed, B, T, V, rest):
    """Draft rows with 1 on the first child's token and `rest` x [0.2, 1) on one token in four."""
    c = Case(seed, B, T, V)
    rng = np.random.Generator(np.random.PCG64(seed + 1))
    c.parents[:, 1:] = 0
    c.tokens[:, 1:] = np.argsort(rng.random((B, V)), 1)[:, :T - 1]
    q = np.where(rng.random((B, T, V)) < 0.25, rng.uniform(0.2, 1.0, (B, T, V)) * rest, 0.0)
    np.put_along_axis(q[:, 0], c.tokens[:, 2:], rng.uniform(0.2, 1.0, (B, T - 2)) * rest, -1)
    q[np.arange(B), 0, c.tokens[:, 1]] = 1.0
    c.q = q.astype(np.float32)
    c.r[:] = rng.uniform(0.9, 1.0, c.r.shape)
    return c


@pytest.mark.parametrize("rest", [1e-43, 1e-41, 1e-39, 1e-37, 1e-30, 1e-20])
@pytest.mark.parametrize("V", [70, 3001])
def test_what_is_left_of_a_peaked_draft(rest, V):
    c = peaked(8900, 40, 5, V, rest)
    _, count, _ = c.check()
    assert (count == 1).any()


@pytest.mark.parametrize("rest", [1e-42, 1e-39])
def test_children_that_the_rest_accepts(rest):
    # the second child has most of the target: accepted against the rest's own share
    c = peaked(8910, 60, 4, 50, rest)
    for b in range(30):
        c.p[b, 0, c.tokens[b, 2]] = np.float32(0.9)
    _, count, _ = c.check()
    assert (count[:30] > 1).any() and (count[30:] == 1).any()


def test_probabilities_below_the_normal_range_are_compared_as_they_are():
    # r Q(x) against P(x), both some 1e-41: the products are not rounded to fp32's steps there
    B = 200
    c = Case(8920, B, 2, 40)
    rng = np.random.Generator(np.random.PCG64(8921))
    x, at = c.tokens[:, 1], np.arange(B)
    q = (rng.integers(20, 3000, B) * 2.0 ** -149).astype(np.float32)
    c.r[:, 1] = rng.random(B, np.float32)
    half = np.float32(0.5)
    exact = clean(q) * c.r[:, 1].astype(np.float64)  # r q in 64 bits
    c.r[0, 1] = half
    p = (np.ceil(exact / 2.0 ** -149) * 2.0 ** -149).astype(np.float32)  # the next fp32 above: accepted by less than a step
    c.p[at, 0, x], c.q[at, 0, x] = p, q
    _, count, _ = c.check()
    assert (count == 2).sum() > B // 2


def test_values_above_one_stay_finite():
    # a row that is no distribution: its removed token holds 1e30
    c = peaked(8930, 20, 4, 300, 1e-41)
    c.q[np.arange(20), 0, c.tokens[:, 1]] = np.float32(1e30)
    c.check()
    assert pkv.read_device_error() == 0


def test_large_target_rows_without_draft_rows():
    # rows that are no distributions: what is left after a rejection is their own
    c = Case(8940, 20, 6, 300, draft=False)
    c.parents[:, 1:] = 0
    c.p = (c.p * np.float32(1e33)).astype(np.float32)
    c.p[np.arange(20)[:, None], 0, c.tokens[:, 1:]] *= np.float32(1e-34)
    c.r[:] = np.float32(0.999)
    _, count, _ = c.check()
    assert (count == 1).any()
    assert pkv.read_device_error() == 0


def test_children_that_the_draft_row_denies():
    # Q(x) = 0: accepted against anything that is left of P(x), however small its product with Y
    B = 40
    c = peaked(8950, B, 4, 60, 1e-40)
    at, x = np.arange(B), c.tokens[:, 2]
    c.q[at, 0, x] = 0.0
    c.p[at, 0, x] = 10.0 ** -np.linspace(5, 37, B)
    _, count, _ = c.check()
    assert (count == 2).sum() > B // 2
