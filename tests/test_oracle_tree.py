"""Pins of the tree operators' oracle: chains, closed forms, brute force, and the distribution that is kept."""

import random
from fractions import Fraction

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import e4m3 as oe4m3
from oracle import tree as otree
from oracle import verify as over
from paged_mla_decode_gb300 import workloads as wl

from .tree_util import chain, random_tree


def test_a_chain_attends_as_causal_drafts():
    rng = np.random.default_rng(1)
    L, N, H = 70, 4, 3
    bits = wl.f32_to_bf16_bits(rng.standard_normal((128, 576), dtype=np.float32))
    q_bits = wl.f32_to_bf16_bits(rng.standard_normal((1, N, H, 576), dtype=np.float32))
    want = oatt.decode(q_bits, bits.reshape(2, 64, 576), np.array([[0, 1]]), [L], 0.05, 1.0, oatt.KV_BF16)
    got = otree.decode(oe4m3.bf16_bits_to_f64(q_bits), [oe4m3.bf16_bits_to_f64(bits)[:L]], [chain(N)], [N], 0.05)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_masked_rows_by_brute_force():
    rng = np.random.default_rng(2)
    k, q = rng.standard_normal((6, 576)), rng.standard_normal((1, 3, 2, 576))
    out, lse = otree.decode(q, [k], [[0b001, 0b101, 0b010]], [3], 0.1)
    for j, seen in enumerate(([0, 1, 2, 3], [0, 1, 2, 3, 5], [0, 1, 2, 4])):
        for h in range(2):
            o, l = oatt.dense_bruteforce(q[0, j, h], k[seen], 0.1)
            assert np.allclose(out[0, j, h], o, rtol=0, atol=1e-12) and abs(lse[0, j, h] - l) < 1e-12
    out, lse = otree.decode(q, [k[:3]], [[0, 1, 2]], [3], 0.1)  # no context
    assert not out[0, 0].any() and np.isneginf(lse[0, 0]).all() and np.array_equal(out[0, 2, 0], k[1, :512])


def test_a_chain_is_verified_as_drafts():
    r = random.Random(3)
    for trial in range(300):
        V, N = r.randint(1, 6), r.randint(1, 5)
        row = lambda: [r.choice([0, 0, 1, 2, 3]) / 8 for _ in range(V)]  # noqa: E731
        p, q = [row() for _ in range(N)], [row() for _ in range(N)]
        x, u = [r.randint(-1, V) for _ in range(N)], [r.random() for _ in range(N)]
        n = r.randint(1, N)
        for draft in (None, q):
            got = otree.verify(p, draft, x, chain(N), u, n)
            want = over.verify(p, None if draft is None else q[:N - 1], x[1:], u[1:] + u[:1], n - 1)
            assert got[0] == want[0] and got[2] == want[1], (trial, draft)
            assert got[1] == list(range(got[2] + 1)) + [-1] * (N - got[2] - 1)


@pytest.mark.parametrize("certain", [False, True])
def test_the_first_token_has_the_targets_distribution(certain):
    """Three children of node 0, drawn independently from q (or fixed, two of them equal): the token that
    is emitted first is p's, up to the spread of the draws (five standard deviations)."""
    r = random.Random(4)
    p, q = [0.125, 0.5, 0.25, 0.125], [0.5, 0.125, 0.0, 0.375]
    masks, count, draws = [1, 3, 5, 9], np.zeros(4), 20000
    rows = [p, q, q, p]  # the children's own rows do not matter for the first token
    for _ in range(draws):
        x = [0, 1, 3, 1] if certain else [0] + r.choices(range(4), q, k=3)
        out, path, a = otree.verify(rows, None if certain else [q] * 4, x, masks, [r.random() for _ in range(4)], 4)
        count[out[0]] += 1
        assert out[0] == (x[path[1]] if a else out[0])
    for v in range(4):
        assert abs(count[v] - draws * p[v]) <= 5 * (draws * p[v] * (1 - p[v])) ** 0.5, (v, count / draws)


def test_what_rejections_leave_folds_into_one_number():
    """max(max(p - a q, 0) - b q, 0) = max(p - (a + b) q, 0), the kernel's form of a node's later rejections."""
    r = random.Random(5)
    for _ in range(50):
        V = r.randint(1, 6)
        p, q = ([Fraction(r.randint(0, 8), 16) for _ in range(V)] for _ in range(2))
        left, weight, c = p, Fraction(1), Fraction(0)
        for _ in range(4):
            left = [max(a - weight * b, 0) for a, b in zip(left, q)]
            c += weight
            assert left == [max(a - c * b, Fraction(0)) for a, b in zip(p, q)]
            weight = sum(left)


def test_verification_by_hand():
    third = [0.25, 0.5, 0.25]
    rows = [third, [1.0, 0.0, 0.0], [0.0, 0.0, 1.0], [0.0, 1.0, 0.0]]
    masks = [1, 3, 5, 13]  # 0-1, 0-2-3
    # child 1 (token 0, 1/4) rejected at u = 1/4, child 2 (token 1) kept below 1/2 / (3/4), its child kept
    assert otree.verify(rows, None, [9, 0, 1, 2], masks, [0.0, 0.25, 0.66, 0.99], 4) == ([1, 2, 1, -1], [0, 2, 3, -1], 2)
    assert otree.verify(rows, None, [9, 0, 1, 2], masks, [0.0, 0.25, 0.67, 0.99], 4) == ([2, -1, -1, -1], [0, -1, -1, -1], 0)
    # fewer nodes; a token outside the vocabulary; a node that sees nothing before it
    assert otree.verify(rows, None, [9, 0, 1, 2], masks, [0.5, 0.25, 0.0, 0.0], 2)[0] == [1, -1, -1, -1]
    assert otree.verify(rows, None, [9, 3, 1, 2], [1, 3, 4, 13], [0.9, 0.0, 0.0, 0.0], 4) == ([2, -1, -1, -1], [0, -1, -1, -1], 0)
    assert otree.verify(rows, None, [9, 0, 1, 2], masks, [0.0] * 4, 0) == ([-1] * 4, [-1] * 4, -1)


def test_probabilities_by_hand():
    x = [1.0, -1.0, 2.0, 0.0]
    e = np.exp([0.5, -1.0, 2.0, 0.0])
    assert np.allclose(otree.probabilities(x, prompt=[True, False, False, False], repetition=2.0), e / e.sum(), rtol=1e-14)
    e = np.exp([1.0, -2.0 - 0.25 * 3 - 0.5, 2.0 / 2 - 0.25 - 0.5, 0.0])
    got = otree.probabilities(x, counts=[0, 2, 0, -4], repetition=2.0, frequency=0.25, presence=0.5, path_tokens=[1, 2, 9, -1])
    assert np.allclose(got, e / e.sum(), rtol=1e-14)
    e = np.exp(np.array([1.0 + 3.0, 2.0 - 1.0]) / 0.5)
    got = otree.probabilities(x, 0.5, biases=[(0, 1.0), (2, -1.0), (0, 2.0), (-1, 9.0), (4, 9.0)], allowed=[1, 0, 1, 0])
    assert np.allclose(got, [e[0] / e.sum(), 0, e[1] / e.sum(), 0], rtol=1e-14)
    assert otree.probabilities([3.0, 5.0, 5.0], 0.0).tolist() == [0, 1, 0]
    assert otree.probabilities([np.inf, 5.0, np.inf], 2.0).tolist() == [0.5, 0, 0.5]
    assert otree.probabilities([np.nan, 5.0], 1.0).tolist() == [0, 1]
    assert otree.probabilities([1.0, 5.0], 1.0, allowed=[0, 0]).tolist() == [0, 0]


def test_compaction_reads_before_it_writes():
    rows = np.arange(8)[:, None] * np.ones((1, 2))
    assert otree.compact(rows, 2, [0, 3, 1, 2], 3)[:, 0].tolist() == [0, 1, 2, 5, 3, 4, 6, 7]
    assert otree.compact(rows, 2, [0, 3, 4], 0)[:, 0].tolist() == list(range(8))


def test_random_trees_are_closed_under_ancestors():
    for n in (1, 2, 17, 64):
        masks = random_tree(random.Random(n), n)
        for i in range(1, n):
            assert masks[i] == masks[otree.parent(masks[i], i)] | 1 << i and masks[i] & 1
