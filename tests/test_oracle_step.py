"""The allocation and verification oracles are pinned by invariants and enumeration (CPU)."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import paging, verify


@pytest.mark.parametrize("seed", range(6))
def test_alloc_gives_disjoint_pages_and_consecutive_slots(seed):
    rng = np.random.default_rng(seed)
    B, width, pages = 9, 12, 90
    lens = rng.integers(0, 300, B)
    held = -(-lens // 64) + rng.integers(0, 2, B)
    new = rng.integers(0, 300, B)
    perm = rng.permutation(pages)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = perm[at:]
    tags = rng.integers(0, 1 << 30, pages)
    got = paging.alloc(lens, new, held, free, len(free), pages, table, int(new.sum()) + 3, tags,
                       np.zeros((B, width), np.int64))
    taken = []
    for b in range(B):
        if got["request_status"][b]:
            assert got["seq_lens_out"][b] == -1 and got["pages_held_out"][b] == held[b]
            continue
        n = int(got["seq_lens_out"][b])
        assert n == lens[b] + new[b] and got["pages_held_out"][b] >= -(-n // 64)
        row = got["block_table"][b, :got["pages_held_out"][b]]
        taken += row.tolist()
        slots = got["slot_mapping"][got["cu_tokens"][b]:got["cu_tokens"][b + 1]]
        pos = np.arange(lens[b], n)
        assert np.array_equal(slots, row[pos // 64] * 64 + pos % 64)
        for j in range(held[b], got["pages_held_out"][b]):
            assert got["expected_tags"][b, j] == got["page_tags"][row[j]] == tags[row[j]] + 1
    assert len(set(taken)) == len(taken)
    assert got["free_count_out"] == len(free) - (got["pages_held_out"] - held).sum()


def test_alloc_refusals():
    table = np.full((5, 2), 7)
    got = paging.alloc([-1, 10, 100, 0, 64], [1, -1, 60, 64, 1], [0, 1, 2, 0, 1], [3], 1, 9, table, 200)
    assert got["request_status"].tolist() == [paging.BAD_LENGTH, paging.BAD_LENGTH, paging.TABLE_FULL, 0,
                                              paging.NO_PAGES]
    assert got["cu_tokens"].tolist() == [0, 1, 1, 61, 125, 126]
    assert got["slot_mapping"][61:125].tolist() == list(range(3 * 64, 4 * 64))


@pytest.mark.parametrize("seed", range(3))
def test_first_token_follows_the_target(seed):
    """Summed over drafts (with their probabilities) and an even grid of uniforms, the first
    token's probability is the target's, up to the grid's resolution."""
    rng = np.random.default_rng(seed)
    V, grid = 4, 64
    p = rng.dirichlet(np.ones(V))
    q = rng.dirichlet(np.ones(V))
    mass = np.zeros(V)
    for x in range(V):
        for u in (np.arange(grid) + 0.5) / grid:
            for s in (np.arange(grid) + 0.5) / grid:
                out, _ = verify.verify([p, p], [q], [x], [u, s])
                mass[out[0]] += q[x] / grid ** 2
    assert np.abs(mass - p).max() < 4.0 / grid


def test_edges():
    p, q = [0.5, 0.5, 0.0], [0.0, 1.0, 0.0]
    assert verify.verify([p, p], [q], [1], [0.75, 0.1]) == ([0, -1], 0)       # rejected: only token 0 is left
    assert verify.verify([p, p], [q], [1], [0.25, 0.6]) == ([1, 1], 1)        # kept, then a bonus token
    assert verify.verify([p, p], [q], [9], [0.0, 0.0]) == ([0, -1], 0)        # no such token
    assert verify.verify([p, p], [p], [2], [0.0, 0.7]) == ([1, -1], 0)        # p = q: the target itself
    assert verify.verify([[0.0] * 3], [], [], [0.3]) == ([-1], 0)
    assert verify.verify([p, p], None, [1], [0.5, 0.9]) == ([0, -1], 0)       # a certain drafter, u = p
    assert verify.verify([p, p], None, [1], [0.4, 0.9], num_drafts=0) == ([1, -1], 0)
    assert verify.verify([p, p], None, [1], [0.4, 0.9], num_drafts=2) == ([-1, -1], -1)
    assert verify.sample([Fraction(1), Fraction(0), Fraction(1)], 0.5) == 2   # the border goes up
