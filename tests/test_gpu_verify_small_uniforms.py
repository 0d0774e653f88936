"""The sampled token at a border that a uniform below 2^-41 decides: u times the total of the
weights lies on an integer number of 2^-60, or just above it (GPU, whole numbers)."""

import random

import numpy as np
import pytest
import torch

from oracle import verify as over

from .test_gpu_verify import _run

pytestmark = pytest.mark.gpu


def _border(r):
    """A uniform u = m 2^-s and weights in units of 2^-60, the first being floor(u * total), where
    u cut off at 2^-64 would give less."""
    while True:
        s, m = r.randint(66, 80), r.randrange(1 << 23, 1 << 24) | 1
        rest = [r.randrange(1 << 22, 1 << 23) << 36 for _ in range(r.randint(1, 3))]
        first = 0
        for _ in range(4):
            first = (m * (sum(rest) + first)) >> s
        total = sum(rest) + first
        if first and (m * total) >> s == first and (((m << 64) >> s) * total) >> 64 < first:
            return m * 2.0 ** -s, [first, *rest]


def test_the_first_token_ends_on_the_border(cuda_device):
    r = random.Random(540)
    found = [_border(r) for _ in range(64)]
    p = np.zeros((64, 1, 8), np.float32)
    u = np.zeros((64, 1), np.float32)
    for b, (x, weights) in enumerate(found):
        u[b] = x
        p[b, 0, :len(weights)] = [w * 2.0 ** -60 for w in weights]
        assert float(u[b, 0]) == x and [int(v * 2.0 ** 60) for v in p[b, 0].tolist()][:len(weights)] == weights
    out, acc, _ = _run(cuda_device, torch.from_numpy(p), None, np.zeros((64, 0)), u)
    want = [over.verify(p[b], None, [], u[b])[0] for b in range(64)]
    assert out.tolist() == want and (acc == 0).all() and all(w == [1] for w in want)


@pytest.mark.parametrize("u", [2.0 ** -149, 2.0 ** -126, 2.0 ** -64, 2.0 ** -61, 2.0 ** -60, 2.0 ** -59, 2.0 ** -41, 0.0])
def test_uniforms_down_to_the_smallest(cuda_device, u):
    """Beside a first token of weight 2^-60, in rows whose total is 1 to within it and in short ones."""
    p = np.zeros((3, 1, 5), np.float32)
    p[0, 0, :3] = [2.0 ** -60, 0.5, 0.5]
    p[1, 0, 1:3] = [2.0 ** -60, 2.0 ** -40]
    p[2, 0, 4] = 2.0 ** -60
    us = np.full((3, 1), u, np.float32)
    out, _, _ = _run(cuda_device, torch.from_numpy(p), None, np.zeros((3, 0)), us)
    assert out.tolist() == [over.verify(p[b], None, [], us[b])[0] for b in range(3)]
