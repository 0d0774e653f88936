"""Verification of drafted tokens in exact rational arithmetic (oracle; test infrastructure only).

[K2.6] "How to serve trillions of tokens for trillion-parameter coding agents", section "Use
custom speculative decoding ...": drafts are verified in parallel without changing the
target's distribution. The rule is rejection sampling: draft x of q is kept with
probability min(1, p(x) / q(x)); a rejection draws from max(p - q, 0), normalised.
"""

from __future__ import annotations

import math
from fractions import Fraction


def _weight(x) -> Fraction:
    x = float(x)
    if math.isnan(x) or x <= 0.0:
        return Fraction(0)
    return Fraction(min(x, 1.0))


def _unit(u) -> Fraction:
    u = float(u)
    if math.isnan(u) or u <= 0.0:
        return Fraction(0)
    return Fraction(min(u, 1.0 - 2.0 ** -24))


def sample(weights, u) -> int:
    """Smallest i with w_0 + .. + w_i > u * sum(w); -1 if all weights are zero."""
    total = sum(weights)
    if total == 0:
        return -1
    at, run = _unit(u) * total, Fraction(0)
    for i, w in enumerate(weights):
        run += w
        if run > at:
            return i
    raise AssertionError("u < 1 always finds one")


def verify(target, draft, tokens, uniforms, num_drafts=None):
    """One request: ``target [K + 1][V]``, ``draft [K][V]`` or None, ``tokens [K]``, ``uniforms [K + 1]``.

    Returns ``(out_tokens [K + 1], accepted)``; left out: all -1 and -1.
    """
    most, vocab = len(target) - 1, len(target[0])
    k = most if num_drafts is None else int(num_drafts)
    if not 0 <= k <= most:
        return [-1] * (most + 1), -1
    a = 0
    while a < k:
        x = int(tokens[a])
        if not 0 <= x < vocab:
            break
        q = Fraction(1) if draft is None else _weight(draft[a][x])
        if not _unit(uniforms[a]) * q < _weight(target[a][x]):
            break
        a += 1
    p = [_weight(v) for v in target[a]]
    rest = p
    if a < k:
        if draft is None:
            rest = [Fraction(0) if i == int(tokens[a]) else v for i, v in enumerate(p)]
        else:
            rest = [max(v - _weight(w), Fraction(0)) for v, w in zip(p, draft[a])]
        if sum(rest) == 0:
            rest = p
    out = [int(t) for t in tokens[:a]] + [sample(rest, uniforms[most])]
    return out + [-1] * (most - a), a
