"""Operators of a tree-speculative step (oracle; test infrastructure only).

[K2.6] "How to serve trillions of tokens for trillion-parameter coding agents", section "Use
custom speculative decoding ...": drafted tokens are verified in parallel without changing the
target's distribution. Here the drafts form a tree. Node 0 is the last sampled token; bit i of a
node's mask says that it sees node i, for a tree its ancestors and itself.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

from . import attention
from .verify import _unit, _weight, sample


def sees(mask, i: int) -> bool:
    return bool(int(mask) >> i & 1)


def decode(q: np.ndarray, entries, masks, nodes, sm_scale: float):
    """Attention of every node: ``q [B, N, H, 576]`` and ``entries[b] [L_b, 576]`` float64, ``masks [B, N]``.

    The last ``nodes[b]`` entries are the nodes'. Returns ``(out [B, N, H, 512], lse [B, N, H])``.
    """
    B, N, H, _ = q.shape
    out, lse = np.zeros((B, N, H, attention.D_LATENT)), np.full((B, N, H), -np.inf)
    for b in range(B):
        n = int(nodes[b])
        context = len(entries[b]) - n
        for j in range(n):
            seen = list(range(context)) + [context + i for i in range(n) if sees(masks[b][j], i)]
            out[b, j], lse[b, j] = attention.attend(q[b, j], entries[b][seen], sm_scale)
    return out, lse


def probabilities(logits, temperature=1.0, counts=None, prompt=None, repetition=1.0, frequency=0.0, presence=0.0,
                  path_tokens=(), biases=(), allowed=None):
    """One row of logits to probabilities, float64.

    ``counts [V]`` how often each token was generated, ``path_tokens`` more of them (drafts before this row),
    ``prompt [V]`` whether a token is in the prompt, ``biases`` pairs (token, value), ``allowed [V]`` a grammar's mask.
    """
    x = np.asarray(logits, np.float64).copy()
    V = len(x)
    count = np.zeros(V) if counts is None else np.maximum(np.asarray(counts, np.float64), 0)
    for t in path_tokens:
        if 0 <= t < V:
            count[t] += 1
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(V):
            if count[i] > 0 or (prompt is not None and prompt[i]):
                x[i] = x[i] / repetition if x[i] > 0 else x[i] * repetition
            if count[i] > 0:
                x[i] -= frequency * count[i]
                x[i] -= presence
        for t, v in biases:
            if 0 <= t < V:
                x[t] += v
    if allowed is not None:
        x[~np.asarray(allowed, bool)] = -np.inf
    x[np.isnan(x)] = -np.inf
    top, p = x.max(), np.zeros(V)
    if top == -np.inf:
        return p
    if not temperature > 0:
        p[int(np.argmax(x))] = 1.0
        return p
    if top == np.inf:
        p[x == np.inf] = 1.0
    else:
        some = x > -np.inf
        p[some] = np.exp((x[some] - top) / temperature)
    return p / p.sum()


def parent(mask, i: int) -> int:
    """The last node before i that it sees; -1: none."""
    return (int(mask) & ((1 << i) - 1)).bit_length() - 1


def verify(target, draft, tokens, masks, uniforms, n: int):
    """One request: ``target [N][V]``, ``draft [N][V]`` or None, ``tokens``, ``masks`` and ``uniforms [N]``.

    From node 0 on: its children are tried in order; one is kept with probability min(1, left / drafted) of its token,
    where `left` is what the rejected ones left of the target (each takes the drafter's distribution off, or,
    without one, its own token). Returns ``(out_tokens [N], path [N], accepted)``; left out: -1.
    """
    N, V = len(target), len(target[0])
    if not 1 <= n <= N:
        return [-1] * N, [-1] * N, -1
    here, out, path = 0, [], [0]
    while True:
        p = [_weight(v) for v in target[here]]
        q = None if draft is None else [_weight(v) for v in draft[here]]
        left, weight, kept = p, Fraction(1), None
        for i in range(here + 1, n):
            if parent(masks[i], i) != here:
                continue
            x = int(tokens[i])
            if 0 <= x < V and _unit(uniforms[i]) * (Fraction(1) if q is None else q[x]) * weight < left[x]:
                kept = i
                break
            if q is None:
                if 0 <= x < V:
                    weight = max(weight - left[x], Fraction(0))
                    left = [Fraction(0) if k == x else v for k, v in enumerate(left)]
            else:
                left = [max(a - weight * c, Fraction(0)) for a, c in zip(left, q)]
                weight = sum(left)
        if kept is None:
            break
        here = kept
        out.append(int(tokens[kept]))
        path.append(kept)
    out.append(sample(left if sum(left) > 0 else p, uniforms[0]))
    a = len(path) - 1
    return out + [-1] * (N - len(out)), path + [-1] * (N - len(path)), a


def compact(rows: np.ndarray, context: int, path, accepted: int) -> np.ndarray:
    """One request's cached rows (tokens first): the kept nodes' rows behind the context."""
    got = rows.copy()
    for i in range(1, accepted + 1):
        got[context + i] = rows[context + int(path[i])]
    return got
