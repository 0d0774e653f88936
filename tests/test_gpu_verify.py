"""mla_verify_drafts equals the rational-arithmetic oracle in every output (GPU, whole numbers).

The kernel's sums are exact for probabilities of 2^-37 and above; smaller ones here (a row
holds at most 131,072) move a border by less than 2^-43 of the total, and the uniforms are
multiples of 2^-24.
"""

import numpy as np
import pytest
import torch

from oracle import verify as over
from paged_mla_decode_gb300 import binding

pytestmark = pytest.mark.gpu


def _probs(rng, shape, sharp=3.0):
    z = rng.standard_normal(shape) * sharp
    p = np.exp(z - z.max(-1, keepdims=True))
    return np.maximum((p / p.sum(-1, keepdims=True)), 0).astype(np.float32)


def _bf16(x):
    return torch.from_numpy(x).bfloat16()


def _run(dev, p, q, tokens, u, k=None, lens=None, pad=(0, 0), stream=None):
    """p, q: CPU tensors [B, K+1, V], [B, K, V] or None; pad: extra elements per row."""
    def put(t, extra):
        if t is None:
            return None
        wide = torch.full((*t.shape[:2], t.shape[2] + extra), float("nan"), dtype=t.dtype, device=dev)
        view = wide[..., :t.shape[2]]
        view.copy_(t)
        return view
    B, rows, _ = p.shape
    i32 = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    out = torch.full((B, rows), -7, dtype=torch.int32, device=dev)
    acc = torch.full((B,), -7, dtype=torch.int32, device=dev)
    lens_out = None if lens is None else torch.full((B,), -7, dtype=torch.int32, device=dev)
    tok = i32(tokens).reshape(B, rows - 1)
    binding.mla_verify_drafts(put(p, pad[0]), put(q, pad[1]), tok, torch.from_numpy(u).to(dev), out, acc,
                              num_drafts=i32(k), seq_lens=i32(lens), seq_lens_out=lens_out, stream=stream)
    torch.cuda.synchronize()
    return out.cpu().numpy(), acc.cpu().numpy(), None if lens is None else lens_out.cpu().numpy()


def _check(dev, p, q, tokens, u, k=None, lens=None, **kw):
    out, acc, lens_out = _run(dev, p, q, tokens, u, k, lens, **kw)
    pf, qf = p.float().numpy(), None if q is None else q.float().numpy()
    for b in range(p.shape[0]):
        if lens is not None and lens[b] < 0:
            want, a, n = [-1] * p.shape[1], -1, lens[b]
        else:
            kb = p.shape[1] - 1 if k is None else int(k[b])
            want, a = over.verify(pf[b], None if q is None else qf[b], tokens[b], u[b], kb)
            n = None if lens is None else int(lens[b]) - (kb - a if a >= 0 else 0)
        assert out[b].tolist() == want, f"request {b}"
        assert acc[b] == a
        if lens is not None:
            assert lens_out[b] == n


def _draws(rng, q, B, K, V):
    """Drafts drawn from q (uniform without one), so that some are kept and some not."""
    if q is None:
        return rng.integers(0, V, (B, K))
    c = np.cumsum(q.astype(np.float64), -1)
    r = rng.random((B, K, 1)) * c[..., -1:]
    return np.minimum((c <= r).sum(-1), V - 1)


@pytest.mark.parametrize("K", [0, 1, 3, 31])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4099])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_matches_oracle(cuda_device, K, V, dtype):
    rng = np.random.default_rng(100 * K + V)
    B = 5
    p = _probs(rng, (B, K + 1, V))
    q = np.abs(p[:, :K] * (1 + 0.5 * rng.standard_normal((B, K, V)).astype(np.float32)))
    tokens = _draws(rng, q, B, K, V)
    u = rng.random((B, K + 1)).astype(np.float32)
    u[0] *= 0.05  # a request that keeps most
    cast = (lambda x: torch.from_numpy(x)) if dtype == "f32" else _bf16
    _check(cuda_device, cast(p), cast(q), tokens, u, lens=rng.integers(K + 1, 999, B))
    _check(cuda_device, cast(p), None, tokens, u, k=rng.integers(-1, K + 2, B), pad=(3, 0))


@pytest.mark.parametrize("pad", [(0, 0), (1, 0), (0, 1), (2, 7), (4, 8), (5, 5)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9001, 40000])
def test_padded_rows_and_alignments(cuda_device, pad, dtype, V):
    """Row strides of every alignment, for p and q apart; the padding holds NaN."""
    rng = np.random.default_rng(sum(pad) + V)
    B, K = 3, 2
    p, q = _probs(rng, (B, K + 1, V), 6.0), _probs(rng, (B, K, V), 6.0)
    tokens, u = _draws(rng, q, B, K, V), rng.random((B, K + 1)).astype(np.float32)
    cast = (lambda x: torch.from_numpy(x)) if dtype == "f32" else _bf16
    _check(cuda_device, cast(p), cast(q), tokens, u, pad=pad)


@pytest.mark.parametrize("B,V", [(1, 131072), (40, 20000), (300, 700)])
def test_batches_and_large_vocabularies(cuda_device, B, V):
    rng = np.random.default_rng(B)
    K = 3
    p = _probs(rng, (B, K + 1, V))
    q = np.roll(p[:, :K], 1, axis=2)
    tokens, u = _draws(rng, q, B, K, V), rng.random((B, K + 1)).astype(np.float32)
    lens = rng.integers(4, 999, B)
    lens[B // 2] = -1
    k = rng.integers(0, K + 1, B)
    _check(cuda_device, torch.from_numpy(p), torch.from_numpy(q), tokens, u, k=k, lens=lens)


def test_edges(cuda_device):
    """Borders of the comparison, p = q, empty rows, values that are no probabilities."""
    nan, inf = float("nan"), float("inf")
    p = np.float32([[[0.5, 0.5, 0.0, 0.0]] * 2, [[0.5, 0.5, 0.0, 0.0]] * 2, [[0.25] * 4] * 2, [[0.0] * 4] * 2,
                    [[nan, -1.0, inf, 0.5]] * 2, [[0.5, 0.25, 0.25, 0.0]] * 2, [[0.5, 0.25, 0.25, 0.0]] * 2,
                    [[0.0, 0.0, 0.0, 1.0]] * 2])
    q = np.float32([[[0.0, 1.0, 0.0, 0.0]], [[0.0, 1.0, 0.0, 0.0]], [[0.25] * 4], [[0.0, 0.0, 1.0, 0.0]],
                    [[0.1, nan, 2.0, 0.1]], [[0.5, 0.25, 0.25, 0.0]], [[0.5, 0.25, 0.25, 0.0]], [[0.0] * 4]])
    tokens = np.array([[1], [1], [-1], [2], [2], [3], [0], [3]])
    u = np.float32([[0.5, 0.0], [0.4999, 0.5], [0.0, 0.999], [0.0, 0.5], [0.99, 0.7], [0.0, 0.5], [nan, 2.0],
                    [1.5, -1.0]])
    _check(cuda_device, torch.from_numpy(p), torch.from_numpy(q), tokens, u)
    _check(cuda_device, torch.from_numpy(p), None, tokens, u)


def test_in_place_lengths_captured_on_a_side_stream(cuda_device):
    rng = np.random.default_rng(9)
    B, K, V = 6, 3, 500
    p, q = _probs(rng, (B, K + 1, V)), _probs(rng, (B, K, V))
    tokens, u = _draws(rng, q, B, K, V), rng.random((B, K + 1)).astype(np.float32)
    dev = cuda_device
    tp, tq, tu = torch.from_numpy(p).to(dev), torch.from_numpy(q).to(dev), torch.from_numpy(u).to(dev)
    tt = torch.from_numpy(tokens.astype(np.int32)).to(dev)
    lens = torch.full((B,), 50, dtype=torch.int32, device=dev)
    out, acc = torch.empty((B, K + 1), dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        binding.mla_verify_drafts(tp, tq, tt, tu, out, acc, seq_lens=lens, seq_lens_out=lens)
    graph.replay()
    tu.copy_(torch.from_numpy(u[::-1].copy()))
    graph.replay()
    length = np.full(B, 50)
    for uu in (u, u[::-1]):
        want = [over.verify(p[b], q[b], tokens[b], uu[b]) for b in range(B)]
        length -= K - np.array([a for _, a in want])
    assert out.cpu().tolist() == [w for w, _ in want] and acc.cpu().tolist() == [a for _, a in want]
    assert lens.cpu().tolist() == length.tolist()


def test_sampled_tokens_follow_the_target(cuda_device):
    """The accepted or resampled first token of 200,000 requests against the target: each count
    within 6 standard deviations of its binomial."""
    rng = np.random.default_rng(10)
    B, V = 200_000, 8
    p1, q1 = _probs(rng, (V,), 1.0), _probs(rng, (V,), 1.0)
    p = torch.from_numpy(p1).expand(B, 2, V).contiguous()
    q = torch.from_numpy(q1).expand(B, 1, V).contiguous()
    tokens = rng.choice(V, size=(B, 1), p=q1.astype(np.float64) / q1.sum(dtype=np.float64))
    u = rng.random((B, 2)).astype(np.float32)
    out, _, _ = _run(cuda_device, p, q, tokens, u)
    count = np.bincount(out[:, 0], minlength=V)
    want = p1.astype(np.float64) / p1.sum(dtype=np.float64)
    assert (np.abs(count - B * want) <= 6 * np.sqrt(B * want * (1 - want)) + 1).all()
