"""mla_verify_tree against the rational oracle (GPU): tokens, paths, lengths and counts are equal."""

import random

import numpy as np
import pytest
import torch

from oracle import tree as otree
from paged_mla_decode_gb300 import binding

from .tree_util import chain, i32, mask_tensor, random_tree

pytestmark = pytest.mark.gpu


def bf16_round(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().float().numpy()


class Case:
    """B random requests; `p` and `q` [B, N, V] as the kernel sees them."""

    def __init__(self, seed, B, N, V, dtype="f32", drafter=True, kind="soft", ragged=True):
        rng, r = np.random.default_rng(seed), random.Random(seed)
        if kind == "soft":
            p, q = rng.dirichlet(np.full(V, 0.5), (B, N)), rng.dirichlet(np.full(V, 0.5), (B, N))
            q = 0.5 * (p + q)
        else:  # eighths, zeros among them: many equal and empty weights
            p, q = rng.integers(0, 3, (B, N, V)) / 8.0, rng.integers(0, 3, (B, N, V)) / 8.0
        self.p, self.q = np.asarray(p, np.float32), np.asarray(q, np.float32)
        if dtype == "bf16":
            self.p, self.q = bf16_round(self.p), bf16_round(self.q)
        self.drafter, self.dtype = drafter, torch.float32 if dtype == "f32" else torch.bfloat16
        self.B, self.N, self.V = B, N, V
        self.masks = [random_tree(r, N) for _ in range(B)]
        self.tokens = rng.integers(-1 if V > 3 else 0, V + (V > 3), (B, N))
        for b in range(B):
            for i in range(1, N):  # as drawn from the parent's row
                if r.random() < 0.8:
                    w = self.q[b, otree.parent(self.masks[b][i], i)].astype(np.float64)
                    if w.sum() > 0:
                        self.tokens[b, i] = rng.choice(V, p=w / w.sum())
        self.u = rng.random((B, N), dtype=np.float32)
        self.u[rng.random((B, N)) < 0.05] = 0.0
        self.nodes = rng.integers(0, N + 2, B) if ragged else np.full(B, N)
        self.lens = rng.integers(0, 500, B) + N
        if ragged:
            self.lens[::7] = rng.integers(-1, N, len(self.lens[::7]))
        self.counts = rng.integers(0, 5, (B, V))

    def run(self, dev, in_place=False, stride=0, bare=False):
        def rows(a):
            wide = torch.full((self.B, self.N, self.V + stride), 0.5, dtype=self.dtype, device=dev)
            wide[..., :self.V] = torch.from_numpy(a).to(dev)
            return wide[..., :self.V]

        out, path = i32(np.full((self.B, self.N), 77), dev), i32(np.full((self.B, self.N), 77), dev)
        acc, lens, counts = i32(np.full(self.B, 77), dev), i32(self.lens, dev), i32(self.counts, dev)
        lens_out = lens if in_place else i32(np.full(self.B, 77), dev)
        kw = {} if bare else dict(num_nodes=i32(self.nodes, dev), seq_lens=lens, seq_lens_out=lens_out, token_counts=counts)
        binding.mla_verify_tree(rows(self.p), rows(self.q) if self.drafter else None, i32(self.tokens, dev),
                                mask_tensor(self.masks, dev), torch.from_numpy(self.u).to(dev), out, path, acc, **kw)
        torch.cuda.synchronize()
        return [t.cpu().numpy() for t in (out, path, acc, lens_out, counts)]

    def check(self, got, bare=False):
        out, path, acc, lens, counts = got
        for b in range(self.B):
            n, L = (self.N, self.N) if bare else (int(self.nodes[b]), int(self.lens[b]))
            if L < n:
                n = 0
            if self.p[b].astype(np.float64).sum(-1).max() >= 16:  # outside the contract: some tokens of the vocabulary
                assert ((out[b] >= -1) & (out[b] < self.V)).all() and -1 <= acc[b] < self.N
                continue
            want = otree.verify(self.p[b], self.q[b] if self.drafter else None, self.tokens[b], self.masks[b], self.u[b], n)
            assert (out[b].tolist(), path[b].tolist(), int(acc[b])) == (want[0], want[1], want[2]), (b, n)
            if not bare:
                assert lens[b] == (L - n + want[2] + 1 if want[2] >= 0 else L)
                c = self.counts[b].copy()
                for t in want[0]:
                    if t >= 0:
                        c[t] += 1
                assert np.array_equal(counts[b], c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("kind", ["soft", "eighths"])
@pytest.mark.parametrize("N,V", [(1, 5), (2, 1), (3, 2), (4, 7), (8, 33), (16, 64), (64, 20), (12, 300)])
def test_random_trees(cuda_device, dtype, drafter, kind, N, V):
    c = Case(N * V, 30, N, V, dtype, drafter, kind)
    c.check(c.run(cuda_device))


@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("stride", [0, 1, 4])
def test_without_lengths_in_place_and_rows_apart(cuda_device, drafter, stride):
    c = Case(stride, 12, 6, 40, drafter=drafter, ragged=False)
    c.check(c.run(cuda_device, stride=stride, bare=True), bare=True)
    c.check(c.run(cuda_device, stride=stride, in_place=True))


def wide_verify(p, q, tokens, masks, u, n):
    """The rule in float64 with arrays (rows of a large vocabulary)."""
    weight = lambda a: np.clip(np.nan_to_num(a.astype(np.float64)), 0.0, 1.0)  # noqa: E731
    here, out, path = 0, [], [0]
    while True:
        left, w, kept = weight(p[here]), 1.0, None
        qv = None if q is None else weight(q[here])
        for i in range(here + 1, n):
            if otree.parent(masks[i], i) != here:
                continue
            x = int(tokens[i])
            if float(u[i]) * (1.0 if qv is None else qv[x]) * w < left[x]:
                kept = i
                break
            if qv is None:
                w = max(w - left[x], 0.0)
                left[x] = 0.0
            else:
                left = np.maximum(left - w * qv, 0.0)
                w = left.sum()
        if kept is None:
            break
        here = kept
        out.append(int(tokens[kept]))
        path.append(kept)
    if left.sum() == 0:
        left = weight(p[here])
    cum = left.cumsum()
    out.append(int(np.searchsorted(cum, float(u[0]) * cum[-1], side="right")))
    return out, path


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("V", [4095, 4096, 32768, 131072, 163840, 163841])
def test_large_vocabularies(cuda_device, dtype, drafter, V):
    """Wide trees, so that a node's fourth child and more are reached; every size of cluster."""
    dev, B, N = cuda_device, 6, 14
    g = torch.Generator().manual_seed(V)
    logits = torch.randn(B, N, V, generator=g) * 2
    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    p, q = torch.softmax(logits, -1).to(kind), torch.softmax(logits + torch.randn(B, N, V, generator=g), -1).to(kind)
    masks = [[1] + [1 | 1 << i for i in range(1, 9)] + [1 | 2 | 1 << i for i in range(9, 14)]] * 3 + [chain(N)] * 3
    tokens = np.zeros((B, N), np.int64)
    for b in range(B):
        for i in range(1, N):
            tokens[b, i] = torch.multinomial(q[b, otree.parent(masks[b][i], i)].float(), 1, generator=g)
    u = torch.rand(B, N, generator=g)
    out, path, acc = i32(np.zeros((B, N)), dev), i32(np.zeros((B, N)), dev), i32(np.zeros(B), dev)
    binding.mla_verify_tree(p.to(dev), q.to(dev) if drafter else None, i32(tokens, dev), mask_tensor(masks, dev), u.to(dev),
                            out, path, acc)
    torch.cuda.synchronize()
    for b in range(B):
        want, kept = wide_verify(p[b].float().numpy(), q[b].float().numpy() if drafter else None, tokens[b], masks[b], u[b].numpy(), N)
        assert out[b].tolist() == want + [-1] * (N - len(want)) and path[b].tolist() == kept + [-1] * (N - len(kept))
        assert int(acc[b]) == len(kept) - 1


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafter", [True, False])
def test_a_chain_is_mla_verify_drafts(cuda_device, dtype, drafter):
    dev, B, N, V = cuda_device, 64, 5, 3000
    g = torch.Generator(device=dev).manual_seed(1)
    logits = torch.randn(B, N, V, generator=g, device=dev)
    p, q = torch.softmax(logits, -1).to(dtype), torch.softmax(logits + torch.randn(B, N, V, generator=g, device=dev), -1).to(dtype)
    tokens = torch.multinomial(q.float().flatten(0, 1), 1, generator=g).view(B, N).roll(1, 1).int()
    u = torch.rand(B, N, generator=g, device=dev)
    out, path, acc = (torch.empty((B, N), dtype=torch.int32, device=dev) for _ in range(3))
    acc = acc[:, 0].contiguous()
    binding.mla_verify_tree(p, q if drafter else None, tokens, mask_tensor([chain(N)] * B, dev), u, out, path, acc)
    want, kept = torch.empty_like(out), torch.empty_like(acc)
    binding.mla_verify_drafts(p, q[:, :N - 1].contiguous() if drafter else None, tokens[:, 1:].contiguous(), u.roll(-1, 1).contiguous(),
                              want, kept)
    assert torch.equal(acc, kept) and torch.equal(out, want)


def test_nans_infinities_and_nothing_left(cuda_device):
    """Rows of NaN, infinities and zeros: weights within [0, 1], the token -1 where there is none."""
    V, N = 6, 4
    c = Case(3, 4, N, V, ragged=False)
    c.p[0] = np.nan
    c.p[1] = 0.0
    c.p[2, 0] = [np.inf, -1, 0, 0, 0, 0]
    c.q[2, 0] = [np.nan, 1, 0, 0, 0, 0]
    c.p[3] = c.q[3]
    c.check(c.run(cuda_device))
    assert (c.run(cuda_device)[0][:2] == -1).all()


@pytest.mark.parametrize("drafter", [True, False])
def test_masks_that_are_no_trees(cuda_device, drafter):
    """Nodes without an ancestor are not reached; bits of later nodes mean nothing."""
    c = Case(9, 8, 6, 30, drafter=drafter, ragged=False)
    full = (1 << 64) - 1
    c.masks = [[0, 2, 4, 8, 16, 32], [full] * 6, [0] * 6, [1, 1, 1, 1, 1, 1], [1, 3, 2, 6, 1 << 63, 33],
               [0, 1, 3, 7, 15, 31], [full, full - 1, full - 3, 1, 2, 4], [5, 7, 1, 2, 8, 9]]
    c.check(c.run(cuda_device))


def test_captured_step_and_two_streams(cuda_device):
    cs = [Case(70 + k, 9, 8, 900) for k in range(2)]
    for k in range(2):
        cs[k].check(cs[k].run(cuda_device))
    dev = cuda_device
    bufs = []
    for c in cs:
        bufs.append([torch.from_numpy(c.p).to(dev), torch.from_numpy(c.q).to(dev), i32(c.tokens, dev), mask_tensor(c.masks, dev),
                     torch.from_numpy(c.u).to(dev), i32(np.zeros((9, 8)), dev), i32(np.zeros((9, 8)), dev), i32(np.zeros(9), dev)])
    kws = [dict(num_nodes=i32(c.nodes, dev), seq_lens=i32(c.lens, dev), token_counts=i32(c.counts, dev)) for c in cs]
    for k in range(2):
        kws[k]["seq_lens_out"] = kws[k]["seq_lens"].clone()
    streams = [torch.cuda.Stream(dev) for _ in cs]
    torch.cuda.synchronize()
    for k in range(2):
        binding.mla_verify_tree(*bufs[k], stream=streams[k], **kws[k])
    torch.cuda.synchronize()
    for k in range(2):
        cs[k].check([t.cpu().numpy() for t in (*bufs[k][5:], kws[k]["seq_lens_out"], kws[k]["token_counts"])])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.mla_verify_tree(*bufs[0], **kws[0])
    for a, b in zip(bufs[0][:5], bufs[1][:5]):
        a.copy_(b)
    for key in ("num_nodes", "seq_lens"):
        kws[0][key].copy_(kws[1][key])
    kws[0]["token_counts"].copy_(i32(cs[1].counts, dev))
    graph.replay()
    torch.cuda.synchronize()
    cs[1].check([t.cpu().numpy() for t in (*bufs[0][5:], kws[0]["seq_lens_out"], kws[0]["token_counts"])])


def test_refusals(cuda_device):
    dev = cuda_device
    good = dict(target_probs=torch.rand(2, 3, 50, device=dev), draft_probs=torch.rand(2, 3, 50, device=dev),
                node_tokens=i32(np.zeros((2, 3)), dev), tree_mask=mask_tensor([chain(3)] * 2, dev), uniforms=torch.rand(2, 3, device=dev),
                out_tokens=i32(np.zeros((2, 3)), dev), path=i32(np.zeros((2, 3)), dev), num_accepted=i32([0, 0], dev))
    binding.mla_verify_tree(**good)
    for kw in (dict(target_probs=good["target_probs"].half()), dict(draft_probs=good["draft_probs"][:, :2]),
               dict(draft_probs=good["draft_probs"].bfloat16()), dict(node_tokens=good["node_tokens"].long()),
               dict(tree_mask=good["tree_mask"][:, :2]), dict(uniforms=good["uniforms"].double()), dict(uniforms=good["uniforms"][:1]),
               dict(path=good["path"][:1]), dict(out_tokens=good["out_tokens"].cpu()), dict(num_accepted=i32([0], dev)),
               dict(seq_lens_out=i32([0, 0], dev)), dict(num_nodes=i32([0], dev)), dict(token_counts=i32(np.zeros((2, 49)), dev))):
        with pytest.raises(AssertionError):
            binding.mla_verify_tree(**{**good, **kw})
    torch.cuda.synchronize()
