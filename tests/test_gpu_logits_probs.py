"""mla_logits_to_probs against the float64 oracle (GPU).

Tolerance. The penalties, the bias and the subtraction of the maximum round at most eight times
to fp32, each by 2^-24 of a magnitude of at most X; divided by the temperature these move the
exponent by 8 * 2^-24 * X / T. The scale log2(e) / T and its product with x - max (at most 2 X)
round three times: 3 * 2^-24 * 2 X / T. exp2 is good to 2^-22, a sum of up to 4,096 terms a thread
group adds less than 2^-17 and the two factors behind it 2^-22. A bf16 result is off by another
2^-8. Results below the smallest normal float may be 0.
"""

import numpy as np
import pytest
import torch

from oracle import tree as otree
from paged_mla_decode_gb300 import binding

from .tree_util import chain, i32, mask_tensor, random_tree

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def words(bits):
    """Truth values [..., V] as 32-bit words [..., ceil(V / 32)]."""
    V = bits.shape[-1]
    wide = np.zeros((*bits.shape[:-1], -(-V // 32) * 32), np.uint64)
    wide[..., :V] = bits
    return (wide.reshape(*bits.shape[:-1], -1, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


class Case:
    def __init__(self, seed, B, R, V, penalties=True, tree=True, biases=5, grammar=0.5, scale=3.0, in_type=F32, dev=None):
        rng = np.random.default_rng(seed)
        x = torch.from_numpy((rng.standard_normal((B, R, V)) * scale).astype(np.float32)).to(in_type)
        self.x, self.B, self.R, self.V, self.dev = x, B, R, V, dev
        self.temperature = rng.uniform(0.3, 1.5, B).astype(np.float32)
        self.temperature[::3] = 0.0
        self.host, self.kw = {}, {"temperature": torch.from_numpy(self.temperature).to(dev)}
        if penalties:
            self.host["counts"] = rng.integers(-1, 4, (B, V)) * (rng.random((B, V)) < 0.3)
            self.host["prompt"] = rng.random((B, V)) < 0.2
            for k, lo, hi in (("repetition", 0.7, 1.5), ("frequency", -0.5, 0.7), ("presence", -0.5, 1.0)):
                self.host[k] = rng.uniform(lo, hi, B).astype(np.float32)
                self.kw[k] = torch.from_numpy(self.host[k]).to(dev)
            self.kw["token_counts"] = i32(self.host["counts"], dev)
            self.kw["prompt_mask"] = torch.from_numpy(words(self.host["prompt"])).to(dev)
        if tree:
            import random
            r = random.Random(seed)
            self.masks = [random_tree(r, R) for _ in range(B)]
            self.tokens = rng.integers(-1, V + 1, (B, R))
            if V > 3:
                self.tokens[:, R // 2:] = rng.integers(0, 3, (B, R - R // 2))  # the same ones again
            self.kw |= {"node_tokens": i32(self.tokens, dev), "tree_mask": mask_tensor(self.masks, dev)}
        self.biases = biases
        if biases:
            self.bias_tokens = rng.integers(-1, V, (B, biases))
            self.bias_tokens[:, -1] = self.bias_tokens[:, 0]  # one twice
            self.bias = (rng.standard_normal((B, biases)) * 4).astype(np.float32)
            self.kw |= {"bias_tokens": i32(self.bias_tokens, dev), "biases": torch.from_numpy(self.bias).to(dev)}
        self.allowed = None
        if grammar:
            self.allowed = rng.random((B, R, V)) < grammar
            self.kw["allowed"] = torch.from_numpy(words(self.allowed)).to(dev)

    def run(self, out_type=F32, stride=None):
        x = self.x.to(self.dev)
        p = torch.full((self.B, self.R, self.V), 7.0, dtype=out_type, device=self.dev)
        if stride:
            wide = torch.full((self.B, self.R, self.V + stride), 9.0, dtype=x.dtype, device=self.dev)
            wide[..., :self.V] = x
            x = wide[..., :self.V]
            p = torch.full((self.B, self.R, self.V + stride), 7.0, dtype=out_type, device=self.dev)[..., :self.V]
        binding.mla_logits_to_probs(x, p, **self.kw)
        torch.cuda.synchronize()
        return p.float().cpu().numpy()

    def row(self, b, j):
        h = {k: v[b] for k, v in self.host.items()}
        path = [] if not hasattr(self, "masks") else [int(self.tokens[b, i]) for i in range(1, self.R)
                                                      if otree.sees(self.masks[b][j], i)]
        return otree.probabilities(self.x[b, j].float().numpy(), self.temperature[b], path_tokens=path if self.host else (),
                                   biases=[(int(t), float(v)) for t, v in zip(self.bias_tokens[b], self.bias[b])] if self.biases
                                   else (), allowed=None if self.allowed is None else self.allowed[b, j], **h)

    def check(self, got, rows=None, out_type=F32):
        for b, j in rows or [(b, j) for b in range(self.B) for j in range(self.R)]:
            want, X, T = self.row(b, j), self.magnitude(b, j), self.temperature[b]
            tol = 0.0 if T == 0 else (8 + 6) * 2.0 ** -24 * X / T + 2.0 ** -17 + 2.0 ** -21
            tol += 2.0 ** -8 if out_type is BF16 else 0.0
            err = np.abs(got[b, j] - want)
            assert (err <= tol * want + 2.0 ** -125).all(), (b, j, (err / np.maximum(want, 1e-30)).max(), tol)
            assert np.array_equal(got[b, j] == 0, want == 0) or (want[got[b, j] == 0] < 2.0 ** -100).all()

    def magnitude(self, b, j):
        x = self.x[b, j].float().numpy()
        X = np.abs(x[np.isfinite(x)]).max(initial=0.0) * 1.5
        if self.host:
            X += abs(self.host["frequency"][b]) * (self.host["counts"][b].max() + self.R) + abs(self.host["presence"][b])
        if self.biases:
            X += np.abs(self.bias[b]).sum()
        return float(X)


@pytest.mark.parametrize("in_type,out_type", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 257, 1000, 4095, 4096, 8200])
def test_every_setting(cuda_device, in_type, out_type, V):
    c = Case(V, 4, 5, V, in_type=in_type, dev=cuda_device)
    c.check(c.run(out_type), out_type=out_type)


@pytest.mark.parametrize("penalties,tree,biases,grammar", [(False, False, 0, 0), (True, False, 0, 0), (False, True, 0, 0),
                                                           (True, True, 0, 0), (False, False, 3, 0), (False, False, 0, 0.01),
                                                           (True, True, 1024, 0), (False, True, 7, 0.9)])
def test_each_setting_by_itself(cuda_device, penalties, tree, biases, grammar):
    c = Case(11, 3, 4, 5000, penalties, tree, biases, grammar, dev=cuda_device)
    c.check(c.run())


@pytest.mark.parametrize("V,stride", [(64, 3), (1000, 8), (999, 9), (4099, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_apart(cuda_device, V, stride, dtype):
    """Padded rows, aligned and not; what lies between them stays."""
    c = Case(V, 2, 3, V, in_type=dtype, dev=cuda_device)
    c.check(c.run(dtype, stride), out_type=dtype)


@pytest.mark.parametrize("V", [131072, 163840, 262147, 393216])
def test_large_vocabularies(cuda_device, V):
    c = Case(V, 2, 2, V, in_type=BF16, biases=300, dev=cuda_device)
    c.check(c.run(), rows=[(0, 1), (1, 0)])


@pytest.mark.parametrize("R", [1, 64])
def test_many_rows(cuda_device, R):
    c = Case(R, 8, R, 640, dev=cuda_device)
    c.check(c.run())


def test_rows_without_a_tree_may_be_many(cuda_device):
    c = Case(5, 2, 130, 96, tree=False, dev=cuda_device)
    c.check(c.run())


def test_in_place(cuda_device):
    c = Case(21, 3, 4, 9000, dev=cuda_device)
    x = c.x.to(cuda_device)
    binding.mla_logits_to_probs(x, x, **c.kw)
    c.check(x.cpu().numpy())


def test_rows_that_are_left_as_they_were(cuda_device):
    c = Case(22, 4, 5, 300, dev=cuda_device)
    p = torch.full((4, 5, 300), 7.0, device=cuda_device)
    n = [0, 5, 2, -3]
    binding.mla_logits_to_probs(c.x.to(cuda_device), p, num_rows=i32(n, cuda_device), **c.kw)
    got = p.cpu().numpy()
    c.check(got, rows=[(b, j) for b in range(4) for j in range(max(n[b], 0))])
    for b in range(4):
        assert (got[b, max(n[b], 0):] == 7.0).all()


@pytest.mark.parametrize("temperature", [1e-30, 1e-40, 0.0, -1.0, float("nan"), 1.0, 1e30, float("inf")])
def test_infinities_nans_and_rows_without_a_token(cuda_device, temperature):
    V = 5000
    x = np.random.default_rng(1).standard_normal((1, 7, V)).astype(np.float32)
    x[0, 0, 4321] = np.inf
    x[0, 1, [5, 4000]] = np.inf
    x[0, 2, ::2] = -np.inf
    x[0, 3, 1::2] = np.nan
    x[0, 4] = -np.inf
    x[0, 5] = np.nan
    x[0, 6, :] = -3e38
    x[0, 6, 77] = 3e38
    d = torch.from_numpy(x).to(cuda_device)
    p = torch.empty_like(d)
    binding.mla_logits_to_probs(d, p, temperature=torch.tensor([temperature], device=cuda_device))
    got = p.cpu().numpy()
    for j in range(7):
        t = float(np.float32(temperature))
        want = otree.probabilities(x[0, j], t if t > 0 else 0.0)
        assert (np.abs(got[0, j] - want) <= (2.0 ** -16 + 14 * 2.0 ** -24 * (0 if t <= 0 or t != t else 10 / max(t, 1e-2))) * want + 1e-37).all(), j
    assert got[0, 0, 4321] == 1.0 and not got[0, 4].any() and not got[0, 5].any()


def test_lowest_of_equal_maxima(cuda_device):
    """Ties over blocks, warps and inside a vector; a bias that makes or breaks one."""
    V = 40000
    x = torch.zeros((4, 1, V), device=cuda_device)
    x[0, 0, [39999, 20001, 20000, 31]] = 2.0
    x[1, 0, [39999, 20001]] = 2.0
    x[2, 0, 30000] = 2.0
    p = torch.empty_like(x)
    binding.mla_logits_to_probs(x, p, temperature=torch.zeros(4, device=cuda_device),
                                bias_tokens=i32([[31], [5], [7], [-1]], cuda_device),
                                biases=torch.tensor([[-0.5], [2.0], [2.5], [9.0]], device=cuda_device))
    assert p.argmax(-1).flatten().tolist() == [20000, 5, 7, 0] and p.sum(-1).flatten().tolist() == [1.0] * 4


def test_the_grammar_hides_the_maximum(cuda_device):
    c = Case(31, 2, 1, 70000, penalties=False, tree=False, biases=0, grammar=0.0, dev=cuda_device)
    c.x[0, 0, 60000], c.x[1, 0, 3] = 60.0, 60.0
    c.allowed = np.zeros((2, 1, 70000), bool)
    c.allowed[0, 0, [1, 65000]] = True
    c.kw["allowed"] = torch.from_numpy(words(c.allowed)).to(cuda_device)
    c.temperature[:] = 1.0
    c.kw["temperature"] = torch.ones(2, device=cuda_device)
    got = c.run()
    c.check(got)
    assert not got[1].any() and np.count_nonzero(got[0]) == 2


def test_captured_and_on_two_streams(cuda_device):
    cs = [Case(41 + k, 2, 3, 6000, dev=cuda_device) for k in range(2)]
    xs, ps = [c.x.to(cuda_device) for c in cs], [torch.empty((2, 3, 6000), device=cuda_device) for _ in cs]
    streams = [torch.cuda.Stream(cuda_device) for _ in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for k in range(2):
            binding.mla_logits_to_probs(xs[k], ps[k], stream=streams[k], **cs[k].kw)
    torch.cuda.synchronize()
    for k in range(2):
        cs[k].check(ps[k].cpu().numpy())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.mla_logits_to_probs(xs[0], ps[0], **cs[0].kw)
    xs[0].copy_(xs[1])
    for k, t in cs[0].kw.items():
        t.copy_(cs[1].kw[k])
    graph.replay()
    torch.cuda.synchronize()
    cs[1].check(ps[0].cpu().numpy())


def test_refusals(cuda_device):
    dev, c = cuda_device, Case(51, 2, 3, 100, dev=cuda_device)
    x, p = c.x.to(dev), torch.empty((2, 3, 100), device=dev)
    binding.mla_logits_to_probs(x, p, **c.kw)
    for kw in (dict(probs=p[:1]), dict(probs=p.double()), dict(logits=x.half()), dict(probs=p.cpu()),
               dict(temperature=c.kw["temperature"][:1]), dict(temperature=c.kw["temperature"].double()), dict(node_tokens=None),
               dict(node_tokens=i32(np.zeros((2, 2)), dev)), dict(token_counts=i32(np.zeros((2, 99)), dev)),
               dict(prompt_mask=i32(np.zeros((2, 3)), dev)), dict(allowed=i32(np.zeros((2, 4)), dev)), dict(biases=None),
               dict(biases=torch.zeros(2, 4, device=dev)), dict(num_rows=i32([1], dev)), dict(repetition=torch.ones(2))):
        with pytest.raises(AssertionError):
            binding.mla_logits_to_probs(**{"logits": x, "probs": p, **c.kw, **kw})
    torch.cuda.synchronize()
