"""mla_kv_compact moves stored entries bit for bit, and nothing else (GPU)."""

import numpy as np
import pytest
import torch

from oracle import tree as otree
from paged_mla_decode_gb300 import binding

from .tree_util import i32

pytestmark = pytest.mark.gpu

CACHES = ["e4m3", "e2m1", "bf16"]


def rows_of(pool, cache):
    """A layer's pages [pages, ...] as bytes [slots, entry bytes], whatever the layout."""
    if cache != "e2m1":
        return pool.reshape(pool.shape[0] * 64, -1)
    codes = pool[:, :18432].reshape(-1, 18, 64, 16).transpose(0, 2, 1, 3).reshape(-1, 288)
    return np.concatenate([codes, pool[:, 18432:].reshape(-1, 9, 64).transpose(0, 2, 1).reshape(-1, 9)], 1)


def random_pool(rng, cache, layers, pages):
    size = {"e4m3": 36864, "e2m1": 19008, "bf16": 73728}[cache]
    return rng.integers(0, 256, (layers, pages, size)).astype(np.uint8)


def as_tensor(raw, cache, dev):
    t = torch.from_numpy(raw).to(dev)
    if cache == "e4m3":
        return t.view(*raw.shape[:2], 64, 576)
    return t.view(torch.bfloat16).view(*raw.shape[:2], 64, 576) if cache == "bf16" else t


def expected(raw, cache, table, lens, path, accepted):
    want = []
    pages, N = raw.shape[1], len(path[0])
    for layer in range(raw.shape[0]):
        rows = rows_of(raw[layer], cache).copy()
        old = rows.copy()
        for b, (L, a) in enumerate(zip(lens, accepted)):
            if a < 1 or a >= N or L < a + 1 or L > 64 * len(table[b]):
                continue
            for i in range(1, a + 1):
                src, dst = L - a - 1 + path[b][i], L - a - 1 + i
                if not 0 <= path[b][i] < N or src >= 64 * len(table[b]):
                    continue
                ps, pd = table[b][src // 64], table[b][dst // 64]
                if 0 <= ps < pages and 0 <= pd < pages:
                    rows[pd * 64 + dst % 64] = old[ps * 64 + src % 64]
        want.append(rows)
    return want


def check(raw, cache, table, lens, path, accepted, dev, one=False):
    pool = as_tensor(raw, cache, dev)
    binding.mla_kv_compact(pool[0] if one else pool, i32(table, dev), i32(lens, dev), i32(path, dev), i32(accepted, dev))
    torch.cuda.synchronize()
    got = pool.view(torch.uint8).cpu().numpy().reshape(raw.shape)
    for layer, want in enumerate(expected(raw, cache, table, lens, path, accepted)):
        assert np.array_equal(rows_of(got[layer], cache), want), layer


def requests(rng, B, N, width, pages):
    table = np.full((B, width), -1)
    perm = rng.permutation(pages)
    for b in range(B):
        table[b] = perm[b * width:(b + 1) * width]
    path, accepted, lens = np.full((B, N), -1), np.zeros(B, int), np.zeros(B, int)
    for b in range(B):
        a = int(rng.integers(0, N))
        accepted[b] = a
        path[b, :a + 1] = [0] + sorted(rng.choice(np.arange(1, N), a, replace=False))
        lens[b] = int(rng.integers(0, width * 64 - N + 1)) + a + 1
    return table, lens, path, accepted


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("N", [2, 3, 8, 31, 64])
@pytest.mark.parametrize("layers", [1, 2, 61])
def test_kept_nodes_of_every_layer(cuda_device, cache, N, layers):
    rng = np.random.default_rng(N * layers)
    B = 2 if layers == 61 else 20
    table, lens, path, accepted = requests(rng, B, N, 3, 3 * B + 2)
    raw = random_pool(rng, cache, layers, 3 * B + 2)
    check(raw, cache, table, lens, path, accepted, cuda_device, one=layers == 1)


@pytest.mark.parametrize("cache", CACHES)
def test_all_nodes_over_a_page_border(cuda_device, cache):
    """63 moves of one request, every entry read and overwritten; a path that turns around."""
    rng = np.random.default_rng(1)
    raw = random_pool(rng, cache, 2, 6)
    path = np.zeros((2, 64), int)
    path[0, 1:] = np.arange(63, 0, -1)
    path[1, 1:] = np.roll(np.arange(1, 64), 1)
    check(raw, cache, [[4, 1, 3], [0, 2, 5]], [101, 192], path, [63, 63], cuda_device)


@pytest.mark.parametrize("cache", CACHES)
def test_what_is_left_alone(cuda_device, cache):
    """Nothing kept, failed requests, bad counts and lengths, paths and pages out of range."""
    rng = np.random.default_rng(2)
    raw = random_pool(rng, cache, 1, 20)
    N = 5
    table = rng.permutation(20).reshape(10, 2)
    table[7, 1] = 20
    table[8, 0] = -1
    good = [0, 2, 4, -1, -1]
    path = [good, good, good, good, good, [0, -1, 5, 4, -1], [0, 4, 2, 3, 1], [0, 2, 4, -1, -1], [0, 2, 4, -1, -1], [0, 3, 4, -1, -1]]
    accepted = [0, -1, 5, 2, 2, 3, 4, 2, 2, 2]
    lens = [50, -1, 50, 2, 129, 60, 70, 66, 66, 128]
    check(raw, cache, table, lens, path, accepted, cuda_device, one=True)


def test_layers_apart_and_far(cuda_device):
    """Padded layers; offsets beyond 32 bits."""
    dev, rng = cuda_device, np.random.default_rng(3)
    raw = random_pool(rng, "e4m3", 3, 6)
    wide = torch.full((3, 9, 64, 576), 7, dtype=torch.uint8, device=dev)
    wide[:, :6] = as_tensor(raw, "e4m3", dev)
    table, lens, path, accepted = requests(rng, 2, 9, 3, 6)
    binding.mla_kv_compact(wide[:, :6], i32(table, dev), i32(lens, dev), i32(path, dev), i32(accepted, dev))
    for layer, want in enumerate(expected(raw, "e4m3", table, lens, path, accepted)):
        assert np.array_equal(rows_of(wide[layer, :6].cpu().numpy(), "e4m3"), want)
    assert (wide[:, 6:] == 7).all()
    del wide
    pages = (1 << 32) // 36864 + 10
    far = torch.zeros((2, pages, 64, 576), dtype=torch.uint8, device=dev)
    raw = random_pool(rng, "e4m3", 2, 2)
    far[:, -2:] = as_tensor(raw, "e4m3", dev)
    args = [[0, 3, 5, 8], [0, 9, 8, 7]]
    binding.mla_kv_compact(far, i32([[pages - 1, pages - 2]] * 1, dev), i32([66], dev), i32(args[:1], dev), i32([3], dev))
    for layer, want in enumerate(expected(raw, "e4m3", [[1, 0]], [66], args[:1], [3])):
        assert np.array_equal(rows_of(far[layer, -2:].cpu().numpy(), "e4m3"), want)
    assert not far[:, :-2].any()


def test_oracle_agrees(cuda_device):
    rng = np.random.default_rng(4)
    raw = random_pool(rng, "bf16", 1, 2)
    rows = rows_of(raw[0], "bf16")
    assert np.array_equal(expected(raw, "bf16", [[0, 1]], [70], [[0, 2, 5, 6]], [3])[0],
                          otree.compact(rows, 66, [0, 2, 5, 6], 3)) is False  # node 5 and 6 are outside four nodes
    path = [[0, 2, 5, 6, -1, -1, -1]]
    assert np.array_equal(expected(raw, "bf16", [[0, 1]], [70], path, [3])[0], otree.compact(rows, 66, path[0], 3))
    check(raw, "bf16", [[0, 1]], [70], path, [3], cuda_device)


def test_refusals(cuda_device):
    dev = cuda_device
    pool = torch.zeros((2, 4, 64, 576), dtype=torch.uint8, device=dev)
    t, l, p, a = i32([[0, 1]], dev), i32([5], dev), i32([[0, 1, 2]], dev), i32([1], dev)
    binding.mla_kv_compact(pool, t, l, p, a)
    for bad in ((pool[..., :575], t, l, p, a), (pool.transpose(1, 2), t, l, p, a), (pool[:0], t, l, p, a), (pool, t[0], l, p, a),
                (pool, t, l.long(), p, a), (pool, t, l, p[0], a), (pool, t, l, p, a.cpu()), (pool.cpu(), t, l, p, a),
                (pool, t, torch.cat([l, l]), p, a)):
        with pytest.raises(AssertionError):
            binding.mla_kv_compact(*bad)
    torch.cuda.synchronize()
