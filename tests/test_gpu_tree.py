"""mla_decode_tree against the float64 oracle (GPU).

Tolerance: the stated one of mla_decode (gpu_util.assert_close), whose arithmetic it has; a
row that sees nothing is exact (zeros, -inf).
"""

import random

import numpy as np
import pytest
import torch

from oracle import e4m3 as oe4m3
from oracle import tree as otree
from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .gpu_util import assert_close, bf16_tensor
from .tree_util import SCALE, Cache, chain, gpu_tree, i32, mask_tensor, queries, random_tree

pytestmark = pytest.mark.gpu

CACHES = ["e4m3", "e2m1", "bf16"]
NAN, INF = 0x7FC0, 0x7F80  # bfloat16 bits


def check(c, q_bits, masks, nodes, num_ctas=0, status=0):
    out, lse, ws = gpu_tree(c, q_bits, masks, nodes, num_ctas)
    n = [q_bits.shape[1]] * len(c.lens) if nodes is None else nodes
    ref_out, ref_lse = otree.decode(oe4m3.bf16_bits_to_f64(q_bits), c.entries(), masks, n, wl.SM_SCALE)
    empty = np.isneginf(ref_lse)
    assert np.isneginf(lse[empty]).all() and not out[empty].any()
    if not empty.all():
        assert_close(out[~empty], lse[~empty], ref_out[~empty], ref_lse[~empty], what=c.cache)
    assert binding.read_device_status(ws) == status
    return out, lse


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("N", [1, 2, 3, 5, 8, 13, 64])
def test_trees_of_every_size(cuda_device, cache, heads, N):
    """Rows that fill, half fill and overflow a tile; trees inside a page, over its border, alone in a request."""
    r = random.Random(N * heads)
    lens = [N, N + 1, N + 63, 64 + N // 2, 128, 300 + N]
    lens = [max(n, N) for n in lens]
    c = Cache(cache, lens, 7 * N + heads, cuda_device)
    check(c, queries(N, len(lens), N, heads), [random_tree(r, N) for _ in lens], None)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("num_ctas", [1, 3, 0, 400])
@pytest.mark.parametrize("heads,N", [(16, 7), (32, 5), (64, 6)])
def test_ragged_nodes_and_splits(cuda_device, cache, num_ctas, heads, N):
    r = random.Random(num_ctas)
    nodes = [0, 1, N, N - 1, 2, N, 3, 0]
    lens = [500, 1, N, 64, 130, 1000, 65, 0]
    c = Cache(cache, lens, 11 + num_ctas, cuda_device)
    masks = [random_tree(r, N) for _ in lens]
    check(c, queries(3, len(lens), N, heads), masks, nodes, num_ctas)


@pytest.mark.parametrize("cache", CACHES)
def test_any_set_of_nodes(cuda_device, cache):
    """Masks that are no tree's: nothing at all, later nodes only, nodes that the request does not have."""
    N, nodes, lens = 9, [9, 5, 9], [9, 70, 256]
    full = (1 << 64) - 1
    masks = [[0, 1 << 8, full, 0, 3, 1 << 1, 0x155, 1 << 63, 0],
             [full - 0x1F, 1 << 4, 0, full, 1, 0, 0, full, 1],
             [1 << 2, 0, full, 1, 1 << 7, 0x1FF, 0, 1 << 8, 1 << 0]]
    c = Cache(cache, lens, 21, cuda_device)
    for heads in (16, 64):
        out, lse = check(c, queries(5, 3, N, heads), masks, nodes)
        assert np.isneginf(lse[0, [0, 3, 7, 8]]).all()  # no context, no visible node
        assert np.isfinite(lse[1, :5]).all() and np.isneginf(lse[1, 5:]).all()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("heads", [16, 64])
def test_a_chain_is_mla_decode(cuda_device, cache, heads):
    """Causal drafts as a chain: mla_decode's results within both calls' tolerance."""
    N, lens = 4, [4, 66, 320, 1000]
    c, q = Cache(cache, lens, 31, cuda_device), queries(6, 4, N, heads)
    out, lse, _ = gpu_tree(c, q, [chain(N)] * 4)
    a = torch.empty((4, N, heads, 512), dtype=torch.bfloat16, device=cuda_device)
    l = torch.empty((4, N, heads), device=cuda_device)
    ws = torch.zeros(binding.mla_decode_workspace_size(4, N, heads), dtype=torch.uint8, device=cuda_device)
    binding.mla_decode(bf16_tensor(q, cuda_device), c.pool, i32(c.table, cuda_device), i32(lens, cuda_device), wl.SM_SCALE,
                       SCALE[cache], a, l, ws)
    a = a.float().cpu().numpy()
    assert np.abs(out - a).max() <= 2 * (1e-2 * np.abs(a).max() + 1e-3)
    assert np.abs(lse - l.cpu().numpy()).max() <= 2e-3


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("dim", [0, 300, 511, 540])
def test_nan_in_a_node_reaches_the_rows_that_see_it(cuda_device, cache, bad, dim):
    """And no others, in its tile or another. (The two 8- and 4-bit caches saturate infinities.)"""
    N, heads, lens, nodes = 6, 32, [70, 6, 128], [6, 6, 4]
    masks = [[1, 3, 5, 11, 21, 35]] * 3  # 0-1-3, 0-2-4, 1-5
    c, q = Cache(cache, lens, 41, cuda_device), queries(7, 3, N, heads)
    ref_out, ref_lse = otree.decode(oe4m3.bf16_bits_to_f64(q), c.entries(), masks, nodes, wl.SM_SCALE)
    row = np.zeros((1, 576), np.uint16)
    row[0, dim] = bad
    for b, n in zip(range(3), nodes):
        c.put(b, [lens[b] - n + 1], row)  # node 1
    out, lse, _ = gpu_tree(c, q, masks, nodes)
    see = np.array([[j < n and m >> 1 & 1 for j, m in enumerate(ms)] for ms, n in zip(masks, nodes)], bool)
    live = np.array([[j < n for j in range(N)] for n in nodes])
    if bad == NAN:
        assert np.isnan(lse[see]).all() and np.isnan(out[see]).all()
    assert_close(out[live & ~see], lse[live & ~see], ref_out[live & ~see], ref_lse[live & ~see], what=cache)
    assert np.isneginf(lse[~live]).all() and not out[~live].any()


@pytest.mark.parametrize("cache", CACHES)
def test_nan_in_a_query_row_and_behind_the_last_node(cuda_device, cache):
    N, heads, lens, nodes = 5, 16, [90, 200], [3, 5]
    masks = [chain(N)] * 2
    c, q = Cache(cache, lens, 51, cuda_device), queries(8, 2, N, heads)
    ref_out, ref_lse = otree.decode(oe4m3.bf16_bits_to_f64(q), c.entries(), masks, nodes, wl.SM_SCALE)
    q[0, 3:] = NAN          # rows of nodes that the request does not have
    q[1, 2, 5, 100] = NAN   # one head of one node
    row = np.full((1, 576), NAN, np.uint16)
    for b in range(2):      # tokens behind the last one
        for t in range(lens[b], -(-lens[b] // 64) * 64):
            c.put(b, [t], row)
    out, lse, _ = gpu_tree(c, q, masks, nodes)
    assert np.isnan(lse[1, 2, 5]) and np.isnan(out[1, 2, 5]).all()
    assert np.isneginf(lse[0, 3:]).all() and not out[0, 3:].any()
    good = np.ones((2, N, heads), bool)
    good[0, 3:] = False
    good[1, 2, 5] = False
    assert_close(out[good], lse[good], ref_out[good], ref_lse[good], what=cache)


@pytest.mark.parametrize("cache", CACHES)
def test_bad_requests_and_pages(cuda_device, cache):
    """Bad lengths, node counts and page ids: zeros, -inf and the status word; the others stand."""
    N, heads, lens = 4, 32, [200, 100, 100, 100, 130]
    c, q, masks = Cache(cache, lens, 61, cuda_device), queries(9, 5, N, heads), [chain(N)] * 5
    nodes, seq_lens = [4, 5, -1, 4, 4], [200, 100, 100, 3, 130]
    table = c.table.copy()
    table[4, 1] = c.num_pages
    out, lse, ws = gpu_tree(c, q, masks, nodes, seq_lens=seq_lens, table=table)
    ref_out, ref_lse = otree.decode(oe4m3.bf16_bits_to_f64(q[:1]), c.entries()[:1], masks[:1], [4], wl.SM_SCALE)
    assert_close(out[:1], lse[:1], ref_out, ref_lse, what=cache)
    assert np.isneginf(lse[1:]).all() and not out[1:].any()
    assert binding.read_device_status(ws) == binding.MLA_DEVICE_ERR_BAD_LENGTH | binding.MLA_DEVICE_ERR_BAD_PAGE
    seq_lens[0] = 64 * c.table.shape[1] + 1
    _, lse, ws = gpu_tree(c, q, masks, [4] * 5, seq_lens=seq_lens, table=table)
    assert np.isneginf(lse[0]).all()


@pytest.mark.parametrize("cache", CACHES)
def test_scores_far_apart(cuda_device, cache):
    """Pages whose maxima rise and fall by hundreds: the running maximum follows for every row by itself."""
    N, heads, lens = 8, 64, [900, 2000]
    c, q = Cache(cache, lens, 71, cuda_device), queries(10, 2, N, heads)
    q = wl.f32_to_bf16_bits(oe4m3.bf16_bits_to_f64(q).astype(np.float32) * 30.0)
    check(c, q, [random_tree(random.Random(1), N)] * 2, None)


def test_long_context_and_one_row(cuda_device):
    """One request over every SM, and the same rows one node at a time."""
    c, N = Cache("e4m3", [20000], 81, cuda_device), 12
    q, masks = queries(11, 1, N, 64), [random_tree(random.Random(2), N)]
    check(c, q, masks, None)


@pytest.mark.parametrize("cache", CACHES)
def test_captured_streams_and_workspace(cuda_device, cache):
    """Captured once, replayed with other inputs; two streams with a workspace each; one workspace call after call."""
    dev, N, heads = cuda_device, 6, 32
    c = Cache(cache, [300, 77], 91, dev)
    d = {"table": i32(c.table, dev), "lens": i32(c.lens, dev), "nodes": i32([6, 2], dev)}
    sets = []
    for k in range(2):
        r = random.Random(k)
        sets.append((queries(20 + k, 2, N, heads), [random_tree(r, N), random_tree(r, N)]))
    size = binding.mla_decode_tree_workspace_size(2, N, heads)
    run = []
    for k in range(2):
        q, m = bf16_tensor(sets[k][0], dev), mask_tensor(sets[k][1], dev)
        out, lse = torch.empty((2, N, heads, 512), dtype=torch.bfloat16, device=dev), torch.empty((2, N, heads), device=dev)
        run.append((q, m, out, lse, torch.zeros(size, dtype=torch.uint8, device=dev)))

    def call(k, stream=None):
        q, m, out, lse, ws = run[k]
        binding.mla_decode_tree(q, c.pool, d["table"], d["lens"], m, wl.SM_SCALE, SCALE[cache], out, lse, ws,
                                num_nodes=d["nodes"], stream=stream)

    want = []
    for q, m in sets:
        want.append(otree.decode(oe4m3.bf16_bits_to_f64(q), c.entries(), m, [6, 2], wl.SM_SCALE))

    def good(k, out, lse):
        out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
        live = np.isfinite(want[k][1])
        assert_close(out[live], lse[live], want[k][0][live], want[k][1][live], what=f"set {k}")
        assert np.isneginf(lse[~live]).all() and not out[~live].any()

    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for k in range(2):
            call(k, streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        good(k, run[k][2], run[k][3])
    call(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for k in (1, 0, 1):
        run[0][0].copy_(bf16_tensor(sets[k][0], dev))
        run[0][1].copy_(mask_tensor(sets[k][1], dev))
        run[0][2].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        good(k, run[0][2], run[0][3])


def test_refusals(cuda_device):
    dev, c = cuda_device, Cache("e4m3", [70, 80], 95, cuda_device)
    N, heads = 3, 16
    good = dict(q=torch.zeros((2, N, heads, 576), dtype=torch.bfloat16, device=dev), kv_pages=c.pool, block_table=i32(c.table, dev),
                seq_lens=i32(c.lens, dev), tree_mask=mask_tensor([chain(N)] * 2, dev), sm_scale=0.1, kv_scale=1.0,
                out=torch.zeros((2, N, heads, 512), dtype=torch.bfloat16, device=dev), lse=torch.zeros((2, N, heads), device=dev),
                workspace=torch.zeros(binding.mla_decode_tree_workspace_size(2, N, heads), dtype=torch.uint8, device=dev))
    binding.mla_decode_tree(**good)
    for k, v in (("tree_mask", good["tree_mask"].int()), ("tree_mask", good["tree_mask"][:1]), ("tree_mask", good["tree_mask"].cpu()),
                 ("tree_mask", good["tree_mask"].t().contiguous().t()), ("num_nodes", i32([1], dev)),
                 ("num_nodes", torch.ones(2, dtype=torch.int64, device=dev)), ("num_nodes", torch.ones(2, dtype=torch.int32)),
                 ("q", good["q"].float()), ("out", good["out"][:, :2])):
        with pytest.raises(AssertionError):
            binding.mla_decode_tree(**{**good, k: v})
    for k, v in (("workspace", good["workspace"][:-256]), ("kv_scale", 0.0), ("sm_scale", float("nan"))):
        with pytest.raises(binding.MlaError):
            binding.mla_decode_tree(**{**good, k: v})
    torch.cuda.synchronize()
