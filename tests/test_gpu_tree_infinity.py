"""mla_decode_tree with a NaN or an infinity in a cached entry, of the context or a node's (GPU).

Only a bf16 cache holds infinities. A row's score of such an entry is +-inf by the sign of its query
there: with +inf the row is NaN; with -inf the entry has no weight, so the reference is the oracle's
without it, at mla_decode's stated tolerance (gpu_util.assert_close), but for the latent dim at which a
context token holds the infinity, where 0 * inf is allowed.
"""

import numpy as np
import pytest

from oracle import e4m3 as oe4m3
from oracle import tree as otree
from paged_mla_decode_gb300 import workloads as wl

from .gpu_util import assert_close
from .tree_util import Cache, chain, gpu_tree, queries

pytestmark = pytest.mark.gpu

NAN, INF = 0x7FC0, 0x7F80
N, HEADS, LENS, NODES = 5, 32, [200, 70, 300], [5, 5, 3]
MASKS = [chain(N)] * 3


@pytest.mark.parametrize("num_ctas", [0, 1])
@pytest.mark.parametrize("dim", [0, 300, 511, 540])
@pytest.mark.parametrize("cache", ["e4m3", "e2m1", "bf16"])
def test_nan_in_a_context_token(cuda_device, cache, dim, num_ctas):
    """Every row of that request sees it; the other requests stand."""
    c, q = Cache(cache, LENS, 43, cuda_device), queries(17, 3, N, HEADS)
    ref_out, ref_lse = otree.decode(oe4m3.bf16_bits_to_f64(q), c.entries(), MASKS, NODES, wl.SM_SCALE)
    row = np.zeros((1, 576), np.uint16)
    row[0, dim] = NAN
    c.put(0, [66], row)
    c.put(2, [LENS[2] - NODES[2] - 1], row)  # just before the nodes, in a page with them
    out, lse, _ = gpu_tree(c, q, MASKS, NODES, num_ctas)
    assert np.isnan(out[0]).all() and np.isnan(lse[0]).all()
    assert np.isnan(out[2, :3]).all() and np.isnan(lse[2, :3]).all()
    assert np.isneginf(lse[2, 3:]).all() and not out[2, 3:].any()
    assert_close(out[1], lse[1], ref_out[1], ref_lse[1], what=cache)


@pytest.mark.parametrize("num_ctas", [0, 1])
@pytest.mark.parametrize("dim", [0, 300, 511, 540])
@pytest.mark.parametrize("where", ["context", "before the nodes", "node"])
def test_infinity(cuda_device, where, dim, num_ctas):
    c, q = Cache("bf16", LENS, 44, cuda_device), queries(18, 3, N, HEADS)
    values = oe4m3.bf16_bits_to_f64(q)
    assert (values[..., dim] != 0).all()
    at = [{"context": 5, "before the nodes": n - k - 1, "node": n - k + 1}[where] for n, k in zip(LENS, NODES)]
    row = np.zeros((1, 576), np.uint16)
    row[0, dim] = INF
    for b in range(3):
        c.put(b, [at[b]], row)
    masks, nodes, entries = MASKS, NODES, c.entries()
    if where == "node":
        masks = [[m & ~2 for m in ms] for ms in MASKS]
        sees = np.array([[j < k and m >> 1 & 1 for j, m in enumerate(ms)] for ms, k in zip(MASKS, NODES)], bool)
    else:
        entries = [np.delete(e, t, 0) for e, t in zip(entries, at)]
        sees = np.array([[j < k for j in range(N)] for k in NODES], bool)
    ref_out, ref_lse = otree.decode(values, entries, masks, nodes, wl.SM_SCALE)
    out, lse, _ = gpu_tree(c, q, MASKS, NODES, num_ctas)
    nan = sees[..., None] & (values[..., dim] > 0)
    empty = np.isneginf(ref_lse)
    assert nan.any() and (sees[..., None] & ~nan).any()
    assert np.isnan(out[nan]).all() and np.isnan(lse[nan]).all()
    assert np.isneginf(lse[empty]).all() and not out[empty].any()
    good = ~nan & ~empty
    assert np.isfinite(lse[good]).all()
    if where != "node" and dim < 512:
        ok = np.isnan(out[..., dim]) | (np.abs(out[..., dim] - ref_out[..., dim]) <= 1e-2 * np.abs(ref_out[good]).max() + 1e-3)
        assert ok[good].all()
        out[..., dim] = ref_out[..., dim]
    assert_close(out[good], lse[good], ref_out[good], ref_lse[good], what=where)
