"""NaN in the cache or in a query reaches every row that sees it, whatever the cache's type and
the split, and no other row (GPU)."""

import numpy as np
import pytest
import torch

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .e2m1_util import append, buffers, fill, reference
from .gpu_util import assert_close, bf16_tensor, gpu_decode, gpu_fill_cache, oracle_decode, oracle_fill_cache

pytestmark = pytest.mark.gpu

CACHES = ["e2m1", "e4m3", "bf16", "f16 operands"]
NAN = 0x7FC0  # bfloat16 bits


def _caches(w, cache, dev):
    """The device's pages, the oracle's (out, lse), and what gpu_decode takes for the type."""
    if cache == "e2m1":
        pages, ref = fill(w, dev)
        return pages, reference(w, ref), {}
    dtype = "bf16" if cache == "bf16" else "e4m3"
    ref = oracle_decode(w, oracle_fill_cache(w, dtype), dtype)
    kw = {"kv_scale": 1.0} if dtype == "bf16" else {}
    return gpu_fill_cache(w, dev, dtype), ref, {**kw, "f16_operands": cache == "f16 operands"}


def _put_nan(w, pages, cache, request, token, dev):
    bits = np.zeros((1, 576), np.uint16)
    bits[0, 100] = NAN
    slot = int(w.block_table[request, token // 64]) * 64 + token % 64
    append(pages, bits, [slot], 1.0 if cache == "bf16" else w.kv_scale, dev)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("num_ctas", [1, 3, 0, 400])
@pytest.mark.parametrize("token", [0, 69, 1999])
def test_nan_token_makes_its_rows_nan(cuda_device, cache, num_ctas, token):
    w = wl.make_lengths_workload("nan", 500, [2000, 150], num_heads=16)
    pages, (ref_out, ref_lse), kw = _caches(w, cache, cuda_device)
    _put_nan(w, pages, cache, 0, token, cuda_device)
    out, lse, ws = gpu_decode(w, pages, cuda_device, num_ctas=num_ctas, **kw)
    assert binding.read_device_status(ws) == 0
    assert np.isnan(lse[0]).all() and np.isnan(out[0]).all()
    assert_close(out[1:], lse[1:], ref_out[1:], ref_lse[1:], what="the other request")


@pytest.mark.parametrize("cache", CACHES)
def test_a_draft_before_the_nan_token_stands(cuda_device, cache):
    """The last draft's own entry is NaN: only that draft sees it."""
    w = wl.make_lengths_workload("nan", 501, [300, 257], num_heads=32, num_queries=3)
    pages, (ref_out, ref_lse), kw = _caches(w, cache, cuda_device)
    _put_nan(w, pages, cache, 0, 299, cuda_device)
    _put_nan(w, pages, cache, 1, 256, cuda_device)  # the first token of a page
    out, lse, _ = gpu_decode(w, pages, cuda_device, **kw)
    assert np.isnan(lse[:, 2]).all() and np.isnan(out[:, 2]).all()
    assert_close(out[:, :2], lse[:, :2], ref_out[:, :2], ref_lse[:, :2], what="drafts before it")


@pytest.mark.parametrize("cache", CACHES)
def test_nan_in_a_query_head(cuda_device, cache):
    """Only that head's row is NaN."""
    w = wl.make_lengths_workload("nan", 502, [2000, 150], num_heads=16)
    pages, (ref_out, ref_lse), kw = _caches(w, cache, cuda_device)
    q = w.q_bits.copy()
    q[0, 0, 5, 33] = NAN
    out, lse, _ = gpu_decode(w, pages, cuda_device, q_bits=q, **kw)
    assert np.isnan(lse[0, 0, 5]) and np.isnan(out[0, 0, 5]).all()
    rest = [h for h in range(16) if h != 5]
    assert_close(out[0, 0, rest], lse[0, 0, rest], ref_out[0, 0, rest], ref_lse[0, 0, rest], what="the other heads")
    assert_close(out[1], lse[1], ref_out[1], ref_lse[1], what="the other request")


@pytest.mark.parametrize("cache", CACHES)
def test_nan_behind_the_last_token_is_not_seen(cuda_device, cache):
    w = wl.make_lengths_workload("nan", 503, [200, 70, 1], num_heads=16)
    pages, (ref_out, ref_lse), kw = _caches(w, cache, cuda_device)
    for b, n in enumerate(w.seq_lens):
        for token in range(int(n), -(-int(n) // 64) * 64):
            _put_nan(w, pages, cache, b, token, cuda_device)
    out, lse, _ = gpu_decode(w, pages, cuda_device, **kw)
    assert_close(out, lse, ref_out, ref_lse, what=cache)


@pytest.mark.parametrize("cache", ["e2m1", "e4m3"])
@pytest.mark.parametrize("shared", [True, False])
def test_grouped(cuda_device, cache, shared):
    """In the shared prefix for every fork of the group, behind it for its own request."""
    w = wl.prefix_shared(seed=504, groups=2, forks=3, prefix=640, suffix_median=150.0, suffix_max=700, num_heads=16)
    rows, token = ((0, 1, 2), 10) if shared else ((1,), int(w.seq_lens[1]) - 1)
    pages, (ref_out, ref_lse), _ = _caches(w, cache, cuda_device)
    _put_nan(w, pages, cache, 1, token, cuda_device)
    out, lse, ws = buffers(w.batch, 1, 16, cuda_device,
                           binding.mla_decode_grouped_workspace_size(w.batch, 1, 16, 0))
    binding.mla_decode_grouped(bf16_tensor(w.q_bits, cuda_device), pages,
                               torch.from_numpy(w.block_table).to(cuda_device),
                               torch.from_numpy(w.seq_lens).to(cuda_device), 3,
                               torch.from_numpy(w.extra["prefix_pages"]).to(cuda_device), w.sm_scale, w.kv_scale,
                               out, lse, ws)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    hit = list(rows)
    assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    rest = [b for b in range(w.batch) if b not in rows]
    assert_close(out[rest], lse[rest], ref_out[rest], ref_lse[rest], what="the other requests")
