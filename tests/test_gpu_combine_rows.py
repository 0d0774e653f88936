"""The merge of a decode's pieces, many rows of few pieces (a warp per unit) and few rows of
many (a block per unit): both match the float64 oracle, for every cache type (GPU).

The worker count decides which merge a call takes (rows against CTAs), so the same
requests run through both; rows that are empty or bad keep out = 0, lse = -inf.
"""

import numpy as np
import pytest

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .e2m1_util import fill, reference
from .gpu_util import assert_close, gpu_decode, gpu_fill_cache, oracle_decode, oracle_fill_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["e2m1", "e4m3", "bf16"])
@pytest.mark.parametrize("nq,num_ctas", [(1, 0), (4, 0), (1, 7), (2, 40), (2, 400)])
def test_both_merges_match_oracle(cuda_device, cache, nq, num_ctas):
    """A request of 60 pages among short ones: up to 60 pieces in one row, one in the others."""
    lengths = [3840] + [nq + (37 * i) % 130 for i in range(19)]
    w = wl.make_lengths_workload("merge", 300 + nq, lengths, num_heads=16, num_queries=nq)
    table, lens = w.block_table.copy(), w.seq_lens.copy()
    lens[5] = -1
    table[7, 0] = w.num_pages
    if cache == "e2m1":
        pages, ref_pages = fill(w, cuda_device)
        ref_out, ref_lse = reference(w, ref_pages)
    else:
        pages, ref_pages = gpu_fill_cache(w, cuda_device, cache), oracle_fill_cache(w, cache)
        ref_out, ref_lse = oracle_decode(w, ref_pages, cache)
    out, lse, ws = gpu_decode(w, pages, cuda_device, num_ctas=num_ctas, seq_lens=lens, block_table=table,
                              kv_scale=1.0 if cache == "bf16" else None)
    assert binding.read_device_status(ws) == binding.MLA_DEVICE_ERR_BAD_PAGE | binding.MLA_DEVICE_ERR_BAD_LENGTH
    good = [b for b in range(w.batch) if b not in (5, 7)]
    assert_close(out[good], lse[good], ref_out[good], ref_lse[good], what=f"{cache} Q={nq} G={num_ctas}")
    for b in (5, 7):
        assert (out[b] == 0).all() and np.isneginf(lse[b]).all()
