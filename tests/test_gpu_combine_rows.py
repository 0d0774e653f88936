"""The merge of a decode's pieces, many rows of few pieces (a warp per unit) and few rows of
many (a block per unit): both match the float64 oracle, for every cache type (GPU).

The worker count decides which merge a call takes (rows against CTAs), so the same
requests run through both; rows that are empty or bad keep out = 0, lse = -inf.
"""

import numpy as np
import pytest
import torch

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .e2m1_util import buffers, fill, reference
from .gpu_util import assert_close, bf16_tensor, gpu_decode, gpu_fill_cache, oracle_decode, oracle_fill_cache

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


@pytest.mark.parametrize("forks,groups,num_ctas", [(2, 14, 0), (8, 6, 0), (2, 14, 40)])
def test_forks_of_a_long_prefix_among_short_groups(cuda_device, forks, groups, num_ctas):
    """The forks of one group share 60 pages, each with as many pieces as the prefix has; the
    other groups share one page, so the call has more rows than can be of many pieces."""
    w = wl.prefix_shared(seed=330 + forks, groups=groups, forks=forks, prefix=3840, suffix_median=90.0,
                         suffix_max=200, num_heads=16)
    pages, ref_pages = fill(w, cuda_device)
    prefix = np.array([60] + [1] * (groups - 1), np.int32)
    w.seq_lens[forks:] = 65 + np.arange(w.batch - forks) * 11 % 150
    out, lse, ws = buffers(w.batch, 1, 16, cuda_device,
                           size=binding.mla_decode_grouped_workspace_size(w.batch, 1, 16, num_ctas))
    binding.mla_decode_grouped(bf16_tensor(w.q_bits, cuda_device), pages, torch.from_numpy(w.block_table).to(cuda_device),
                               torch.from_numpy(w.seq_lens).to(cuda_device), forks,
                               torch.from_numpy(prefix).to(cuda_device), w.sm_scale, w.kv_scale, out, lse, ws,
                               num_ctas=num_ctas)
    torch.cuda.synchronize()
    assert binding.read_device_status(ws) == 0
    assert_close(out.float().cpu().numpy(), lse.cpu().numpy(), *reference(w, ref_pages), what=f"{groups}x{forks}")
