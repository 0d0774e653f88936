"""The two merges on either side of the rule between them: a block per unit while the rows are no
more than the worker CTAs' ranges can cut into more than 16 pieces (CTAs / 15; twice that in a
grouped decode), a warp per unit and blocks for the rows of many pieces beyond (GPU)."""

import numpy as np
import pytest
import torch

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .e2m1_util import buffers, fill, reference
from .gpu_util import assert_close, bf16_tensor, gpu_decode, gpu_fill_cache, oracle_decode, oracle_fill_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["e2m1", "e4m3", "bf16"])
@pytest.mark.parametrize("num_ctas", [400, 300, 299, 315, 314])
@pytest.mark.parametrize("long", [1, 4])
def test_rows_at_the_border(cuda_device, cache, num_ctas, long):
    """20 rows (and 21 with an empty one): blocks from 300 (315) CTAs on, warps below. `long` of
    them have 60 pages, the others up to three."""
    lengths = [3840] * long + [1 + (37 * i) % 130 for i in range(20 - long)]
    w = wl.make_lengths_workload("border", 560 + long, lengths, num_heads=16)
    table, lens, q = w.block_table, w.seq_lens, w.q_bits
    if num_ctas in (315, 314):
        table, lens = np.concatenate([table, table[:1]]), np.concatenate([lens, [0]]).astype(np.int32)
        q = np.concatenate([q, q[:1]])
    if cache == "e2m1":
        pages, ref_pages = fill(w, cuda_device)
        ref = reference(w, ref_pages)
    else:
        pages, ref = gpu_fill_cache(w, cuda_device, cache), oracle_decode(w, oracle_fill_cache(w, cache), cache)
    out, lse, _ = gpu_decode(w, pages, cuda_device, num_ctas=num_ctas, seq_lens=lens, block_table=table, q_bits=q,
                             kv_scale=1.0 if cache == "bf16" else None)
    assert_close(out[:20], lse[:20], *ref, what=f"{cache} G={num_ctas}")
    assert (out[20:] == 0).all() and np.isneginf(lse[20:]).all()


@pytest.mark.parametrize("num_ctas", [150, 149, 152])
@pytest.mark.parametrize("forks", [2, 10])
def test_grouped_rows_at_the_border(cuda_device, num_ctas, forks):
    """20 rows of a grouped decode: blocks from 150 CTAs on, warps below."""
    w = wl.prefix_shared(seed=565 + forks, groups=20 // forks, forks=forks, prefix=3840, suffix_median=90.0,
                         suffix_max=200, num_heads=16)
    pages, ref_pages = fill(w, cuda_device)
    out, lse, ws = buffers(20, 1, 16, cuda_device, size=binding.mla_decode_grouped_workspace_size(20, 1, 16, num_ctas))
    binding.mla_decode_grouped(bf16_tensor(w.q_bits, cuda_device), pages, torch.from_numpy(w.block_table).to(cuda_device),
                               torch.from_numpy(w.seq_lens).to(cuda_device), forks,
                               torch.from_numpy(w.extra["prefix_pages"]).to(cuda_device), w.sm_scale, w.kv_scale, out, lse,
                               ws, num_ctas=num_ctas)
    assert binding.read_device_status(ws) == 0
    assert_close(out.float().cpu().numpy(), lse.cpu().numpy(), *reference(w, ref_pages), what=f"{forks} forks")
