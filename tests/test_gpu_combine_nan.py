"""mla_decode_combine of partials with a NaN: a decode's NaN row, held by one of several shards,
makes the merged row NaN (GPU)."""

import numpy as np
import pytest
import torch

from paged_mla_decode_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("num_parts,at", [(1, 0), (2, 1), (7, 3), (300, 299)])
@pytest.mark.parametrize("others", ["finite", "empty"])
def test_nan_part(cuda_device, num_parts, at, others):
    rng = np.random.default_rng(530 + num_parts)
    part_out = rng.standard_normal((num_parts, 4, 512)).astype(np.float32)
    part_lse = rng.standard_normal((num_parts, 4)).astype(np.float32)
    if others == "empty":
        part_lse[:, 1:3] = -np.inf
    part_out[at, 1], part_lse[at, 1] = np.nan, np.nan   # as mla_decode gives it
    part_lse[at, 2] = np.nan
    out = torch.empty((4, 512), dtype=torch.bfloat16, device=cuda_device)
    lse = torch.empty(4, dtype=torch.float32, device=cuda_device)
    binding.mla_decode_combine(torch.from_numpy(part_out).to(cuda_device), torch.from_numpy(part_lse).to(cuda_device),
                               out, lse)
    assert torch.isnan(out[1:3]).all() and torch.isnan(lse[1:3]).all()
    assert torch.isfinite(out[[0, 3]]).all() and torch.isfinite(lse[[0, 3]]).all()
