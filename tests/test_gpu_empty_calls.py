"""Decodes without a single page, each followed at once by a full one in the same workspace (GPU).

The empty call's kernels must all have ended before the next call's write the workspace: the full call's
results are those that it gives in a workspace of its own, bit for bit.
"""

import numpy as np
import pytest
import torch

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .tree_util import SCALE, Cache, chain, i32, mask_tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call,cache", [("mla_decode", "e4m3"), ("mla_decode", "e2m1"), ("mla_decode", "bf16"),
                                        ("mla_decode_grouped", "e4m3"), ("mla_decode_grouped", "e2m1"),
                                        ("mla_decode_tree", "e4m3"), ("mla_decode_tree", "e2m1"), ("mla_decode_tree", "bf16")])
def test_empty_then_full(cuda_device, call, cache):
    dev, B, N, H = cuda_device, 96, 4, 64
    rng = np.random.default_rng(6)
    c = Cache(cache, rng.integers(4, 200, B).tolist(), 66, dev)
    g = torch.Generator(device=dev).manual_seed(7)
    q = torch.randn(B, N, H, 576, generator=g, device=dev).bfloat16()
    other = torch.full_like(q, 100.0)
    table, lens, none = i32(c.table, dev), i32(c.lens, dev), i32([0] * B, dev)
    kw = {"mla_decode": {}, "mla_decode_grouped": dict(forks=2, prefix_pages=i32([0] * (B // 2), dev)),
          "mla_decode_tree": dict(tree_mask=mask_tensor([chain(N)] * B, dev))}[call]
    none_kw = dict(kw, num_nodes=i32([0] * B, dev)) if call == "mla_decode_tree" else kw
    size = getattr(binding, call + "_workspace_size")(B, N, H)
    out, lse = torch.empty(B, N, H, 512, dtype=torch.bfloat16, device=dev), torch.empty(B, N, H, device=dev)
    e_out, e_lse = torch.empty_like(out), torch.empty_like(lse)

    def run(q, lens, out, lse, ws, kw):
        getattr(binding, call)(q=q, kv_pages=c.pool, block_table=table, seq_lens=lens, sm_scale=wl.SM_SCALE,
                               kv_scale=SCALE[cache], out=out, lse=lse, workspace=ws, **kw)

    run(q, lens, out, lse, torch.zeros(size, dtype=torch.uint8, device=dev), kw)
    want = out.clone(), lse.clone()
    assert torch.isfinite(want[1]).all()
    ws = torch.zeros(size, dtype=torch.uint8, device=dev)
    for _ in range(20):
        out.fill_(7.0)
        run(other, none, e_out, e_lse, ws, none_kw)
        run(q, lens, out, lse, ws, kw)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert not e_out.any() and torch.isneginf(e_lse).all()
