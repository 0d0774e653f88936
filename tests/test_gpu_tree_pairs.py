"""mla_decode_tree by pairs of CTAs whose last tile of rows is one CTA's only, over many pages (GPU).

Tolerance: the stated one of mla_decode (gpu_util.assert_close), whose arithmetic it has.
"""

import random

import numpy as np
import pytest
import torch

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .gpu_util import bf16_tensor
from .test_gpu_tree import check
from .tree_util import SCALE, Cache, i32, mask_tensor, queries, random_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("num_ctas", [0, 2, 5])
@pytest.mark.parametrize("N", [13, 15])
def test_odd_tiles(cuda_device, cache, num_ctas, N):
    r = random.Random(N)
    lens, nodes = [3000, 700, 2111, 64], [N, N - 1, 1, N]
    c = Cache(cache, lens, 5 + N, cuda_device)
    masks = [random_tree(r, N) for _ in lens]
    check(c, queries(N, len(lens), N, 64), masks, nodes, num_ctas)


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_two_streams_at_once(cuda_device, cache):
    """Two calls in flight, each with its own workspace, give what each gives alone, bit for bit."""
    r, N, lens = random.Random(4), 14, [1500, 900, 4000]
    c = Cache(cache, lens, 31, cuda_device)
    mask = mask_tensor([random_tree(r, N) for _ in lens], cuda_device)
    q = [bf16_tensor(queries(s, len(lens), N, 64), cuda_device) for s in (1, 2)]
    table, lens_t = i32(c.table, cuda_device), i32(lens, cuda_device)
    size = binding.mla_decode_tree_workspace_size(len(lens), N, 64)

    def call(k, stream=None):
        out = torch.zeros((len(lens), N, 64, 512), dtype=torch.bfloat16, device=cuda_device)
        lse = torch.zeros((len(lens), N, 64), device=cuda_device)
        ws = torch.zeros(size, dtype=torch.uint8, device=cuda_device)
        torch.cuda.synchronize()
        return out, lse, ws, lambda: binding.mla_decode_tree(q[k], c.pool, table, lens_t, mask, wl.SM_SCALE, SCALE[cache],
                                                             out, lse, ws, stream=stream)

    alone = [call(k) for k in range(2)]
    for a in alone:
        a[3]()
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=cuda_device) for _ in range(2)]
    both = [call(k, streams[k]) for k in range(2)]
    for _ in range(3):
        for b in both:
            b[3]()
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(a[0], b[0]) and np.array_equal(a[1].cpu().numpy(), b[1].cpu().numpy())
        assert binding.read_device_status(b[2]) == 0
