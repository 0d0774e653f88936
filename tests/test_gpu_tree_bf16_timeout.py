"""A wait of the bf16 tree decode that runs out (GPU).

As test_gpu_tree_timeout.py: the test library's QK issuer waits, before its third page, on a barrier that
nothing completes, with waits between roles limited to 20 ms. By then the TMA warp has pages in flight
and the other roles wait for this one: the call must end, set the status bit and leave the device usable.
"""

import pytest
import torch

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import build as mla_build
from paged_mla_decode_gb300 import workloads as wl

from .gpu_util import bf16_tensor
from .test_gpu_tree import check
from .tree_util import Cache, chain, i32, mask_tensor, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nodes", [1, 3])  # of 64 heads: a tile of rows each
def test_wait_timeout(cuda_device, nodes):
    dev = cuda_device
    stall = binding.open_library(mla_build.STALL_LIB_PATH)
    lens, ctas = [1900, 1200], 4  # every CTA holds more than two pages, so every one reaches the stall
    c, q_bits, masks = Cache("bf16", lens, 63, dev), queries(64, 2, nodes, 64), [chain(nodes)] * 2
    q, mask, table, seq_lens = bf16_tensor(q_bits, dev), mask_tensor(masks, dev), i32(c.table, dev), i32(lens, dev)
    out = torch.zeros((2, nodes, 64, 512), dtype=torch.bfloat16, device=dev)
    lse = torch.zeros((2, nodes, 64), dtype=torch.float32, device=dev)
    ws = torch.zeros(stall.mla_decode_tree_workspace_size(2, nodes, 64, ctas), dtype=torch.uint8, device=dev)
    st = stall.mla_decode_tree(q.data_ptr(), c.pool.data_ptr(), c.pool.shape[0], 64, binding.MLA_KV_BF16, table.data_ptr(),
                               table.shape[1], seq_lens.data_ptr(), mask.data_ptr(), None, 2, nodes, 64, wl.SM_SCALE, 1.0,
                               ctas, ws.data_ptr(), ws.numel(), out.data_ptr(), lse.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
    assert st == binding.MLA_OK
    torch.cuda.synchronize()  # the call ends: no wait is left running
    assert binding.read_device_status(ws) & binding.MLA_DEVICE_ERR_TIMEOUT
    check(c, q_bits, masks, None, num_ctas=ctas)  # the product's, against the oracle, with no status bit
