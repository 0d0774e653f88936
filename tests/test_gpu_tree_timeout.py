"""A wait of the tree decode that runs out (GPU), in one CTA and in a pair of them.

The test library's QK issuer waits, before its third page, on a barrier that nothing completes, with waits between
roles limited to 20 ms: the call must end, set the status bit and leave the device usable.
"""

import numpy as np
import pytest
import torch

from oracle import e4m3
from oracle import tree as otree
from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import build as mla_build
from paged_mla_decode_gb300 import workloads as wl

from .gpu_util import bf16_tensor, gpu_fill_cache, oracle_fill_cache
from .tree_util import mask_tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nodes", [1, 2], ids=["single", "pair"])  # of 64 heads: one tile of rows, or two
def test_wait_timeout(cuda_device, nodes):
    dev = cuda_device
    stall = binding.open_library(mla_build.STALL_LIB_PATH)
    w = wl.make_lengths_workload("stall", 62, [5000, 3000], num_heads=64)
    pages = gpu_fill_cache(w, dev)
    q_one = bf16_tensor(w.q_bits, dev)  # [2, 1, 64, 576]
    q = q_one.repeat(1, nodes, 1, 1).contiguous()
    table = torch.from_numpy(w.block_table).to(dev)
    lens = torch.from_numpy(w.seq_lens).to(dev)
    chain = [[(1 << (i + 1)) - 1 for i in range(nodes)]] * 2
    mask = mask_tensor(chain, dev)
    out = torch.zeros((2, nodes, 64, 512), dtype=torch.bfloat16, device=dev)
    lse = torch.zeros((2, nodes, 64), dtype=torch.float32, device=dev)
    ctas = 4  # every worker holds more than two pages, so every one reaches the stall
    ws = torch.zeros(stall.mla_decode_tree_workspace_size(2, nodes, 64, ctas), dtype=torch.uint8, device=dev)
    st = stall.mla_decode_tree(q.data_ptr(), pages.data_ptr(), pages.shape[0], 64, binding.MLA_KV_E4M3, table.data_ptr(),
                               table.shape[1], lens.data_ptr(), mask.data_ptr(), None, 2, nodes, 64, w.sm_scale,
                               w.kv_scale, ctas, ws.data_ptr(), ws.numel(), out.data_ptr(), lse.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
    assert st == binding.MLA_OK
    torch.cuda.synchronize()
    assert binding.read_device_status(ws) & binding.MLA_DEVICE_ERR_TIMEOUT

    ws = torch.zeros(binding.mla_decode_tree_workspace_size(2, nodes, 64, ctas), dtype=torch.uint8, device=dev)
    binding.mla_decode_tree(q, pages, table, lens, mask, w.sm_scale, w.kv_scale, out, lse, ws, num_ctas=ctas)
    assert binding.read_device_status(ws) == 0
    values = e4m3.decode(oracle_fill_cache(w)) * w.kv_scale
    entries = [values.reshape(-1, 64, 576)[w.block_table[b]].reshape(-1, 576)[: w.seq_lens[b]] for b in range(2)]
    want, want_lse = otree.decode(e4m3.bf16_bits_to_f64(w.q_bits).reshape(2, 1, 64, 576).repeat(nodes, 1), entries,
                                  np.array(chain), [nodes] * 2, w.sm_scale)
    # the output's own rounding, and operands in two terms (2^-8 of the largest value covers both)
    assert np.abs(out.float().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max() * 2
    assert np.abs(lse.cpu().numpy() - want_lse).max() <= 1e-3
