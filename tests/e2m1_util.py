"""Helpers of the 4-bit cache's GPU tests: pools filled by the library and by the oracle."""

import numpy as np
import torch

from oracle import attention as oatt
from oracle import e2m1 as oe2m1
from oracle import e4m3 as oe4m3
from paged_mla_decode_gb300 import binding

from .gpu_util import bf16_tensor


def append(pages, bits, slots, scale, dev):
    """mla_kv_append of bf16 bit patterns [n, 576] at slots [n]."""
    x = bf16_tensor(bits, dev)
    binding.mla_kv_append(x[:, :512].contiguous(), x[:, 512:].contiguous(),
                          torch.from_numpy(np.asarray(slots, np.int32)).to(dev), pages, scale)


def fill(w, dev):
    """Both sides' 4-bit pools holding every segment of workload ``w``: (device, oracle bytes)."""
    pages = torch.zeros((w.num_pages, binding.MLA_E2M1_PAGE_BYTES), dtype=torch.uint8, device=dev)
    ref = np.zeros((w.num_pages, oe2m1.PAGE_BYTES), dtype=np.uint8)
    for si in range(len(w.segments)):
        bits, slots = w.segment_latent(si), w.segment_slots(si)
        append(pages, bits, slots, w.kv_scale, dev)
        oe2m1.store(ref, slots, *oe2m1.encode(oe4m3.bf16_bits_to_f64(bits), w.kv_scale))
    return pages, ref


def reference(w, ref_pages, q_bits=None, seq_lens=None, rows=None):
    values = oe2m1.decode_pages(ref_pages, w.kv_scale)
    return oatt.decode(w.q_bits if q_bits is None else q_bits, values, w.block_table,
                       w.seq_lens if seq_lens is None else seq_lens, w.sm_scale, 1.0,
                       kv_dtype=oatt.KV_VALUES, rows=rows)


def buffers(B, Q, H, dev, size=None):
    out = torch.full((B, Q, H, 512), float("nan"), dtype=torch.bfloat16, device=dev)
    lse = torch.full((B, Q, H), float("nan"), dtype=torch.float32, device=dev)
    n = binding.mla_decode_workspace_size(B, Q, H) if size is None else size
    return out, lse, torch.zeros(n, dtype=torch.uint8, device=dev)
