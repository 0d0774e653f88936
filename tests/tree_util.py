"""Helpers of the tree operators' tests: random trees, caches of every type with their float64 entries."""

import random

import numpy as np
import torch

from oracle import attention as oatt
from oracle import e2m1 as oe2m1
from oracle import e4m3 as oe4m3
from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .gpu_util import bf16_tensor

SCALE = {"e4m3": wl.KV_SCALE, "e2m1": wl.KV_SCALE, "bf16": 1.0}


def random_tree(rng: random.Random, n: int, back: int = 4):
    """Masks of a tree of n nodes; a node's parent is one of the `back` before it."""
    masks = [1]
    for i in range(1, n):
        masks.append(masks[rng.randint(max(0, i - back), i - 1)] | 1 << i)
    return masks


def chain(n: int):
    return [(2 << j) - 1 for j in range(n)]


def mask_tensor(masks, dev):
    return torch.from_numpy(np.array(masks, dtype=np.uint64).view(np.int64)).to(dev)


def i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(dev)


class Cache:
    """Requests of the given lengths in a pool of shuffled pages, filled through mla_kv_append."""

    def __init__(self, cache, lens, seed, dev, spare=3):
        rng = np.random.default_rng(seed)
        counts = [-(-n // 64) for n in lens]
        self.cache, self.lens, self.dev = cache, list(lens), dev
        self.num_pages = sum(counts) + spare
        perm = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), max(1, max(counts))), -1, np.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = perm[at:at + c]
            at += c
        shape, dtype = {"e4m3": ((self.num_pages, 64, 576), torch.uint8), "bf16": ((self.num_pages, 64, 576), torch.bfloat16),
                        "e2m1": ((self.num_pages, binding.MLA_E2M1_PAGE_BYTES), torch.uint8)}[cache]
        self.pool = torch.zeros(shape, dtype=dtype, device=dev)
        self.bits = [wl.f32_to_bf16_bits(rng.standard_normal((n, 576), dtype=np.float32) * 0.5) for n in lens]
        for b in range(len(lens)):
            self.put(b, np.arange(lens[b]), self.bits[b])

    def slots(self, b, tokens):
        tokens = np.asarray(tokens)
        return self.table[b, tokens // 64] * 64 + tokens % 64

    def put(self, b, tokens, bits):
        """Appends bf16 bit patterns [n, 576] as these tokens of request b."""
        if len(bits) == 0:
            return
        x = bf16_tensor(bits, self.dev)
        binding.mla_kv_append(x[:, :512].contiguous(), x[:, 512:].contiguous(), i32(self.slots(b, tokens), self.dev),
                              self.pool, SCALE[self.cache])

    def entries(self):
        """The stored values by the oracle's codecs, float64 [L, 576] a request."""
        got = []
        for bits in self.bits:
            x = oe4m3.bf16_bits_to_f64(bits)
            if self.cache == "bf16":
                got.append(x)
            elif self.cache == "e4m3":
                got.append(oatt.dequant(oe4m3.encode(x, SCALE["e4m3"]), oatt.KV_E4M3, SCALE["e4m3"]))
            else:
                got.append(oe2m1.values(*oe2m1.encode(x, SCALE["e2m1"]), SCALE["e2m1"]) if len(x) else x)
        return got


def queries(seed, B, N, H):
    return wl.f32_to_bf16_bits(np.random.default_rng(seed).standard_normal((B, N, H, 576), dtype=np.float32))


def gpu_tree(c: Cache, q_bits, masks, nodes=None, num_ctas=0, workspace=None, seq_lens=None, table=None):
    dev = c.dev
    B, N, H, _ = q_bits.shape
    out = torch.full((B, N, H, 512), float("nan"), dtype=torch.bfloat16, device=dev)
    lse = torch.full((B, N, H), float("nan"), device=dev)
    if workspace is None:
        workspace = torch.zeros(binding.mla_decode_tree_workspace_size(B, N, H, num_ctas), dtype=torch.uint8, device=dev)
    binding.mla_decode_tree(bf16_tensor(q_bits, dev), c.pool, i32(c.table if table is None else table, dev),
                            i32(c.lens if seq_lens is None else seq_lens, dev), mask_tensor(masks, dev), wl.SM_SCALE,
                            SCALE[c.cache], out, lse, workspace, num_nodes=None if nodes is None else i32(nodes, dev),
                            num_ctas=num_ctas)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy(), workspace
