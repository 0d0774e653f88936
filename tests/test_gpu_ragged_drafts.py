"""Speculative steps whose requests have different numbers of drafts: all are allocated, appended and
decoded with the most queries, padded behind their drafts, and verified with their own (GPU)."""

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import e2m1 as oe2m1
from oracle import e4m3 as oe4m3
from oracle import verify as over
from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .e2m1_util import buffers
from .gpu_util import assert_close, bf16_tensor

pytestmark = pytest.mark.gpu


def test_steps_with_fewer_drafts_in_some_requests(cuda_device):
    dev, rng = cuda_device, np.random.default_rng(550)
    B, K, H, V, width, steps = 6, 3, 16, 97, 4, 5
    Q, pages = K + 1, B * width
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(dev)  # noqa: E731
    lens = np.array([0, 60, 61, 63, 64, 130])
    held = -(-lens // 64)
    table = np.full((B, width), -1)
    perm = rng.permutation(pages)
    at = np.concatenate([[0], np.cumsum(held)])
    for b in range(B):
        table[b, :held[b]] = perm[at[b]:at[b + 1]]
    pool = torch.zeros((pages, binding.MLA_E2M1_PAGE_BYTES), dtype=torch.uint8, device=dev)
    entries = [wl.f32_to_bf16_bits(rng.standard_normal((n, 576)).astype(np.float32) * 0.5) for n in lens]
    for b in range(B):  # the cached contexts
        x, t = bf16_tensor(entries[b], dev), np.arange(lens[b])
        binding.mla_kv_append(x[:, :512].contiguous(), x[:, 512:].contiguous(),
                              i32(table[b, t // 64] * 64 + t % 64), pool, wl.KV_SCALE)
    d_lens, d_held, d_count, d_table, d_free = i32(lens), i32(held), i32([pages - at[-1]]), i32(table), i32(perm[at[-1]:])
    d_cu, d_slots, d_status, d_padded = i32([0] * (B + 1)), i32([0] * B * Q), i32([0] * B), i32([0] * B)
    out, lse, ws = buffers(B, Q, H, dev)
    tokens, acc = i32(np.zeros((B, Q))), i32([0] * B)
    for s in range(steps):
        k = rng.integers(0, K + 1, B)
        bits = wl.f32_to_bf16_bits(rng.standard_normal((B, Q, 576)).astype(np.float32) * 0.5)
        for b in range(B):  # the padding may be anything: here NaN, which no true row may see
            bits[b, k[b] + 1:] = 0x7FC0
        q_bits = wl.f32_to_bf16_bits(rng.standard_normal((B, Q, H, 576)).astype(np.float32))
        z = np.exp(rng.standard_normal((B, Q, V)).astype(np.float32))
        p = z / z.sum(-1, keepdims=True)
        dq = np.roll(p[:, :K], 1, axis=2)
        draft, u = rng.integers(0, V, (B, K)), rng.random((B, Q)).astype(np.float32) * np.float32(0.6)
        x = bf16_tensor(bits.reshape(B * Q, 576), dev)
        binding.mla_kv_alloc(d_lens, i32([Q] * B), d_held, d_free, d_count, pages, d_table, d_padded, d_held, d_count,
                             d_cu, d_slots, d_status)
        binding.mla_kv_append(x[:, :512].contiguous(), x[:, 512:].contiguous(), d_slots, pool, wl.KV_SCALE)
        binding.mla_decode(bf16_tensor(q_bits, dev), pool, d_table, d_padded, wl.SM_SCALE, wl.KV_SCALE, out, lse, ws)
        d_k = i32(k)
        binding.mla_verify_drafts(torch.from_numpy(p).to(dev), torch.from_numpy(dq).to(dev), i32(draft),
                                  torch.from_numpy(u).to(dev), tokens, acc, num_drafts=d_k,
                                  seq_lens=d_padded - (K - d_k), seq_lens_out=d_lens)
        assert (d_status == 0).all() and d_padded.tolist() == (lens + Q).tolist()
        o, e = out.float().cpu().numpy(), lse.cpu().numpy()
        for b in range(B):
            entries[b] = np.concatenate([entries[b][:lens[b]], bits[b, :k[b] + 1]])
            n = k[b] + 1  # this request alone, with its own number of queries
            values = oe2m1.values(*oe2m1.encode(oe4m3.bf16_bits_to_f64(entries[b]), wl.KV_SCALE), wl.KV_SCALE)
            one = np.zeros((width, 64, 576))
            one.reshape(-1, 576)[:len(values)] = values
            ref = oatt.decode(q_bits[b:b + 1, :n], one, np.arange(width)[None], np.array([len(values)]), wl.SM_SCALE, 1.0,
                              kv_dtype=oatt.KV_VALUES)
            assert_close(o[b, :n], e[b, :n], ref[0][0], ref[1][0], what=f"step {s}, request {b}")
            want, a = over.verify(p[b], dq[b], draft[b], u[b], k[b])
            assert tokens[b].tolist() == want and int(acc[b]) == a
            lens[b] += a + 1
        assert d_lens.tolist() == lens.tolist()
