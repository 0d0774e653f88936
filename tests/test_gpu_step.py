"""A speculative serving loop over a 4-bit cache, captured once and replayed (GPU).

Each replay allocates pages and slots, appends the step's entries, checks the pages' tags,
decodes, verifies the drafts and hands the lengths that stay to the next step. Every
output of every step is compared with the oracles run in the same order.
"""

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import e2m1 as oe2m1
from oracle import e4m3 as oe4m3
from oracle import integrity as oig
from oracle import paging, verify as over
from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .e2m1_util import buffers
from .gpu_util import assert_close, bf16_tensor

pytestmark = pytest.mark.gpu


def test_captured_speculative_loop(cuda_device):
    dev, rng = cuda_device, np.random.default_rng(1)
    B, Q, H, V, width, pages, steps = 5, 3, 16, 257, 6, 24, 12
    K = Q - 1
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(dev)  # noqa: E731
    lens, held = np.array([0, 62, 130, -1, 5]), np.array([0, 1, 3, 2, 1])
    perm = rng.permutation(pages)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free, count = perm[at:], pages - at
    tags = rng.integers(0, 1 << 31, pages).astype(np.uint32)
    expected = np.where(table >= 0, tags[np.clip(table, 0, None)], 0).astype(np.uint32)
    new = np.full(B, Q)
    pool = np.zeros((pages, oe2m1.PAGE_BYTES), np.uint8)
    # the cached tokens before the first step
    first = wl.f32_to_bf16_bits(rng.standard_normal((pages * 64, 576)).astype(np.float32) * 0.5)
    oe2m1.store(pool, np.arange(pages * 64), *oe2m1.encode(oe4m3.bf16_bits_to_f64(first), wl.KV_SCALE))

    d_pool, d_table, d_free = torch.from_numpy(pool).to(dev), i32(table), i32(free)
    d_lens, d_held, d_count, d_new = i32(lens), i32(held), i32([count]), i32(new)
    d_tags, d_expected = i32(tags.view(np.int32)), i32(expected.view(np.int32))
    d_cu, d_slots, d_status, d_check = i32([0] * (B + 1)), i32([0] * (B * Q)), i32([0] * B), i32([0] * B)
    d_len2, d_checked = i32([0] * B), i32([0] * B)
    lat = torch.zeros((B * Q, 512), dtype=torch.bfloat16, device=dev)
    rope = torch.zeros((B * Q, 64), dtype=torch.bfloat16, device=dev)
    q = torch.zeros((B, Q, H, 576), dtype=torch.bfloat16, device=dev)
    out, lse, ws = buffers(B, Q, H, dev)
    d_p, d_q = torch.zeros((B, Q, V), device=dev), torch.zeros((B, K, V), device=dev)
    d_draft, d_u = i32(np.zeros((B, K))), torch.zeros((B, Q), device=dev)
    d_tokens, d_acc = i32(np.zeros((B, Q))), i32([0] * B)

    def step():
        binding.mla_kv_alloc(d_lens, d_new, d_held, d_free, d_count, pages, d_table, d_len2, d_held, d_count, d_cu,
                             d_slots, d_status, page_tags=d_tags, expected_tags=d_expected)
        binding.mla_kv_append(lat, rope, d_slots, d_pool, wl.KV_SCALE)
        binding.mla_kv_check(d_tags, d_table, d_expected, d_len2, d_check, d_checked)
        binding.mla_decode(q, d_pool, d_table, d_checked, wl.SM_SCALE, wl.KV_SCALE, out, lse, ws)
        binding.mla_verify_drafts(d_p, d_q, d_draft, d_u, d_tokens, d_acc, seq_lens=d_checked, seq_lens_out=d_lens)

    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for s in range(steps):
        bits = wl.f32_to_bf16_bits(rng.standard_normal((B * Q, 576)).astype(np.float32) * 0.5)
        q_bits = wl.f32_to_bf16_bits(rng.standard_normal((B, Q, H, 576)).astype(np.float32))
        z = rng.standard_normal((B, Q, V)).astype(np.float32)
        p = np.exp(z) / np.exp(z).sum(-1, keepdims=True)
        dq = np.roll(p[:, :K], 1, axis=2)
        draft, u = rng.integers(0, V, (B, K)), rng.random((B, Q)).astype(np.float32) * np.float32(0.6)
        x = bf16_tensor(bits, dev)
        lat.copy_(x[:, :512])
        rope.copy_(x[:, 512:])
        q.copy_(bf16_tensor(q_bits, dev))
        d_p.copy_(torch.from_numpy(p))
        d_q.copy_(torch.from_numpy(dq))
        d_draft.copy_(torch.from_numpy(draft.astype(np.int32)))
        d_u.copy_(torch.from_numpy(u))
        if s == 7:  # a page of request 2 is handed to somebody else
            stolen = int(table[2, 0])
            tags[stolen] += np.uint32(1)
            d_tags.copy_(i32(tags.view(np.int32)))
        graph.replay()

        got = paging.alloc(lens, new, held, free, count, pages, table, B * Q, tags, expected)
        table, tags, expected = got["block_table"], got["page_tags"], got["expected_tags"]
        held, count, len2 = got["pages_held_out"], got["free_count_out"], got["seq_lens_out"]
        oe2m1.store(pool, got["slot_mapping"], *oe2m1.encode(oe4m3.bf16_bits_to_f64(bits), wl.KV_SCALE))
        status, checked = oig.kv_check(tags, table, expected, len2)
        assert np.array_equal(d_slots.cpu().numpy(), got["slot_mapping"]), s
        assert np.array_equal(d_status.cpu().numpy(), got["request_status"])
        assert np.array_equal(d_table.cpu().numpy(), table) and int(d_count) == count
        assert np.array_equal(d_checked.cpu().numpy(), checked)
        assert np.array_equal(d_pool.cpu().numpy(), pool)
        good = [b for b in range(B) if checked[b] >= Q]
        values = oe2m1.decode_pages(pool, wl.KV_SCALE)
        ref_out, ref_lse = oatt.decode(q_bits[good], values, table[good], checked[good], wl.SM_SCALE, 1.0,
                                       kv_dtype=oatt.KV_VALUES)
        o, e = out.float().cpu().numpy(), lse.cpu().numpy()
        assert_close(o[good], e[good], ref_out, ref_lse, what=f"step {s}")
        for b in set(range(B)) - set(good):
            assert (o[b] == 0).all() and np.isneginf(e[b]).all()
        lens = np.array(checked, dtype=np.int64)
        for b in range(B):
            if checked[b] < 0:
                assert (d_tokens[b] == -1).all() and int(d_acc[b]) == -1
                continue
            want, a = over.verify(p[b], dq[b], draft[b], u[b])
            assert d_tokens[b].cpu().tolist() == want and int(d_acc[b]) == a
            lens[b] -= K - a
        assert np.array_equal(d_lens.cpu().numpy(), lens)
    assert checked[2] == -1 and count < pages - at  # the theft was seen, and pages were taken
