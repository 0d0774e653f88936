"""A tree-speculative serving loop, captured once and replayed (GPU).

Each replay allocates the nodes' pages and slots, appends their entries, decodes the tree, turns
logits into probabilities, walks down the tree, moves the kept entries together in two layers' caches
and hands lengths, counts and caches to the next step. Every output of every step is compared with
the oracles run in the same order.
"""

import random

import numpy as np
import pytest
import torch

from oracle import e4m3 as oe4m3
from oracle import e2m1 as oe2m1
from oracle import paging
from oracle import tree as otree
from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .gpu_util import assert_close, bf16_tensor
from .tree_util import SCALE, i32, mask_tensor, random_tree
from .test_gpu_kv_compact import rows_of
from .test_gpu_logits_probs import words

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,H", [("e4m3", 64), ("e2m1", 16), ("bf16", 32)])
def test_captured_tree_loop(cuda_device, cache, H):
    dev, rng = cuda_device, np.random.default_rng(5)
    B, N, V, width, pages, steps = 4, 7, 523, 6, 20, 8
    lens, held = np.array([0, 60, 130, 5]), np.array([0, 1, 3, 1])
    perm = rng.permutation(pages)
    table, at = np.full((B, width), -1), 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free, count = perm[at:], pages - at
    shape = {"e4m3": (2, pages, 64, 576), "bf16": (2, pages, 64, 576), "e2m1": (2, pages, binding.MLA_E2M1_PAGE_BYTES)}[cache]
    pool = torch.zeros(shape, dtype=torch.bfloat16 if cache == "bf16" else torch.uint8, device=dev)
    entries = [np.zeros((0, 576), np.uint16) for _ in range(B)]

    def append(slots, bits):
        x = bf16_tensor(bits, dev)
        for layer in range(2):
            binding.mla_kv_append(x[:, :512].contiguous(), x[:, 512:].contiguous(), i32(slots, dev), pool[layer], SCALE[cache])

    for b in range(B):
        if lens[b]:
            entries[b] = wl.f32_to_bf16_bits(rng.standard_normal((lens[b], 576), dtype=np.float32) * 0.5)
            t = np.arange(lens[b])
            append(table[b, t // 64] * 64 + t % 64, entries[b])

    d_table, d_free, d_count = i32(table, dev), i32(free, dev), i32([count], dev)
    d_lens, d_held, d_new = i32(lens, dev), i32(held, dev), i32([N] * B, dev)
    d_len2, d_cu, d_slots, d_status = i32(lens, dev), i32([0] * (B + 1), dev), i32([0] * (B * N), dev), i32([0] * B, dev)
    lat = torch.zeros((B * N, 512), dtype=torch.bfloat16, device=dev)
    rope = torch.zeros((B * N, 64), dtype=torch.bfloat16, device=dev)
    q = torch.zeros((B, N, H, 576), dtype=torch.bfloat16, device=dev)
    out, lse = torch.zeros((B, N, H, 512), dtype=torch.bfloat16, device=dev), torch.zeros((B, N, H), device=dev)
    ws = torch.zeros(binding.mla_decode_tree_workspace_size(B, N, H), dtype=torch.uint8, device=dev)
    d_mask = mask_tensor([[0] * N] * B, dev)
    logits = torch.zeros((2, B, N, V), dtype=torch.bfloat16, device=dev)  # the target's and the drafter's
    probs = torch.zeros((2, B, N, V), device=dev)
    d_tok, d_u = i32(np.zeros((B, N)), dev), torch.zeros((B, N), device=dev)
    counts, prompt = np.zeros((B, V), int), rng.random((B, V)) < 0.1
    temperature = np.float32([0.7, 0.0, 1.0, 1.2])
    settings = {"repetition": np.float32([1.2, 1.0, 1.1, 1.3]), "frequency": np.float32([0.3, 0.0, 0.2, 0.5]),
                "presence": np.float32([0.1, 0.4, 0.0, 0.3])}
    d_counts, d_allowed = i32(counts, dev), i32(np.zeros((B, N, -(-V // 32))), dev)
    kw = {k: torch.from_numpy(v).to(dev) for k, v in settings.items()}
    kw |= dict(temperature=torch.from_numpy(temperature).to(dev), prompt_mask=torch.from_numpy(words(prompt)).to(dev),
               token_counts=d_counts, node_tokens=d_tok, tree_mask=d_mask)
    tokens, path, acc = i32(np.zeros((B, N)), dev), i32(np.zeros((B, N)), dev), i32([0] * B, dev)

    def step():
        binding.mla_kv_alloc(d_lens, d_new, d_held, d_free, d_count, pages, d_table, d_len2, d_held, d_count, d_cu, d_slots, d_status)
        for layer in range(2):
            binding.mla_kv_append(lat, rope, d_slots, pool[layer], SCALE[cache])
        binding.mla_decode_tree(q, pool[1], d_table, d_len2, d_mask, wl.SM_SCALE, SCALE[cache], out, lse, ws)
        binding.mla_logits_to_probs(logits[0], probs[0], allowed=d_allowed, **kw)
        binding.mla_logits_to_probs(logits[1], probs[1], **kw)
        binding.mla_verify_tree(probs[0], probs[1], d_tok, d_mask, d_u, tokens, path, acc, seq_lens=d_len2, seq_lens_out=d_lens,
                                token_counts=d_counts)
        binding.mla_kv_compact(pool, d_table, d_lens, path, acc)

    graph = torch.cuda.CUDAGraph()
    keep = [t.clone() for t in (d_table, d_count, d_lens, d_held, d_counts, pool)]
    step()  # (warm: nothing that a capture may not do is left)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for t, k in zip((d_table, d_count, d_lens, d_held, d_counts, pool), keep):
        t.copy_(k)
    some_kept = 0
    for s in range(steps):
        r = random.Random(s)
        masks = [random_tree(r, N, 3) for _ in range(B)]
        bits = wl.f32_to_bf16_bits(rng.standard_normal((B * N, 576), dtype=np.float32) * 0.5)
        q_bits = wl.f32_to_bf16_bits(rng.standard_normal((B, N, H, 576), dtype=np.float32))
        x = torch.from_numpy(rng.standard_normal((B, N, V)).astype(np.float32) * 2)
        x = torch.stack([x, x + 0.3 * torch.from_numpy(rng.standard_normal((B, N, V)).astype(np.float32))]).bfloat16()
        allowed = rng.random((B, N, V)) < 0.95
        drafted = np.zeros((B, N), int)
        q_rows = np.zeros((B, N, V))
        xf = x.float().numpy()

        def row(which, b, j):
            on_path = [int(drafted[b, i]) for i in range(1, N) if otree.sees(masks[b][j], i)]
            return otree.probabilities(xf[which, b, j], temperature[b], counts[b], prompt[b], path_tokens=on_path,
                                       allowed=allowed[b, j] if which == 0 else None, **{k: v[b] for k, v in settings.items()})

        for b in range(B):  # the drafter's rows in node order: a node's own token counts in its row
            for i in range(N):
                if i > 0:
                    drafted[b, i] = rng.choice(V, p=q_rows[b, otree.parent(masks[b][i], i)])
                q_rows[b, i] = row(1, b, i)
        u = rng.random((B, N), dtype=np.float32)
        xb = bf16_tensor(bits, dev)
        lat.copy_(xb[:, :512])
        rope.copy_(xb[:, 512:])
        q.copy_(bf16_tensor(q_bits, dev))
        logits.copy_(x.to(dev))
        d_mask.copy_(mask_tensor(masks, dev))
        d_tok.copy_(i32(drafted, dev))
        d_u.copy_(torch.from_numpy(u))
        d_allowed.copy_(torch.from_numpy(words(allowed)))
        graph.replay()
        torch.cuda.synchronize()

        want = paging.alloc(lens, [N] * B, held, free, count, pages, table, B * N)
        assert np.array_equal(d_slots.cpu().numpy(), want["slot_mapping"]) and (want["seq_lens_out"] >= 0).all()
        table, held, count = want["block_table"], want["pages_held_out"], want["free_count_out"]
        assert np.array_equal(d_table.cpu().numpy(), table) and int(d_count) == count
        for b in range(B):
            entries[b] = np.concatenate([entries[b], bits[b * N:(b + 1) * N]])
        values = []
        for e in entries:
            v = oe4m3.bf16_bits_to_f64(e)
            if cache == "e4m3":
                v = oe4m3.decode(oe4m3.encode(v, SCALE[cache])) * np.float64(np.float32(SCALE[cache]))
            values.append(oe2m1.values(*oe2m1.encode(v, SCALE[cache]), SCALE[cache]) if cache == "e2m1" else v)
        ref = otree.decode(oe4m3.bf16_bits_to_f64(q_bits), values, masks, [N] * B, wl.SM_SCALE)
        assert_close(out.float().cpu().numpy(), lse.cpu().numpy(), *ref, what=f"step {s}")
        got = probs.cpu().numpy()
        for b in range(B):
            for j in range(N):
                for which in range(2):
                    p = row(which, b, j)
                    assert np.abs(got[which, b, j] - p).max() <= 1e-4 * p.max(), (s, b, j)
            # the walk over the library's own probabilities: equal
            toks, kept, a = otree.verify(got[0, b], got[1, b], drafted[b], masks[b], u[b], N)
            assert (tokens[b].tolist(), path[b].tolist(), int(acc[b])) == (toks, kept, a)
            some_kept += a
            for t in toks:
                if t >= 0:
                    counts[b, t] += 1
            entries[b] = otree.compact(entries[b], len(entries[b]) - N, kept, a)[:len(entries[b]) - N + a + 1]
            lens[b] = len(entries[b])
        assert np.array_equal(d_lens.cpu().numpy(), lens) and np.array_equal(d_counts.cpu().numpy(), counts)
        # both layers hold the kept entries, as an append of them alone would have left them
        raw = pool.view(torch.uint8).cpu().numpy().reshape(2, pages, -1)
        for b in range(B):
            fresh = torch.zeros(pool.shape[1:], dtype=pool.dtype, device=dev)
            t = np.arange(lens[b])
            slots = table[b, t // 64] * 64 + t % 64
            xb = bf16_tensor(entries[b], dev)
            binding.mla_kv_append(xb[:, :512].contiguous(), xb[:, 512:].contiguous(), i32(slots, dev), fresh, SCALE[cache])
            fresh = rows_of(fresh.view(torch.uint8).cpu().numpy().reshape(pages, -1), cache)
            for layer in range(2):
                assert np.array_equal(rows_of(raw[layer], cache)[slots], fresh[slots])
    assert some_kept >= steps  # (trees are walked, not only left at node 0)
    assert binding.read_device_status(ws) == 0
