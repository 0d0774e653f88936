"""The 4-bit cache: append is bit-exact, decode matches the float64 oracle (GPU).

Decode tolerance: the stated one of mla_decode (test_gpu_decode.py), against the oracle's
own 4-bit encoding; the two pools are compared byte for byte first. The 4-bit values are
e4m3 numbers, so the same cache written out as e4m3 codes must give mla_decode's results.
"""

import numpy as np
import pytest
import torch

from oracle import e2m1 as oe2m1
from oracle import e4m3 as oe4m3
from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .e2m1_util import append, buffers, fill, reference
from .gpu_util import assert_close, bf16_tensor, gpu_decode

pytestmark = pytest.mark.gpu

SCALE = wl.KV_SCALE


def _check_append(bits, slots, num_pages, scale, dev):
    pages = torch.full((num_pages, binding.MLA_E2M1_PAGE_BYTES), 0xA5, dtype=torch.uint8, device=dev)
    ref = np.full((num_pages, oe2m1.PAGE_BYTES), 0xA5, dtype=np.uint8)
    append(pages, bits, slots, scale, dev)
    oe2m1.store(ref, slots, *oe2m1.encode(oe4m3.bf16_bits_to_f64(bits), scale))
    assert np.array_equal(pages.cpu().numpy(), ref)


@pytest.mark.parametrize("n", [0, 1, 2, 17, 64, 1000])
@pytest.mark.parametrize("scale", [SCALE, 1.0, 2.0 ** -100, 2.0 ** 100])
def test_append_random_tokens(cuda_device, n, scale):
    """Random tokens at shuffled slots, among them skipped and out-of-range ones."""
    rng = np.random.default_rng(n)
    x = (rng.standard_normal((n, 576)) * np.ldexp(56.0 * scale, rng.integers(-12, 6, (n, 1)))).astype(np.float32)
    pages = 20
    slots = rng.permutation(pages * 64)[:n]
    slots[::7] = -1
    if n > 2:
        slots[2] = pages * 64
    _check_append(wl.f32_to_bf16_bits(x), slots, pages, scale, cuda_device)


@pytest.mark.parametrize("scale", [SCALE, 1.0, float(np.float32(1.0 / 3.0)), float(np.float32(0.7)), 2.0 ** -100,
                                   1.875, 1.875 * 2.0 ** -8, 1.5, 0.1875])
def test_append_every_bf16(cuda_device, scale):
    """All 65,536 bf16 values, neighbours sharing blocks: ties, near ties (an e2m1 midpoint
    times the default scale is within one float32 ulp of bf16 values), subnormals,
    infinities and NaNs."""
    order = np.arange(1 << 16, dtype=np.uint16)
    bits = np.zeros(114 * 576, dtype=np.uint16)
    bits[:1 << 16] = order
    _check_append(bits.reshape(114, 576), np.arange(114), 2, scale, cuda_device)
    # each value beside a large one, so that every code of a fixed power is met
    one = np.tile(wl.f32_to_bf16_bits(np.float32([6.0 * scale]))[0], 3640 * 576)
    wide = one.reshape(-1, 32)
    wide[:2115, 1:] = np.resize(order, 2115 * 31).reshape(2115, 31)
    small = oe4m3.bf16_bits_to_f64(wide)
    wide[~(np.abs(small) <= 6.0 * scale)] = 0
    _check_append(one.reshape(3640, 576), np.arange(3640), 57, scale, cuda_device)


@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("num_ctas", [1, 3, 0, 400])
def test_ragged_lengths_and_splits(cuda_device, heads, num_ctas):
    lengths = [1, 2, 63, 64, 65, 129, 777, 1000]
    w = wl.make_lengths_workload("e2m1", 70 + heads, lengths, num_heads=heads)
    pages, ref_pages = fill(w, cuda_device)
    assert np.array_equal(pages.cpu().numpy(), ref_pages)
    out, lse, ws = gpu_decode(w, pages, cuda_device, num_ctas=num_ctas)
    assert binding.read_device_status(ws) == 0
    assert_close(out, lse, *reference(w, ref_pages), what=f"H={heads} G={num_ctas}")


@pytest.mark.parametrize("nq", [2, 3, 4])
def test_draft_queries(cuda_device, nq):
    w = wl.make_lengths_workload("e2m1", 80 + nq, [nq, nq + 1, 64 + nq - 1, 300, 1031], num_heads=64,
                                 num_queries=nq)
    pages, ref_pages = fill(w, cuda_device)
    out, lse, _ = gpu_decode(w, pages, cuda_device)
    assert_close(out, lse, *reference(w, ref_pages), what=f"Q={nq}")


def test_matches_the_e4m3_cache_of_the_same_values(cuda_device):
    """A long request (many pages a CTA) and a large score range: the expanded pages written
    as e4m3 codes give the same attention, to the order of the tensor core's additions."""
    w = wl.make_lengths_workload("e2m1", 91, [30000, 12345], num_heads=64)
    q = wl.f32_to_bf16_bits(oe4m3.bf16_bits_to_f64(w.q_bits).astype(np.float32) * 6)
    pages, ref_pages = fill(w, cuda_device)
    codes, nibs = oe2m1.load(ref_pages)
    wide = oe4m3.encode(oe2m1.values(codes, nibs, 1.0), 1.0)
    same = torch.from_numpy(wide).to(cuda_device)
    a_out, a_lse, _ = gpu_decode(w, pages, cuda_device, q_bits=q)
    b_out, b_lse, _ = gpu_decode(w, same, cuda_device, q_bits=q)
    # out: one bf16 rounding each (2^-8 relative) of sums that differ by fp32 additions
    assert np.abs(a_out - b_out).max() <= 2.0 ** -7 * np.abs(b_out).max()
    assert np.abs(a_lse - b_lse).max() <= 1e-5 * np.abs(b_lse).max()


def test_nan_block_reaches_only_its_request(cuda_device):
    w = wl.make_lengths_workload("e2m1", 92, [200, 150], num_heads=16)
    pages, ref_pages = fill(w, cuda_device)
    bits = np.zeros((1, 576), np.uint16)
    bits[0, 100] = 0x7FC0
    append(pages, bits, [int(w.block_table[0, 1]) * 64 + 5], w.kv_scale, cuda_device)
    out, lse, _ = gpu_decode(w, pages, cuda_device)
    ref_out, ref_lse = reference(w, ref_pages)
    assert np.isnan(lse[0]).all() and np.isnan(out[0]).all()
    assert_close(out[1:], lse[1:], ref_out[1:], ref_lse[1:], what="the other request")


def test_bad_pages_and_lengths(cuda_device):
    """As for an e4m3 cache: the rows get out = 0, lse = -inf and a status bit; others stand.
    Tokens behind the last one of a page (NaN blocks here) are never seen."""
    w = wl.make_lengths_workload("e2m1", 93, [200, 150, 100, 70], num_heads=32)
    pages, ref_pages = fill(w, cuda_device)
    pages.view(w.num_pages, -1)[int(w.block_table[3, 1]), oe2m1.CODE_BYTES:].view(9, 64)[:, 6:] = 0xFF
    table, lens = w.block_table.copy(), w.seq_lens.copy()
    table[0, 1] = w.num_pages
    table[1, 2] = -5
    lens[2] = -1
    out, lse, ws = gpu_decode(w, pages, cuda_device, block_table=table, seq_lens=lens)
    assert binding.read_device_status(ws) == binding.MLA_DEVICE_ERR_BAD_PAGE | binding.MLA_DEVICE_ERR_BAD_LENGTH
    assert (out[:3] == 0).all() and np.isneginf(lse[:3]).all()
    ref_out, ref_lse = reference(w, ref_pages)
    assert_close(out[3:], lse[3:], ref_out[3:], ref_lse[3:], what="the good request")


@pytest.mark.parametrize("groups,forks,prefix,nq,num_ctas", [(3, 4, 640, 1, 0), (2, 3, 1280, 2, 7), (5, 1, 320, 4, 0)])
def test_grouped(cuda_device, groups, forks, prefix, nq, num_ctas):
    w = wl.prefix_shared(seed=95 + groups, groups=groups, forks=forks, prefix=prefix, suffix_median=150.0,
                         suffix_max=700, num_queries=nq)
    pages, ref_pages = fill(w, cuda_device)
    B, H = w.batch, w.num_heads
    out, lse, ws = buffers(B, nq, H, cuda_device, binding.mla_decode_grouped_workspace_size(B, nq, H, num_ctas))
    binding.mla_decode_grouped(bf16_tensor(w.q_bits, cuda_device), pages,
                               torch.from_numpy(w.block_table).to(cuda_device),
                               torch.from_numpy(w.seq_lens).to(cuda_device), forks,
                               torch.from_numpy(w.extra["prefix_pages"]).to(cuda_device), w.sm_scale,
                               w.kv_scale, out, lse, ws, num_ctas=num_ctas)
    torch.cuda.synchronize()
    assert binding.read_device_status(ws) == 0
    assert_close(out.float().cpu().numpy(), lse.cpu().numpy(), *reference(w, ref_pages), what="grouped")


def test_static_scratch_and_stream(cuda_device):
    """The entry without a workspace, and a call on another stream than the inputs'."""
    w = wl.make_lengths_workload("e2m1", 97, [333, 64, 1000], num_heads=64, num_queries=2)
    pages, ref_pages = fill(w, cuda_device)
    q, table = bf16_tensor(w.q_bits, cuda_device), torch.from_numpy(w.block_table).to(cuda_device)
    lens = torch.from_numpy(w.seq_lens).to(cuda_device)
    out, lse, _ = buffers(w.batch, 2, 64, cuda_device)
    ref = reference(w, ref_pages)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    binding.mla_decode_static_scratch(q, pages, table, lens, w.sm_scale, w.kv_scale, out, lse, stream=side)
    side.synchronize()
    assert_close(out.float().cpu().numpy(), lse.cpu().numpy(), *ref, what="static scratch")


def test_graph_replay_follows_lengths(cuda_device):
    """One captured append + decode, replayed as a request grows over a page border."""
    w = wl.make_lengths_workload("e2m1", 98, [130], num_heads=64)
    pages, ref_pages = fill(w, cuda_device)
    q, table = bf16_tensor(w.q_bits, cuda_device), torch.from_numpy(w.block_table).to(cuda_device)
    bits = w.segment_latent(0)
    x = bf16_tensor(bits[:1], cuda_device)
    lat, rope = x[:, :512].contiguous(), x[:, 512:].contiguous()
    lens = torch.tensor([0], dtype=torch.int32, device=cuda_device)
    slot = torch.tensor([-1], dtype=torch.int32, device=cuda_device)
    out, lse, ws = buffers(1, 1, 64, cuda_device)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        binding.mla_decode(q, pages, table, lens, w.sm_scale, w.kv_scale, out, lse, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        binding.mla_kv_append(lat, rope, slot, pages, w.kv_scale)
        binding.mla_decode(q, pages, table, lens, w.sm_scale, w.kv_scale, out, lse, ws)
    pages.zero_()
    ws.zero_()
    for t in range(70):
        y = bf16_tensor(bits[t:t + 1], cuda_device)
        lat.copy_(y[:, :512])
        rope.copy_(y[:, 512:])
        slot.fill_(int(w.block_table[0, t // 64]) * 64 + t % 64)
        lens.fill_(t + 1)
        graph.replay()
        if t in (0, 1, 63, 64, 69):
            torch.cuda.synchronize()
            ref = reference(w, ref_pages, seq_lens=np.array([t + 1]))
            assert_close(out.float().cpu().numpy(), lse.cpu().numpy(), *ref, what=f"length {t + 1}")
