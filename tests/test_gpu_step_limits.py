"""Offsets beyond 32 bits, calls in flight on two streams, and the 4-bit pipeline's timeout (GPU).

The large buffers are allocated and left as they are but for the parts a test uses.
"""

import numpy as np
import pytest
import torch

from oracle import e2m1 as oe2m1
from oracle import e4m3 as oe4m3
from oracle import verify as over
from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import build as mla_build
from paged_mla_decode_gb300 import workloads as wl

from .e2m1_util import append, buffers, fill, reference
from .gpu_util import assert_close, bf16_tensor

pytestmark = pytest.mark.gpu


def _i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(dev)


def test_pool_larger_than_4_gib(cuda_device):
    """Append, gather and decode over the last pages of a 4.6 GB pool."""
    dev, pages = cuda_device, 240_000
    w = wl.make_lengths_workload("far", 401, [300, 64, 130], num_heads=16, num_queries=2)
    _, ref_pages = fill(w, dev)
    pool = torch.empty((pages, binding.MLA_E2M1_PAGE_BYTES), dtype=torch.uint8, device=dev)
    far = pages - w.num_pages
    for si in range(len(w.segments)):
        append(pool, w.segment_latent(si), w.segment_slots(si) + 64 * far, w.kv_scale, dev)
    table = np.where(w.block_table >= 0, w.block_table + far, -1)
    out, lse, ws = buffers(w.batch, 2, 16, dev)
    binding.mla_decode(bf16_tensor(w.q_bits, dev), pool, _i32(table, dev), _i32(w.seq_lens, dev), w.sm_scale, w.kv_scale,
                       out, lse, ws)
    assert_close(out.float().cpu().numpy(), lse.cpu().numpy(), *reference(w, ref_pages), what="far pages")
    total = int(w.seq_lens.sum())
    latent = torch.empty((total, 512), dtype=torch.bfloat16, device=dev)
    rope = torch.empty((total, 64), dtype=torch.bfloat16, device=dev)
    cu = np.concatenate([[0], np.cumsum(w.seq_lens)])
    binding.mla_kv_gather(pool, w.kv_scale, _i32(table, dev), _i32(cu, dev), latent, rope)
    got = torch.cat([latent, rope], 1).view(torch.int16).cpu().numpy().view(np.uint16)
    values = oe2m1.decode_pages(ref_pages, 1.0).reshape(-1, 576)
    want = np.concatenate([values[(w.block_table[b, np.arange(n) // 64] * 64 + np.arange(n) % 64)]
                           for b, n in enumerate(w.seq_lens)])
    assert np.array_equal(got, wl.f32_to_bf16_bits(want.astype(np.float32) * np.float32(w.kv_scale)))


def test_gather_from_a_large_e4m3_pool(cuda_device):
    dev, pages = cuda_device, 130_000                    # 4.8 GB
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 0x7F, (2, 64, 576)).astype(np.uint8)
    pool = torch.empty((pages, 64, 576), dtype=torch.uint8, device=dev)
    pool[-2:] = torch.from_numpy(codes).to(dev)
    latent = torch.empty((100, 512), dtype=torch.bfloat16, device=dev)
    rope = torch.empty((100, 64), dtype=torch.bfloat16, device=dev)
    binding.mla_kv_gather(pool, 1.0, _i32([[pages - 1, pages - 2]], dev), _i32([0, 100], dev), latent, rope,
                          starts=_i32([20], dev))
    want = oe4m3.decode(codes[::-1]).reshape(-1, 576)[20:120]
    assert np.array_equal(torch.cat([latent, rope], 1).float().cpu().numpy(), want)  # 4 bits: exact in bf16


def test_block_table_beyond_2_31_entries(cuda_device):
    """The last of 65 requests with the widest block table there is."""
    dev, width, B = cuda_device, 0x7FFFFFFF // 64, 65
    table = torch.empty((B, width), dtype=torch.int32, device=dev)
    table[B - 1, :2] = torch.tensor([7, 3], dtype=torch.int32, device=dev)
    lens, new, held = np.zeros(B), np.zeros(B), np.zeros(B)
    lens[-1], new[-1], held[-1] = 100, 200, 2
    slots, cu = _i32(np.zeros(201), dev), _i32(np.zeros(B + 1), dev)
    lens_out, held_out, count_out, status = (_i32(np.zeros(n), dev) for n in (B, B, 1, B))
    binding.mla_kv_alloc(_i32(lens, dev), _i32(new, dev), _i32(held, dev), _i32([11, 12, 13, 14, 15], dev), _i32([5], dev),
                         16, table, lens_out, held_out, count_out, cu, slots, status)
    pos = np.arange(100, 300)
    want = np.array([7, 3, 15, 14, 13])[pos // 64] * 64 + pos % 64
    assert np.array_equal(slots.cpu().numpy(), np.append(want, -1))
    assert table[B - 1, :5].tolist() == [7, 3, 15, 14, 13] and int(count_out) == 2
    assert (status == 0).all() and int(lens_out[-1]) == 300 and int(held_out[-1]) == 5


@pytest.mark.parametrize("dtype,stride", [(torch.float32, 1_100_000_004), (torch.bfloat16, 2_200_000_001)])
def test_probability_rows_far_apart(cuda_device, dtype, stride):
    dev, V = cuda_device, 1000
    rng = np.random.default_rng(3)
    p = torch.from_numpy(rng.dirichlet(np.ones(V), (1, 3)).astype(np.float32)).to(dtype)
    q = torch.from_numpy(rng.dirichlet(np.ones(V), (1, 2)).astype(np.float32)).to(dtype)
    wide = torch.empty(2 * stride + V, dtype=dtype, device=dev)
    tp, tq = wide.as_strided((1, 3, V), (3 * stride, stride, 1)), wide.as_strided((1, 2, V), (2 * stride, stride, 1), V)
    tp.copy_(p)
    tq.copy_(q)
    tokens = np.array([[5, 6]])
    for u in ([0.0, 0.0, 0.7], [0.0, 1.0, 0.4], [1.0, 0.0, 0.2]):
        out, acc = _i32([[0, 0, 0]], dev), _i32([0], dev)
        binding.mla_verify_drafts(tp, tq, _i32(tokens, dev), torch.tensor([u], device=dev), out, acc)
        want, a = over.verify(p[0].float().numpy(), q[0].float().numpy(), tokens[0], np.float32(u))
        assert out.tolist() == [want] and acc.tolist() == [a]


def test_rows_that_sum_past_16_end_with_a_token_or_none(cuda_device):
    """Not probabilities, but nothing is left unwritten or out of range."""
    p = torch.ones((4, 2, 9000), device=cuda_device)
    q = torch.zeros((4, 1, 9000), device=cuda_device)
    for u in (0.0, 0.5, 0.999):
        out, acc = _i32(np.full((4, 2), -7), cuda_device), _i32([-7] * 4, cuda_device)
        binding.mla_verify_drafts(p, q, _i32([[3]] * 4, cuda_device), torch.full((4, 2), u, device=cuda_device), out, acc)
        assert ((out >= -1) & (out < 9000)).all() and (acc >= 0).all()


def test_two_streams_at_once(cuda_device):
    """Independent calls in flight together, each with its own outputs and workspace."""
    dev = cuda_device
    work = []
    for k in range(2):
        w = wl.make_lengths_workload("two", 410 + k, [3000, 500, 64 + k], num_heads=64)
        pages, ref_pages = fill(w, dev)
        work.append((w, pages, ref_pages, bf16_tensor(w.q_bits, dev), _i32(w.block_table, dev), _i32(w.seq_lens, dev),
                     buffers(w.batch, 1, 64, dev), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for w, pages, _, q, table, lens, (out, lse, ws), stream in work:
            binding.mla_decode(q, pages, table, lens, w.sm_scale, w.kv_scale, out, lse, ws, stream=stream)
    torch.cuda.synchronize()
    for w, _, ref_pages, _, _, _, (out, lse, ws), _ in work:
        assert binding.read_device_status(ws) == 0
        assert_close(out.float().cpu().numpy(), lse.cpu().numpy(), *reference(w, ref_pages), what="two streams")


def test_stalled_4_bit_pipeline_ends(cuda_device):
    """The test build whose QK issuer never passes its third page: every role, the expanders
    among them, gives up (waits of 20 ms), the status says so and the device stays usable."""
    dev = cuda_device
    stall = binding.open_library(mla_build.STALL_LIB_PATH)
    w = wl.make_lengths_workload("stall", 420, [5000, 3000], num_heads=64)
    pages, ref_pages = fill(w, dev)
    q, table, lens = bf16_tensor(w.q_bits, dev), _i32(w.block_table, dev), _i32(w.seq_lens, dev)
    ctas = 4  # every CTA holds more than two pages, so every CTA reaches the stall
    out, lse, ws = buffers(w.batch, 1, 64, dev, binding.mla_decode_workspace_size(w.batch, 1, 64, ctas))
    st = stall.mla_decode(q.data_ptr(), pages.data_ptr(), pages.shape[0], 64, binding.MLA_KV_E2M1, table.data_ptr(),
                          table.shape[1], lens.data_ptr(), w.batch, 1, 64, w.sm_scale, w.kv_scale, ctas, ws.data_ptr(),
                          ws.numel(), out.data_ptr(), lse.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == binding.MLA_OK
    torch.cuda.synchronize()
    assert binding.read_device_status(ws) & binding.MLA_DEVICE_ERR_TIMEOUT
    ws.zero_()
    binding.mla_decode(q, pages, table, lens, w.sm_scale, w.kv_scale, out, lse, ws, num_ctas=ctas)
    assert binding.read_device_status(ws) == 0
    assert_close(out.float().cpu().numpy(), lse.cpu().numpy(), *reference(w, ref_pages), what="after the stall")
