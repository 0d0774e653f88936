"""mla_kv_gather equals the stored values rounded to bfloat16 (GPU).

value * kv_scale is one float32 product (4 or fewer significant bits times 24) rounded to
bf16: bit for bit the same in numpy, so no tolerance is needed.
"""

import numpy as np
import pytest
import torch

from oracle import e2m1 as oe2m1
from oracle import e4m3 as oe4m3
from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .gpu_util import bf16_tensor

pytestmark = pytest.mark.gpu


def _pool(rng, cache, pages, dev):
    """Random stored bytes of every kind, and their values as float32 [pages, 64, 576]."""
    if cache == "bf16":
        bits = rng.integers(0, 1 << 16, (pages, 64, 576)).astype(np.uint16)
        return bf16_tensor(bits, dev), bits
    if cache == "e4m3":
        codes = rng.integers(0, 256, (pages, 64, 576)).astype(np.uint8)
        return torch.from_numpy(codes).to(dev), oe4m3.decode(codes).astype(np.float32)
    raw = rng.integers(0, 256, (pages, oe2m1.PAGE_BYTES)).astype(np.uint8)
    return torch.from_numpy(raw).to(dev), oe2m1.decode_pages(raw, 1.0).astype(np.float32)


def _case(dev, cache, lens, starts, seed=0, tail=3, scale=wl.KV_SCALE):
    rng = np.random.default_rng(seed)
    scale = 1.0 if cache == "bf16" else scale
    s = [0] * len(lens) if starts is None else starts
    need = [-(-(a + n) // 64) for a, n in zip(s, lens)]
    pages = sum(need) + 2
    perm = rng.permutation(pages)
    table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    pool, values = _pool(rng, cache, pages, dev)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    total = int(cu[-1])
    latent = torch.full((total + tail, 512), 7.0, dtype=torch.bfloat16, device=dev)
    rope = torch.full((total + tail, 64), 7.0, dtype=torch.bfloat16, device=dev)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=dev)
    binding.mla_kv_gather(pool, scale, torch.from_numpy(table).to(dev), torch.from_numpy(cu).to(dev), latent, rope,
                          starts=st)
    got = torch.cat([latent, rope], 1).view(torch.int16).cpu().numpy().view(np.uint16)
    want = []
    for b, n in enumerate(lens):
        pos = s[b] + np.arange(n)
        want.append(values[table[b, pos // 64], pos % 64])
    want = np.concatenate(want) if want else np.zeros((0, 576), values.dtype)
    if cache != "bf16":
        nan = np.isnan(want)
        want = wl.f32_to_bf16_bits(np.where(nan, 0, want) * np.float32(scale))
        assert ((got[:total] & 0x7FFF) > 0x7F80)[nan].all()
        assert np.array_equal(got[:total][~nan], want[~nan])
    else:
        assert np.array_equal(got[:total], want)
    assert (got[total:] == 0x40E0).all()  # rows behind the last range keep their 7.0


@pytest.mark.parametrize("cache", ["e2m1", "e4m3", "bf16"])
@pytest.mark.parametrize("lens,starts", [([1], None), ([64], [64]), ([65, 0, 1, 130], [3, 700, 63, 0]),
                                         ([0, 0], None), ([777, 1024, 5], [0, 11, 62]), ([9000, 20000], None)])
def test_ranges(cuda_device, cache, lens, starts):
    _case(cuda_device, cache, lens, starts)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -100, 2.0 ** 100, 0.3])
def test_scales(cuda_device, scale):
    _case(cuda_device, "e2m1", [100, 30], [5, 60], scale=float(np.float32(scale)))


def test_many_requests(cuda_device):
    rng = np.random.default_rng(4)
    _case(cuda_device, "e2m1", rng.integers(0, 4, 1500).tolist(), rng.integers(0, 70, 1500).tolist())


def test_pages_outside_the_cache_and_beyond_the_table_are_zero_rows(cuda_device):
    pool = torch.full((4, binding.MLA_E2M1_PAGE_BYTES), 0x77, dtype=torch.uint8, device=cuda_device)
    table = torch.tensor([[0, 4], [-1, 3]], dtype=torch.int32, device=cuda_device)
    cu = torch.tensor([0, 130, 200], dtype=torch.int32, device=cuda_device)
    latent = torch.full((190, 512), 7.0, dtype=torch.bfloat16, device=cuda_device)
    rope = torch.full((190, 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    starts = torch.tensor([0, -6], dtype=torch.int32, device=cuda_device)
    binding.mla_kv_gather(pool, 1.0, table, cu, latent, rope, starts=starts)
    zero = (latent == 0).all(1).cpu().numpy() & (rope == 0).all(1).cpu().numpy()
    assert not zero[:64].any() and zero[64:].all()          # page 4, the table's end, token -6, page -1
    binding.mla_kv_gather(pool, 1.0, table, cu, latent, rope, starts=torch.tensor([0, 64], dtype=torch.int32,
                                                                                device=cuda_device))
    zero = (latent == 0).all(1).cpu().numpy()
    assert zero[64:130].all() and not zero[130:].any()      # the last rows of the second range are cut


def test_captured_and_side_stream(cuda_device):
    rng = np.random.default_rng(6)
    raw = rng.integers(0, 225, (3, oe2m1.PAGE_BYTES)).astype(np.uint8) & 0x77
    pool = torch.from_numpy(raw).to(cuda_device)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=cuda_device)
    cu = torch.tensor([0, 150], dtype=torch.int32, device=cuda_device)
    latent = torch.zeros((150, 512), dtype=torch.bfloat16, device=cuda_device)
    rope = torch.zeros((150, 64), dtype=torch.bfloat16, device=cuda_device)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        binding.mla_kv_gather(pool, 1.0, table, cu, latent, rope)
    for order in ([2, 0, 1], [1, 2, 0]):
        table.copy_(torch.tensor([order], dtype=torch.int32))
        graph.replay()
        want = oe2m1.decode_pages(raw[order], 1.0).reshape(-1, 576)[:150]
        got = torch.cat([latent, rope], 1).float().cpu().numpy()
        assert np.array_equal(got, want)  # at most 2 significant bits: exact in bf16
