"""Query heads of every magnitude that bfloat16 has (GPU)."""

import numpy as np
import pytest

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import workloads as wl

from .e2m1_util import fill, reference
from .gpu_util import assert_close, gpu_decode, gpu_fill_cache, oracle_decode, oracle_fill_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["e2m1", "e4m3", "f16 operands"])
@pytest.mark.parametrize("scale", ["as usual", "large"])
def test_tiny_heads(cuda_device, cache, scale):
    """Heads whose largest element is 2^-119 .. 2^-133 (every other element zero, the rest
    within 2^-6 of the largest): uniform attention at the usual scale, and the scores of an
    ordinary head where sm_scale makes up for it."""
    w = wl.make_lengths_workload("tiny heads", 520, [700, 65], num_heads=16)
    rng = np.random.default_rng(521)
    q = np.zeros((2, 1, 16, 576), np.float64)
    for h in range(16):
        top = -119 - h if h < 15 else -133
        steps = min(64, 2 ** (top + 133))
        q[:, :, h] = rng.integers(-steps, steps + 1, (2, 1, 576)) * (2.0 ** top / steps)
        q[:, :, h, ::2] = 0
        q[:, :, h, 1] = 2.0 ** top
    w.q_bits[:] = np.sign(q).astype(np.float32).view(np.uint32) >> 16 & 0x8000
    w.q_bits |= (np.abs(q).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    if scale == "large":
        w.sm_scale = float(np.float32(2.0 ** 122))
    if cache == "e2m1":
        pages, ref_pages = fill(w, cuda_device)
        ref = reference(w, ref_pages)
    else:
        pages, ref = gpu_fill_cache(w, cuda_device), oracle_decode(w, oracle_fill_cache(w))
    assert np.isfinite(ref[1]).all() and (np.abs(ref[1][0] - np.log(700)).max() > 0.1) == (scale == "large")
    out, lse, ws = gpu_decode(w, pages, cuda_device, f16_operands=cache == "f16 operands")
    assert binding.read_device_status(ws) == 0
    assert_close(out, lse, *ref, what=f"{cache}, {scale} scale")


@pytest.mark.parametrize("cache", ["e2m1", "e4m3", "bf16", "f16 operands"])
@pytest.mark.parametrize("bits", [0x7F80, 0xFF80])
def test_infinity_in_a_head(cuda_device, cache, bits):
    """Its scores are infinities of both signs, whose differences are NaN: its row alone is NaN."""
    w = wl.make_lengths_workload("infinite head", 522, [2000, 150], num_heads=16)
    kw = {"f16_operands": cache == "f16 operands"}
    if cache == "e2m1":
        pages, ref_pages = fill(w, cuda_device)
        ref_out, ref_lse = reference(w, ref_pages)
    else:
        dtype = "bf16" if cache == "bf16" else "e4m3"
        pages = gpu_fill_cache(w, cuda_device, dtype)
        ref_out, ref_lse = oracle_decode(w, oracle_fill_cache(w, dtype), dtype)
        if dtype == "bf16":
            kw["kv_scale"] = 1.0
    q = w.q_bits.copy()
    q[0, 0, 5, 33] = bits
    out, lse, _ = gpu_decode(w, pages, cuda_device, q_bits=q, **kw)
    assert np.isnan(lse[0, 0, 5]) and np.isnan(out[0, 0, 5]).all()
    rest = [h for h in range(16) if h != 5]
    assert_close(out[0, 0, rest], lse[0, 0, rest], ref_out[0, 0, rest], ref_lse[0, 0, rest], what="the other heads")
    assert_close(out[1], lse[1], ref_out[1], ref_lse[1], what="the other request")
