"""The binding refuses, for every entry point, tensors whose pointer the library cannot use: host
tensors, strided ones, arrays that are too short."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from paged_mla_decode_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _check_args(dev):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    return [i32(4), i32(2, 3), i32(2, 3), i32(2), i32(2), i32(2)]


def _combine_args(dev):
    return [torch.zeros(3, 2, 512, device=dev), torch.zeros(3, 2, device=dev),
            torch.zeros(2, 512, dtype=torch.bfloat16, device=dev), torch.zeros(2, device=dev)]


@pytest.mark.parametrize("call,args", [(binding.mla_kv_check, _check_args), (binding.mla_decode_combine, _combine_args)])
def test_host_tensors(call, args):
    with pytest.raises(AssertionError):
        call(*args("cpu"))


@pytest.mark.gpu
@pytest.mark.parametrize("call,args", [(binding.mla_kv_check, _check_args), (binding.mla_decode_combine, _combine_args)])
def test_each_tensor_of_the_small_calls(cuda_device, call, args):
    good = args(cuda_device)
    call(*good)
    for k, t in enumerate(good):
        wide = torch.zeros((*t.shape, 2), dtype=t.dtype, device=cuda_device)[..., 0]
        for bad in (t.cpu(), wide):
            with pytest.raises(AssertionError):
                call(*good[:k], bad, *good[k + 1:])
    torch.cuda.synchronize()


def _decode_args(dev, heads=16):
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    return {"q": torch.zeros(4, 1, heads, 576, dtype=torch.bfloat16, device=dev),
            "kv_pages": torch.zeros(8, 64, 576, dtype=torch.uint8, device=dev), "block_table": i32(np.arange(8).reshape(4, 2)),
            "seq_lens": i32([70, 64, 1, 100]), "sm_scale": 0.1, "kv_scale": 1.0,
            "out": torch.zeros(4, 1, heads, 512, dtype=torch.bfloat16, device=dev), "lse": torch.zeros(4, 1, heads, device=dev)}


@pytest.mark.gpu
def test_prefix_pages_of_a_grouped_decode(cuda_device):
    a = _decode_args(cuda_device)
    ws = torch.zeros(binding.mla_decode_grouped_workspace_size(4, 1, 16), dtype=torch.uint8, device=cuda_device)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    call = lambda p, forks=2: binding.mla_decode_grouped(**a, forks=forks, prefix_pages=p, workspace=ws)  # noqa: E731
    call(i32([0, 0]))
    for bad in (i32([0]), i32([]), torch.zeros(2, dtype=torch.int32), i32([0, 0, 0, 0])[::2], i32([0, 0]).long()):
        with pytest.raises(AssertionError):
            call(bad)
    for forks in (0, 3, 400):  # groups that cannot be cut: the library's refusal
        with pytest.raises(binding.MlaError):
            call(i32([0] * 4), forks)
    torch.cuda.synchronize()
    assert binding.read_device_status(ws) == 0


@pytest.mark.gpu
def test_device_status_of_the_static_scratch(cuda_device):
    a = _decode_args(cuda_device)
    status = torch.full((1,), 9, dtype=torch.int32, device=cuda_device)
    binding.mla_decode_static_scratch(**a, device_status=status)
    assert int(status) == 0
    for bad in (status.cpu(), status[:0], status.long()):
        with pytest.raises(AssertionError):
            binding.mla_decode_static_scratch(**a, device_status=bad)


def test_refusals_stand_without_assert_statements():
    """python -O drops assert statements; the checks stay. (Host tensors, so that no call could
    reach a kernel.)"""
    code = """
import torch
from paged_mla_decode_gb300 import binding as b
bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
f32 = lambda *s: torch.zeros(s)
pages = torch.zeros(2, 64, 576, dtype=torch.uint8)
dec = (bf(1, 1, 16, 576), pages, i32(1, 2), i32(1))
out = (bf(1, 1, 16, 512), f32(1, 1, 16))
ws = torch.zeros(9, dtype=torch.uint8)
calls = {
    "append": lambda: b.mla_kv_append(bf(3, 512), bf(3, 64), i32(3), pages, 1.0),
    "decode": lambda: b.mla_decode(*dec, 0.1, 1.0, *out, ws),
    "grouped": lambda: b.mla_decode_grouped(*dec, 1, i32(1), 0.1, 1.0, *out, ws),
    "static": lambda: b.mla_decode_static_scratch(*dec, 0.1, 1.0, *out),
    "combine": lambda: b.mla_decode_combine(f32(2, 3, 512), f32(2, 3), bf(3, 512), f32(3)),
    "check": lambda: b.mla_kv_check(i32(2), i32(1, 2), i32(1, 2), i32(1), i32(1), i32(1)),
    "gather": lambda: b.mla_kv_gather(pages, 1.0, i32(1, 2), i32(2), bf(3, 512), bf(3, 64)),
    "alloc": lambda: b.mla_kv_alloc(i32(1), i32(1), i32(1), i32(4), i32(1), 4, i32(1, 2), i32(1), i32(1), i32(1),
                                    i32(2), i32(3), i32(1)),
    "verify": lambda: b.mla_verify_drafts(f32(1, 2, 5), None, i32(1, 1), f32(1, 2), i32(1, 2), i32(1)),
    "pages": lambda: b.kv_dtype_code(pages[:, :, :575]),
    "stride": lambda: b._row_stride(f32(2, 3, 10)[..., ::2]),
}
b.load_library = lambda *a: print("reached the library")
for name, call in calls.items():
    try:
        call()
    except AssertionError as e:
        print(name, "refused")
"""
    for flags in ([], ["-O"]):
        run = subprocess.run([sys.executable, *flags, "-c", code], capture_output=True, text=True, cwd=ROOT)
        got = run.stdout.split("\n")[:-1]
        assert run.returncode == 0 and len(got) == 11, run.stdout + run.stderr
        assert all(line.endswith(" refused") for line in got), got
