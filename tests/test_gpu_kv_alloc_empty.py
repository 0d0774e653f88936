"""mla_kv_alloc with tags and no request, or no page: arrays without an entry, whose address may
be NULL, are not taken for missing ones (GPU)."""

import pytest
import torch

from paged_mla_decode_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slots", [0, 7])
def test_no_request(cuda_device, slots):
    i32 = lambda *s: torch.full(s, 3, dtype=torch.int32, device=cuda_device)  # noqa: E731
    none, count, cu, out, tags = i32(0), i32(1), i32(1), i32(slots), i32(9)
    binding.mla_kv_alloc(none, none, none, i32(9), count, 9, i32(0, 4), none, none, count, cu, out, none,
                         page_tags=tags, expected_tags=i32(0, 4))
    assert int(count) == 3 and int(cu) == 0 and (out == -1).all() and (tags == 3).all()


def test_no_page(cuda_device):
    """Every free-list entry is outside a cache without pages."""
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    table, expected = i32([[-1, -1], [-1, -1]]), i32([[5, 5], [5, 5]])
    count, cu, slots, status, lens, held = i32([2]), i32([0] * 3), i32([9] * 8), i32([9] * 2), i32([0, 0]), i32([0, 0])
    binding.mla_kv_alloc(lens, i32([3, 2]), held, i32([4, 6]), count, 0, table, lens, held, count, cu, slots, status,
                         page_tags=i32([]), expected_tags=expected)
    assert table.tolist() == [[6, -1], [4, -1]] and (expected == 5).all() and (slots == -1).all()
    assert cu.tolist() == [0, 3, 5] and lens.tolist() == [3, 2] and held.tolist() == [1, 1] and int(count) == 0
    assert (status == 0).all()
