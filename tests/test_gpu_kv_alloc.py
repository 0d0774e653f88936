"""mla_kv_alloc equals the request-by-request oracle in every output (GPU, whole numbers)."""

import numpy as np
import pytest
import torch

from oracle import paging
from paged_mla_decode_gb300 import binding

pytestmark = pytest.mark.gpu


def _inputs(seed, B, cached, new, spare=50, num_slots=None, tags=True, width=None, bad=0):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, cached + 1, B)
    n = rng.integers(0, new + 1, B)
    held = -(-lens // 64) + rng.integers(0, 2, B)
    need = int(np.maximum(-(-(lens + n) // 64) - held, 0).sum())
    free = max(0, need + spare)
    pages = int(held.sum()) + free + 2
    perm = rng.permutation(pages)
    w = int(max(held.max(initial=0), (-(-(lens + n) // 64)).max(initial=0), 1)) if width is None else width
    table = np.full((B, w), -1, np.int64)
    at = 0
    for b in range(B):
        k = min(int(held[b]), w)
        table[b, :k] = perm[at:at + k]
        at += k
    pool = perm[at:at + free + 1]  # one entry more than is free
    for b in rng.integers(0, B, bad):
        kind = rng.integers(0, 4)
        if kind == 0:
            lens[b] = -1
        elif kind == 1:
            n[b] = -3
        elif kind == 2:
            held[b] = w + 1
        else:
            held[b], lens[b] = 0, 70
    return {"lens": lens, "new": n, "held": held, "free": pool, "count": free, "pages": pages, "table": table,
            "slots": int(np.maximum(n, 0).sum()) + 3 if num_slots is None else num_slots,
            "tags": rng.integers(0, 1 << 32, pages).astype(np.uint32) if tags else None,
            "expected": rng.integers(0, 1 << 32, (B, w)).astype(np.uint32) if tags else None}


def _device(c, dev):
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(dev)  # noqa: E731
    B = len(c["lens"])
    d = {"lens": i32(c["lens"]), "new": i32(c["new"]), "held": i32(c["held"]), "free": i32(c["free"]),
         "count": i32([c["count"]]), "table": i32(c["table"]).reshape(B, -1), "lens_out": i32([-9] * B), "held_out": i32([-9] * B),
         "count_out": i32([-9]), "cu": i32([-9] * (B + 1)), "slots": i32([-9] * c["slots"]), "status": i32([-9] * B),
         "tags": None, "expected": None}
    if c["tags"] is not None:
        d["tags"], d["expected"] = i32(c["tags"].view(np.int32)), i32(c["expected"].view(np.int32))
    return d


def _call(c, d, stream=None):
    binding.mla_kv_alloc(d["lens"], d["new"], d["held"], d["free"], d["count"], c["pages"], d["table"], d["lens_out"],
                         d["held_out"], d["count_out"], d["cu"], d["slots"], d["status"], page_tags=d["tags"],
                         expected_tags=d["expected"], stream=stream)


def _oracle(c):
    return paging.alloc(c["lens"], c["new"], c["held"], c["free"], c["count"], c["pages"], c["table"], c["slots"],
                        c["tags"], c["expected"])


def _same(d, want, what=""):
    for key, name in (("lens_out", "seq_lens_out"), ("held_out", "pages_held_out"), ("count_out", "free_count_out"),
                      ("cu", "cu_tokens"), ("slots", "slot_mapping"), ("status", "request_status"),
                      ("table", "block_table"), ("tags", "page_tags"), ("expected", "expected_tags")):
        if d[key] is None:
            continue
        got = d[key].cpu().numpy()
        ref = np.asarray(want[name])
        got = got.view(np.uint32) if ref.dtype == np.uint32 else got
        assert np.array_equal(got.reshape(ref.shape), ref), f"{what}: {name}"


@pytest.mark.parametrize("B,cached,new", [(1, 0, 1), (1, 64, 0), (1, 100000, 70000), (3, 200, 4), (7, 5000, 300),
                                          (256, 1000, 4), (1023, 100, 5), (1024, 100, 5), (1025, 100, 5),
                                          (2500, 300, 9), (33, 3000, 9000), (5000, 64, 40)])
@pytest.mark.parametrize("spare", [40, -7])
def test_matches_oracle(cuda_device, B, cached, new, spare):
    c = _inputs(B + 100 + spare, B, cached, new, spare=spare, tags=B % 2 == 1)
    d = _device(c, cuda_device)
    _call(c, d)
    _same(d, _oracle(c), f"B={B}")


@pytest.mark.parametrize("B,new,num_slots,width", [(40, 200, 1500, None), (40, 200, None, 4), (40, 200, 0, None),
                                                   (1500, 60, 20000, 3), (64, 6000, 150000, 60)])
def test_refusals_and_bad_requests(cuda_device, B, new, num_slots, width):
    c = _inputs(B + new, B, 400 if width is None else 64 * width, new, num_slots=num_slots, width=width, bad=B // 4)
    c["free"][::5] = -1
    c["free"][1::7] = c["pages"] + 3
    d = _device(c, cuda_device)
    _call(c, d)
    want = _oracle(c)
    assert len(set(want["request_status"].tolist())) > 1
    _same(d, want)


@pytest.mark.parametrize("B,new,num_slots,bad", [(2, 30000, None, 0), (6, 30000, None, 3), (9, 20000, 70000, 2),
                                                 (3, 13000, None, 1)])
def test_long_requests(cuda_device, B, new, num_slots, bad):
    """Runs of rows within one or two long requests, some of them refused, with bad free pages."""
    c = _inputs(B + new, B, 3000, new, num_slots=num_slots, bad=bad)
    c["free"][::9] = -1
    c["free"][4::11] = c["pages"]
    d = _device(c, cuda_device)
    _call(c, d)
    want = _oracle(c)
    assert len(want["slot_mapping"]) >= 4096 * B and (want["slot_mapping"] >= 0).any()
    _same(d, want)


@pytest.mark.parametrize("count", [-5, 0, 10 ** 6])
def test_free_count_is_clamped_to_the_list(cuda_device, count):
    c = _inputs(3, 5, 100, 200)
    c["count"] = count
    d = _device(c, cuda_device)
    _call(c, d)
    _same(d, _oracle(c))


def test_in_place_and_captured(cuda_device):
    """Outputs on their inputs, replayed: the requests grow step by step, twice over a stream."""
    c = _inputs(11, 70, 500, 3, spare=400)
    c["table"] = np.concatenate([c["table"], np.full((70, 8), -1)], 1)
    c["expected"] = np.zeros_like(c["table"], dtype=np.uint32)
    d = _device(c, cuda_device)
    d["lens_out"], d["held_out"], d["count_out"] = d["lens"], d["held"], d["count"]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        _call(c, d)
    for step in range(40):
        graph.replay()
        want = _oracle(c)
        _same(d, want, f"step {step}")
        c.update(lens=want["seq_lens_out"], held=want["pages_held_out"], count=want["free_count_out"],
                 table=want["block_table"], tags=want["page_tags"], expected=want["expected_tags"])


def test_large_call_in_place(cuda_device):
    """Whole contexts admitted at once, outputs on their inputs, two calls in a row."""
    c = _inputs(12, 48, 0, 20000, spare=2000)
    c["table"] = np.concatenate([c["table"], np.full((48, 400), -1)], 1)
    c["expected"] = np.zeros_like(c["table"], dtype=np.uint32)
    d = _device(c, cuda_device)
    d["lens_out"], d["held_out"], d["count_out"] = d["lens"], d["held"], d["count"]
    for step in range(2):
        _call(c, d)
        want = _oracle(c)
        _same(d, want, f"call {step}")
        c.update(lens=want["seq_lens_out"], held=want["pages_held_out"], count=want["free_count_out"],
                 table=want["block_table"], tags=want["page_tags"], expected=want["expected_tags"])


def test_empty_batch(cuda_device):
    i32 = lambda *s: torch.full(s, 5, dtype=torch.int32, device=cuda_device)  # noqa: E731
    count, cu, slots = i32(1), i32(1), i32(4)
    none = i32(0)
    binding.mla_kv_alloc(none, none, none, i32(9), count, 9, i32(0, 3), none, none, count, cu, slots, none)
    assert int(count) == 5 and int(cu) == 0 and (slots == -1).all()
