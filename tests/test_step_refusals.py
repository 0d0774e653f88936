"""Refusals of the step's operators, before anything is enqueued (CPU; no CUDA call is made)."""

import ctypes

import pytest
import torch

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import build as mbuild

FAKE = ctypes.c_void_p(1 << 20)      # never dereferenced: the checks fail first
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return binding.load_library()


def test_e2m1_append_and_decode(lib):
    app = lambda n, dt, scale, kv=FAKE: lib.mla_kv_append(FAKE, FAKE, FAKE, n, kv, 10, 64, dt, scale, None)  # noqa: E731
    assert app(0, 2, 1.0) == 0
    for scale in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 101):
        assert app(0, 2, scale) == 1
    assert app(0, 2, 2.0 ** -100) == 0 and app(0, 2, 2.0 ** 100) == 0
    assert app(1, 2, 1.0, kv=ctypes.c_void_p((1 << 20) + 8)) == 1
    assert app(1, 3, 1.0) == 1
    dec = lambda fn, scale, dt=2: fn(FAKE, FAKE, 10, 64, dt, FAKE, 4, FAKE, 0, 1, 64, 0.1, scale, 0,  # noqa: E731
                                     None, 0, FAKE, FAKE, None)
    assert dec(lib.mla_decode, 1.0) == 0
    assert dec(lib.mla_decode, 2.0 ** 101) == 1
    assert dec(lib.mla_decode, 1.0, dt=3) == 1
    assert dec(lib.mla_decode_f16_operands, 1.0) == 2


def _gather(lib, **kw):
    a = dict(kv=FAKE, pages=10, ps=64, dt=2, scale=1.0, table=FAKE, mp=4, starts=None, cu=FAKE, batch=1, n=0,
             lat=FAKE, rope=FAKE)
    a.update(kw)
    return lib.mla_kv_gather(a["kv"], a["pages"], a["ps"], a["dt"], a["scale"], a["table"], a["mp"], a["starts"],
                             a["cu"], a["batch"], a["n"], a["lat"], a["rope"], None)


def test_gather(lib):
    assert _gather(lib) == 0 and _gather(lib, batch=0, n=5) == 0
    for bad in (dict(batch=-1), dict(n=-1), dict(pages=-1), dict(mp=0), dict(dt=3), dict(scale=0.0),
                dict(scale=float("nan")), dict(dt=1, scale=0.5), dict(scale=2.0 ** 101),
                dict(n=1, kv=None), dict(n=1, table=None), dict(n=1, cu=None), dict(n=1, lat=None),
                dict(n=1, rope=None), dict(n=1, kv=ODD), dict(n=1, lat=ODD), dict(n=1, cu=ODD), dict(n=1, starts=ODD)):
        assert _gather(lib, **bad) == 1, bad
    assert _gather(lib, ps=32) == 2
    assert _gather(lib, n=1 << 31) == 2


def _alloc(lib, **kw):
    a = dict(lens=FAKE, new=FAKE, batch=1, ps=64, held=FAKE, free=FAKE, count=FAKE, cap=4, pages=10, table=FAKE, mp=4,
             tags=None, expected=None, lo=FAKE, ho=FAKE, co=FAKE, cu=FAKE, slots=FAKE, n=4, status=FAKE)
    a.update(kw)
    return lib.mla_kv_alloc(*[a[k] for k in ("lens", "new", "batch", "ps", "held", "free", "count", "cap", "pages",
                                             "table", "mp", "tags", "expected", "lo", "ho", "co", "cu", "slots", "n",
                                             "status")], None)


def test_alloc(lib):
    for bad in [dict(batch=-1), dict(cap=-1), dict(pages=-1), dict(mp=0), dict(n=-1), dict(tags=FAKE),
                dict(expected=FAKE), dict(slots=ODD)] + [{k: None} for k in
                                                         ("lens", "new", "held", "free", "count", "table", "lo", "ho",
                                                          "co", "cu", "slots", "status")]:
        assert _alloc(lib, **bad) == 1, bad
    for bad in (dict(ps=16), dict(pages=1 << 26), dict(n=1 << 31), dict(mp=1 << 26)):
        assert _alloc(lib, **bad) == 2, bad


def _verify(lib, **kw):
    a = dict(p=FAKE, ps=100, q=FAKE, qs=100, dt=0, tok=FAKE, u=FAKE, k=None, lens=None, batch=1, drafts=3, vocab=100,
             out=FAKE, acc=FAKE, lo=None)
    a.update(kw)
    return lib.mla_verify_drafts(*[a[k] for k in ("p", "ps", "q", "qs", "dt", "tok", "u", "k", "lens", "batch",
                                                  "drafts", "vocab", "out", "acc", "lo")], None)


def test_verify(lib):
    assert _verify(lib, batch=0) == 0
    for bad in [dict(batch=-1), dict(drafts=-1), dict(drafts=32), dict(vocab=0), dict(dt=2), dict(ps=99), dict(qs=99),
                dict(lo=FAKE), dict(p=ODD), dict(q=ODD), dict(dt=1, p=ctypes.c_void_p((1 << 20) + 1)), dict(u=ODD),
                dict(out=ODD)] + [{k: None} for k in ("p", "tok", "u", "out", "acc")]:
        assert _verify(lib, **bad) == 1, bad


def test_binding_refuses_what_the_library_cannot_see():
    """Host tensors, wrong types, shapes and strides never reach a kernel."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    page = torch.zeros((2, binding.MLA_E2M1_PAGE_BYTES), dtype=torch.uint8)
    assert binding.kv_dtype_code(page) == binding.MLA_KV_E2M1
    for bad in (page[:, :-1].contiguous(), torch.zeros((2, 2 * binding.MLA_E2M1_PAGE_BYTES), dtype=torch.uint8)[:, ::2]):
        with pytest.raises(AssertionError):
            binding.kv_dtype_code(bad)
    with pytest.raises(AssertionError):
        binding.mla_kv_gather(page, 1.0, i32(1, 2), i32(2), torch.zeros(3, 512).bfloat16(), torch.zeros(3, 64).bfloat16())
    with pytest.raises(AssertionError):
        binding.mla_kv_alloc(i32(1), i32(1), i32(1), i32(4), i32(1), 4, i32(1, 2), i32(1), i32(1), i32(1), i32(2), i32(3),
                             i32(1))
    with pytest.raises(AssertionError):
        binding.mla_verify_drafts(torch.zeros(1, 2, 5), None, i32(1, 1), torch.zeros(1, 2), i32(1, 2), i32(1))
    bf = lambda *s: torch.zeros(s).bfloat16()  # noqa: E731
    with pytest.raises(AssertionError):
        binding.mla_kv_append(bf(3, 512), bf(3, 64), i32(3), page, 1.0)
    with pytest.raises(AssertionError):
        binding.mla_decode(bf(1, 1, 16, 576), page, i32(1, 2), i32(1), 0.1, 1.0, bf(1, 1, 16, 512), torch.zeros(1, 1, 16),
                           torch.zeros(9, dtype=torch.uint8))
    probs = torch.zeros(2, 3, 10)
    assert binding._row_stride(probs) == 10 and binding._row_stride(probs[..., :7]) == 10
    assert binding._row_stride(probs[:, :1]) == 30
    for bad in (probs[..., ::2], probs.transpose(0, 1), probs[:, :2]):
        with pytest.raises(AssertionError):
            binding._row_stride(bad)
