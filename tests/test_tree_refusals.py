"""Refusals of the tree operators, before anything is enqueued (CPU; no kernel is launched)."""

import ctypes

import pytest
import torch

from paged_mla_decode_gb300 import binding
from paged_mla_decode_gb300 import build as mbuild

FAKE = ctypes.c_void_p(1 << 20)      # never dereferenced: the checks fail first
ODD = ctypes.c_void_p((1 << 20) + 2)
FOUR = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return binding.load_library()


def _call(fn, defaults, **kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values(), None)


def _tree(lib, **kw):
    return _call(lib.mla_decode_tree, dict(
        q=FAKE, kv=FAKE, pages=10, ps=64, dt=0, table=FAKE, mp=4, lens=FAKE, mask=FAKE, nodes=None, batch=1, n=8, heads=64,
        sm=0.1, scale=1.0, ctas=16, ws=FAKE, bytes=1 << 40, out=FAKE, lse=FAKE), **kw)


def test_decode_tree(lib):
    for bad in [dict(batch=-1), dict(pages=-1), dict(mp=0), dict(ctas=-1), dict(n=0), dict(n=65), dict(dt=3), dict(scale=0.0),
                dict(scale=float("inf")), dict(sm=float("nan")), dict(dt=2, scale=2.0 ** 101), dict(q=ODD), dict(kv=ODD),
                dict(table=ODD), dict(lens=ODD), dict(mask=FOUR), dict(nodes=ODD), dict(out=ODD), dict(lse=ODD)] + [
                    {k: None} for k in ("q", "kv", "table", "lens", "mask", "out", "lse")]:
        assert _tree(lib, **bad) == 1, bad
    for bad in (dict(heads=48), dict(heads=128), dict(ps=32), dict(mp=1 << 30, batch=4), dict(pages=1 << 26)):
        assert _tree(lib, **bad) == 2, bad
    for bad in (dict(ws=None), dict(ws=FOUR), dict(bytes=1000)):
        assert _tree(lib, **bad) == 3, bad
    assert _tree(lib, batch=0, q=None, ws=None) == 0
    size = lib.mla_decode_tree_workspace_size
    assert 0 < size(1, 1, 16, 8) <= size(1, 4, 16, 8) < size(1, 5, 16, 8) < size(2, 5, 16, 8) < size(2, 64, 64, 8)
    for bad in ((-1, 4, 64, 8), (1, 0, 64, 8), (1, 65, 64, 8), (1, 4, 48, 8), (1, 4, 64, -1)):
        assert size(*bad) == 0


def _probs(lib, **kw):
    return _call(lib.mla_logits_to_probs, dict(
        x=FAKE, xs=100, xt=0, p=ctypes.c_void_p(1 << 24), ps=100, pt=0, batch=1, rows=4, vocab=100, temp=None, nrows=None,
        tok=None, mask=None, counts=None, prompt=None, rep=None, freq=None, pres=None, bt=None, bv=None, nb=0, allowed=None), **kw)


def test_logits_to_probs(lib):
    for bad in [dict(batch=-1), dict(rows=0), dict(vocab=0), dict(nb=-1), dict(xt=2), dict(pt=-1), dict(xs=99), dict(ps=99),
                dict(tok=FAKE), dict(mask=FAKE), dict(tok=FAKE, mask=FAKE, rows=65), dict(tok=FAKE, mask=FOUR), dict(nb=1),
                dict(nb=1, bt=FAKE), dict(x=None), dict(p=None), dict(x=ODD), dict(p=ODD), dict(p=FAKE, pt=1),
                dict(p=FAKE, ps=104)] + [{k: ODD} for k in ("temp", "nrows", "counts", "prompt", "rep", "freq", "pres", "allowed")]:
        assert _probs(lib, **bad) == 1, bad
    for bad in (dict(vocab=393217, xs=393217, ps=393217), dict(nb=1025, bt=FAKE, bv=FAKE), dict(batch=1 << 28)):
        assert _probs(lib, **bad) == 2, bad
    assert _probs(lib, batch=0, x=None) == 0


def _verify(lib, **kw):
    return _call(lib.mla_verify_tree, dict(
        p=FAKE, ps=100, q=FAKE, qs=100, dt=0, tok=FAKE, mask=FAKE, u=FAKE, nodes=None, lens=None, batch=1, n=4, vocab=100,
        out=FAKE, path=FAKE, acc=FAKE, lo=None, counts=None), **kw)


def test_verify_tree(lib):
    for bad in [dict(batch=-1), dict(n=0), dict(n=65), dict(vocab=0), dict(dt=2), dict(ps=99), dict(qs=99), dict(lo=FAKE),
                dict(p=ODD), dict(q=ODD), dict(mask=FOUR)] + [{k: None} for k in ("p", "tok", "mask", "u", "out", "path", "acc")] + [
                    {k: ODD} for k in ("tok", "u", "nodes", "out", "path", "acc", "counts")]:
        assert _verify(lib, **bad) == 1, bad
    assert _verify(lib, vocab=(1 << 30) + 1, ps=1 << 31, qs=1 << 31) == 2
    assert _verify(lib, batch=1 << 29) == 2
    assert _verify(lib, batch=0, p=None) == 0


def _compact(lib, **kw):
    return _call(lib.mla_kv_compact, dict(
        kv=FAKE, layers=2, stride=10 * 36864, pages=10, ps=64, dt=0, table=FAKE, mp=4, lens=FAKE, path=FAKE, acc=FAKE,
        batch=1, n=4), **kw)


def test_kv_compact(lib):
    for bad in [dict(batch=-1), dict(layers=-1), dict(pages=-1), dict(mp=0), dict(n=0), dict(n=65), dict(dt=3),
                dict(stride=10 * 36864 - 16), dict(stride=10 * 36864 + 8), dict(dt=1), dict(kv=ODD), dict(lens=ODD)] + [
                    {k: None} for k in ("kv", "table", "lens", "path", "acc")]:
        assert _compact(lib, **bad) == 1, bad
    for bad in (dict(ps=16), dict(pages=1 << 26, stride=1 << 50), dict(layers=65536), dict(mp=1 << 30, batch=4)):
        assert _compact(lib, **bad) == 2, bad
    assert _compact(lib, batch=0) == 0 and _compact(lib, layers=0) == 0


def test_binding_refuses_host_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    mask = torch.zeros(2, 3, dtype=torch.int64)
    p = torch.zeros(2, 3, 10)
    for call in (lambda: binding.mla_logits_to_probs(p, p.clone()),
                 lambda: binding.mla_verify_tree(p, None, i32(2, 3), mask, torch.zeros(2, 3), i32(2, 3), i32(2, 3), i32(2)),
                 lambda: binding.mla_kv_compact(torch.zeros(4, 64, 576, dtype=torch.uint8), i32(2, 2), i32(2), i32(2, 3), i32(2)),
                 lambda: binding.mla_decode_tree(torch.zeros(2, 3, 16, 576, dtype=torch.bfloat16),
                                                 torch.zeros(4, 64, 576, dtype=torch.uint8), i32(2, 2), i32(2), mask, 0.1, 1.0,
                                                 torch.zeros(2, 3, 16, 512, dtype=torch.bfloat16), torch.zeros(2, 3, 16),
                                                 torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(AssertionError):
            call()
