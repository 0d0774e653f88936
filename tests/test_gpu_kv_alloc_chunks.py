"""mla_kv_alloc over several chunks of 1,024 requests with a slot map of 4,096 entries a request
and more, where a warp takes 512 rows at once: chunks without new tokens, and chunks behind the
map's end (GPU, whole numbers against the oracle)."""

import numpy as np
import pytest

from .test_gpu_kv_alloc import _call, _device, _oracle, _same

pytestmark = pytest.mark.gpu


def _step(seed, lens, new, num_slots, free, width=16):
    """Requests in the middle of their lives (no page beyond their tokens' own)."""
    rng = np.random.default_rng(seed)
    lens, new = np.asarray(lens), np.asarray(new)
    held = -(-lens // 64)
    pages = int(held.sum()) + free + 3
    perm = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int64)
    at = np.concatenate([[0], np.cumsum(held)])
    for b in range(len(lens)):
        table[b, :held[b]] = perm[at[b]:at[b + 1]]
    return {"lens": lens, "new": new, "held": held, "free": perm[at[-1]:at[-1] + free + 1], "count": free, "pages": pages,
            "table": table, "slots": num_slots, "tags": rng.integers(0, 1 << 32, pages).astype(np.uint32),
            "expected": rng.integers(0, 1 << 32, table.shape).astype(np.uint32)}


def _check(c, dev):
    d = _device(c, dev)
    _call(c, d)
    _same(d, _oracle(c))


@pytest.mark.parametrize("rows", [0, 1, 100, 511, 512, 1000])
@pytest.mark.parametrize("free", [0, 26, 40, 2000])
def test_second_chunk_without_new_tokens(cuda_device, rows, free):
    """1,024 requests with `rows` new tokens in all, then 1,024 with none, one page each."""
    new = np.zeros(2048, np.int64)
    new[:1000] = np.diff(np.linspace(0, rows, 1001).astype(int))
    lens = np.full(2048, 64)
    lens[:1024] = np.arange(1024) % 130
    _check(_step(400 + rows, lens, new, 4096 * 2048, free), cuda_device)


@pytest.mark.parametrize("idle", [(0,), (1,), (2,), (1, 2), (0, 1, 2, 3, 4)])
def test_idle_chunks_among_five(cuda_device, idle):
    """5,000 requests; the chunks named have no new token (some of a negative number of them)."""
    rng = np.random.default_rng(410 + sum(idle))
    new, lens = rng.integers(0, 6, 5000), rng.integers(0, 700, 5000)
    for k in idle:
        new[1024 * k:1024 * (k + 1)] = -(np.arange(len(new[1024 * k:1024 * (k + 1)])) % 3 == 1).astype(int)
    c = _step(410, lens, new, 4096 * 5000, free=300)
    c["free"][::9] = -1
    _check(c, cuda_device)


@pytest.mark.parametrize("beyond", [-1, 0, 1, 200, 400])
@pytest.mark.parametrize("later", [0, 3])
def test_rows_of_the_first_chunk_end_at_or_beyond_the_map(cuda_device, beyond, later):
    """Its second request asks for nearly all rows there are (and is refused for its table row);
    `beyond` rows lie behind the map's end, which is inside a run of 512 rows. The chunks
    behind have no new token, or `later` each."""
    num_slots = 4096 * 2100 + 100
    new, lens = np.full(2100, later), np.arange(2100) % 200
    new[:1024] = 0
    new[0], new[1] = 70, num_slots - 70 + beyond
    _check(_step(420, lens, new, num_slots, free=50), cuda_device)
