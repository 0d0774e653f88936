"""Operators of a speculative serving step over the paged latent cache, as measured workloads.

Five operators, each as a user's program calls it:

* ``append``  -- quantise new tokens into the 4-bit (e2m1) page pool and read the stored values back
  (mla_kv_append, mla_kv_gather);
* ``gather``  -- read ragged ranges of cached entries back as bfloat16 rows (mla_kv_gather);
* ``decode``  -- split-KV attention over the 4-bit page pool (mla_decode);
* ``alloc``   -- extend requests by new tokens: pages off the free list, block-table rows, page tags
  and the slot map (mla_kv_alloc);
* ``verify``  -- accept or reject drafted tokens against the target's probabilities and sample the
  next one (mla_verify_drafts).

4-bit page of 64 tokens (19,008 bytes): codes ``[18 blocks][64 tokens][16 bytes]`` (32 e2m1 codes per
block and token, the even element in the low nibble), then exponents ``[9][64]`` (byte i of a token:
block 2i in the low nibble, block 2i + 1 in the high one). A block's value is
``e2m1(code) * 2**(n - 8) * kv_scale`` with n its exponent nibble; n = 15 marks a block that held a NaN.
"""

import math
import random

import torch

own = False

PAGE = 64
ENTRY, LATENT, ROPE = 576, 512, 64
BLOCK = 32
BLOCKS = ENTRY // BLOCK
CODE_BYTES = BLOCKS * PAGE * 16
PAGE_BYTES = CODE_BYTES + BLOCKS // 2 * PAGE
TOKEN_BYTES = PAGE_BYTES / PAGE
KV_SCALE = 0.0089285718277096748  # float32(4 / 448)
SM_SCALE = 0.072168782353401184   # float32(1 / sqrt(192))
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDPOINTS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # between neighbouring e2m1 values

LATENT_BYTES = {"e2m1": TOKEN_BYTES, "e4m3": ENTRY, "bf16": 2 * ENTRY}


def listed():
    return [
        # one decode step's new tokens: 32 requests, a sampled token and three drafts each
        {"name": "append step 32x4", "op": "append", "batch": 32, "lo": 4, "hi": 4},
        # prompts of a few thousand tokens admitted together (ragged)
        {"name": "append prompts 16x<=4k", "op": "append", "batch": 16, "lo": 500, "hi": 4000},
        # the context of a short second chunk, from an FP8 pool
        {"name": "gather 3x<=777 e4m3", "op": "gather", "batch": 3, "lo": 65, "hi": 777, "cache": "e4m3", "offset": True},
        # long contexts read back for a prefill chunk, from the 4-bit pool
        {"name": "gather 4x<=100k e2m1", "op": "gather", "batch": 4, "lo": 60000, "hi": 100000, "cache": "e2m1", "offset": False},
        # two short requests, 16 heads: the smallest call
        {"name": "decode 2 short h16", "op": "decode", "batch": 2, "queries": 1, "heads": 16, "lo": 777, "hi": 1024, "aborted": 0},
        # one agent session of 100k tokens
        {"name": "decode 1x100k", "op": "decode", "batch": 1, "queries": 1, "heads": 64, "lo": 100000, "hi": 100000, "aborted": 0},
        # 32 sessions of 60k to 140k tokens, one of them failed by the integrity check
        {"name": "decode 32x60k-140k", "op": "decode", "batch": 32, "queries": 1, "heads": 64, "lo": 60000, "hi": 140000, "aborted": 1},
        # 32 sessions, four causal drafts each
        {"name": "decode 32x<=256k q4", "op": "decode", "batch": 32, "queries": 4, "heads": 64, "lo": 32000, "hi": 256000, "aborted": 0},
        # page bookkeeping of one speculative step of 256 requests
        {"name": "alloc step 256x4", "op": "alloc", "batch": 256, "cached": 140000, "lo": 4, "hi": 4, "tags": True, "short": False},
        # 32 long contexts admitted at once, the last ones past the free pages
        {"name": "alloc admit 32x<=140k", "op": "alloc", "batch": 32, "cached": 0, "lo": 60000, "hi": 140000, "tags": True, "short": True},
        # one request, three drafts, 128k tokens in the vocabulary
        {"name": "verify 1x3 128k", "op": "verify", "batch": 1, "drafts": 3, "vocab": 131072, "dtype": "f32", "drafter": True, "ragged": False, "gap": 1.0},
        # 128 requests, three drafts, 160k tokens in the vocabulary
        {"name": "verify 128x3 160k", "op": "verify", "batch": 128, "drafts": 3, "vocab": 163840, "dtype": "f32", "drafter": True, "ragged": True, "gap": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "alloc", "verify"])
    batch = _log_int(rng, 1, 32)
    if op == "append":
        hi = _log_int(rng, 1, min(4000, 64000 // batch))
        return {"op": op, "batch": batch, "lo": rng.randint(0, hi), "hi": hi}
    if op == "gather":
        hi = _log_int(rng, 1, min(100000, 300000 // batch))
        return {"op": op, "batch": batch, "lo": rng.randint(0, hi), "hi": hi,
                "cache": rng.choice(["e2m1", "e4m3", "bf16"]), "offset": rng.random() < 0.5}
    if op == "decode":
        queries = rng.randint(1, 4)
        hi = _log_int(rng, queries, 140000)
        return {"op": op, "batch": batch, "queries": queries, "heads": rng.choice([16, 32, 64]),
                "lo": rng.randint(queries, hi), "hi": hi, "aborted": rng.choice([0, 0, 1])}
    if op == "alloc":
        batch = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, min(140000, 3000000 // batch))
        return {"op": op, "batch": batch, "cached": rng.choice([0, _log_int(rng, 1, 140000)]), "lo": rng.randint(0, hi),
                "hi": hi, "tags": rng.random() < 0.5, "short": rng.random() < 0.5}
    batch = _log_int(rng, 1, 128)
    return {"op": op, "batch": batch, "drafts": rng.randint(0, 3), "vocab": _log_int(rng, 1000, 163840),
            "dtype": rng.choice(["f32", "bf16"]), "drafter": rng.random() < 0.7, "ragged": rng.random() < 0.5,
            "gap": rng.uniform(0.1, 3.0)}


def _lengths(case, salt=0):
    """The requests' lengths: part of the case, so that its work is known without its inputs."""
    r = random.Random("%d %d %d %d" % (case["batch"], case["lo"], case["hi"], salt))
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _pages(n):
    return -(-n // PAGE)


def _pages_of(lens):
    return sum(_pages(n) for n in lens)


def _offset(case, b):
    return (37 * b + 11) % 200 if case["offset"] else 0


# ---- the 4-bit format, plainly ----


def _quantise(x, scale):
    """Codes [..., 18, 32] (0..15) and exponent nibbles [..., 18] of entries x [..., 576], in 64 bits."""
    x = x.double().unflatten(-1, (BLOCKS, BLOCK))
    a = x.abs()
    amax = a.amax(-1)  # NaN if the block holds one
    e = torch.arange(-8, 6, device=x.device, dtype=torch.float64)
    n = (amax[..., None] > 7.0 * scale * torch.exp2(e)).sum(-1)
    bad = torch.isnan(amax)
    y = a * torch.exp2(8.0 - n)[..., None]
    code = torch.zeros_like(y, dtype=torch.int32)
    for i, m in enumerate(MIDPOINTS):  # ties go to the even code
        code += (y >= m * scale) if i % 2 else (y > m * scale)
    code += 8 * torch.signbit(x)
    code = torch.where(bad[..., None], 0, code)
    return code.to(torch.uint8), torch.where(bad, 15, n).to(torch.uint8)


def _store(pool, slots, code, nib):
    """Scatters tokens' codes and exponents into the page pool; slots < 0 are skipped."""
    keep = slots >= 0
    slot, code, nib = slots[keep].long(), code[keep], nib[keep]
    page, off = slot // PAGE, slot % PAGE
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    exps = nib[..., 0::2] | (nib[..., 1::2] << 4)
    pool[:, :CODE_BYTES].unflatten(1, (BLOCKS, PAGE, 16))[page, :, off] = packed
    pool[:, CODE_BYTES:].unflatten(1, (BLOCKS // 2, PAGE))[page, :, off] = exps


def _tables(device):
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=device)
    byte = torch.arange(256, device=device)
    pair = torch.stack([value[byte & 15], value[byte >> 4]], -1)
    power = torch.exp2(torch.arange(16, device=device, dtype=torch.float32) - 8.0)
    power[15] = float("nan")
    return pair, torch.stack([power[byte & 15], power[byte >> 4]], -1)


def _values(pool, pages, scale):
    """The entries of `pages` [...] as float32 [..., 64, 576]."""
    pair, power = _tables(pool.device)
    raw = pool[pages]
    code, exps = raw[..., :CODE_BYTES], raw[..., CODE_BYTES:]
    v = pair.index_select(0, code.reshape(-1).int()).view(*code.shape[:-1], BLOCKS, PAGE, BLOCK)
    p = power.index_select(0, exps.reshape(-1).int()).view(*exps.shape[:-1], BLOCKS // 2, PAGE, 2)
    v = v.movedim(-3, -2).unflatten(-2, (BLOCKS // 2, 2)) * p.movedim(-3, -2)[..., None]
    return v.flatten(-3) * scale


def _decoded(pool, pages, cache, scale):
    if cache == "e2m1":
        return _values(pool, pages, scale)
    if cache == "e4m3":
        return pool[pages].view(torch.float8_e4m3fn).float() * scale
    return pool[pages].float()


# ---- inputs ----


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _entries(g, n):
    return (torch.randn(n, ENTRY, generator=g, device="cuda") * 0.5).bfloat16()


def _pool(g, num_pages, cache):
    """A page pool filled with quantised normal entries."""
    if cache == "bf16":
        return _entries(g, num_pages * PAGE).view(num_pages, PAGE, ENTRY)
    if cache == "e4m3":
        return (_entries(g, num_pages * PAGE).float() / KV_SCALE).to(torch.float8_e4m3fn).view(torch.uint8).view(num_pages, PAGE, ENTRY)
    pool = torch.empty(num_pages, PAGE_BYTES, dtype=torch.uint8, device="cuda")
    for at in range(0, num_pages, 4096):
        n = min(4096, num_pages - at)
        code, nib = _quantise(_entries(g, n * PAGE), KV_SCALE)
        _store(pool[at:at + n], torch.arange(n * PAGE, device="cuda"), code, nib)
    return pool


def _block_table(g, lens, num_pages):
    """Random pages of the pool, row by row; entries past a request's pages are -1."""
    counts = torch.tensor([_pages(n) for n in lens], device="cuda")
    width = max(1, max(_pages(n) for n in lens))
    order = torch.randperm(num_pages, generator=g, device="cuda")
    first = counts.cumsum(0) - counts
    at = torch.arange(width, device="cuda")
    held = at[None] < counts[:, None]
    return torch.where(held, order[torch.where(held, first[:, None] + at[None], 0)], -1).int()


def _starts(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    return {"case": case, **globals()["_prepare_" + case["op"]](case, g)}


def _prepare_append(case, g):
    lens = _lengths(case)
    total = sum(lens)
    # the new tokens follow 37 b + 11 cached ones, so that they start inside a page
    starts = [(37 * b + 11) % 200 for b in range(case["batch"])]
    ends = [s + n for s, n in zip(starts, lens)]
    num_pages = _pages_of(ends) + 3
    table = _block_table(g, ends, num_pages)
    x = _entries(g, total)
    cu, start = _starts(lens), torch.tensor(starts, dtype=torch.int32, device="cuda")
    row = torch.arange(total, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), row.int(), right=True)
    pos = start[b] + row - cu[b]
    return {"latent": x[:, :LATENT].contiguous(), "rope": x[:, LATENT:].contiguous(),
            "slots": (table[b, pos // PAGE] * PAGE + pos % PAGE).int(), "cu": cu, "starts": start, "table": table,
            "pool": torch.zeros(num_pages, PAGE_BYTES, dtype=torch.uint8, device="cuda"),
            "latent_out": torch.empty(total, LATENT, dtype=torch.bfloat16, device="cuda"),
            "rope_out": torch.empty(total, ROPE, dtype=torch.bfloat16, device="cuda")}


def _prepare_gather(case, g):
    lens = _lengths(case)
    starts = [_offset(case, b) for b in range(case["batch"])]
    ends = [s + n for s, n in zip(starts, lens)]
    num_pages = _pages_of(ends) + 3
    return {"pool": _pool(g, num_pages, case["cache"]), "table": _block_table(g, ends, num_pages), "cu": _starts(lens),
            "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
            "latent_out": torch.empty(sum(lens), LATENT, dtype=torch.bfloat16, device="cuda"),
            "rope_out": torch.empty(sum(lens), ROPE, dtype=torch.bfloat16, device="cuda")}


def _prepare_decode(case, g):
    lens = _lengths(case)
    num_pages = _pages_of(lens) + 3
    B, Q, H = case["batch"], case["queries"], case["heads"]
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["aborted"]:
        seq[-1] = -1  # as the integrity check marks a request whose pages were handed on
    return {"pool": _pool(g, num_pages, "e2m1"), "table": _block_table(g, lens, num_pages), "lens": seq,
            "q": torch.randn(B, Q, H, ENTRY, generator=g, device="cuda").bfloat16(),
            "out": torch.empty(B, Q, H, LATENT, dtype=torch.bfloat16, device="cuda"),
            "lse": torch.empty(B, Q, H, device="cuda")}


def _alloc_shape(case):
    """Cached and new tokens of each request, and how many pages the free list holds."""
    new, r = _lengths(case), random.Random("%d %d" % (case["batch"], case["cached"]))
    cached = [r.randint(0, case["cached"]) for _ in new]
    held = [_pages(c) + (1 if r.random() < 0.3 else 0) for c in cached]  # a page kept from rejected drafts
    need = [max(0, _pages(c + n) - h) for c, n, h in zip(cached, new, held)]
    free = sum(need) * 9 // 10 if case["short"] else sum(need) + 100
    return cached, new, held, need, free


def _prepare_alloc(case, g):
    cached, new, held, need, free = _alloc_shape(case)
    B = case["batch"]
    num_pages = sum(held) + free + 1
    width = max(1, max(max(h, _pages(c + n)) for c, n, h in zip(cached, new, held)))
    order = torch.randperm(num_pages, generator=g, device="cuda").int()
    at, h = torch.arange(width, device="cuda"), torch.tensor(held, device="cuda")
    first, have = h.cumsum(0) - h, at[None] < h[:, None]
    table = torch.where(have, order[torch.where(have, first[:, None] + at[None], 0)], -1).int()
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"seq_lens": torch.tensor(cached, **i32), "new": torch.tensor(new, **i32), "held": torch.tensor(held, **i32),
         "free": order[sum(held):].contiguous(), "free_count": torch.tensor([free], **i32), "table": table,
         "num_pages": num_pages, "seq_lens_out": torch.empty(B, **i32), "held_out": torch.empty(B, **i32),
         "free_count_out": torch.empty(1, **i32), "cu": torch.empty(B + 1, **i32),
         "slots": torch.empty(sum(new) + 5, **i32), "status": torch.empty(B, **i32), "tags": None, "expected": None}
    if case["tags"]:
        s["tags"] = torch.randint(0, 1 << 30, (num_pages,), generator=g, **i32)
        s["expected"] = torch.where(table >= 0, s["tags"][table.clamp(min=0).long()], 0)
    return s


def _prepare_verify(case, g):
    B, K, V = case["batch"], case["drafts"], case["vocab"]
    dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    logits = torch.randn(B, K + 1, V, generator=g, device="cuda") * 3.0
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits[:, :K] + case["gap"] * torch.randn(B, K, V, generator=g, device="cuda"), -1).to(dtype)
    race = torch.rand(B, K, V, generator=g, device="cuda").clamp_(min=1e-20).log_().neg_()
    draft = (q.float() / race).argmax(-1).int()
    drafts = torch.randint(0, K + 1, (B,), generator=g, device="cuda").int() if case["ragged"] else None
    i32 = dict(dtype=torch.int32, device="cuda")
    return {"p": p, "q": q if case["drafter"] else None, "draft": draft, "drafts": drafts,
            "u": torch.rand(B, K + 1, generator=g, device="cuda"),
            "lens": torch.randint(K + 1, 140000, (B,), generator=g, device="cuda").int(),
            "tokens": torch.empty(B, K + 1, **i32), "accepted": torch.empty(B, **i32), "lens_out": torch.empty(B, **i32)}


# ---- one pass ----


def run(state):
    return globals()["_run_" + state["case"]["op"]](state)


def _plain_gather(s, cache, scale):
    row = torch.arange(s["latent_out"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].contiguous(), row.int(), right=True)
    pos = s["starts"][b] + row - s["cu"][b]
    page, off = s["table"][b, pos // PAGE].long(), pos % PAGE
    if cache == "e2m1":
        pair, power = _tables("cuda")
        code = s["pool"][:, :CODE_BYTES].unflatten(1, (BLOCKS, PAGE, 16))[page, :, off].long()
        exps = s["pool"][:, CODE_BYTES:].unflatten(1, (BLOCKS // 2, PAGE))[page, :, off].long()
        v = (pair[code].view(-1, BLOCKS, BLOCK) * power[exps].view(-1, BLOCKS, 1) * scale).flatten(1)
    else:
        v = s["pool"][page, off]
        v = v.view(torch.float8_e4m3fn).float() * scale if cache == "e4m3" else v.float()
    v = v.bfloat16()
    return {"latent": v[:, :LATENT], "rope": v[:, LATENT:]}


def _run_append(s):
    if own:
        from paged_mla_decode_gb300 import binding

        binding.mla_kv_append(s["latent"], s["rope"], s["slots"], s["pool"], KV_SCALE)
        binding.mla_kv_gather(s["pool"], KV_SCALE, s["table"], s["cu"], s["latent_out"], s["rope_out"], starts=s["starts"])
        return {"latent": s["latent_out"], "rope": s["rope_out"]}
    code, nib = _quantise(torch.cat([s["latent"], s["rope"]], 1), KV_SCALE)
    _store(s["pool"], s["slots"], code, nib)
    return _plain_gather(s, "e2m1", KV_SCALE)


def _run_gather(s):
    cache = s["case"]["cache"]
    scale = 1.0 if cache == "bf16" else KV_SCALE
    if own:
        from paged_mla_decode_gb300 import binding

        binding.mla_kv_gather(s["pool"], scale, s["table"], s["cu"], s["latent_out"], s["rope_out"], starts=s["starts"])
        return {"latent": s["latent_out"], "rope": s["rope_out"]}
    return _plain_gather(s, cache, scale)


def _run_decode(s):
    if own:
        from paged_mla_decode_gb300 import binding

        if "workspace" not in s:
            B, Q, H = s["q"].shape[:3]
            s["workspace"] = torch.zeros(binding.mla_decode_workspace_size(B, Q, H), dtype=torch.uint8, device="cuda")
        binding.mla_decode(s["q"], s["pool"], s["table"], s["lens"], SM_SCALE, KV_SCALE, s["out"], s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    q, lens = s["q"], s["lens"]
    B, Q, H = q.shape[:3]
    kv = _values(s["pool"], s["table"].clamp(min=0).long(), KV_SCALE).flatten(1, 2)  # [B, T, 576]
    score = torch.bmm(q.float().flatten(1, 2), kv.transpose(1, 2)).mul_(SM_SCALE).view(B, Q, H, -1)
    # draft j of a request of L tokens sees the first L - Q + j + 1 of them; L < Q leaves none
    seen = lens[:, None] - Q + 1 + torch.arange(Q, device="cuda")
    seen = torch.where(lens[:, None] >= Q, seen, 0)
    t = torch.arange(kv.shape[1], device="cuda")
    score.masked_fill_((t >= seen[..., None])[:, :, None], -math.inf)
    top = score.amax(-1)
    score = torch.exp(score.sub_(top.clamp(min=-3e38)[..., None]))
    total = score.sum(-1)
    out = torch.bmm(score.flatten(1, 2), kv[..., :LATENT]).view(B, Q, H, LATENT)
    return {"out": (out / total.clamp(min=1e-30)[..., None]).bfloat16(), "lse": top + torch.log(total)}


def _run_alloc(s):
    if own:
        from paged_mla_decode_gb300 import binding

        binding.mla_kv_alloc(s["seq_lens"], s["new"], s["held"], s["free"], s["free_count"], s["num_pages"], s["table"],
                             s["seq_lens_out"], s["held_out"], s["free_count_out"], s["cu"], s["slots"], s["status"],
                             page_tags=s["tags"], expected_tags=s["expected"])
        keys = ("seq_lens_out", "held_out", "free_count_out", "cu", "slots", "status", "table", "tags", "expected")
        return {k: s[k] for k in keys if s[k] is not None}
    L, n, held, table = s["seq_lens"].long(), s["new"].long(), s["held"].long(), s["table"]
    width, count = table.shape[1], s["free_count"].long()
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    fits = (L + n + PAGE - 1) // PAGE
    full = fits > width
    need = torch.where(full, 0, (fits - held).clamp(min=0))
    ends = need.cumsum(0)
    first = ends - need
    out_of_pages = (need > 0) & (ends > count)
    fail = full | out_of_pages
    need = torch.where(fail, 0, need)
    # pages come off the end of the free list, one request after the other
    at = torch.arange(width, device="cuda")
    k = at[None] - held[:, None]
    fresh = (k >= 0) & (k < need[:, None])
    page = s["free"][torch.where(fresh, count - 1 - first[:, None] - k, 0)]
    table.copy_(torch.where(fresh, page, table))
    got = {}
    if s["tags"] is not None:
        s["tags"].scatter_add_(0, torch.where(fresh, page, 0).long().flatten(), fresh.int().flatten())
        s["expected"].copy_(torch.where(fresh, s["tags"][page.long()], s["expected"]))
        got = {"tags": s["tags"], "expected": s["expected"]}
    row = torch.arange(s["slots"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    inside = b < L.shape[0]
    b = b.clamp(max=L.shape[0] - 1)
    pos = L[b] + row - cu[b]
    live = inside & ~fail[b]
    slot = table[b, torch.where(live, pos // PAGE, 0)].long() * PAGE + pos % PAGE
    return {"seq_lens_out": torch.where(fail, -1, L + n).int(), "held_out": (held + need).int(),
            "free_count_out": (count - need.sum()).int(), "cu": cu.int(), "slots": torch.where(live, slot, -1).int(),
            "status": (2 * full.int() + 8 * out_of_pages.int()).int(), "table": table, **got}


def _weight(p):
    return torch.where(p > 0, p.double().clamp(max=1.0), 0.0)


def _run_verify(s):
    if own:
        from paged_mla_decode_gb300 import binding

        binding.mla_verify_drafts(s["p"], s["q"], s["draft"], s["u"], s["tokens"], s["accepted"], num_drafts=s["drafts"],
                                  seq_lens=s["lens"], seq_lens_out=s["lens_out"])
        return {"tokens": s["tokens"], "accepted": s["accepted"], "lens": s["lens_out"]}
    p, q, draft, u = s["p"], s["q"], s["draft"].long(), s["u"].double()
    B, K = draft.shape
    each = torch.arange(B, device="cuda")
    drafts = torch.full((B,), K, device="cuda") if s["drafts"] is None else s["drafts"].long()
    px = _weight(p[:, :K].gather(2, draft[..., None])[..., 0])
    qx = _weight(q.gather(2, draft[..., None])[..., 0]) if q is not None else torch.ones_like(px)
    # 64 bits hold the product of two 32-bit numbers exactly
    ok = (u[:, :K] * qx < px) & (torch.arange(K, device="cuda") < drafts[:, None])
    a = ok.long().cumprod(1).sum(1)
    w = _weight(p[each, a])
    if K > 0:
        rejected = a < drafts
        j = a.clamp(max=K - 1)
        less = _weight(q[each, j]) if q is not None else torch.zeros_like(w).scatter_(1, draft[each, j][:, None], math.inf)
        rest = torch.where(rejected[:, None], (w - less).clamp(min=0.0), w)
        w = torch.where((rest.sum(1) > 0)[:, None], rest, w)
    cum = w.cumsum(1)
    total = cum[:, -1:]
    token = torch.searchsorted(cum, u[:, K:] * total, right=True)[:, 0].clamp(max=w.shape[1] - 1)
    token = torch.where(total[:, 0] > 0, token, -1)
    i = torch.arange(K + 1, device="cuda")
    padded = torch.cat([draft, draft.new_full((B, 1), -1)], 1)
    tokens = torch.where(i < a[:, None], padded, torch.where(i == a[:, None], token[:, None], -1))
    return {"tokens": tokens.int(), "accepted": a.int(), "lens": (s["lens"] - (drafts - a)).int()}


# ---- what a pass cannot do without ----


def work(case):
    op = case["op"]
    if op == "append":
        n = sum(_lengths(case))
        return {"bytes": 8 * case["batch"] + n * (2 * ENTRY + 4 + 2 * TOKEN_BYTES + 2 * ENTRY), "flops": 0}
    if op == "gather":
        n = sum(_lengths(case))
        return {"bytes": 8 * case["batch"] + n * (LATENT_BYTES[case["cache"]] + 2 * ENTRY), "flops": 0}
    if op == "decode":
        lens = _lengths(case)
        lens = lens[:-1] if case["aborted"] else lens
        Q, H = case["queries"], case["heads"]
        seen = sum(Q * n - Q * (Q - 1) // 2 for n in lens)
        rows = case["batch"] * Q * H
        return {"bytes": sum(lens) * TOKEN_BYTES + 4 * _pages_of(lens) + rows * (2 * ENTRY + 2 * LATENT + 4),
                "flops": seen * H * 2 * (ENTRY + LATENT)}
    if op == "alloc":
        cached, new, held, need, free = _alloc_shape(case)
        pages = min(sum(need), free)
        return {"bytes": 4 * (sum(new) + 5) + pages * (20 if case["tags"] else 8) + 28 * case["batch"], "flops": 0}
    # one row of p is summed and searched, and one of q where a draft is rejected (most requests of three drafts)
    size = 4 if case["dtype"] == "f32" else 2
    rows = 2 if case["drafter"] and case["drafts"] else 1
    return {"bytes": case["batch"] * rows * case["vocab"] * size, "flops": 0}


# ---- the definition in 64 bits ----


def _exact_grid():
    """The 256 values of a byte pair (code, exponent nibble), from the format's definition."""
    grid = torch.zeros(16, 16, dtype=torch.float64)
    for code in range(16):
        m, e = code & 1, (code >> 1) & 3
        v = 0.5 * m if e == 0 else (1.0 + 0.5 * m) * 2.0 ** (e - 1)
        for n in range(16):
            grid[code, n] = math.nan if n == 15 else (-v if code & 8 else v) * 2.0 ** (n - 8)
    return grid.cuda()


def _exact_entries(pool, table, upto, grid):
    """The first `upto` entries of one request as float64 [upto, 576], block by block."""
    raw = pool[table[: _pages(upto)].long()]
    got = torch.empty(raw.shape[0] * PAGE, ENTRY, dtype=torch.float64, device="cuda")
    for blk in range(BLOCKS):
        code = raw[:, blk * 1024:(blk + 1) * 1024].reshape(-1, 16).long()
        nib = raw[:, CODE_BYTES + (blk // 2) * PAGE:CODE_BYTES + (blk // 2 + 1) * PAGE].reshape(-1).long()
        nib = (nib >> 4 if blk % 2 else nib & 15)[:, None]
        got[:, blk * BLOCK:(blk + 1) * BLOCK:2] = grid[code & 15, nib]
        got[:, blk * BLOCK + 1:(blk + 1) * BLOCK:2] = grid[code >> 4, nib]
    return got[:upto] * KV_SCALE


def exact(case, seed):
    if case["op"] in ("alloc", "verify"):
        return None  # whole numbers
    s = prepare(case, seed)
    lens = _lengths(case)
    if case["op"] == "append":
        x = torch.cat([s["latent"], s["rope"]], 1).double().unflatten(1, (BLOCKS, BLOCK))
        amax = x.abs().amax(2, keepdim=True)
        step = torch.full_like(amax, 2.0 ** 6)
        for e in range(5, -9, -1):
            step = torch.where(amax <= 7 * 2.0 ** e * KV_SCALE, 2.0 ** e, step)
        # the nearest of the eight magnitudes; the even code of two equally near ones
        near = torch.full(x.shape, 9.0, dtype=torch.float64, device="cuda")
        best = torch.zeros_like(x)
        for code in (0, 2, 4, 6, 1, 3, 5, 7):
            far = (x.abs() / (step * KV_SCALE) - E2M1[code]).abs()
            best = torch.where(far < near, E2M1[code], best)
            near = torch.minimum(far, near)
        v = (torch.copysign(best, x) * step * KV_SCALE).flatten(1)
        return {"latent": v[:, :LATENT], "rope": v[:, LATENT:]}
    grid = _exact_grid()
    if case["op"] == "gather":
        rows = []
        for b, n in enumerate(lens):
            lo = _offset(case, b)
            if case["cache"] == "e2m1":
                rows.append(_exact_entries(s["pool"], s["table"][b], lo + n, grid)[lo:])
            else:
                v = s["pool"][s["table"][b, : _pages(lo + n)].long()].flatten(0, 1)[lo:lo + n]
                v = v.view(torch.float8_e4m3fn).double() * KV_SCALE if case["cache"] == "e4m3" else v.double()
                rows.append(v)
        v = torch.cat(rows)
        return {"latent": v[:, :LATENT], "rope": v[:, LATENT:]}
    if work(case)["flops"] > 3e12:
        return None
    q = s["q"].double()
    B, Q, H = q.shape[:3]
    out = torch.zeros(B, Q, H, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, L in enumerate(lens):
        if case["aborted"] and b == B - 1:
            continue
        kv = _exact_entries(s["pool"], s["table"][b], L, grid)
        for j in range(Q):
            k = kv[:L - Q + j + 1]
            score = (q[b, j] @ k.T) * SM_SCALE
            lse[b, j] = torch.logsumexp(score, 1)
            out[b, j] = torch.exp(score - lse[b, j][:, None]) @ k[:, :LATENT]
    return {"out": out, "lse": lse}
