"""Operators of a tree-speculative serving step over the paged latent cache, as measured workloads.

A request's drafter proposes a tree of tokens. Node 0 is its last sampled token, node i > 0 a draft whose
parent is an earlier node; ``tree_mask[b][j]`` is a 64-bit word, bit i set where node j sees node i (its
ancestors and itself). One step, as a user's program runs it:

* ``tree``    -- attention of the nodes over the cached context and the nodes that each one sees, whose
  entries lie behind the context in node order (mla_decode_tree);
* ``probs``   -- the nodes' logits to probabilities: penalties for repeated tokens (the tokens on a node's own
  path count too), biases, a grammar's mask, the temperature (mla_logits_to_probs);
* ``verify``  -- walk down from node 0, keep a child by rejection sampling or try the next one, sample the
  token behind the last kept node (mla_verify_tree);
* ``compact`` -- move the kept nodes' cache entries to the front of the tree's, in every layer's cache
  (mla_kv_compact).

The cache's formats are those of ``operators.py`` beside this file: e4m3 codes or bfloat16 ``[pages, 64, 576]``,
4-bit pages of 19,008 bytes: ``[18 blocks][64 tokens][16 bytes]`` of e2m1 codes, then exponents ``[9][64]``.
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
KV_SCALE = 0.0089285718277096748  # float32(4 / 448)
SM_SCALE = 0.072168782353401184   # float32(1 / sqrt(192))
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

LATENT_BYTES = {"e2m1": PAGE_BYTES / PAGE, "e4m3": ENTRY, "bf16": 2 * ENTRY}


def listed():
    return [
        # a short chat, a small tree, 16 heads: the smallest attention
        {"name": "tree 1x900 n6 h16 e4m3", "op": "tree", "cache": "e4m3", "batch": 1, "nodes": 6, "ragged": False, "heads": 16, "lo": 900, "hi": 900},
        # one agent session of 100k tokens, the last token and 15 drafts
        {"name": "tree 1x100k n16 e4m3", "op": "tree", "cache": "e4m3", "batch": 1, "nodes": 16, "ragged": False, "heads": 64, "lo": 100000, "hi": 100000},
        # 16 sessions of 32k to 140k tokens, trees of up to 12 nodes
        {"name": "tree 16x32k-140k n<=12 e4m3", "op": "tree", "cache": "e4m3", "batch": 16, "nodes": 12, "ragged": True, "heads": 64, "lo": 32000, "hi": 140000},
        # 8 sessions over the 4-bit cache
        {"name": "tree 8x20k-100k n8 e2m1", "op": "tree", "cache": "e2m1", "batch": 8, "nodes": 8, "ragged": False, "heads": 64, "lo": 20000, "hi": 100000},
        # many short requests with large trees, a bfloat16 cache, a rank's 32 heads
        {"name": "tree 32x<=4k n<=31 h32 bf16", "op": "tree", "cache": "bf16", "batch": 32, "nodes": 31, "ragged": True, "heads": 32, "lo": 100, "hi": 4000},
        # one request's four rows, 128k tokens in the vocabulary, a grammar
        {"name": "probs 1x4 128k", "op": "probs", "batch": 1, "rows": 4, "vocab": 131072, "in": "bf16", "out": "f32", "tree": True, "penalties": False, "biases": 0, "grammar": True},
        # 32 requests, trees of eight nodes, everything at once
        {"name": "probs 32x8 160k", "op": "probs", "batch": 32, "rows": 8, "vocab": 163840, "in": "bf16", "out": "f32", "tree": True, "penalties": True, "biases": 100, "grammar": True},
        # a plain decode step of 128 requests
        {"name": "probs 128x1 160k", "op": "probs", "batch": 128, "rows": 1, "vocab": 163840, "in": "f32", "out": "f32", "tree": False, "penalties": True, "biases": 16, "grammar": False},
        # one request, a tree of 16 nodes from a drafter's most likely tokens
        {"name": "verify 1x16 128k", "op": "verify", "batch": 1, "nodes": 16, "ragged": False, "vocab": 131072, "dtype": "f32", "drafter": False, "gap": 1.0},
        # 64 requests, trees of up to 16 nodes drawn from a drafter
        {"name": "verify 64x<=16 160k", "op": "verify", "batch": 64, "nodes": 16, "ragged": True, "vocab": 163840, "dtype": "f32", "drafter": True, "gap": 1.0},
        # kept nodes of 32 requests in the caches of 61 layers
        {"name": "compact 32x16 61 layers e4m3", "op": "compact", "cache": "e4m3", "batch": 32, "nodes": 16, "layers": 61},
        # kept nodes of 16 requests in one 4-bit cache, read back
        {"name": "compact 16x32 e2m1", "op": "compact", "cache": "e2m1", "batch": 16, "nodes": 32, "layers": 1},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "probs", "verify", "compact"])
    if op == "tree":
        batch, nodes, heads = _log_int(rng, 1, 32), _log_int(rng, 1, 64), rng.choice([16, 32, 64])
        hi = _log_int(rng, nodes, max(nodes, min(140000, 400000000 // (batch * nodes * heads))))
        return {"op": op, "cache": rng.choice(["e4m3", "e4m3", "e2m1", "bf16"]), "batch": batch, "nodes": nodes,
                "ragged": rng.random() < 0.5, "heads": heads, "lo": rng.randint(nodes, hi), "hi": hi}
    if op == "probs":
        batch, rows = _log_int(rng, 1, 64), _log_int(rng, 1, 32)
        return {"op": op, "batch": batch, "rows": rows, "vocab": _log_int(rng, 1000, min(163840, 40000000 // (batch * rows))),
                "in": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "f32", "bf16"]), "tree": rng.random() < 0.5,
                "penalties": rng.random() < 0.7, "biases": rng.choice([0, _log_int(rng, 1, 300)]), "grammar": rng.random() < 0.5}
    if op == "verify":
        batch, nodes = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        return {"op": op, "batch": batch, "nodes": nodes, "ragged": rng.random() < 0.5,
                "vocab": _log_int(rng, 1000, min(163840, 160000000 // (batch * nodes))), "dtype": rng.choice(["f32", "bf16"]),
                "drafter": rng.random() < 0.5, "gap": rng.uniform(0.1, 3.0)}
    cache = rng.choice(["e4m3", "e2m1", "bf16"])
    return {"op": op, "cache": cache, "batch": _log_int(rng, 1, 32), "nodes": rng.randint(2, 64),
            "layers": 1 if cache == "e2m1" else _log_int(rng, 1, 30)}


def _pages(n):
    return -(-n // PAGE)


def _pages_of(lens):
    return sum(_pages(n) for n in lens)


def _shape_rng(case, salt):
    return random.Random("%s %d %d" % (salt, case["batch"], case["nodes"]))


def _nodes(case):
    """The requests' tree sizes: part of the case, so that its work is known without its inputs."""
    r = _shape_rng(case, "nodes")
    return [r.randint(1, case["nodes"]) if case["ragged"] else case["nodes"] for _ in range(case["batch"])]


def _lengths(case):
    """Cached tokens of each request, its tree's nodes included."""
    r = _shape_rng(case, "lengths")
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _kept(case):
    """A compaction's requests: tokens before the tree, and the kept nodes, node 0 first."""
    r = _shape_rng(case, "kept")
    base = [r.randint(0, 200) for _ in range(case["batch"])]
    return base, [[0] + sorted(r.sample(range(1, case["nodes"]), r.randint(0, min(7, case["nodes"] - 1)))) for _ in base]


def _tree(r, n):
    """Parents and masks of a random tree of n nodes (a node's parent is one of the last few before it)."""
    parent, mask = [-1], [1]
    for i in range(1, n):
        parent.append(r.randint(max(0, i - 4), i - 1))
        mask.append(mask[parent[i]] | 1 << i)
    return parent, mask


def _words(masks):
    return [m - (1 << 64) if m >> 63 else m for m in masks]


# ---- the 4-bit format, plainly ----


def _tables():
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    byte = torch.arange(256, device="cuda")
    power = torch.exp2(torch.arange(16, device="cuda", dtype=torch.float32) - 8.0)
    power[15] = math.nan
    return torch.stack([value[byte & 15], value[byte >> 4]], -1), torch.stack([power[byte & 15], power[byte >> 4]], -1)


def _code_view(pool):
    return pool[..., :CODE_BYTES].unflatten(-1, (BLOCKS, PAGE, 16))


def _exps_view(pool):
    return pool[..., CODE_BYTES:].unflatten(-1, (BLOCKS // 2, PAGE))


def _page_values(pool, pages, cache):
    """The entries of `pages` [...] as float32 [..., 64, 576]."""
    if cache == "e4m3":
        return pool[pages].view(torch.float8_e4m3fn).float().mul_(KV_SCALE)
    if cache == "bf16":
        return pool[pages].float()
    pair, power = _tables()
    raw = pool[pages]
    code, exps = raw[..., :CODE_BYTES], raw[..., CODE_BYTES:]
    v = pair.index_select(0, code.reshape(-1).int()).view(*code.shape[:-1], BLOCKS, PAGE, BLOCK)
    p = power.index_select(0, exps.reshape(-1).int()).view(*exps.shape[:-1], BLOCKS // 2, PAGE, 2)
    v = v.movedim(-3, -2).unflatten(-2, (BLOCKS // 2, 2)) * p.movedim(-3, -2)[..., None]
    return v.flatten(-3).mul_(KV_SCALE)


# ---- inputs ----


def _entries(g, n):
    return (torch.randn(n, ENTRY, generator=g, device="cuda") * 0.5).bfloat16()


def _pool(g, num_pages, cache):
    """Pages full of entries as an append leaves them."""
    if cache == "bf16":
        return _entries(g, num_pages * PAGE).view(num_pages, PAGE, ENTRY)
    if cache == "e4m3":
        return (_entries(g, num_pages * PAGE).float() / KV_SCALE).to(torch.float8_e4m3fn).view(torch.uint8).view(num_pages, PAGE, ENTRY)
    pool = torch.empty(num_pages, PAGE_BYTES, dtype=torch.uint8, device="cuda")
    bounds = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for at in range(0, num_pages, 4096):
        n = min(4096, num_pages - at)
        x = _entries(g, n * PAGE).float().view(n, PAGE, BLOCKS, BLOCK)
        top = x.abs().amax(-1)
        e = torch.ceil(torch.log2(top / (7 * KV_SCALE))).clamp(-8, 6)
        code = torch.bucketize(x.abs() / (torch.exp2(e) * KV_SCALE)[..., None], bounds) + 8 * (x < 0)
        code, e = code.to(torch.uint8), (e + 8).to(torch.uint8)
        _code_view(pool)[at:at + n] = (code[..., 0::2] | code[..., 1::2] << 4).transpose(1, 2)
        _exps_view(pool)[at:at + n] = (e[..., 0::2] | e[..., 1::2] << 4).transpose(1, 2)
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


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _masks(trees):
    return torch.tensor([_words(mask) for _, mask in trees], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"case": case, **globals()["_prepare_" + case["op"]](case, g, random.Random(seed))}


def _prepare_tree(case, g, r):
    B, N, H = case["batch"], case["nodes"], case["heads"]
    lens = _lengths(case)
    num_pages = _pages_of(lens) + 3
    return {"pool": _pool(g, num_pages, case["cache"]), "table": _block_table(g, lens, num_pages), "lens": _i32(lens),
            "mask": _masks([_tree(r, N) for _ in range(B)]), "nodes": _i32(_nodes(case)) if case["ragged"] else None,
            "q": torch.randn(B, N, H, ENTRY, generator=g, device="cuda").bfloat16(),
            "out": torch.empty(B, N, H, LATENT, dtype=torch.bfloat16, device="cuda"),
            "lse": torch.empty(B, N, H, device="cuda")}


def _prepare_probs(case, g, r):
    B, R, V = case["batch"], case["rows"], case["vocab"]
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}
    words = -(-V // 32)
    s = {"logits": (torch.randn(B, R, V, generator=g, device="cuda") * 3.0).to(kind[case["in"]]),
         "probs": torch.empty(B, R, V, dtype=kind[case["out"]], device="cuda"),
         # an eighth of the requests decode greedily
         "temperature": torch.tensor([0.0 if r.random() < 0.125 else r.uniform(0.3, 1.2) for _ in range(B)], device="cuda")}
    if case["tree"]:
        s["tokens"] = torch.randint(0, V, (B, R), generator=g, device="cuda").int()
        s["mask"] = _masks([_tree(r, R) for _ in range(B)])
    if case["penalties"]:
        counts = torch.zeros(B, V, dtype=torch.int32, device="cuda")
        written = (torch.rand(B, 2000, generator=g, device="cuda") ** 3 * V).long().clamp(max=V - 1)
        s["counts"] = counts.scatter_add_(1, written, torch.ones_like(written, dtype=torch.int32))
        bits = torch.rand(B, words, 32, generator=g, device="cuda") < 0.02
        s["prompt"] = (bits.int() << torch.arange(32, device="cuda", dtype=torch.int32)).sum(-1).int()
        s["repetition"], s["frequency"], s["presence"] = (
            torch.tensor([r.uniform(lo, hi) for _ in range(B)], device="cuda") for lo, hi in ((1.0, 1.3), (0.0, 0.5), (0.0, 0.8)))
    if case["biases"]:
        ids = torch.randint(0, V, (B, case["biases"]), generator=g, device="cuda").int()
        used = torch.randint(0, case["biases"] + 1, (B, 1), generator=g, device="cuda")
        s["bias_tokens"] = torch.where(torch.arange(case["biases"], device="cuda") < used, ids, -1)
        s["biases"] = torch.randn(B, case["biases"], generator=g, device="cuda") * 4.0
    if case["grammar"]:
        # some rows may go on with anything, some with a few tokens
        share = torch.rand(B, R, 1, 1, generator=g, device="cuda") ** 4
        bits = torch.rand(B, R, words, 32, generator=g, device="cuda") >= share
        s["allowed"] = (bits.int() << torch.arange(32, device="cuda", dtype=torch.int32)).sum(-1).int()
    return s


def _prepare_verify(case, g, r):
    B, N, V = case["batch"], case["nodes"], case["vocab"]
    dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    trees = [_tree(r, N) for _ in range(B)]
    parent = torch.tensor([p for p, _ in trees], device="cuda")
    logits = torch.randn(B, N, V, generator=g, device="cuda") * 3.0
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits + case["gap"] * torch.randn(B, N, V, generator=g, device="cuda"), -1).to(dtype)
    del logits
    each, tokens = torch.arange(B, device="cuda"), torch.zeros(B, N, dtype=torch.int32, device="cuda")
    for i in range(1, N):
        race = torch.rand(B, V, generator=g, device="cuda").clamp_(min=1e-20).log_().neg_()
        tokens[:, i] = (q[each, parent[:, i]].float() / race).argmax(-1).int()
    i32 = dict(dtype=torch.int32, device="cuda")
    return {"p": p, "q": q if case["drafter"] else None, "tokens": tokens, "mask": _masks(trees),
            "nodes": _i32(_nodes(case)) if case["ragged"] else None,
            "u": torch.rand(B, N, generator=g, device="cuda"),
            "lens": torch.randint(N, 140000, (B,), generator=g, device="cuda").int(),
            "counts": torch.randint(0, 3, (B, V), generator=g, **i32),
            "out_tokens": torch.empty(B, N, **i32), "path": torch.empty(B, N, **i32), "accepted": torch.empty(B, **i32),
            "lens_out": torch.empty(B, **i32)}


def _prepare_compact(case, g, r):
    base, kept = _kept(case)
    N, L = case["nodes"], case["layers"]
    lens = [c + N for c in base]
    num_pages = _pages_of(lens) + 3
    pool = _pool(g, L * num_pages, case["cache"])
    pool = pool.view(L, num_pages, *pool.shape[1:]) if L > 1 else pool
    s = {"pool": pool, "table": _block_table(g, lens, num_pages), "path": _i32([k + [-1] * (N - len(k)) for k in kept]),
         "accepted": _i32([len(k) - 1 for k in kept]), "lens": _i32([c + len(k) for c, k in zip(base, kept)])}
    if case["cache"] == "e2m1":
        cu = [0]
        for k in kept:
            cu.append(cu[-1] + len(k))
        s |= {"cu": _i32(cu), "starts": _i32(base), "latent": torch.empty(cu[-1], LATENT, dtype=torch.bfloat16, device="cuda"),
              "rope": torch.empty(cu[-1], ROPE, dtype=torch.bfloat16, device="cuda")}
    return s


# ---- one pass ----


def run(state):
    return globals()["_run_" + state["case"]["op"]](state)


def _bits(mask, count):
    """Bits 0 .. count - 1 of 64-bit words, as a last axis of truth values."""
    return (mask[..., None] >> torch.arange(count, device=mask.device) & 1).bool()


def _run_tree(s):
    case, q, lens = s["case"], s["q"], s["lens"]
    if own:
        from paged_mla_decode_gb300 import binding

        scale = 1.0 if case["cache"] == "bf16" else KV_SCALE
        if "workspace" not in s:
            size = binding.mla_decode_tree_workspace_size(*q.shape[:3])
            s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        binding.mla_decode_tree(q, s["pool"], s["table"], lens, s["mask"], SM_SCALE, scale, s["out"], s["lse"], s["workspace"],
                                num_nodes=s["nodes"])
        return {"out": s["out"], "lse": s["lse"]}
    B, N, H = q.shape[:3]
    kv = _page_values(s["pool"], s["table"].clamp(min=0).long(), case["cache"]).flatten(1, 2)  # [B, T, 576]
    score = torch.bmm(q.float().flatten(1, 2), kv.transpose(1, 2)).mul_(SM_SCALE).view(B, N, H, -1)
    n = s["nodes"] if s["nodes"] is not None else torch.full_like(lens, N)
    t = torch.arange(kv.shape[1], device="cuda")
    node = t - (lens - n)[:, None]  # [B, T]: negative for the context
    seen = (s["mask"][:, :, None] >> node.clamp(0, 63)[:, None] & 1).bool() | (node < 0)[:, None]
    seen &= (node < n[:, None])[:, None] & (torch.arange(N, device="cuda") < n[:, None])[:, :, None]
    score.masked_fill_(~seen[:, :, None], -math.inf)
    top = score.amax(-1)
    score = score.sub_(top.clamp(min=-3e38)[..., None]).exp_()
    total = score.sum(-1)
    out = torch.bmm(score.flatten(1, 2), kv[..., :LATENT]).view(B, N, H, LATENT)
    return {"out": (out / total.clamp(min=1e-30)[..., None]).bfloat16(), "lse": top + torch.log(total)}


def _run_probs(s):
    case, x = s["case"], s["logits"]
    if own:
        from paged_mla_decode_gb300 import binding

        binding.mla_logits_to_probs(x, s["probs"], temperature=s["temperature"], node_tokens=s.get("tokens"),
                                    tree_mask=s.get("mask"), token_counts=s.get("counts"), prompt_mask=s.get("prompt"),
                                    repetition=s.get("repetition"), frequency=s.get("frequency"), presence=s.get("presence"),
                                    bias_tokens=s.get("bias_tokens"), biases=s.get("biases"), allowed=s.get("allowed"))
        return {"probs": s["probs"]}
    B, R, V = x.shape
    x, v = x.float(), torch.arange(V, device="cuda")
    if case["penalties"]:
        count = s["counts"][:, None].expand(B, R, V)
        if case["tree"]:
            on_path = _bits(s["mask"], R).int()
            on_path[:, :, 0] = 0  # node 0's token is among the counted
            count = count.clone().scatter_add_(2, s["tokens"].long()[:, None].expand(B, R, R), on_path)
        seen = (count > 0) | (s["prompt"][:, None, v // 32] >> v % 32 & 1).bool()
        factor = s["repetition"][:, None, None]
        x = torch.where(seen, torch.where(x > 0, x / factor, x * factor), x)
        x = x - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0)
    if case["biases"]:
        at = s["bias_tokens"].long()
        add = torch.zeros(B, V, device="cuda").scatter_add_(1, at.clamp(min=0), torch.where(at >= 0, s["biases"], 0.0))
        x = x + add[:, None]
    if case["grammar"]:
        x = torch.where((s["allowed"][:, :, v // 32] >> v % 32 & 1).bool(), x, -math.inf)
    t = s["temperature"][:, None, None]
    top = x.amax(-1, keepdim=True)
    w = torch.exp((x - top.clamp(min=-3e38)) / torch.where(t > 0, t, 1.0))
    p = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
    first = torch.where(x == top, v, V).amin(-1, keepdim=True)  # ties go to the lowest index
    greedy = ((v == first) & (top > -math.inf)).float()
    return {"probs": torch.where(t > 0, p, greedy).to(s["probs"].dtype)}


def _weight(p):
    return torch.where(p > 0, p.double().clamp(max=1.0), 0.0)


def _run_verify(s):
    if own:
        from paged_mla_decode_gb300 import binding

        binding.mla_verify_tree(s["p"], s["q"], s["tokens"], s["mask"], s["u"], s["out_tokens"], s["path"], s["accepted"],
                                num_nodes=s["nodes"], seq_lens=s["lens"], seq_lens_out=s["lens_out"], token_counts=s["counts"])
        return {k: s[k] for k in ("out_tokens", "path", "accepted", "lens_out", "counts")}
    p, q, u, tokens = s["p"], s["q"], s["u"].double(), s["tokens"].long()
    B, N, V = p.shape
    each, i64 = torch.arange(B, device="cuda"), dict(dtype=torch.int64, device="cuda")
    n = s["nodes"].long() if s["nodes"] is not None else torch.full((B,), N, **i64)
    at = torch.arange(N, device="cuda")
    seen = _bits(s["mask"], N) & (at < at[:, None])
    parent = torch.where(seen, at, -1).amax(-1)  # the last node before it that a node sees
    # node by node: which one the walk stands at, its kept nodes, what its rejected children left of p
    here, kept = torch.zeros(B, **i64), torch.zeros(B, **i64)
    out, path = torch.full((B, N), -1, **i64), torch.full((B, N), -1, **i64)
    path[:, 0] = 0
    left = torch.ones(B, dtype=torch.float64, device="cuda")  # its weight; of the whole p: 1
    less = torch.zeros(B, dtype=torch.float64, device="cuda")  # how many times q has been taken off
    gone = torch.zeros(B, V, dtype=torch.bool, device="cuda")  # without q: rejected tokens

    def rest():
        w = _weight(p[each, here])
        if q is None:
            return torch.where(gone, 0.0, w)
        return (w - less[:, None] * _weight(q[each, here])).float().clamp(min=0.0).double()

    for i in range(1, N):
        tries = (parent[:, i] == here) & (i < n)
        x, w = tokens[:, i], rest()
        wx = w[each, x]
        qx = _weight(q[each, here, x]) if q is not None else torch.ones_like(wx)
        keep = tries & (u[:, i] * qx * left < wx)
        drop = tries & ~keep
        # kept: the walk goes on from node i, with its whole p
        out[each, kept] = torch.where(keep, x, out[each, kept])
        kept = kept + keep.long()
        path[each, kept] = torch.where(keep, i, path[each, kept])
        here = torch.where(keep, i, here)
        gone = (gone | (drop[:, None] & (torch.arange(V, device="cuda") == x[:, None]))) & ~keep[:, None]
        less = torch.where(keep, 0.0, torch.where(drop, (less + left).float().double(), less))
        remain = rest().sum(1) if q is not None else (left - wx).clamp(min=0.0)
        left = torch.where(keep, 1.0, torch.where(drop, remain, left))
    w = rest()
    w = torch.where((w.sum(1) > 0)[:, None], w, _weight(p[each, here]))
    cum = w.cumsum(1)
    total = cum[:, -1:]
    token = torch.searchsorted(cum, u[:, :1] * total, right=True)[:, 0].clamp(max=V - 1)
    out[each, kept] = torch.where(total[:, 0] > 0, token, -1)
    emitted = out >= 0
    s["counts"].scatter_add_(1, out.clamp(min=0), emitted.int())
    return {"out_tokens": out.int(), "path": path.int(), "accepted": kept.int(), "lens_out": (s["lens"] - n + kept + 1).int(),
            "counts": s["counts"]}


def _run_compact(s):
    case, pool, table = s["case"], s["pool"], s["table"]
    four_bit = case["cache"] == "e2m1"
    if own:
        from paged_mla_decode_gb300 import binding

        binding.mla_kv_compact(pool, table, s["lens"], path=s["path"], num_accepted=s["accepted"])
        if four_bit:
            binding.mla_kv_gather(pool, KV_SCALE, table, s["cu"], s["latent"], s["rope"], starts=s["starts"])
            return {"latent": s["latent"], "rope": s["rope"]}
        return {"pool": pool.view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else pool}
    path = s["path"].long()
    b, i = torch.nonzero(path >= 0, as_tuple=True)
    base = (s["lens"] - s["accepted"] - 1).long()[b]
    src, dst = base + path[b, i], base + i
    ps, pd = table[b, src // PAGE].long(), table[b, dst // PAGE].long()
    if four_bit:
        for view in (_code_view(pool), _exps_view(pool)):
            view[pd, :, dst % PAGE] = view[ps, :, src % PAGE]
        pair, power = _tables()
        code = _code_view(pool)[pd, :, dst % PAGE].long()
        exps = _exps_view(pool)[pd, :, dst % PAGE].long()
        v = (pair[code].view(-1, BLOCKS, BLOCK) * power[exps].view(-1, BLOCKS, 1) * KV_SCALE).flatten(1).bfloat16()
        return {"latent": v[:, :LATENT], "rope": v[:, LATENT:]}
    slots = pool.view(-1, pool.shape[-3] * PAGE, ENTRY)  # [layers, slots, 576]
    slots[:, pd * PAGE + dst % PAGE] = slots[:, ps * PAGE + src % PAGE]
    return {"pool": pool.view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else pool}


# ---- what a pass cannot do without ----


def work(case):
    op, B = case["op"], case["batch"]
    if op == "tree":
        lens, nodes, H = _lengths(case), _nodes(case), case["heads"]
        rows = sum(nodes) * H
        return {"bytes": sum(lens) * LATENT_BYTES[case["cache"]] + 4 * _pages_of(lens) + rows * 2 * ENTRY + 8 * sum(nodes)
                + B * case["nodes"] * H * (2 * LATENT + 4),
                "flops": sum(n * (L - n + 1) for n, L in zip(nodes, lens)) * H * 2 * (ENTRY + LATENT)}
    if op == "probs":
        size, V, rows = {"f32": 4, "bf16": 2}, case["vocab"], B * case["rows"]
        return {"bytes": rows * V * (size[case["in"]] + size[case["out"]]) + (rows * V // 8 if case["grammar"] else 0)
                + (B * (4 * V + V // 8) if case["penalties"] else 0) + B * case["biases"] * 8, "flops": 0}
    if op == "verify":
        # one row of p is summed and searched, and one of q where a draft is rejected (most requests)
        rows = 2 if case["drafter"] and case["nodes"] > 1 else 1
        return {"bytes": B * rows * case["vocab"] * (4 if case["dtype"] == "f32" else 2) + B * case["nodes"] * 24, "flops": 0}
    base, kept = _kept(case)
    moved = sum(sum(1 for i, v in enumerate(k) if v != i) for k in kept)
    back = sum(len(k) for k in kept) * (LATENT_BYTES["e2m1"] + 2 * ENTRY) if case["cache"] == "e2m1" else 0
    return {"bytes": case["layers"] * moved * 2 * LATENT_BYTES[case["cache"]] + back + 8 * sum(len(k) for k in kept) + 8 * B, "flops": 0}


# ---- the definition in 64 bits ----


def _exact_grid():
    """The 256 values of a code and an exponent nibble, from the format's definition."""
    grid = torch.zeros(16, 16, dtype=torch.float64)
    for code in range(16):
        m, e = code & 1, (code >> 1) & 3
        v = 0.5 * m if e == 0 else (1.0 + 0.5 * m) * 2.0 ** (e - 1)
        for n in range(16):
            grid[code, n] = math.nan if n == 15 else (-v if code & 8 else v) * 2.0 ** (n - 8)
    return grid.cuda()


def _exact_entries(pool, table, upto, cache, grid):
    """The first `upto` entries of one request as float64 [upto, 576]."""
    raw = pool[table[:_pages(upto)].long()]
    if cache == "bf16":
        return raw.flatten(0, 1)[:upto].double()
    if cache == "e4m3":
        return raw.view(torch.float8_e4m3fn).flatten(0, 1)[:upto].double() * KV_SCALE
    got = torch.empty(raw.shape[0] * PAGE, ENTRY, dtype=torch.float64, device="cuda")
    for blk in range(BLOCKS):
        code = raw[:, blk * 1024:(blk + 1) * 1024].reshape(-1, 16).long()
        nib = raw[:, CODE_BYTES + (blk // 2) * PAGE:CODE_BYTES + (blk // 2 + 1) * PAGE].reshape(-1).long()
        nib = (nib >> 4 if blk % 2 else nib & 15)[:, None]
        got[:, blk * BLOCK:(blk + 1) * BLOCK:2] = grid[code & 15, nib]
        got[:, blk * BLOCK + 1:(blk + 1) * BLOCK:2] = grid[code >> 4, nib]
    return got[:upto] * KV_SCALE


def _exact_tree(case, s):
    if work(case)["flops"] > 3e12:
        return None
    q, grid = s["q"].double(), _exact_grid()
    B, N, H = q.shape[:3]
    out = torch.zeros(B, N, H, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(_lengths(case), _nodes(case))):
        kv = _exact_entries(s["pool"], s["table"][b], L, case["cache"], grid)
        for j in range(n):
            m = int(s["mask"][b, j])
            k = torch.cat([kv[:L - n], kv[[L - n + i for i in range(n) if m >> i & 1]]])
            score = (q[b, j] @ k.T) * SM_SCALE
            lse[b, j] = torch.logsumexp(score, 1)
            out[b, j] = torch.exp(score - lse[b, j][:, None]) @ k[:, :LATENT]
    return {"out": out, "lse": lse}


def _exact_probs(case, s):
    B, R, V = s["logits"].shape
    probs = torch.zeros(B, R, V, dtype=torch.float64, device="cuda")
    for b in range(B):
        for j in range(R):
            x = s["logits"][b, j].double()
            if case["penalties"]:
                count = s["counts"][b].double()
                if case["tree"]:
                    m = int(s["mask"][b, j])
                    for i in range(1, R):
                        if m >> i & 1:
                            count[int(s["tokens"][b, i])] += 1
                prompt = (s["prompt"][b][:, None] >> torch.arange(32, device="cuda") & 1).flatten()[:V].bool()
                theta = float(s["repetition"][b])
                scaled = torch.where(x > 0, x / theta, x * theta)
                x = torch.where(prompt | (count > 0), scaled, x)
                x = x - float(s["frequency"][b]) * count - float(s["presence"][b]) * (count > 0).double()
            if case["biases"]:
                for v, c in zip(s["bias_tokens"][b].tolist(), s["biases"][b].tolist()):
                    if v >= 0:
                        x[v] += c
            if case["grammar"]:
                words = s["allowed"][b, j][:, None] >> torch.arange(32, device="cuda")
                x = x.masked_fill((words & 1).flatten()[:V] == 0, -math.inf)
            t = float(s["temperature"][b])
            if bool((x == -math.inf).all()):
                continue
            if t == 0:
                probs[b, j, int((x == x.max()).nonzero()[0])] = 1.0
            else:
                probs[b, j] = torch.softmax(x / t, 0)
    return {"probs": probs}


def exact(case, seed):
    if case["op"] in ("verify", "compact"):
        return None  # whole numbers, and values that are moved
    if case["op"] == "probs" and case["batch"] * (case["rows"] + case["biases"]) > 8000:
        return None
    s = prepare(case, seed)
    return _exact_tree(case, s) if case["op"] == "tree" else _exact_probs(case, s)
