"""Page allocation for a step, request by request (oracle; test infrastructure only).

The page allocator of [CF] "Smaller, faster, safer: running Kimi and GLM at scale", section
"Protecting a shared KV cache": pages come off a free list, a page's tag changes when it is
handed out again, and a request keeps the tag each of its pages had then. The interface
(requests extended by new tokens, in order, from the end of the list) is ours.
"""

from __future__ import annotations

import numpy as np

PAGE = 64
BAD_LENGTH, TABLE_FULL, SLOTS_FULL, NO_PAGES = 1, 2, 4, 8


def alloc(seq_lens, new_tokens, held, free_pages, free_count, num_pages, block_table, num_slots,
          page_tags=None, expected_tags=None) -> dict:
    """Everything mla_kv_alloc writes, as new arrays. Plain loops over Python integers."""
    table = np.array(block_table)
    width = table.shape[1]
    tags = None if page_tags is None else np.array(page_tags).astype(np.uint32)
    expected = None if expected_tags is None else np.array(expected_tags).astype(np.uint32)
    free = [int(p) for p in free_pages[:max(0, min(int(free_count), len(free_pages)))]]
    start = len(free)
    slots = np.full(num_slots, -1, dtype=np.int64)
    cu, status, lens_out, held_out = [0], [], [], []
    row, asked = 0, 0  # rows and pages asked for by the requests so far
    for b in range(len(seq_lens)):
        length, new, h = int(seq_lens[b]), int(new_tokens[b]), int(held[b])
        rows = max(new, 0)
        first, row = row, row + rows
        cu.append(min(row, 2 ** 31 - 1))
        why = 0
        if length < 0 or new < 0 or not -(-length // PAGE) <= h <= width:
            why = BAD_LENGTH
        elif -(-(length + new) // PAGE) > width:
            why = TABLE_FULL
        elif row > num_slots:
            why = SLOTS_FULL
        else:
            need = max(0, -(-(length + new) // PAGE) - h)
            asked += need
            if need and asked > start:
                why = NO_PAGES
        status.append(why)
        held_out.append(h if why else h + need)
        lens_out.append(-1 if why else length + new)
        if why:
            continue
        for k in range(need):
            page = free.pop()
            table[b, h + k] = page
            if tags is not None and 0 <= page < num_pages:
                tags[page] += np.uint32(1)
                expected[b, h + k] = tags[page]
        for i in range(new):
            page = int(table[b, (length + i) // PAGE])
            if 0 <= page < num_pages:
                slots[first + i] = page * PAGE + (length + i) % PAGE
    return {"seq_lens_out": np.array(lens_out, np.int64), "pages_held_out": np.array(held_out, np.int64),
            "free_count_out": len(free), "cu_tokens": np.array(cu, np.int64), "slot_mapping": slots,
            "request_status": np.array(status, np.int64), "block_table": table, "page_tags": tags,
            "expected_tags": expected}
