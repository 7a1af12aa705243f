"""CPU oracle for the step maps — TEST INFRASTRUCTURE.

Only the tests and the smoke check may use this module.  It shares no code
with the CUDA library.

What it computes, request by request in plain Python, from the definition in
include/ddtree_maps.h: the pages a step takes from the free list, the verify
index layout, and the new tokens' slots, positions and table rows.  A call that
breaks a rule changes nothing.
"""
from __future__ import annotations

from typing import Dict, List, Optional, Sequence


def depth_of(parent: Sequence[int], i: int):
    """(steps from node i up to its root, whether a bad parent cut the walk)."""
    steps = 0
    while True:
        p = parent[i]
        if p == -1:
            return steps, False
        if not 0 <= p < i:
            return steps, True
        steps, i = steps + 1, p


def step_maps(page_table: List[List[int]], prefix_lens: Sequence[int], max_new: int, page_size: int, n_pages: int,
              capacity: Optional[int], table_row: Optional[Sequence[int]] = None,
              new_lens: Optional[Sequence[int]] = None, tree_parent: Optional[Sequence[Sequence[int]]] = None,
              pages_held: Optional[Sequence[int]] = None, free_pages: Sequence[int] = (), free_head: int = 0) -> Dict:
    B = len(prefix_lens)
    rows = list(table_row) if table_row is not None else list(range(B))
    new = list(new_lens) if new_lens is not None else [max_new] * B
    stride = len(page_table[0])
    table = [list(r) for r in page_table]
    held = list(pages_held) if pages_held is not None else [stride] * B
    tokens = B * max_new
    nothing = dict(table=table, held=held, head=free_head, indptr=[0] * (B + 1), indices=None, new_indptr=[0] * (B + 1),
                   slots=[-1] * tokens, positions=[-1] * tokens, rows=[-1] * tokens, bad_index=False, bad_parent=False,
                   bad_length=False, no_pages=False)
    total = 0
    for P, n, r, h in zip(prefix_lens, new, rows, held):
        if P < 0 or not 0 <= n <= max_new or not 0 <= r < len(table) or not 0 <= h <= stride:
            return {**nothing, "bad_length": True}
        if (P + n + page_size - 1) // page_size > stride:
            return {**nothing, "bad_length": True}
        total += P + n
    if total > 2 ** 31 - 1 or (capacity is not None and total > capacity):
        return {**nothing, "bad_length": True}
    need = [max(0, (P + n + page_size - 1) // page_size - h) for P, n, h in zip(prefix_lens, new, held)]
    if pages_held is not None and not (0 <= free_head <= len(free_pages) and sum(need) <= len(free_pages) - free_head):
        return {**nothing, "no_pages": True}
    out = dict(nothing, indptr=[0], new_indptr=[0], indices=[], slots=[], positions=[], rows=[])
    head = free_head
    for b in range(B):
        P, n, row = prefix_lens[b], new[b], table[rows[b]]
        for k in range(held[b], held[b] + need[b]):
            row[k] = free_pages[head]
            out["bad_index"] |= not 0 <= row[k] < n_pages
            head += 1
        where = []
        for j in range(P + n):
            page = row[j // page_size]
            if not 0 <= page < n_pages:
                # Entries that no list asks for are not looked at.
                out["bad_index"] |= capacity is not None or j >= P
                where.append(-1)
            else:
                where.append(page * page_size + j % page_size)
        out["indptr"].append(out["indptr"][-1] + P + n)
        out["new_indptr"].append(out["new_indptr"][-1] + n)
        out["indices"] += where
        out["slots"] += where[P:]
        out["rows"] += [rows[b]] * n
        for i in range(n):
            depth = i
            if tree_parent is not None:
                depth, cut = depth_of(tree_parent[b], i)
                out["bad_parent"] |= cut
            out["positions"].append(P + depth)
    for name in ("slots", "positions", "rows"):
        out[name] += [-1] * (tokens - len(out[name]))
    out["held"] = [h + k for h, k in zip(held, need)]
    out["head"] = head
    return out
