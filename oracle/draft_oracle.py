"""CPU oracle for the drafter's attention — TEST INFRASTRUCTURE.

Only the tests and the smoke check may use this module.  It shares no code
with the CUDA library.  Float64: the visible set is written out key by key, the
rows are gathered, and the softmax is the plain one.
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence

import torch


def visible_keys(position: int, window: int, n_sinks: int) -> List[int]:
    return [j for j in range(position + 1) if window == 0 or j > position - window or j < n_sinks]


def draft_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                    token_rows: Optional[Sequence[int]], positions: Sequence[int], window: int, n_sinks: int,
                    sm_scale: float, out: torch.Tensor, lse: torch.Tensor):
    """(out, lse) in float64, starting from the given buffers (padding tokens
    keep them).  Also the sum of |p_j v_j| for every output, which its rounding
    errors are relative to, and the largest sum of |scaled product| terms."""
    out, lse = out.to(torch.float64), lse.to(torch.float64)
    mass, terms = torch.zeros_like(out), torch.zeros_like(lse)
    page, kvh = int(k_cache.shape[1]), int(k_cache.shape[2])
    group = int(q.shape[1]) // kvh
    for n, pos in enumerate(positions):
        if pos == -1:
            continue
        row = n if token_rows is None else int(token_rows[n])
        out[n], lse[n] = 0.0, -math.inf
        if pos < -1 or not 0 <= row < page_table.shape[0] or pos // page >= page_table.shape[1]:
            continue
        keys = torch.tensor(visible_keys(pos, window, n_sinks))
        pages = page_table[row][keys // page].long()
        good = (pages >= 0) & (pages < k_cache.shape[0])
        keys, pages = keys[good], pages[good]
        if not len(keys):
            continue
        k = k_cache[pages, keys % page].to(torch.float64)
        v = v_cache[pages, keys % page].to(torch.float64)
        for h in range(int(q.shape[1])):
            kh, qh = k[:, h // group], q[n, h].to(torch.float64)
            s = sm_scale * (kh @ qh)
            p = torch.exp(s - s.max())
            total = p.sum()
            lse[n, h] = s.max() + torch.log(total)
            out[n, h] = (p / total) @ v[:, h // group]
            mass[n, h] = (p / total) @ v[:, h // group].abs()
            terms[n, h] = abs(sm_scale) * float((kh.abs() @ qh.abs()).max())
    return out, lse, mass, terms
