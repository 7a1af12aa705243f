"""CPU oracle for the attention over whole prompts — TEST INFRASTRUCTURE.

Only the tests and the smoke check may use this module.  It shares no code
with the CUDA library.  Float64, one sequence and head at a time with the
visible pairs as a mask.  A value that is no number counts for the rows that
see it alone.
"""
from __future__ import annotations

import math
from typing import Sequence

import torch


def visible(n_queries: int, n_keys: int, window: int, n_sinks: int) -> torch.Tensor:
    """[queries, keys]: which keys each query sees; the queries are the last of the keys."""
    p = torch.arange(n_queries)[:, None] + (n_keys - n_queries)
    j = torch.arange(n_keys)[None, :]
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < n_sinks)
    return seen


def prompt_attention(q, k, v, q_indptr: Sequence[int], k_indptr: Sequence[int], window: int, n_sinks: int, sm_scale: float, out, lse):
    """(out, lse) in float64 from the given buffers (rows of no sequence keep
    them); the sum of |p_j v_j| of every output, and the largest sum of
    |scaled product| terms of its row."""
    out, lse = out.to(torch.float64), lse.to(torch.float64)
    mass, terms = torch.zeros_like(out), torch.zeros_like(lse)
    group = q.shape[1] // k.shape[1]
    for b in range(len(q_indptr) - 1):
        rows, keys = slice(q_indptr[b], q_indptr[b + 1]), slice(k_indptr[b], k_indptr[b + 1])
        n, m = q_indptr[b + 1] - q_indptr[b], k_indptr[b + 1] - k_indptr[b]
        if n == 0:
            continue
        seen = visible(n, m, window, n_sinks)
        some = seen.any(-1)
        for h in range(q.shape[1]):
            if m == 0:
                out[rows, h], lse[rows, h] = 0.0, -math.inf
                continue
            qh, kh, vh = q[rows, h].to(torch.float64), k[keys, h // group].to(torch.float64), v[keys, h // group].to(torch.float64)
            s = (sm_scale * (qh @ kh.T)).masked_fill(~seen, -math.inf)
            top = s.amax(-1).masked_fill(~some, 0.0)
            p = torch.exp(s - top[:, None])
            total = p.sum(-1)
            p = p / torch.where(some, total, torch.ones_like(total))[:, None]
            odd = ~torch.isfinite(vh).all(-1)
            clean = torch.where(odd[:, None], torch.zeros_like(vh), vh)
            o = p @ clean
            for j in odd.nonzero().flatten().tolist():
                see = seen[:, j]
                o[see] += p[see, j, None] * vh[j]
            out[rows, h] = o
            lse[rows, h] = torch.where(some, top + torch.log(total), torch.full_like(total, -math.inf))
            mass[rows, h] = p @ clean.abs()
            size = abs(sm_scale) * (qh.abs() @ kh.abs().T)
            terms[rows, h] = size.masked_fill(~seen, 0.0).amax(-1)
    return out, lse, mass, terms
