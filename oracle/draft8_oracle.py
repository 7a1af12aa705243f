"""CPU oracle for the drafter's 8-bit cache — TEST INFRASTRUCTURE.

Only the tests and the smoke check may use this module.  It shares no code
with the CUDA library.  Float64; e4m3 is a table of its 256 numbers, and
rounding looks the nearest one up.
"""
from __future__ import annotations

import math
from typing import Sequence

import torch


def e4m3_table() -> torch.Tensor:
    """The number of every code: sign, exponent - 7, three bits; 0x7f and 0xff are NaN."""
    out = []
    for code in range(256):
        sign, e, m = -1.0 if code & 0x80 else 1.0, code >> 3 & 15, code & 7
        value = math.nan if code & 0x7F == 0x7F else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out.append(sign * value)
    return torch.tensor(out, dtype=torch.float64)


TABLE = e4m3_table()
_NUMBERS = TABLE[:127].contiguous()                  # 0 .. 448, ascending
_BORDERS = (_NUMBERS[1:] + _NUMBERS[:-1]) / 2        # between code i and i + 1


def values(codes: torch.Tensor) -> torch.Tensor:
    """Numbers of the codes (uint8 or float8_e4m3fn)."""
    return TABLE[codes.view(torch.uint8).long()]


def codes_of(x: torch.Tensor) -> torch.Tensor:
    """Nearest code, ties to the even one, 448 beyond the range, NaN for NaN."""
    a = x.to(torch.float64).abs()
    code = torch.searchsorted(_BORDERS, a)           # a border itself belongs to the lower code ...
    up = torch.searchsorted(_BORDERS, a, right=True)  # ... or to the upper one
    code = torch.where(code % 2 == 0, code, up).clamp_max(126)
    code = torch.where(torch.isnan(a), torch.full_like(code, 127), code)
    sign = torch.signbit(x).long() * 128
    return (code + sign).to(torch.uint8)


def scale_for(top: float) -> float:
    """Least power of two s with top <= 448 s, from 2^-64 to 2^96; 1 for 0."""
    if top == 0:
        return 1.0
    e = -64
    while e < 96 and top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def scale_ok(s: float) -> bool:
    return 2.0 ** -64 <= s <= 2.0 ** 96


def write_rows(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, block: int, positions: Sequence[int],
               slots: Sequence[int]) -> None:
    """Rows x [tokens, heads, dim] (float64) into codes [pages, page, heads,
    dim] (uint8) and scales [pages, blocks, heads] (float64), in place."""
    pages, page = codes.shape[:2]
    runs = {}
    for n, s in enumerate(slots):
        if positions[n] >= 0 and 0 <= s < pages * page:
            runs.setdefault((s // page, s % page // block), []).append((n, s % page))
    for (p, b), rows in runs.items():
        inside = [t for _, t in rows]
        others = [t for t in range(b * block, min((b + 1) * block, page)) if t not in inside]
        for h in range(codes.shape[2]):
            mags = torch.stack([x[n, h] for n, _ in rows]).abs()
            mags = mags[torch.isfinite(mags)]
            top = float(mags.max()) if mags.numel() else 0.0
            old = float(scales[p, b, h])
            begun = b * block not in inside and scale_ok(old)
            new = old if begun and top <= 448 * old else scale_for(top)
            if begun and new != old:
                for t in others:
                    codes[p, t, h] = codes_of(TABLE[codes[p, t, h].long()] * old / new)
            for n, t in rows:
                codes[p, t, h] = codes_of(x[n, h] / new)
            scales[p, b, h] = new


def dequantised(codes: torch.Tensor, scales: torch.Tensor, block: int) -> torch.Tensor:
    """[pages, page, heads, dim] in float64; rows whose scale is out of range are NaN."""
    at = torch.arange(codes.shape[1]) // block
    s = scales.to(torch.float64)[:, at]
    good = (s >= 2.0 ** -64) & (s <= 2.0 ** 96)
    return values(codes) * torch.where(good, s, torch.full_like(s, math.nan))[..., None]


def read_rows(codes, scales, block: int, slots: Sequence[int], out: torch.Tensor) -> torch.Tensor:
    """Rows in float64, starting from the buffer `out` (slots outside keep it; bad scales give 0)."""
    out, pages, page = out.to(torch.float64), *codes.shape[:2]
    full = dequantised(codes, scales, block)
    for n, s in enumerate(slots):
        if 0 <= s < pages * page:
            row = full[s // page, s % page]
            ok = torch.tensor([scale_ok(float(v)) for v in scales[s // page, s % page // block]])
            out[n] = torch.where(ok[:, None], row, torch.zeros_like(row))
    return out



def attention(q, k_codes, v_codes, k_scale, v_scale, block: int, page_table, token_rows, positions, window: int, n_sinks: int,
              sm_scale: float, out, lse):
    """The drafter's attention over the dequantised cache, as
    draft_oracle.draft_attention gives it: (out, lse) in float64 from the given
    buffers, the sum of |p_j v_j| of every output and the largest sum of
    |scaled product| terms.  Keys whose scale is out of range are dropped."""
    out, lse = out.to(torch.float64), lse.to(torch.float64)
    mass, terms = torch.zeros_like(out), torch.zeros_like(lse)
    pages, page, kvh = k_codes.shape[:3]
    k_all, v_all = dequantised(k_codes, k_scale, block), dequantised(v_codes, v_scale, block)
    at = torch.arange(page) // block
    good = [(s >= 2.0 ** -64) & (s <= 2.0 ** 96) for s in (k_scale.to(torch.float64)[:, at], v_scale.to(torch.float64)[:, at])]
    good = good[0] & good[1]
    group = q.shape[1] // kvh
    for n, pos in enumerate(positions):
        if pos == -1:
            continue
        row = n if token_rows is None else int(token_rows[n])
        out[n], lse[n] = 0.0, -math.inf
        if pos < -1 or not 0 <= row < page_table.shape[0] or pos // page >= page_table.shape[1]:
            continue
        seen = torch.tensor([j for j in range(pos + 1) if window == 0 or j > pos - window or j < n_sinks])
        where = page_table[row][seen // page].long()
        here = (where >= 0) & (where < pages)
        seen, where = seen[here], where[here]
        for h in range(q.shape[1]):
            kh = h // group
            live = good[where, seen % page, kh]
            if not bool(live.any()):
                continue
            k, v = (c[where[live], seen[live] % page, kh] for c in (k_all, v_all))
            qh = q[n, h].to(torch.float64)
            s = sm_scale * (k @ qh)
            p = torch.exp(s - s.max())
            total = p.sum()
            lse[n, h] = s.max() + torch.log(total)
            out[n, h] = (p / total) @ v
            mass[n, h] = (p / total) @ v.abs()
            terms[n, h] = abs(sm_scale) * float((k.abs() @ qh.abs()).max())
    return out, lse, mass, terms
