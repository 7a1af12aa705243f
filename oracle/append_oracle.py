"""CPU oracle for the cache appends — TEST INFRASTRUCTURE.

Only the tests and the smoke check may use this module.  It shares no code
with the CUDA library.

Float64 throughout: the rotation is a product of complex numbers at angles
p * f_i, the norm the plain formula.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

PLAIN, LINEAR, YARN = 0, 1, 2


def frequencies(rot_dim: int, theta: float, scaling: int = PLAIN, factor: float = 1.0, original: int = 1,
                beta_fast: float = 32.0, beta_slow: float = 1.0) -> torch.Tensor:
    """Radians per position of every pair."""
    out = []
    for i in range(rot_dim // 2):
        f = theta ** (-2.0 * i / rot_dim)
        if scaling == LINEAR:
            f /= factor
        elif scaling == YARN:
            def index_of(beta):
                # theta^(-2 i / rot) * original / 2 pi = beta, solved for i
                return rot_dim * math.log(original / (2 * math.pi * beta)) / (2 * math.log(theta))
            low = max(0, math.floor(index_of(beta_fast)))
            high = min(rot_dim - 1, math.ceil(index_of(beta_slow)))
            share = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f = share * f / factor + (1.0 - share) * f
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotate(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, interleaved: bool, mscale: float = 1.0) -> torch.Tensor:
    """x [tokens, heads, width]: the first 2 * len(freqs) columns turned."""
    x = x.to(torch.float64)
    half = len(freqs)
    turn = torch.polar(torch.full((1,), mscale, dtype=torch.float64), positions.to(torch.float64)[:, None] * freqs)[:, None, :]
    y = x.clone()
    if interleaved:
        z = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2]) * turn
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def pair_lengths(x: torch.Tensor, half: int, interleaved: bool) -> torch.Tensor:
    """|(a, b)| of every rotated column's pair, |x| of the others: what a
    rotation's rounding errors are relative to."""
    x = x.to(torch.float64)
    r = x.abs()
    if interleaved:
        z = torch.hypot(x[..., 0:2 * half:2], x[..., 1:2 * half:2])
        r[..., 0:2 * half:2], r[..., 1:2 * half:2] = z, z
    else:
        z = torch.hypot(x[..., :half], x[..., half:2 * half])
        r[..., :half], r[..., half:2 * half] = z, z
    return r


def norm(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float) -> torch.Tensor:
    x = x.to(torch.float64)
    if weight is None:
        return x
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.to(torch.float64)


def mla_append(kv: torch.Tensor, weight, eps, q, positions, slots, pool, freqs, interleaved, mscale=1.0):
    """(pool in float64 with the new rows, rotated queries or None)."""
    kv = kv.to(torch.float64)
    out = pool.to(torch.float64)
    rows = torch.cat([norm(kv[:, :512], weight, eps), rotate(kv[:, None, 512:], positions, freqs, interleaved, mscale)[:, 0]], 1)
    for n, s in enumerate(slots.tolist()):
        if 0 <= s < len(out) and int(positions[n]) >= 0:
            out[s] = rows[n]
    return out, None if q is None else rotate(q, positions, freqs, interleaved, mscale)


def draft_append(q, k, v, wq, wk, eps, positions, slots, k_cache, v_cache, freqs, interleaved, mscale=1.0):
    """(rotated queries, key cache, value cache) in float64; caches are
    [pages, page_size, heads, dim]."""
    kc, vc = k_cache.to(torch.float64), v_cache.to(torch.float64)
    keys = rotate(norm(k, wk, eps), positions, freqs, interleaved, mscale)
    page = kc.shape[1]
    for n, s in enumerate(slots.tolist()):
        if s >= 0 and int(positions[n]) >= 0:
            kc[s // page, s % page] = keys[n]
            vc[s // page, s % page] = v[n].to(torch.float64)
    return rotate(norm(q, wq, eps), positions, freqs, interleaved, mscale), kc, vc
