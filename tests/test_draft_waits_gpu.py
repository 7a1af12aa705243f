"""Waits of the drafter's attention that run out (groups through tensor memory).

A bound of 1 us makes waits on copies and products expire: the call ends, says
TIMEOUT, writes nothing outside its buffers nor for padding tokens, and the same
buffers serve the next call with the default bound."""
import random

import pytest
import torch

from speculative_decode_tree_gb300 import binding as B
from test_draft_attn_gpu import Case

pytestmark = pytest.mark.gpu

SHAPES = [(d, t) for d in (64, 128, 256) for t in (torch.bfloat16, torch.float16)]


def _guarded(t, fill):
    """A contiguous copy of `t` between two stretches of `fill`."""
    pad, n = 4096, t.numel()
    whole = torch.full((n + 2 * pad,), fill, dtype=t.dtype, device=t.device)
    inner = whole[pad:pad + n].view(t.shape)
    inner.copy_(t)
    return inner, (whole[:pad], whole[pad + n:])


@pytest.mark.parametrize("dim,dtype", SHAPES)
@pytest.mark.parametrize("lengths", ["long", "many", "one"])
def test_expired_waits_end_the_call(lengths, dim, dtype):
    r = random.Random(dim)
    positions = {"long": [40000, 5, -1, 9000], "many": [r.choice([-1, 0, 40, 100, r.randint(0, 400)]) for _ in range(203)],
                 "one": [700]}[lengths]
    c = Case(positions, 120 if lengths == "long" else 40, 3 if lengths == "long" else 1, dim, dtype=dtype, seed=61)
    c.device()
    (out, og), (lse, lg), (ws, wg) = (_guarded(t, f) for t, f in ((c.out, 3.0), (c.lse, 3.0), (c.ws, 0x5A)))
    assert ws.data_ptr() % 256 == 0 and out.data_ptr() % 16 == 0
    args, kw = c.args[:6] + (out, ws), dict(c.kw, lse=lse)
    seen = 0
    for limit in (1, 2, 5, 20):
        c.plan.wait_limit_us = limit
        B.ddtree_draft_attention(*args, **kw)
        bits = B.ddtree_verify_mla_check(ws)
        assert bits & ~B.DDTREE_ST_TIMEOUT == 0
        seen |= bits
        for n, p in enumerate(positions):
            if p == -1:
                assert torch.equal(out[n].cpu(), c.out0[n]) and torch.equal(lse[n].cpu(), c.lse0[n])
        assert all(bool((g == 3.0).all()) for g in og + lg) and all(bool((g == 0x5A).all()) for g in wg)
    assert seen == B.DDTREE_ST_TIMEOUT
    c.plan.wait_limit_us = 0
    B.ddtree_draft_attention(*args, **kw)
    assert B.ddtree_verify_mla_check(ws) == 0
    c.out, c.lse = out, lse
    c.compare()
