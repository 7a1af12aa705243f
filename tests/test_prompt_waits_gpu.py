"""Waits of the prompt attention with bounds that may run out.

Whatever bound is set, the call ends, says TIMEOUT or nothing, writes nothing
outside its rows and buffers, and the same buffers serve the next call."""
import pytest
import torch

from speculative_decode_tree_gb300 import binding as B
from test_draft_waits_gpu import _guarded
from test_prompt_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[4000], [30] * 40, [5, 900, 0, 300], [30] * 1000, [700] * 40])
def test_short_bounds_end_the_call(lens, dim, dtype):
    c = Case(lens, 8, 2, dim, dtype=dtype, seed=61)
    c.device()
    (out, og), (lse, lg), (ws, wg) = (_guarded(t, f) for t, f in ((c.out, 3.0), (c.lse, 3.0), (c.ws, 0x5A)))
    assert ws.data_ptr() % 256 == 0 and out.data_ptr() % 16 == 0
    args = c.args[:7] + (out, ws)
    for limit in (1, 2, 5, 20):
        c.plan.wait_limit_us = limit
        out.copy_(c.out0), lse.copy_(c.lse0)
        B.ddtree_prompt_attention(*args, lse=lse)
        assert B.ddtree_verify_mla_check(ws) & ~B.DDTREE_ST_TIMEOUT == 0
        assert torch.equal(out[c.qp[-1]:].cpu(), c.out0[c.qp[-1]:]) and torch.equal(lse[c.qp[-1]:].cpu(), c.lse0[c.qp[-1]:])
        assert all(bool((g == 3.0).all()) for g in og + lg) and all(bool((g == 0x5A).all()) for g in wg)
    c.plan.wait_limit_us = 0
    out.copy_(c.out0), lse.copy_(c.lse0)
    B.ddtree_prompt_attention(*args, lse=lse)
    assert B.ddtree_verify_mla_check(ws) == 0
    c.out, c.lse = out, lse
    if sum(lens) < 2000:
        c.compare()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_expired_waits_are_reported(dim, dtype):
    # A call whose status is 0 has the bits of a call without a bound, whatever the bound was; of 1 us some do not hold.
    seen = 0
    for lens, ctx in (([4000], [0]), ([30] * 40, [0] * 40), ([5, 900, 0, 300], [40] * 4), ([30] * 1000, [0] * 1000), ([2, 70], [40000, 300])):
        c = Case(lens, 8, 2, dim, ctx=ctx, dtype=dtype, seed=62)
        c.device()
        B.ddtree_prompt_attention(*c.args, **c.kw)
        assert B.ddtree_verify_mla_check(c.ws) == 0
        out, lse = c.out.clone(), c.lse.clone()
        for limit in (1, 2, 5, 20, 100, 999, 1000):
            c.plan.wait_limit_us = limit
            for _ in range(3):
                c.out.copy_(c.out0), c.lse.copy_(c.lse0)
                B.ddtree_prompt_attention(*c.args, **c.kw)
                bits = B.ddtree_verify_mla_check(c.ws)
                assert bits in (0, B.DDTREE_ST_TIMEOUT)
                seen |= bits
                if bits == 0:
                    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
        c.plan.wait_limit_us = 0
        c.out.copy_(c.out0), c.lse.copy_(c.lse0)
        B.ddtree_prompt_attention(*c.args, **c.kw)
        assert B.ddtree_verify_mla_check(c.ws) == 0
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    assert seen == B.DDTREE_ST_TIMEOUT
