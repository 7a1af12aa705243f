"""Fields of the drafter-attention plan that the caller sets (no GPU)."""
import ctypes

import pytest

from speculative_decode_tree_gb300 import binding as B
from test_append_oracle import P, Q, _cache


@pytest.fixture(scope="module")
def lib():
    from speculative_decode_tree_gb300.build import build
    build()
    return B.library()


def test_wait_limit(lib):
    c, plan = _cache(), B.DraftPlan()
    assert lib.ddtree_draft_attention_plan(4, 8, ctypes.addressof(c), 0, 0, 152, ctypes.addressof(plan)) == 0
    assert plan.wait_limit_us == 0

    def call():
        return lib.ddtree_draft_attention(ctypes.addressof(plan), P, ctypes.addressof(c), P, 4, 8, None, P, 0.1, Q, P, P,
                                          plan.workspace_bytes - 1, None)
    # The workspace is looked at after the plan: one byte short of it tells a plan that is taken.
    for limit, code in ((0, B.DDTREE_EWORKSPACE), (1, B.DDTREE_EWORKSPACE), (2 ** 31 - 1, B.DDTREE_EWORKSPACE), (-1, B.DDTREE_EINVAL)):
        plan.wait_limit_us = limit
        assert call() == code, limit


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_scales_whose_product_with_log2_e_overflows(lib, scale):
    c, plan = _cache(), B.DraftPlan()
    assert lib.ddtree_draft_attention_plan(4, 8, ctypes.addressof(c), 0, 0, 152, ctypes.addressof(plan)) == 0
    for s, code in ((scale, B.DDTREE_EINVAL), (scale / 2, B.DDTREE_EWORKSPACE)):
        assert lib.ddtree_draft_attention(ctypes.addressof(plan), P, ctypes.addressof(c), P, 4, 8, None, P, s, Q, P, P,
                                          plan.workspace_bytes - 1, None) == code
