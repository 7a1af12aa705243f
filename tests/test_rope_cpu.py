"""Edges of the rotation's set-up (no GPU)."""
import math

import pytest

from speculative_decode_tree_gb300 import binding as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    from speculative_decode_tree_gb300.build import build
    build()
    return B.library()


def _yarn(original, beta_slow=1.0, rot=64, theta=10000.0):
    return B.ddtree_rope_init(rot, theta=theta, scaling=B.DDTREE_ROPE_YARN, factor=8.0, original_positions=original,
                              beta_fast=32.0, beta_slow=beta_slow)


@pytest.mark.parametrize("original,beta_slow", [(1, 1.0), (6, 1.0), (12, 2.0), (62, 10.0)])
def test_yarn_needs_a_pair_that_turns_slowly_often_enough(original, beta_slow):
    # The fastest pair turns original / (2 pi) times: below beta_slow the ramp has no lower end, and the first pair
    # came out as it was although it turns less often than the pairs that are stretched.
    assert original / (2 * math.pi) < beta_slow
    with pytest.raises(B.DDTreeError) as e:
        _yarn(original, beta_slow)
    assert e.value.code == B.DDTREE_EINVAL


@pytest.mark.parametrize("original,beta_slow", [(7, 1.0), (13, 2.0), (63, 10.0), (4096, 1.0)])
def test_yarn_just_above(original, beta_slow):
    r, plain = _yarn(original, beta_slow), B.ddtree_rope_init(64, theta=10000.0)
    slow = [i for i in range(32) if 10000.0 ** (-i / 32) * original / (2 * math.pi) < beta_slow]
    # One whole pair past the border the ramp has ended.
    for i in slow[1:]:
        assert r.turns[i] == pytest.approx(plain.turns[i] / 8.0, rel=1e-12)
