"""Pins of the step-maps oracle, and the entry point's host-side refusals (no GPU)."""
import ctypes

import pytest

from oracle import step_maps
from speculative_decode_tree_gb300 import binding as B


def test_worked_example():
    # Two requests, pages of 4: P=5, n=2 holds pages 9 and 3 (7 tokens fit); P=4, n=1 holds page 7 and takes one.
    m = step_maps([[9, 3, -1], [7, -1, -1]], [5, 4], 2, 4, 16, 16, new_lens=[2, 1], pages_held=[2, 1],
                  free_pages=[8, 12, 5], free_head=1)
    assert m["indptr"] == [0, 7, 12] and m["new_indptr"] == [0, 2, 3]
    assert m["indices"] == [36, 37, 38, 39, 12, 13, 14, 28, 29, 30, 31, 48]
    assert m["slots"] == [13, 14, 48, -1] and m["positions"] == [5, 6, 4, -1] and m["rows"] == [0, 0, 1, -1]
    assert m["table"] == [[9, 3, -1], [7, 12, -1]] and m["held"] == [2, 2] and m["head"] == 2


def test_tree_depths_and_bad_parents():
    m = step_maps([[0]], [3], 5, 64, 1, None, tree_parent=[[-1, 0, 0, 1, -1]])
    assert m["positions"] == [3, 4, 4, 5, 3] and not m["bad_parent"]
    m = step_maps([[0]], [3], 3, 64, 1, None, tree_parent=[[-1, 2, 1]])
    assert m["positions"] == [3, 3, 4] and m["bad_parent"]


def test_rules_leave_everything():
    t = [[1, -1]]
    assert step_maps(t, [3], 2, 2, 9, 4, pages_held=[1], free_pages=[4, 5], free_head=0)["bad_length"]  # 5 > 4 entries, 3 pages
    m = step_maps(t, [2], 2, 2, 9, 4, pages_held=[1], free_pages=[4], free_head=1)
    assert m["no_pages"] and m["table"] == t and m["slots"] == [-1, -1] and m["held"] == [1] and m["head"] == 1


@pytest.fixture(scope="module")
def lib():
    from speculative_decode_tree_gb300.build import build
    build()
    return B.library()


def test_refusals(lib):
    p = ctypes.c_void_p(1 << 12)
    q = ctypes.c_void_p(1 << 13)
    odd = ctypes.c_void_p((1 << 12) + 2)
    ok = dict(batch=2, max_new=4, page=16, pages=100, table=p, rows=4, stride=8, row=None, prefix=p, new=None, parent=None,
              held=p, free=p, n_free=10, head=p, held_out=q, head_out=q, indptr=p, indices=p, cap=100, nptr=None,
              slots=p, pos=p, trow=None, status=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.ddtree_step_maps(*[a[k] for k in ok], None)
    for bad in (dict(batch=0), dict(batch=1025), dict(max_new=0), dict(max_new=65), dict(page=0), dict(page=65537),
                dict(pages=0), dict(pages=(1 << 31) // 16), dict(rows=0), dict(rows=1), dict(stride=0), dict(table=None),
                dict(table=odd), dict(row=odd), dict(prefix=None), dict(new=odd), dict(parent=odd), dict(held=odd),
                dict(free=None), dict(n_free=-1), dict(head=None), dict(held_out=None), dict(held_out=p),
                dict(head_out=None), dict(head_out=p), dict(held=None), dict(indptr=None), dict(indices=odd),
                dict(cap=-1), dict(indices=None), dict(nptr=odd), dict(slots=None), dict(pos=None), dict(trow=odd),
                dict(status=odd)):
        assert call(**bad) == B.DDTREE_EINVAL, bad
