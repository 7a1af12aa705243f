"""Step maps on the GPU against the oracle, exactly: growth from the free list,
the index layout, slots, positions, rows, and the calls that change nothing."""
import random

import pytest
import torch

from oracle import step_maps
from speculative_decode_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
I32 = torch.int32
GUARD = -77


def _dev(x):
    return None if x is None else torch.tensor(x, dtype=I32, device="cuda")


def _buffers(b, t, capacity):
    full = lambda n: torch.full((n,), GUARD, dtype=I32, device="cuda")  # noqa: E731
    return dict(indptr=full(b + 1), new_indptr=full(b + 1), slots=full(b * t), positions=full(b * t), rows=full(b * t),
                held=full(b), head=full(1), indices=None if capacity is None else full(max(capacity, 1))[:capacity],
                status=torch.zeros(1, dtype=I32, device="cuda"))


def _call(c, table, o, stream=None):
    grow = c["held"] is not None
    B.ddtree_step_maps(table, _dev(c["prefix"]), c["new"], c["page"], c["pages"], o["indptr"], o["indices"], o["slots"],
                       o["positions"], table_row=_dev(c["rows"]), new_lens=_dev(c["new_lens"]),
                       tree_parent=_dev(c["parent"]), pages_held=_dev(c["held"]),
                       free_pages=_dev(c["free"]) if grow else None, free_head=_dev([c["head"]]) if grow else None,
                       pages_held_out=o["held"] if grow else None, free_head_out=o["head"] if grow else None,
                       new_indptr=o["new_indptr"], token_rows=o["rows"], status=o["status"], stream=stream)


def _compare(c, table, o):
    ref = step_maps(c["table"], c["prefix"], c["new"], c["page"], c["pages"], c["capacity"], c["rows"], c["new_lens"],
                    c["parent"], c["held"], c["free"] or (), c["head"])
    torch.cuda.synchronize()
    assert table.tolist() == ref["table"]
    for name in ("indptr", "new_indptr", "slots", "positions", "rows"):
        assert o[name].tolist() == ref[name], name
    if c["held"] is not None:
        assert o["held"].tolist() == ref["held"] and o["head"].tolist() == [ref["head"]]
    if o["indices"] is not None:
        want = ref["indices"] or []
        assert o["indices"].tolist() == want + [GUARD] * (c["capacity"] - len(want))
    bits = (B.DDTREE_ST_BAD_INDEX * ref["bad_index"] | B.DDTREE_ST_BAD_PARENT * ref["bad_parent"] |
            B.DDTREE_ST_BAD_LENGTH * ref["bad_length"] | B.DDTREE_ST_NO_PAGES * ref["no_pages"])
    assert int(o["status"]) == bits
    return ref


def _check(c):
    table = _dev(c["table"])
    o = _buffers(len(c["prefix"]), c["new"], c["capacity"])
    _call(c, table, o)
    return _compare(c, table, o)


def _case(seed, prefixes, new, page, *, ragged=False, tree=False, grow=True, rows=None, spare=3, indices=True):
    r = random.Random(seed)
    b = len(prefixes)
    new_lens = [r.randint(0, new) for _ in prefixes] if ragged else None
    lens = [p + n for p, n in zip(prefixes, new_lens or [new] * b)]
    need = [-(-x // page) for x in lens]
    held = [r.randint(max(0, -(-p // page)), k) if r.random() < 0.9 else k for p, k in zip(prefixes, need)]
    n_rows = rows or b
    where = r.sample(range(n_rows), b) if rows else None
    pages = sum(need) + spare
    perm = list(range(pages))
    r.shuffle(perm)
    stride = max(need + [1]) + 2
    table = [[-1] * stride for _ in range(n_rows)]
    for i in range(b):
        have = held[i] if grow else need[i]
        row = table[where[i] if where else i]
        for k in range(have):
            row[k] = perm.pop()
    head = min(2, spare)
    return dict(table=table, prefix=prefixes, new=new, page=page, pages=pages, rows=where, new_lens=new_lens,
                parent=[[r.randint(-1, i - 1) for i in range(new)] for _ in range(b)] if tree else None,
                held=held if grow else None, free=[0] * head + perm if grow else None, head=head if grow else 0,
                capacity=sum(lens) + r.randint(0, 5) if indices else None)


@pytest.mark.parametrize("page", [1, 2, 7, 16, 64])
@pytest.mark.parametrize("prefixes,new", [([0], 1), ([1], 64), ([256], 4), ([0, 0, 5], 2), ([63, 64, 65], 3),
                                          ([1000, 0, 4097, 1, 31], 33)])
def test_lengths_and_pages(page, prefixes, new):
    _check(_case(page + new, prefixes, new, page))
    _check(_case(page + new + 1, prefixes, new, page, tree=True, rows=len(prefixes) + 4))
    _check(_case(page + new + 2, prefixes, new, page, ragged=True, grow=False))


@pytest.mark.parametrize("batch", [1, 2, 31, 32, 33, 255, 256, 257, 1023, 1024])
def test_batches(batch):
    r = random.Random(batch)
    prefixes = [r.choice([0, 1, 15, 16, 17, r.randint(0, 300)]) for _ in range(batch)]
    _check(_case(batch, prefixes, 5, 16, ragged=True, rows=batch + 3))
    _check(_case(batch, prefixes, 5, 3, tree=True, indices=False))


def test_no_new_tokens_at_all():
    c = _case(5, [3, 0, 9], 4, 4, ragged=True)
    c["new_lens"] = [0, 0, 0]
    _check(c)
    c = _case(6, [0, 0], 4, 4, ragged=True)
    c["new_lens"] = [0, 0]
    _check(c)


def test_chain_trees_of_64_nodes_and_stars():
    c = _case(7, [10, 20, 30], 64, 16, tree=True)
    c["parent"] = [list(range(-1, 63)), [-1] * 64, [-1] + [0] * 63]
    assert _check(c)["positions"][63] == 73


@pytest.mark.parametrize("parent", [[-1, 1, 0], [0, -1, 1], [-1, 5, 1], [-1, -2, 1]])
def test_bad_parents_end_the_walk(parent):
    c = _case(8, [10], 3, 16, tree=True)
    c["parent"] = [parent]
    assert _check(c)["bad_parent"]


def test_bad_pages_become_dropped_rows():
    c = _case(9, [100, 50], 4, 16, grow=False)
    c["table"][0][2] = c["pages"]
    c["table"][1][3] = -5
    assert _check(c)["bad_index"]
    c = _case(10, [100, 50], 40, 16)
    c["held"], c["free"] = [7, 4], [c["pages"] + 9] * 20
    assert _check(c)["bad_index"]


@pytest.mark.parametrize("what", ["negative", "long", "new", "row", "held", "capacity", "dry", "head"])
def test_calls_that_change_nothing(what):
    c = _case(11, [100, 50, 7], 4, 16, ragged=True, rows=5)
    if what == "negative":
        c["prefix"] = [100, -1, 7]
    elif what == "long":
        c["prefix"] = [100, 2 ** 31 - 1, 7]
    elif what == "new":
        c["new_lens"] = [0, 5, 1]
    elif what == "row":
        c["rows"] = [0, 5, 1]
    elif what == "held":
        c["held"] = [-1, 2, 1]
    elif what == "capacity":
        c["capacity"] = sum(c["prefix"]) + sum(c["new_lens"]) - 1
    elif what == "dry":
        c["held"], c["free"], c["head"] = [1, 1, 0], [1] * 11, 3
    else:
        c["head"] = len(c["free"]) + 1
    ref = _check(c)
    assert ref["no_pages"] if what in ("dry", "head") else ref["bad_length"]


def test_indices_at_an_odd_address_and_without_optional_outputs():
    c = _case(12, [37, 5], 3, 4)
    table, o = _dev(c["table"]), _buffers(2, 3, c["capacity"])
    big = torch.full((c["capacity"] + 1,), GUARD, dtype=I32, device="cuda")
    o["indices"] = big[1:]
    _call(c, table, o)
    ref = _compare(c, table, o)
    o2 = _buffers(2, 3, c["capacity"])
    B.ddtree_step_maps(_dev(ref["table"]), _dev(c["prefix"]), 3, 4, c["pages"], o2["indptr"], None, o2["slots"], o2["positions"])
    assert o2["slots"].tolist() == ref["slots"] and o2["positions"].tolist() == ref["positions"]
    assert int(big[0]) == GUARD


def test_captured_step_replays_with_other_lengths():
    c = _case(13, [40, 3, 77], 4, 16, ragged=True)
    table, o = _dev(c["table"]), _buffers(3, 4, c["capacity"] + 60)
    dev = {k: _dev(c[k]) for k in ("prefix", "new_lens", "held", "free")}
    head = _dev([c["head"]])
    args = (table, dev["prefix"], 4, 16, c["pages"], o["indptr"], o["indices"], o["slots"], o["positions"])
    kw = dict(new_lens=dev["new_lens"], pages_held=dev["held"], free_pages=dev["free"], free_head=head,
              pages_held_out=o["held"], free_head_out=o["head"], new_indptr=o["new_indptr"], token_rows=o["rows"],
              status=o["status"])
    bound = B.BoundStepMaps(*args, **kw)
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=st):
        bound()
    for prefix, new in (([40, 3, 77], c["new_lens"]), ([41, 0, 70], [0, 4, 1]), ([32, 16, 80], [4, 4, 4])):
        held = [-(-p // 16) for p in prefix]
        table.copy_(_dev([list(range(3 * i, 3 * i + len(c["table"][0]))) for i in range(3)]))
        start = table.tolist()
        dev["prefix"].copy_(_dev(prefix)), dev["new_lens"].copy_(_dev(new)), dev["held"].copy_(_dev(held))
        dev["free"].fill_(1)
        o["indices"].fill_(GUARD)
        g.replay()
        cc = dict(c, table=start, prefix=prefix, new_lens=new, held=held, free=[1] * len(c["free"]), capacity=c["capacity"] + 60)
        _compare(cc, table, o)


def test_python_refusals():
    c = _case(14, [5], 2, 4, grow=False)
    table, o = _dev(c["table"]), _buffers(1, 2, 10)
    good = (table, _dev(c["prefix"]), 2, 4, c["pages"], o["indptr"], o["indices"], o["slots"], o["positions"])
    for i, bad in ((0, table.long()), (0, table[0]), (0, table.cpu()), (5, o["indptr"][:1]), (7, o["slots"][:1]),
                   (8, o["positions"].float()), (0, _dev([[1, 2, 3, 4]] * 2)[:, ::2])):
        a = list(good)
        a[i] = bad
        with pytest.raises((TypeError, ValueError)):
            B.ddtree_step_maps(*a)
