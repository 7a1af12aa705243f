"""Calls through the binding that its objects and checks have to hold for."""
import pytest
import torch

from speculative_decode_tree_gb300 import binding as B
from test_draft_attn_gpu import Case

pytestmark = pytest.mark.gpu
I32 = torch.int32


def test_bound_attention_keeps_the_plan_it_checked():
    # The strides that were checked against `out` count, whatever becomes of the plan.  (Every place that either
    # stride reaches lies inside the buffer.)
    c = Case([300, 5, 77], 8, 2, 64, seed=71)
    c.device()
    wide = torch.full((3, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.plan.out_stride = 16 * 64
    bound = B.BoundDraftAttention(c.plan, c.q_dev, c.cache, *c.args[3:6], wide[:, :8], c.ws, **c.kw)
    c.plan.out_stride = 0
    bound()
    torch.cuda.synchronize()
    assert bool((wide[:, 8:] == 7.0).all())
    c.out = wide[:, :8].contiguous()
    c.compare()


def test_bound_appends_keep_their_rotation():
    g = torch.Generator().manual_seed(72)
    kv, q = torch.randn(5, 576, generator=g).to(torch.bfloat16).cuda(), torch.randn(5, 3, 64, generator=g).to(torch.bfloat16).cuda()
    pos, slots = torch.arange(1, 6, dtype=I32, device="cuda"), torch.arange(5, dtype=I32, device="cuda")
    pools, outs = [torch.zeros(5, 576, dtype=torch.bfloat16, device="cuda") for _ in range(2)], [torch.zeros_like(q) for _ in range(2)]
    rope = B.ddtree_rope_init(64, theta=1e4, interleaved=True)
    B.ddtree_mla_append(rope, kv, pos, slots, pools[0], q_rope=q, q_out=outs[0])
    bound = B.BoundMlaAppend(rope, kv, pos, slots, pools[1], q_rope=q, q_out=outs[1])
    rope.interleaved = 0
    bound()
    assert torch.equal(pools[0], pools[1]) and torch.equal(outs[0], outs[1])

    caches = [B.DraftCache(torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda"),
                           torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")) for _ in range(2)]
    rope = B.ddtree_rope_init(64, theta=1e4, interleaved=True)
    B.ddtree_draft_append(caches[0], rope, q, q, q, pos, slots, outs[0])
    bound = B.BoundDraftAppend(caches[1], rope, q, q, q, pos, slots, outs[1])
    rope.interleaved = 0
    bound()
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(outs[0], outs[1])


def test_an_empty_index_list_is_too_small_for_any_key():
    def call(prefix):
        table = torch.tensor([[0, -1, -1]], dtype=I32, device="cuda")
        o = {n: torch.full((s,), -9, dtype=I32, device="cuda") for n, s in
             (("indptr", 2), ("slots", 2), ("pos", 2), ("held", 1), ("head", 1))}
        status = torch.zeros(1, dtype=I32, device="cuda")
        new = torch.tensor([2 if prefix else 0], dtype=I32, device="cuda")
        B.ddtree_step_maps(table, torch.tensor([prefix], dtype=I32, device="cuda"), 2, 4, 8, o["indptr"],
                           torch.empty(0, dtype=I32, device="cuda"), o["slots"], o["pos"], new_lens=new,
                           pages_held=torch.ones(1, dtype=I32, device="cuda"),
                           free_pages=torch.arange(1, 8, dtype=I32, device="cuda"),
                           free_head=torch.zeros(1, dtype=I32, device="cuda"), pages_held_out=o["held"],
                           free_head_out=o["head"], status=status)
        return table.tolist(), o["indptr"].tolist(), o["held"].tolist(), o["head"].tolist(), int(status)

    assert call(3) == ([[0, -1, -1]], [0, 0], [1], [0], B.DDTREE_ST_BAD_LENGTH)
    assert call(0) == ([[0, -1, -1]], [0, 0], [1], [0], 0)


def test_reading_a_step_status_leaves_the_next_steps_bits(monkeypatch):
    from speculative_decode_tree_gb300.runner import DeviceStep
    pool = torch.zeros(64, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.full((1, 40), -1, dtype=I32, device="cuda")
    free = torch.arange(8, dtype=I32, device="cuda")
    step = DeviceStep(1, 4, 2, 30, 1, pool, table, free, B.ddtree_rope_init(64, theta=1e4), 0.1)
    step.tree_parent.fill_(-1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step.run(side)
    assert step.status(side) == 0

    # A slow clear, and a step that runs out of pages right behind it on the other stream.
    clear = torch.Tensor.zero_

    def slow(t):
        torch.cuda._sleep(200_000_000)
        return clear(t)
    step.free_head.fill_(6)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.Tensor, "zero_", slow)
    assert step.status(side) == 0
    step.run(side)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert step.status(side) & B.DDTREE_ST_NO_PAGES
    assert step.status(side) & B.DDTREE_ST_NO_PAGES == 0


@pytest.mark.parametrize("page", [16, 48, 8])
@pytest.mark.parametrize("entry", [2 ** 31 - 1, -2 ** 31, -1, 70_000_000])
def test_index_rows_of_table_entries_far_outside_the_pool(page, entry):
    from test_maps_gpu import _case, _check
    c = _case(21 + page, [page * 9 + 5, page * 4], 6, page, grow=False)
    c["table"][0][2] = c["table"][1][1] = c["table"][0][9] = entry
    assert _check(c)["bad_index"]


@pytest.mark.parametrize("heads,kvh,dim", [(8, 2, 64), (24, 1, 64), (8, 1, 256), (40, 1, 128)])
@pytest.mark.parametrize("scale", [0.0, 1e-38, -1e-42])
def test_scales_that_no_score_survives(scale, heads, kvh, dim):
    # Scores up to 1e38: what little the scale leaves of them must not become a weight.
    c = Case([700, 30], heads, kvh, dim, seed=73, scale=scale)
    c.q.mul_(1e17), c.k_raw.mul_(1e17)
    c.q_dev.copy_(c.q)
    assert c.run() == 0
    c.compare()
