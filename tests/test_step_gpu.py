"""The operators of a decode step in a row, as a serving loop runs them: step
maps, latent append, verify attention and acceptance over several steps of one
captured graph, with the page table, the free list and the accepted tokens
carried from step to step; and the drafter's maps, append and attention over
the accepted tokens.  Every stage is checked against its oracle on the inputs
that the GPU stages before it produced."""
import random

import pytest
import torch

from oracle import accept_batched, append_oracle, draft_attention, step_maps, verify_request
from parity_util import assert_within_tolerance
from speculative_decode_tree_gb300 import binding as B
from speculative_decode_tree_gb300.runner import DeviceStep
from test_append_gpu import _bound, _close
from test_draft_attn_gpu import _bounds

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16


def _ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def test_target_steps_from_one_graph():
    r, g = random.Random(3), torch.Generator().manual_seed(3)
    nb, T, H, V, rows, cap = 3, 7, 4, 40, 1024, 160
    scale, eps = 576 ** -0.5, 1e-6
    pool = torch.randn(rows, 576, generator=g).to(BF).cuda()
    free = list(range(rows))
    r.shuffle(free)
    prefix = [90, 0, 33]
    table = [[free.pop() for _ in range(p)] + [-1] * (cap - p) for p in prefix]
    dev_table, dev_free = _ints(table), _ints(free)
    rope = B.ddtree_rope_init(64, theta=10000.0, interleaved=True, scaling=B.DDTREE_ROPE_YARN, factor=4.0, original_positions=64)
    freqs = append_oracle.frequencies(64, 10000.0, append_oracle.YARN, 4.0, 64)
    weight = (1 + 0.1 * torch.randn(512, generator=g)).to(BF)
    step = DeviceStep(nb, T, H, cap - T, 1, pool, dev_table, dev_free, rope, scale, weight.cuda())
    out_i = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")  # noqa: E731
    logits, drafts = torch.zeros(nb, T + 1, V, dtype=BF, device="cuda"), out_i(nb, T)
    acc = [out_i(nb), out_i(nb), out_i(nb, T), out_i(nb, T), out_i(nb, T)]
    aws = torch.zeros(B.ddtree_accept_greedy_workspace_size(nb, T), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
        B.ddtree_accept_greedy(logits, drafts, step.tree_parent, step.kv_indices, step.kv_indptr, step.prefix_lens, *acc, aws)
    head, held = 0, list(prefix)
    taken = 0
    for _ in range(4):
        parents = [[r.randint(-1, i - 1) for i in range(T)] for _ in range(nb)]
        kv, q = torch.randn(nb * T, 576, generator=g).to(BF), torch.randn(nb * T, H, 576, generator=g).to(BF)
        logits.copy_(torch.randn(nb, T + 1, V, generator=g)), drafts.copy_(torch.randint(0, V, (nb, T), generator=g))
        for b in range(nb):  # the first root is always right, later nodes often
            for i in range(T):
                if parents[b][i] == i - 1:
                    drafts[b, i] = int(logits[b, i].float().argmax())
        step.prefix_lens.copy_(_ints(prefix)), step.tree_parent.copy_(_ints(parents)), step.pages_held.copy_(_ints(held))
        step.free_head.fill_(head), step.kv_new.copy_(kv), step.q.copy_(q)
        before = dev_table.tolist()
        pool_before = pool.cpu()
        graph.replay()
        assert step.status() == 0
        m = step_maps(before, prefix, T, 1, rows, nb * cap, tree_parent=parents, pages_held=held, free_pages=free, free_head=head)
        n = m["indptr"][-1]
        assert dev_table.tolist() == m["table"] and step.kv_indptr.tolist() == m["indptr"]
        assert step.kv_indices[:n].tolist() == m["indices"] and step.new_slots.tolist() == m["slots"]
        assert step.positions.tolist() == m["positions"] and int(step.free_head_out) == m["head"]
        pos, slots = step.positions.cpu(), step.new_slots.cpu()
        want, wq = append_oracle.mla_append(kv, weight, eps, q[..., 512:], pos, slots, pool_before, freqs, True, rope.mscale)
        length = torch.cat([want[slots.long()][:, None, :512].abs(), append_oracle.pair_lengths(kv[:, None, 512:], 32, True)], -1)
        _close(pool.cpu()[slots.long()][:, None], want[slots.long()][:, None], _bound(want[slots.long()][:, None], length, pos, BF, rope.mscale), "rows")
        _close(step.q[..., 512:], wq, _bound(wq, append_oracle.pair_lengths(q[..., 512:], 32, True), pos, BF, rope.mscale), "queries")
        assert torch.equal(step.q[..., :512].cpu(), q[..., :512])
        host_pool, host_q = pool.cpu(), step.q.cpu()
        for b in range(nb):
            sl = slice(b * T, (b + 1) * T)
            O, L = verify_request(host_q[sl, :, :512], host_q[sl, :, 512:], host_pool, step.kv_indices[m["indptr"][b]:m["indptr"][b + 1]].cpu(),
                                  prefix[b], parents[b], scale)
            assert_within_tolerance(step.out[sl], step.lse[sl], O, L, f"request {b}")
        ref = accept_batched(logits.cpu(), drafts.cpu(), _ints(parents).cpu(), step.kv_indices.cpu(), step.kv_indptr.cpu(), _ints(prefix).cpu())
        for buf, key in zip(acc, ("accept_len", "next_token", "accepted_nodes", "commit_indices", "freed_indices")):
            assert (buf.cpu().numpy() == ref[key]).all(), key
        # Commit: accepted rows follow the prefix in path order, the others go back to the list.
        head = m["head"]
        for b in range(nb):
            k = int(acc[0][b])
            taken += k
            dev_table[b, prefix[b]:prefix[b] + k] = acc[3][b, :k]
            dev_table[b, prefix[b] + k:prefix[b] + T] = -1
            for i, row in enumerate(acc[4][b, :T - k].tolist()):
                head -= 1
                free[head] = row
            prefix[b] += k
            held[b] = prefix[b]
        dev_free.copy_(_ints(free))
    assert taken >= 4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_drafter_takes_in_accepted_tokens(dtype):
    r, g = random.Random(5), torch.Generator().manual_seed(5)
    nb, T, H, KV, D, page, pages, window, sinks = 3, 5, 6, 2, 128, 16, 60, 40, 3
    prefix, new = [100, 7, 0], [5, 0, 3]
    cap = 12
    perm = list(range(pages))
    r.shuffle(perm)
    held = [-(-p // page) for p in prefix]
    table = [[perm.pop() for _ in range(h)] + [-1] * (cap - h) for h in held]
    kc, vc = (torch.randn(pages, KV, page, D, generator=g).to(dtype).cuda().transpose(1, 2) for _ in range(2))
    cache = B.DraftCache(kc, vc)
    width = (H + 2 * KV) * D
    qkv = torch.randn(nb * T, width, generator=g).to(dtype)
    d = qkv.cuda()
    q, k, v = d[:, :H * D].view(-1, H, D), d[:, H * D:(H + KV) * D].view(-1, KV, D), d[:, (H + KV) * D:].view(-1, KV, D)
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g)).to(dtype) for _ in range(2))
    rope = B.ddtree_rope_init(64, theta=10000.0)
    freqs = append_oracle.frequencies(64, 10000.0)
    dev_table, bufs = _ints(table), {n: torch.full((s,), -9, dtype=I32, device="cuda") for n, s in
                                     (("indptr", nb + 1), ("slots", nb * T), ("pos", nb * T), ("rows", nb * T), ("held", nb), ("head", 1))}
    status = torch.zeros(1, dtype=I32, device="cuda")
    q_out = torch.zeros(nb * T, H, D, dtype=dtype, device="cuda")
    out = torch.full((nb * T, H, D), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((nb * T, H), 7.0, device="cuda")
    plan = B.ddtree_draft_attention_plan(nb * T, H, cache, window, sinks)
    ws = torch.empty(B.ddtree_draft_attention_workspace_size(plan), dtype=torch.uint8, device="cuda")
    host_k, host_v = kc.cpu(), vc.cpu()
    args = dict(prefix=_ints(prefix), new=_ints(new), held=_ints(held), free=_ints(perm), head=_ints([0]), wq=wq.cuda(), wk=wk.cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.ddtree_step_maps(dev_table, args["prefix"], T, page, pages, bufs["indptr"], None, bufs["slots"], bufs["pos"], new_lens=args["new"],
                           pages_held=args["held"], free_pages=args["free"], free_head=args["head"], pages_held_out=bufs["held"],
                           free_head_out=bufs["head"], token_rows=bufs["rows"], status=status)
        B.ddtree_draft_append(cache, rope, q, k, v, bufs["pos"], bufs["slots"], q_out, q_weight=args["wq"], k_weight=args["wk"], status=status)
        B.ddtree_draft_attention(plan, q_out, cache, dev_table, bufs["pos"], D ** -0.5, out, ws, token_rows=bufs["rows"], lse=lse)
    graph.replay()
    graph.replay()  # nothing of a step depends on what the last one left behind
    assert B.ddtree_verify_mla_check(ws) == 0 and int(status) == 0
    m = step_maps(table, prefix, T, page, pages, None, new_lens=new, pages_held=held, free_pages=perm, free_head=0)
    assert dev_table.tolist() == m["table"] and bufs["slots"].tolist() == m["slots"] and bufs["rows"].tolist() == m["rows"]
    pos, slots = torch.tensor(m["positions"], dtype=I32), torch.tensor(m["slots"], dtype=I32)
    cq, ck, cv = (t.cpu() for t in (q, k, v))
    rq, rk, rv = append_oracle.draft_append(cq, ck, cv, wq, wk, 1e-6, pos, slots, host_k, host_v, freqs, False)
    n = sum(new)
    _close(q_out[:n], rq[:n], _bound(rq, append_oracle.pair_lengths(append_oracle.norm(cq, wq, 1e-6), 32, False), pos, dtype, 1.0)[:n], "queries")
    assert torch.equal(vc.cpu().double(), rv)
    ref, rl, mass, terms = draft_attention(q_out.cpu(), kc.cpu(), vc.cpu(), dev_table.cpu(), m["rows"], m["positions"], window, sinks,
                                           D ** -0.5, torch.full((nb * T, H, D), 7.0), torch.full((nb * T, H), 7.0))
    ob, lb = _bounds(ref, rl, mass, terms, D, dtype)
    assert bool(((out.cpu().double() - ref).abs() <= ob).all()) and bool(((lse.cpu().double() - rl).abs() <= lb).all())
    assert bool((out[n:] == 7.0).all()) and bool((lse[n:] == 7.0).all())
