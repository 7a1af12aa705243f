"""The drafter's operators with its cache in 8 bits in a row, as a serving loop
runs them: prompts taken in by chunks (step maps, 8-bit append, the contexts read
back, prompt attention, one captured graph for chunks of any length), then
tokens one at a time (maps, append, one-token attention, another graph).  Every
stage is checked against its oracle on the inputs that the GPU stages before it
produced."""
import random

import pytest
import torch

from oracle import append_oracle, prompt_attention, step_maps
from oracle import draft8_oracle as O
from speculative_decode_tree_gb300 import binding as B
from test_append_gpu import _bound, _close

pytestmark = pytest.mark.gpu
I32 = torch.int32
U = 2.0 ** -24


def _ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,page,block", [(64, 16, 16), (128, 24, 16), (256, 16, 1)])
def test_prompts_by_chunks_then_tokens(dim, page, block, dtype):
    r, g = random.Random(dim), torch.Generator().manual_seed(dim)
    nb, T, H, KV, pages, window, sinks, cap = 3, 40, 6, 2, 40, 50, 3, 12
    free = list(range(pages))
    r.shuffle(free)
    prefix, head = [0, 0, 0], 0
    table = [[-1] * cap for _ in range(nb)]
    dev_table = _ints(table)
    codes = [torch.zeros(pages, page, KV, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages, -(-page // block), KV, device="cuda") for _ in range(2)]
    cache = B.Draft8Cache(*codes, *scales, block)
    rope = B.ddtree_rope_init(dim // 2, theta=10000.0)
    freqs = append_oracle.frequencies(dim // 2, 10000.0)
    wq, wk = ((1 + 0.1 * torch.randn(dim, generator=g)).to(dtype) for _ in range(2))
    dq, dk = wq.cuda(), wk.cuda()
    most = nb * cap * page
    dev = dict(prefix=_ints(prefix), new=_ints([0] * nb), held=_ints([0] * nb), free=_ints(free), head=_ints([0]))
    buf = {n: torch.full((s,), -1, dtype=I32, device="cuda") for n, s in
           (("indptr", nb + 1), ("indices", most), ("slots", nb * T), ("pos", nb * T), ("rows", nb * T), ("held", nb), ("head", 1), ("new", nb + 1))}
    status = torch.zeros(1, dtype=I32, device="cuda")
    x = torch.zeros(nb * T, H + 2 * KV, dim, dtype=dtype, device="cuda")   # one projection
    q_out, out = torch.zeros(nb * T, H, dim, dtype=dtype, device="cuda"), torch.zeros(nb * T, H, dim, dtype=dtype, device="cuda")
    lse = torch.zeros(nb * T, H, device="cuda")
    k_rows, v_rows = (torch.zeros(most, KV, dim, dtype=dtype, device="cuda") for _ in range(2))
    scale = dim ** -0.5
    prompt = B.ddtree_prompt_attention_plan(nb, nb * T, most, H, KV, dim, dtype, window, sinks)
    token = B.ddtree_draft8_attention_plan(nb * T, H, cache, dtype, window, sinks)
    ws = torch.empty(B.ddtree_prompt_attention_workspace_size(prompt), dtype=torch.uint8, device="cuda")
    ws8 = torch.empty(B.ddtree_draft8_attention_workspace_size(token), dtype=torch.uint8, device="cuda")

    def maps_and_append(indices):
        B.ddtree_step_maps(dev_table, dev["prefix"], T, page, pages, buf["indptr"], indices, buf["slots"], buf["pos"], new_lens=dev["new"],
                           pages_held=dev["held"], free_pages=dev["free"], free_head=dev["head"], pages_held_out=buf["held"],
                           free_head_out=buf["head"], new_indptr=buf["new"], token_rows=buf["rows"], status=status)
        B.ddtree_draft8_append(cache, rope, x[:, :H], x[:, H:H + KV], x[:, H + KV:], buf["pos"], buf["slots"], q_out, q_weight=dq, k_weight=dk,
                               status=status)
    graphs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graphs[0]):
        maps_and_append(buf["indices"])
        B.ddtree_draft8_read(cache, buf["indices"], k_rows, v_rows, status=status)
        B.ddtree_prompt_attention(prompt, q_out, k_rows, v_rows, buf["new"], buf["indptr"], scale, out, ws, lse=lse)
    with torch.cuda.graph(graphs[1]):
        maps_and_append(None)
        B.ddtree_draft8_attention(token, q_out, cache, dev_table, buf["pos"], scale, out, ws8, token_rows=buf["rows"], lse=lse)

    for new, graph in (([40, 33, 5], 0), ([30, 0, 40], 0), ([1, 1, 1], 1), ([17, 40, 0], 0), ([1, 0, 1], 1), ([3, 1, 4], 1)):
        proj = torch.randn(nb * T, H + 2 * KV, dim, generator=g)
        proj[torch.rand(nb * T, generator=g) < 0.1] *= 20                  # some tokens make their blocks grow
        x.copy_(proj.to(dtype))
        before = [c.cpu().clone() for c in codes], [s.cpu().double() for s in scales]
        held = [-(-p // page) for p in prefix]
        for n, v in (("prefix", prefix), ("new", new), ("held", held), ("head", [head])):
            dev[n].copy_(_ints(v))
        buf["indices"].fill_(-1), out.fill_(7.0), lse.fill_(7.0)
        graphs[graph].replay()
        torch.cuda.synchronize()
        assert int(status) == 0 and B.ddtree_verify_mla_check(ws8 if graph else ws) == 0
        m = step_maps(table, prefix, T, page, pages, most if graph == 0 else None, new_lens=new, pages_held=held, free_pages=free, free_head=head)
        table, head = m["table"], m["head"]
        assert dev_table.tolist() == table and buf["slots"].tolist() == m["slots"] and buf["new"].tolist()[-1] == sum(new)
        n = sum(new)
        pos = torch.tensor(m["positions"], dtype=I32)
        host = x.cpu()
        # Queries, and the cache's values bit for bit.
        rq = append_oracle.rotate(append_oracle.norm(host[:, :H], wq, 1e-6), pos, freqs, False)
        length = append_oracle.pair_lengths(append_oracle.norm(host[:, :H], wq, 1e-6), len(freqs), False)
        _close(q_out[:n], rq[:n], _bound(rq, length, pos, dtype, 1.0)[:n], "queries")
        O.write_rows(host[:, H + KV:].double(), before[0][1], before[1][1], block, m["positions"], m["slots"])
        assert torch.equal(codes[1].cpu(), before[0][1]) and torch.equal(scales[1].cpu().double(), before[1][1])
        # Attention over what the cache holds, rounded to 16 bits on its way (or not, token by token).
        now_k, now_v = [c.cpu() for c in codes], [s.cpu() for s in scales]
        half = torch.finfo(dtype).eps / 2
        if graph == 0:
            idx = buf["indices"].cpu()
            total = int(buf["indptr"][-1])
            for got, c, s in ((k_rows, now_k[0], now_v[0]), (v_rows, now_k[1], now_v[1])):
                ref = O.read_rows(c, s, block, idx[:total].tolist(), torch.zeros(total, KV, dim))
                assert bool(((got[:total].cpu().double() - ref).abs() <= ref.abs() * (half + U) + 2.0 ** -25).all())
            ref, rl, mass, terms = prompt_attention(q_out.cpu(), k_rows.cpu(), v_rows.cpu(), buf["new"].tolist(), buf["indptr"].tolist(), window, sinks,
                                                    scale, torch.full((nb * T, H, dim), 7.0), torch.full((nb * T, H), 7.0))
            weight, tiny = half, 200 * 2.0 ** -35 * float(v_rows.double().abs().max())
        else:
            ref, rl, mass, terms = O.attention(q_out.cpu(), now_k[0], now_k[1], now_v[0], now_v[1], block, torch.tensor(table, dtype=I32), m["rows"],
                                               m["positions"], window, sinks, scale, torch.full((nb * T, H, dim), 7.0), torch.full((nb * T, H), 7.0))
            weight, tiny = 2.0 ** -11, 200 * 448 * 2.0 ** -35 * float(now_v[1].max())
        score = dim * U * terms + 100 * U
        ob = ref.abs() * half + mass * (weight + 2 * (2 * score + 64 * U)[..., None]) + tiny + 2.0 ** -25
        assert bool(((out.cpu().double() - ref).abs() <= ob).all())
        assert bool(((lse.cpu().double() - rl).abs() <= score + 8 * U * rl.abs() + 64 * U).all())
        assert bool((out[n:] == 7.0).all()) and bool((lse[n:] == 7.0).all())
        prefix = [p + k for p, k in zip(prefix, new)]
