"""The operators around verify attention, as measured calls.

Four operators of one speculative decode step, in their plain form (elementary
torch operations in 32 bits or more, rounded once) and as the library's calls:

  maps          page tables grown from a free list, and from the lengths the
                verify index layout, slots, positions and table rows
  mla_append    a latent KV row per token (norm of the latent, rotation of the
                rope part) written to the pool, and the rotated query rope part
  draft_append  the drafter's head norms and rotation of queries and keys, keys
                and values written to its paged cache
  draft_attn    the drafter's attention of one new token per request over its
                paged cache, with an optional sliding window and sink tokens
"""
import math

import torch

own = False

DEV = "cuda"
INT32 = torch.int32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # The smallest step: one request of the 256-token prefix workload, a 4-node chain, token-granular.
        dict(name="maps_one_request", op="maps", batch=1, lo=256, hi=256, new=4, ragged=False, tree=False,
             page=1, table_rows=4, alloc=True),
        # Eight requests of 1k to 185k tokens with 32-node trees on a churned token-granular pool.
        dict(name="maps_mixed_batch", op="maps", batch=8, lo=1024, hi=189440, new=32, ragged=False, tree=True,
             page=1, table_rows=16, alloc=True),
        # A full batch of short and long contexts whose accepted chains differ in length, pages of 16.
        dict(name="maps_full_batch", op="maps", batch=1024, lo=256, hi=131072, new=9, ragged=True, tree=False,
             page=16, table_rows=1024, alloc=True),
        # One 32-node tree on a rank with 8 heads: latency only.
        dict(name="mla_append_tree", op="mla_append", tokens=32, heads=8, interleaved=True, scaling="yarn",
             far=65536, packed=True, norm=True),
        # Eight 64-node trees with all 128 heads, queries cut out of a wider projection.
        dict(name="mla_append_heads", op="mla_append", tokens=512, heads=128, interleaved=True, scaling="yarn",
             far=189440, packed=True, norm=True),
        # A long prompt's rows written in one call, an odd number of them, the half layout.
        dict(name="mla_append_prompt", op="mla_append", tokens=65521, heads=16, interleaved=False, scaling="none",
             far=65536, packed=False, norm=True),
        # The drafter's step for eight requests.
        dict(name="draft_append_step", op="draft_append", tokens=8, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, scaling="none", far=65536, dtype="bf16", norm=True, page=16, heads_first=False),
        # The drafter taking in a long prompt; a quarter of the head rotated, pages with the heads outside.
        dict(name="draft_append_prompt", op="draft_append", tokens=32749, heads=16, kv_heads=4, dim=64, rot=16,
             interleaved=True, scaling="linear", far=131072, dtype="fp16", norm=False, page=64, heads_first=True),
        # One request far into its context, a 2,048-token window and four sink tokens, token-granular.
        dict(name="draft_attn_window", op="draft_attn", batch=1, lo=65536, hi=65536, heads=32, kv_heads=8, dim=128,
             window=2048, sinks=4, page=1, heads_first=False, dtype="bf16"),
        # One request over its whole 185k context with few key heads: the split over the length is everything.
        dict(name="draft_attn_long", op="draft_attn", batch=1, lo=189440, hi=189440, heads=16, kv_heads=2, dim=256,
             window=0, sinks=0, page=16, heads_first=True, dtype="bf16"),
        # Eight requests of 1k to 185k tokens, no window: the most bytes.
        dict(name="draft_attn_mixed", op="draft_attn", batch=8, lo=1024, hi=189440, heads=32, kv_heads=8, dim=128,
             window=0, sinks=0, page=64, heads_first=False, dtype="bf16"),
        # A served batch of a few thousand tokens each, one key head for eight queries, a page size that is no
        # power of two.
        dict(name="draft_attn_batch", op="draft_attn", batch=61, lo=511, hi=16384, heads=64, kv_heads=8, dim=64,
             window=0, sinks=0, page=48, heads_first=False, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["maps", "mla_append", "draft_append", "draft_attn"])
    scaling = rng.choice(["none", "linear", "yarn"])
    if op == "maps":
        batch = _log(rng, 1, 1024)
        hi = _log(rng, 64, 131072)
        tree = rng.random() < 0.5
        return dict(op=op, batch=batch, lo=max(1, _log(rng, 1, hi)), hi=hi, new=rng.randint(1, 64),
                    ragged=not tree and rng.random() < 0.5, tree=tree, page=rng.choice([1, 1, 16, 33, 64, 256]),
                    table_rows=batch + rng.randint(0, 9), alloc=rng.random() < 0.8) if batch * hi < 1 << 26 else draw(rng)
    if op == "mla_append":
        heads = rng.choice([1, 5, 8, 16, 24, 64, 128])
        return dict(op=op, tokens=_log(rng, 1, min(65536, (1 << 20) // max(heads, 8))), heads=heads,
                    interleaved=rng.random() < 0.5, scaling=scaling, far=_log(rng, 1024, 1 << 20),
                    packed=rng.random() < 0.5, norm=rng.random() < 0.8)
    if op == "draft_append":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 7, 8, 16])
        return dict(op=op, tokens=_log(rng, 1, max(1, (1 << 26) // (dim * (heads + 2 * kv)))), heads=heads,
                    kv_heads=kv, dim=dim, rot=rng.choice([16, dim // 4, dim // 2, dim]),
                    interleaved=rng.random() < 0.5, scaling=scaling, far=_log(rng, 1024, 1 << 20),
                    dtype=rng.choice(["bf16", "fp16"]), norm=rng.random() < 0.7,
                    page=rng.choice([1, 16, 48, 64]), heads_first=rng.random() < 0.5)
    batch = _log(rng, 1, 256)
    dim = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    hi = _log(rng, 16, 189440)
    window = 0 if rng.random() < 0.6 else _log(rng, 1, 8192)
    if batch * hi * kv * dim > 1 << 28:
        return draw(rng)
    return dict(op=op, batch=batch, lo=max(1, _log(rng, 1, hi)), hi=hi, heads=kv * rng.choice([1, 3, 4, 8, 16, 40, 64]),
                kv_heads=kv, dim=dim, window=window, sinks=rng.choice([0, 1, 4, 33]), page=rng.choice([1, 16, 48, 64]),
                heads_first=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))


def _lens(case):
    """Lengths of a batch, spread evenly over their logarithm."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    return [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]


def _visible(case, pos):
    lo = max(0, pos - case["window"] + 1) if case["window"] else 0
    return min(case["sinks"], lo) + pos - lo + 1


def work(case):
    op = case["op"]
    if op == "maps":
        new = [1 + i % case["new"] for i in range(case["batch"])] if case["ragged"] else [case["new"]] * case["batch"]
        total = sum(_lens(case)) + sum(new)
        pages = sum(-(-(p + n) // case["page"]) for p, n in zip(_lens(case), new))
        return {"bytes": 4 * (total + pages + 4 * sum(new) + 8 * case["batch"]), "flops": 0}
    if op == "mla_append":
        n, h = case["tokens"], case["heads"]
        return {"bytes": n * (2 * 1152 + 2 * h * 128 + 8) + 1024, "flops": n * (4 * 512 + (h + 1) * 64 * 3)}
    if op == "draft_append":
        n, d = case["tokens"], case["dim"]
        heads = case["heads"] + 2 * case["kv_heads"]
        return {"bytes": n * (heads * d * 4 + 8), "flops": n * (case["heads"] + case["kv_heads"]) * (4 * d + 3 * case["rot"])}
    seen = sum(_visible(case, p) for p in _lens(case))
    n, d = case["batch"], case["dim"]
    return {"bytes": seen * case["kv_heads"] * d * 4 + 4 * -(-seen // case["page"]) + n * case["heads"] * (d * 4 + 4),
            "flops": 4 * seen * case["heads"] * d}


# ----------------------------------------------------------------- the inputs
def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _rope(case, rot):
    """Arguments of the rotation: base, scaling, factor, original length, mscale."""
    scaling = case["scaling"]
    return dict(rot=rot, interleaved=case["interleaved"], theta=10000.0 if scaling == "yarn" else 500000.0,
                scaling=scaling, factor=1.0 if scaling == "none" else 8.0, original=4096, beta_fast=32.0,
                beta_slow=1.0, mscale=0.1 * math.log(8.0) + 1.0 if scaling == "yarn" else 1.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1_000_003 * seed + 17)
    s = {"case": case, "kept": {}}  # "kept": calls whose buffers stay the same, marshalled once by the program
    op = case["op"]
    if op == "maps":
        b, page = case["batch"], case["page"]
        order = torch.randperm(b, generator=gen, device=DEV)
        prefix = torch.tensor(_lens(case), dtype=INT32, device=DEV)[order]
        new = (1 + torch.arange(b, device=DEV) % case["new"]).to(INT32)[order] if case["ragged"] else \
            torch.full((b,), case["new"], dtype=INT32, device=DEV)
        need = (prefix + new + page - 1) // page
        # Half the requests have room left in their last page only, the others some spare pages.
        held = torch.minimum((prefix + page - 1) // page + torch.randint(0, 2, (b,), generator=gen, device=DEV), need)
        held = (held if case["alloc"] else need).to(INT32)
        stride = (case["hi"] + case["new"] + page - 1) // page + 3
        pages = int(need.sum()) + 64
        perm = torch.randperm(pages, generator=gen, device=DEV).to(INT32)
        rows = torch.randperm(case["table_rows"], generator=gen, device=DEV)[:b]
        col = torch.arange(stride, device=DEV)[None, :]
        first = torch.cumsum(held, 0) - held
        mine = torch.where(col < held[:, None], perm[(first[:, None] + col).clamp_max(pages - 1)], -1)
        table = torch.full((case["table_rows"], stride), -1, dtype=INT32, device=DEV)
        table[rows] = mine.to(INT32)
        t = case["new"]
        parent = (torch.rand((b, t), generator=gen, device=DEV) * (torch.arange(t, device=DEV) + 1)).floor().to(INT32) - 1
        total = int((prefix + new).sum())
        empty = lambda *shape: torch.full(shape, -1, dtype=INT32, device=DEV)  # noqa: E731
        s.update(table=table, rows=rows.to(INT32), prefix=prefix, new=new if case["ragged"] else None,
                 parent=parent if case["tree"] else None, held=held, free=perm[int(held.sum()):].contiguous(),
                 head=torch.tensor([5], dtype=INT32, device=DEV), pages=pages, total=total,
                 indptr=empty(b + 1), indices=empty(total + 7), new_indptr=empty(b + 1), slots=empty(b * t),
                 positions=empty(b * t), token_rows=empty(b * t), held_out=empty(b), head_out=empty(1),
                 status=torch.zeros(1, dtype=INT32, device=DEV))
        return s
    if op == "mla_append":
        n, h = case["tokens"], case["heads"]
        rows = n + n // 8 + 16
        wide = 192 if case["packed"] else 64  # queries are the last 64 columns of a wider projection
        s.update(kv=_normal(gen, (n, 576), torch.bfloat16) * 1.5,
                 weight=(1 + 0.1 * _normal(gen, (512,), torch.float32)).to(torch.bfloat16) if case["norm"] else None,
                 q=_normal(gen, (n, max(h, 1), wide), torch.bfloat16)[:, :h, wide - 64:],
                 positions=torch.randint(0, case["far"], (n,), generator=gen, device=DEV).to(INT32),
                 slots=torch.randperm(rows, generator=gen, device=DEV)[:n].to(INT32),
                 pool=_normal(gen, (rows, 576), torch.bfloat16),
                 q_out=torch.zeros(n, h, 64, dtype=torch.bfloat16, device=DEV), rope=_rope(case, 64),
                 status=torch.zeros(1, dtype=INT32, device=DEV))
        return s
    dtype, d, kvh, page = DTYPES[case["dtype"]], case["dim"], case["kv_heads"], case["page"]

    def cache(pages):
        if case["heads_first"]:
            return _normal(gen, (pages, kvh, page, d), dtype).transpose(1, 2)
        return _normal(gen, (pages, page, kvh, d), dtype)

    if op == "draft_append":
        n, h = case["tokens"], case["heads"]
        pages = -(-n // page) + 3
        qkv = _normal(gen, (n, (h + 2 * kvh) * d), dtype) * 2
        weight = lambda: (1 + 0.1 * _normal(gen, (d,), torch.float32)).to(dtype) if case["norm"] else None  # noqa: E731
        s.update(q=qkv[:, :h * d].view(n, h, d), k=qkv[:, h * d:(h + kvh) * d].view(n, kvh, d),
                 v=qkv[:, (h + kvh) * d:].view(n, kvh, d), wq=weight(), wk=weight(),
                 positions=torch.randint(0, case["far"], (n,), generator=gen, device=DEV).to(INT32),
                 slots=torch.randperm(pages * page, generator=gen, device=DEV)[:n].to(INT32),
                 k_cache=cache(pages), v_cache=cache(pages), q_out=torch.zeros(n, h, d, dtype=dtype, device=DEV),
                 rope=_rope(case, case["rot"]), status=torch.zeros(1, dtype=INT32, device=DEV))
        return s
    b, h = case["batch"], case["heads"]
    lens = torch.tensor(_lens(case), device=DEV)
    pos = lens[torch.randperm(b, generator=gen, device=DEV)]  # the new token stands behind its context
    lo = (pos - case["window"] + 1).clamp_min(0) if case["window"] else torch.zeros_like(pos)
    stride = int(pos.max()) // page + 2
    col = torch.arange(stride, device=DEV)[None, :]
    # Pages that neither the window nor the sinks reach have been given back.
    keep = (col <= pos[:, None] // page) & ((col >= lo[:, None] // page) | (col * page < case["sinks"]))
    pages = int(keep.sum()) + 5
    table = torch.full((b + 2, stride), -1, dtype=INT32, device=DEV)
    token_rows = torch.randperm(b + 2, generator=gen, device=DEV)[:b]
    mine = torch.full((b, stride), -1, dtype=INT32, device=DEV)
    mine[keep] = torch.randperm(pages, generator=gen, device=DEV)[:pages - 5].to(INT32)
    table[token_rows] = mine
    s.update(q=_normal(gen, (b, h, d), dtype) * 2, k_cache=cache(pages), v_cache=cache(pages), table=table,
             token_rows=token_rows.to(INT32), positions=pos.to(INT32), scale=d ** -0.5,
             most=max(_visible(case, p) for p in _lens(case)),
             out=torch.zeros(b, h, d, dtype=dtype, device=DEV), lse=torch.zeros(b, h, dtype=torch.float32, device=DEV))
    return s


# ------------------------------------------------------------ the plain forms
def _reach(r):
    return (r @ r).clamp_max(1.0)


def _plain_maps(s):
    case = s["case"]
    b, t, page = case["batch"], case["new"], case["page"]
    prefix = s["prefix"].long()
    new = s["new"].long() if s["new"] is not None else torch.full_like(prefix, t)
    lens = prefix + new
    held = s["held"].long()
    want = torch.maximum((lens + page - 1) // page, held)
    need = want - held
    off = s["head"].long() + torch.cumsum(need, 0) - need
    rows = s["rows"].long()
    col = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    given = (col >= held[:, None]) & (col < want[:, None])
    at = (off[:, None] + col - held[:, None]).clamp(0, s["free"].numel() - 1)
    s["table"][rows] = torch.where(given, s["free"][at], s["table"][rows])
    s["held_out"].copy_(want)
    s["head_out"].copy_(s["head"] + need.sum())
    ptr = torch.cumsum(lens, 0) - lens
    s["indptr"][0] = 0
    s["indptr"][1:] = torch.cumsum(lens, 0)
    which = torch.repeat_interleave(torch.arange(b, device=DEV), lens, output_size=s["total"])
    j = torch.arange(s["total"], device=DEV) - ptr[which]
    s["indices"][:s["total"]] = s["table"][rows[which], j // page] * page + (j % page).to(INT32)
    nptr = torch.cumsum(new, 0)
    s["new_indptr"][0] = 0
    s["new_indptr"][1:] = nptr
    node = torch.arange(b * t, device=DEV)
    of = torch.searchsorted(nptr, node, right=True)
    live = of < b
    of = of.clamp_max(b - 1)
    i = torch.where(live, node - (nptr - new)[of], 0)
    if s["parent"] is not None:
        parent = s["parent"].long()
        eye = torch.eye(t, device=DEV)
        r = eye + (parent[:, :, None] == torch.arange(t, device=DEV)).float()
        r = _reach(_reach(_reach(_reach(_reach(_reach(r))))))
        depth = (r.sum(-1).long() - 1)[of, i]
    else:
        depth = i
    key = prefix[of] + i
    slot = s["table"][rows[of], key // page].long() * page + key % page
    s["positions"].copy_(torch.where(live, prefix[of] + depth, -1))
    s["slots"].copy_(torch.where(live, slot, -1))
    s["token_rows"].copy_(torch.where(live, rows[of], -1))


def _plain_angles(rope, positions):
    """Angles in radians, in 64 bits: one row per token, one column per pair."""
    half = rope["rot"] // 2
    i = torch.arange(half, device=positions.device, dtype=torch.float64)
    freq = rope["theta"] ** (-2.0 * i / rope["rot"])
    if rope["scaling"] == "linear":
        freq = freq / rope["factor"]
    if rope["scaling"] == "yarn":
        turn = lambda beta: rope["rot"] * math.log(rope["original"] / (beta * 2 * math.pi)) / (2 * math.log(rope["theta"]))  # noqa: E731
        low = max(math.floor(turn(rope["beta_fast"])), 0)
        high = min(math.ceil(turn(rope["beta_slow"])), rope["rot"] - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        freq = freq / rope["factor"] * ramp + freq * (1 - ramp)
    return positions.double()[:, None] * freq


def _plain_rotate(x, rope, positions):
    """x [tokens, heads, width] in 32 bits: its first rope["rot"] columns rotated."""
    angle = _plain_angles(rope, positions)
    cos = (torch.cos(angle) * rope["mscale"]).float()[:, None, :]
    sin = (torch.sin(angle) * rope["mscale"]).float()[:, None, :]
    rot = rope["rot"]
    y = x.clone()
    if rope["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = a * sin + b * cos
    return y


EPS = 1e-6


def _plain_norm(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _plain_mla_append(s):
    x = s["kv"].float()
    latent = _plain_norm(x[:, :512], s["weight"])
    rope = _plain_rotate(x[:, None, 512:], s["rope"], s["positions"])[:, 0]
    s["pool"][s["slots"].long()] = torch.cat([latent, rope], -1).to(s["pool"].dtype)
    s["q_out"].copy_(_plain_rotate(s["q"].float(), s["rope"], s["positions"]))


def _plain_draft_append(s):
    page = s["case"]["page"]
    slot = s["slots"].long()
    q = _plain_rotate(_plain_norm(s["q"].float(), s["wq"]), s["rope"], s["positions"])
    k = _plain_rotate(_plain_norm(s["k"].float(), s["wk"]), s["rope"], s["positions"])
    s["q_out"].copy_(q)
    s["k_cache"][slot // page, slot % page] = k.to(s["k_cache"].dtype)
    s["v_cache"][slot // page, slot % page] = s["v"]


def _plain_draft_attn(s):
    case = s["case"]
    page, kvh = case["page"], case["kv_heads"]
    pos = s["positions"].long()
    lo = (pos - case["window"] + 1).clamp_min(0) if case["window"] else torch.zeros_like(pos)
    first = lo.clamp_max(case["sinks"])
    seen = first + pos - lo + 1
    v = torch.arange(s["most"], device=pos.device)[None, :]
    live = v < seen[:, None]
    key = torch.where(v < first[:, None], v, v - first[:, None] + lo[:, None])
    key = torch.where(live, key, pos[:, None])
    at = s["table"].long()[s["token_rows"].long()[:, None], key // page]
    k = s["k_cache"][at, key % page].float()
    q = s["q"].float().view(pos.numel(), kvh, -1, case["dim"])
    score = torch.einsum("nhgd,nvhd->nhgv", q, k) * s["scale"]
    del k
    score = score.masked_fill(~live[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("nhgv,nvhd->nhgd", p, s["v_cache"][at, key % page].float()) / total
    s["out"].copy_(out.view(s["out"].shape))
    s["lse"].copy_((top + torch.log(total)).view(s["lse"].shape))


# ---------------------------------------------------------- the library's calls
def _own_rope(B, rope):
    scaling = {"none": B.DDTREE_ROPE_PLAIN, "linear": B.DDTREE_ROPE_LINEAR, "yarn": B.DDTREE_ROPE_YARN}[rope["scaling"]]
    return B.ddtree_rope_init(rope["rot"], theta=rope["theta"], interleaved=rope["interleaved"], scaling=scaling,
                              factor=rope["factor"], original_positions=rope["original"],
                              beta_fast=rope["beta_fast"], beta_slow=rope["beta_slow"], mscale=rope["mscale"])


def _own_call(s):
    """The step's call with its buffers, checked and marshalled once, as a decode loop with static buffers keeps it."""
    from speculative_decode_tree_gb300 import binding as B
    case = s["case"]
    if case["op"] == "maps":
        return B.BoundStepMaps(s["table"], s["prefix"], case["new"], case["page"], s["pages"], s["indptr"], s["indices"],
                               s["slots"], s["positions"], table_row=s["rows"], new_lens=s["new"],
                               tree_parent=s["parent"], pages_held=s["held"], free_pages=s["free"],
                               free_head=s["head"], pages_held_out=s["held_out"], free_head_out=s["head_out"],
                               new_indptr=s["new_indptr"], token_rows=s["token_rows"], status=s["status"])
    if case["op"] == "mla_append":
        return B.BoundMlaAppend(_own_rope(B, s["rope"]), s["kv"], s["positions"], s["slots"], s["pool"],
                                latent_weight=s["weight"], eps=EPS, q_rope=s["q"], q_out=s["q_out"], status=s["status"])
    cache = B.DraftCache(s["k_cache"], s["v_cache"])
    if case["op"] == "draft_append":
        return B.BoundDraftAppend(cache, _own_rope(B, s["rope"]), s["q"], s["k"], s["v"], s["positions"], s["slots"],
                                  s["q_out"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS, status=s["status"])
    plan = B.ddtree_draft_attention_plan(case["batch"], case["heads"], cache, window=case["window"], n_sinks=case["sinks"])
    workspace = torch.empty(B.ddtree_draft_attention_workspace_size(plan), dtype=torch.uint8, device=DEV)
    return B.BoundDraftAttention(plan, s["q"], cache, s["table"], s["positions"], s["scale"], s["out"], workspace,
                                 token_rows=s["token_rows"], lse=s["lse"])


PLAIN = {"maps": _plain_maps, "mla_append": _plain_mla_append, "draft_append": _plain_draft_append,
         "draft_attn": _plain_draft_attn}
OUTPUTS = {"maps": ("table", "held_out", "head_out", "indptr", "indices", "new_indptr", "slots", "positions", "token_rows"),
           "mla_append": ("pool", "q_out"), "draft_append": ("q_out", "k_cache", "v_cache"), "draft_attn": ("out", "lse")}


def run(state):
    if own:
        if "call" not in state["kept"]:
            state["kept"]["call"] = _own_call(state)
        state["kept"]["call"]()
    else:
        PLAIN[state["case"]["op"]](state)
    return {k: state[k] for k in OUTPUTS[state["case"]["op"]]}


# ------------------------------------------------------- the definitions, 64 bits
def _frequency(rope, i):
    f = rope["theta"] ** (-2.0 * i / rope["rot"])
    if rope["scaling"] == "linear":
        return f / rope["factor"]
    if rope["scaling"] != "yarn":
        return f
    # Pairs that turn more than beta_fast times over the original length keep their frequency, those that turn
    # less than beta_slow times are stretched, the others are mixed along their index.
    edge = [rope["rot"] * math.log(rope["original"] / (b * 2 * math.pi)) / (2 * math.log(rope["theta"]))
            for b in (rope["beta_fast"], rope["beta_slow"])]
    low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rope["rot"] - 1)
    mix = min(1.0, max(0.0, (i - low) / max(high - low, 1e-3)))
    return f * (1 - mix) + f / rope["factor"] * mix


def _turned(vec, rope, positions):
    """The rotation as a product of complex numbers, in 64 bits."""
    rot, half = rope["rot"], rope["rot"] // 2
    freq = [_frequency(rope, i) for i in range(half)]
    angle = positions.double().unsqueeze(-1) * torch.tensor(freq, dtype=torch.float64, device=positions.device)
    turn = torch.polar(torch.full_like(angle, rope["mscale"]), angle).unsqueeze(1)
    head, rest = vec[..., :rot], vec[..., rot:]
    if rope["interleaved"]:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous()) * turn
        head = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, rest], -1)


def _scaled(vec, weight):
    if weight is None:
        return vec
    return vec / torch.sqrt((vec * vec).sum(-1, keepdim=True) / vec.shape[-1] + EPS) * weight.double()


def exact(case, seed):
    if case["op"] == "maps":
        return None
    s = prepare(case, seed)
    if case["op"] == "mla_append":
        kv = s["kv"].double()
        pool = s["pool"].double()
        row = torch.cat([_scaled(kv[:, :512], s["weight"]), _turned(kv[:, 512:].unsqueeze(1), s["rope"], s["positions"]).squeeze(1)], 1)
        pool.index_copy_(0, s["slots"].long(), row)
        return {"pool": pool, "q_out": _turned(s["q"].double(), s["rope"], s["positions"])}
    if case["op"] == "draft_append":
        keys, values = s["k_cache"].double(), s["v_cache"].double()
        where = s["slots"].long()
        where = (torch.div(where, case["page"], rounding_mode="floor"), where.remainder(case["page"]))
        keys.index_put_(where, _turned(_scaled(s["k"].double(), s["wk"]), s["rope"], s["positions"]))
        values.index_put_(where, s["v"].double())
        return {"q_out": _turned(_scaled(s["q"].double(), s["wq"]), s["rope"], s["positions"]), "k_cache": keys, "v_cache": values}
    out, lse = s["out"].double(), s["lse"].double()
    group = case["heads"] // case["kv_heads"]
    for n, (pos, row) in enumerate(zip(s["positions"].tolist(), s["token_rows"].tolist())):
        keys = [j for j in range(min(case["sinks"], pos + 1)) if case["window"] and j <= pos - case["window"]]
        since = max(0, pos - case["window"] + 1) if case["window"] else 0
        j = torch.cat([torch.tensor(keys, dtype=torch.long, device=DEV), torch.arange(since, pos + 1, device=DEV)])
        page = s["table"][row, j // case["page"]].long()
        k = s["k_cache"][page, j % case["page"]].double()
        v = s["v_cache"][page, j % case["page"]].double()
        for g in range(case["kv_heads"]):
            heads = slice(g * group, (g + 1) * group)
            score = s["q"][n, heads].double() @ k[:, g].T * s["scale"]
            lse[n, heads] = torch.logsumexp(score, -1)
            out[n, heads] = torch.softmax(score, -1) @ v[:, g]
    return {"out": out, "lse": lse}
