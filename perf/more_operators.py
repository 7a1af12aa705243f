"""The drafter's prompt and its cache in 8 bits, as measured calls.

Four operators beside the drafter's append and attention, in their plain form
(elementary torch operations in 32 bits or more, rounded once) and as the
library's calls:

  append8   head norms and rotation of queries and keys; keys and values
            quantised as they are written, e4m3 with a scale for each block of
            tokens and key head, and the touched blocks read back
  read8     rows of that cache read back into 16 bits
  attn8     the drafter's attention of one new token per request over that
            cache, with an optional sliding window and sink tokens
  prompt    causal attention over whole prompts, packed one behind the other,
            each with an optional earlier context
"""
import math

import torch

own = False

DEV = "cuda"
INT32 = torch.int32
FP8 = torch.float8_e4m3fn
TOP = 448.0                    # the largest e4m3 number
LOW, HIGH = -64, 96            # exponents of a scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # The drafter's step for eight requests: one token each, in the middle of a block.
        dict(name="append8_step", op="append8", tokens=8, prompt=False, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, factor=1.0, far=65536, dtype="bf16", norm=True, page=16, block=16, heads_first=False),
        # The accepted tokens of a full batch, token-granular, a scale for each token and head.
        dict(name="append8_tokens", op="append8", tokens=1021, prompt=False, heads=16, kv_heads=4, dim=64, rot=16,
             interleaved=True, factor=8.0, far=131072, dtype="fp16", norm=False, page=1, block=1, heads_first=False),
        # The drafter taking in a long prompt that goes on in a block begun before.
        dict(name="append8_prompt", op="append8", tokens=32749, prompt=True, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, factor=1.0, far=65536, dtype="bf16", norm=True, page=64, block=16, heads_first=False),
        # A short context read back before the next chunk of its prompt.
        dict(name="read8_chunk", op="read8", rows=509, kv_heads=8, dim=128, page=16, block=16, heads_first=False, dtype="bf16"),
        # A 64k context read back, pages with the heads outside.
        dict(name="read8_context", op="read8", rows=65521, kv_heads=4, dim=256, page=64, block=8, heads_first=True, dtype="fp16"),
        # One request far into its context, a 2,048-token window and four sink tokens, token-granular.
        dict(name="attn8_window", op="attn8", batch=1, lo=65536, hi=65536, heads=32, kv_heads=8, dim=128, window=2048,
             sinks=4, page=1, block=1, heads_first=False, dtype="bf16"),
        # One request over its whole 185k context with few key heads: the split over the length is everything.
        dict(name="attn8_long", op="attn8", batch=1, lo=189440, hi=189440, heads=16, kv_heads=2, dim=256, window=0,
             sinks=0, page=16, block=16, heads_first=True, dtype="bf16"),
        # Eight requests of 1k to 185k tokens, no window: the most bytes.
        dict(name="attn8_mixed", op="attn8", batch=8, lo=1024, hi=189440, heads=32, kv_heads=8, dim=128, window=0,
             sinks=0, page=64, block=16, heads_first=False, dtype="bf16"),
        # A served batch of a few thousand tokens each; a page size that is no power of two and no multiple of the block.
        dict(name="attn8_batch", op="attn8", batch=61, lo=511, hi=16384, heads=64, kv_heads=8, dim=64, window=0, sinks=0,
             page=48, block=32, heads_first=False, dtype="fp16"),
        # Short prompts of a served batch, some of one token.
        dict(name="prompt_short", op="prompt", batch=64, lo=1, hi=251, context=0, heads=32, kv_heads=8, dim=128, window=0,
             sinks=0, packed=True, dtype="bf16"),
        # One long prompt: matrix products are everything.
        dict(name="prompt_long", op="prompt", batch=1, lo=16384, hi=16384, context=0, heads=16, kv_heads=2, dim=128,
             window=0, sinks=0, packed=False, dtype="bf16"),
        # Chunks of different lengths behind earlier contexts, a window and sink tokens.
        dict(name="prompt_chunks", op="prompt", batch=5, lo=1031, hi=4099, context=4096, heads=32, kv_heads=8, dim=64,
             window=2048, sinks=4, packed=True, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _block(rng, dim):
    return rng.choice([b for b in (1, 8, 16, 32, 64) if b * dim <= 4096])


def draw(rng):
    op = rng.choice(["append8", "read8", "attn8", "prompt"])
    dim = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([1, 16, 48, 64])
    block = min(page, _block(rng, dim))
    case = dict(op=op, kv_heads=kv, dim=dim, dtype=rng.choice(["bf16", "fp16"]))
    if op == "append8":
        heads = kv * rng.choice([1, 2, 3, 4, 7, 8, 16])
        prompt = rng.random() < 0.5
        most = max(1, min(32749, (1 << 27) // (dim * (heads + 2 * kv))))
        return dict(case, tokens=_log(rng, 1, most if prompt else min(most, 1024)), prompt=prompt, heads=heads,
                    rot=rng.choice([16, dim // 4, dim // 2, dim]), interleaved=rng.random() < 0.5,
                    factor=rng.choice([1.0, 8.0]), far=_log(rng, 1024, 1 << 20), norm=rng.random() < 0.7, page=page,
                    block=block, heads_first=rng.random() < 0.5)
    if op == "read8":
        return dict(case, rows=_log(rng, 1, min(65521, (1 << 26) // (kv * dim))), page=page, block=block,
                    heads_first=rng.random() < 0.5)
    if op == "attn8":
        batch, hi = _log(rng, 1, 256), _log(rng, 16, 189440)
        if batch * hi * kv * dim > 1 << 28:
            return draw(rng)
        return dict(case, batch=batch, lo=max(1, _log(rng, 1, hi)), hi=hi, heads=kv * rng.choice([1, 3, 4, 8, 16, 24]),
                    window=0 if rng.random() < 0.6 else _log(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 33]), page=page,
                    block=block, heads_first=rng.random() < 0.5)
    batch, hi = _log(rng, 1, 64), _log(rng, 1, 16384)
    lo = max(1, _log(rng, 1, hi))
    context = 0 if rng.random() < 0.5 else _log(rng, 1, 4 * lo)  # a chunk is no small part of its context
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    if batch * hi * (hi + context) * heads * dim > 1 << 38:
        return draw(rng)
    return dict(case, batch=batch, lo=lo, hi=hi, context=context, heads=heads,
                window=0 if rng.random() < 0.6 else _log(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 33]),
                packed=rng.random() < 0.5)


def _lens(case):
    """Lengths of a batch, spread evenly over their logarithm."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    return [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]


def _contexts(case):
    """Earlier contexts: none, up to the longest."""
    return [case["context"] * i // max(1, case["batch"] - 1) if case["batch"] > 1 else case["context"] for i in range(case["batch"])]


def _visible(case, pos):
    lo = max(0, pos - case["window"] + 1) if case["window"] else 0
    return min(case["sinks"], lo) + pos - lo + 1


def _touched(case):
    """Rows that an append case reads back, about: of each token's block those up to the token, or a prompt's rows."""
    return case["tokens"] if case["prompt"] else case["tokens"] * (min(case["block"], case["page"]) + 1) // 2


def work(case):
    op, d, kvh = case["op"], case["dim"], case["kv_heads"]
    if op == "append8":
        n, h = case["tokens"], case["heads"]
        return {"bytes": n * ((h + 2 * kvh) * d * 2 + h * d * 2 + 2 * kvh * d + 8) + _touched(case) * 2 * kvh * d * 3,
                "flops": n * (h + kvh) * (4 * d + 3 * case["rot"]) + n * 4 * kvh * d}
    if op == "read8":
        return {"bytes": case["rows"] * (2 * kvh * (3 * d + 4 / case["block"]) + 4), "flops": case["rows"] * 2 * kvh * d}
    if op == "attn8":
        seen = sum(_visible(case, p) for p in _lens(case))
        n = case["batch"]
        return {"bytes": seen * kvh * (2 * d + 8 / case["block"]) + 4 * -(-seen // case["page"]) + n * case["heads"] * (d * 4 + 4),
                "flops": 4 * seen * case["heads"] * d}
    pairs = sum(_visible(case, c + i) for n, c in zip(_lens(case), _contexts(case)) for i in range(n))
    nq, nk = sum(_lens(case)), sum(_lens(case)) + sum(_contexts(case))
    return {"bytes": nq * case["heads"] * (4 * d + 4) + nk * kvh * 4 * d, "flops": 4 * pairs * case["heads"] * d}


# ----------------------------------------------------------------- the inputs
def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _cache(gen, case, pages):
    """A cache that has been written to: codes as a quantiser leaves them, powers of two as scales."""
    kvh, page, d = case["kv_heads"], case["page"], case["dim"]
    blocks = -(-page // case["block"])

    def codes():
        shape = (pages, kvh, page, d) if case["heads_first"] else (pages, page, kvh, d)
        c = torch.empty(shape, dtype=FP8, device=DEV)
        c.copy_((torch.randn(shape, generator=gen, device=DEV, dtype=torch.float16) * 112).clamp(-TOP, TOP))
        return c.transpose(1, 2) if case["heads_first"] else c

    def scales():
        return _power(torch.randint(-9, -4, (pages, blocks, kvh), generator=gen, device=DEV))
    return dict(k_cache=codes(), v_cache=codes(), k_scale=scales(), v_scale=scales())


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1_000_003 * seed + 29)
    s = {"case": case, "kept": {}}  # "kept": calls whose buffers stay the same, marshalled once by the program
    op, d, kvh, dtype = case["op"], case["dim"], case["kv_heads"], DTYPES[case["dtype"]]
    if op == "append8":
        n, h, page, block = case["tokens"], case["heads"], case["page"], case["block"]
        blocks = -(-page // block)
        if case["prompt"]:
            # The prompt goes on where the last chunk ended, within a block; pages come from a free list.
            off = min(page, block) // 2
            pages = -(-(n + off) // page) + 3
            order = torch.randperm(pages, generator=gen, device=DEV)
            at = torch.arange(n + off, device=DEV)
            rows = order[at // page] * page + at % page
            slots, rows = rows[off:], rows
        else:
            # One token for each of n blocks, at places spread over a block (the shortest one's).
            pages = -(-n // blocks) + 3
            of = torch.randperm(pages * blocks, generator=gen, device=DEV)[:n]
            inside = (torch.arange(n, device=DEV) * 7 + 3) % (page - (blocks - 1) * block)
            first = of // blocks * page + of % blocks * block
            slots = first + inside
            all_rows = first[:, None] + torch.arange(block, device=DEV)[None, :]
            rows = all_rows[torch.arange(block, device=DEV)[None, :] <= inside[:, None]]
        qkv = _normal(gen, (n, (h + 2 * kvh) * d), dtype) * 2
        weight = lambda: (1 + 0.1 * _normal(gen, (d,), torch.float32)).to(dtype) if case["norm"] else None  # noqa: E731
        s.update(_cache(gen, case, pages), q=qkv[:, :h * d].view(n, h, d), k=qkv[:, h * d:(h + kvh) * d].view(n, kvh, d),
                 v=qkv[:, (h + kvh) * d:].view(n, kvh, d), wq=weight(), wk=weight(),
                 positions=torch.randint(0, case["far"], (n,), generator=gen, device=DEV).to(INT32),
                 slots=slots.to(INT32), rows=rows.to(INT32), q_out=torch.zeros(n, h, d, dtype=dtype, device=DEV),
                 k_out=torch.zeros(rows.numel(), kvh, d, dtype=torch.bfloat16, device=DEV),
                 v_out=torch.zeros(rows.numel(), kvh, d, dtype=torch.bfloat16, device=DEV),
                 rope=dict(rot=case["rot"], interleaved=case["interleaved"], theta=500000.0, factor=case["factor"]),
                 status=torch.zeros(1, dtype=INT32, device=DEV))
        return s
    if op == "read8":
        n, page = case["rows"], case["page"]
        pages = -(-n // page) + 3
        at = torch.arange(n, device=DEV)
        order = torch.randperm(pages, generator=gen, device=DEV)
        s.update(_cache(gen, case, pages), rows=(order[at // page] * page + at % page).to(INT32),
                 k_out=torch.zeros(n, kvh, d, dtype=dtype, device=DEV), v_out=torch.zeros(n, kvh, d, dtype=dtype, device=DEV),
                 status=torch.zeros(1, dtype=INT32, device=DEV))
        return s
    if op == "attn8":
        b, h, page = case["batch"], case["heads"], case["page"]
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
        s.update(_cache(gen, case, pages), q=_normal(gen, (b, h, d), dtype) * 2, table=table,
                 token_rows=token_rows.to(INT32), positions=pos.to(INT32), scale=d ** -0.5,
                 most=max(_visible(case, p) for p in _lens(case)),
                 out=torch.zeros(b, h, d, dtype=dtype, device=DEV), lse=torch.zeros(b, h, dtype=torch.float32, device=DEV))
        return s
    b, h = case["batch"], case["heads"]
    order = torch.randperm(b, generator=gen, device=DEV)
    new = torch.tensor(_lens(case), device=DEV)[order]
    keys = new + torch.tensor(_contexts(case), device=DEV)[order]
    indptr = lambda x: torch.cat([x.new_zeros(1), torch.cumsum(x, 0)]).to(INT32)  # noqa: E731
    nq, nk = int(new.sum()) + 3, int(keys.sum()) + 3  # three rows behind the last sequence
    if case["packed"] and case["context"] == 0:  # parts of one projection
        qkv = _normal(gen, (nq, h + 2 * kvh, d), dtype) * 1.5
        q, k, v = qkv[:, :h], qkv[:, h:h + kvh], qkv[:, h + kvh:]
    else:
        q = _normal(gen, (nq, h, d), dtype) * 1.5
        k, v = _normal(gen, (nk, kvh, d), dtype) * 1.5, _normal(gen, (nk, kvh, d), dtype) * 1.5
    s.update(q=q, k=k, v=v, q_indptr=indptr(new), k_indptr=indptr(keys), scale=d ** -0.5,
             most_q=max(_lens(case)), most_k=max(n + c for n, c in zip(_lens(case), _contexts(case))), rows=int(new.sum()),
             out=torch.zeros(nq, h, d, dtype=dtype, device=DEV), lse=torch.zeros(nq, h, dtype=torch.float32, device=DEV))
    return s


# ------------------------------------------------------------ the plain forms
def _plain_rotate(x, rope, positions):
    """x [tokens, heads, width] in 32 bits: its first rope["rot"] columns rotated; angles in 64 bits."""
    rot = rope["rot"]
    i = torch.arange(rot // 2, device=positions.device, dtype=torch.float64)
    angle = positions.double()[:, None] * (rope["theta"] ** (-2.0 * i / rot) / rope["factor"])
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
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


def _plain_norm(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _codes(x, scale):
    return (x / scale).clamp(-TOP, TOP).to(FP8)


def _power(e):
    """2^e in 32 bits, exactly."""
    return ((e.to(INT32) + 127) << 23).view(torch.float32)


def _scale_for(top):
    """The least power of two that takes `top` into e4m3's range; 1 for nothing but zeros."""
    _, e = torch.frexp(top / TOP)  # top / 448 = m 2^e, m in [1/2, 1)
    e = torch.where(_power(e.clamp(-125, 127) - 1) * TOP >= top, e - 1, e)
    return torch.where(top > 0, _power(e.clamp(LOW, HIGH)), torch.ones_like(top))


def _bytes(t):
    return t.view(torch.uint8)


def _plain_write(s, cache, scale, x):
    """Rows x [tokens, kv_heads, dim] in 32 bits into the slots; a block's scale grows where it has to."""
    case = s["case"]
    page, block = case["page"], case["block"]
    blocks = -(-page // block)
    slot = s["slots"].long()
    number, token = slot // page, slot % page
    of = number * blocks + token // block
    flat = scale.view(-1, case["kv_heads"])
    top = torch.zeros_like(flat).index_reduce_(0, of, x.abs().amax(-1), "amax")
    # A block that gets its first token starts afresh; others keep their scale or let it grow.
    fresh = torch.zeros(flat.shape[0], device=DEV).index_reduce_(0, of, (token % block == 0).float(), "amax") > 0
    written = torch.zeros(flat.shape[0], device=DEV).index_fill_(0, of, 1.0) > 0
    old, want = flat.clone(), _scale_for(top)
    kept = ~fresh[:, None] & (old * TOP >= top)
    now = torch.where(written[:, None] & ~kept, want, old)
    flat.copy_(now)
    # What a block held before is taken over into its new scale.
    if slot.numel() * block <= page * scale.shape[0]:
        near = (token // block * block)[:, None] + torch.arange(block, device=DEV)[None, :]
        where = number[:, None].expand(near.shape), near.clamp_max(page - 1)
        held = _bytes(cache)[where].view(FP8).float() * old[of][:, None, :, None]
        _bytes(cache)[where] = _bytes(_codes(held, now[of][:, None, :, None]))
    else:
        at = torch.arange(page, device=DEV) // block
        held = cache.float() * old.view(scale.shape)[:, at][..., None]
        cache.copy_(_codes(held, now.view(scale.shape)[:, at][..., None]))
    _bytes(cache)[number, token] = _bytes(_codes(x, now[of][..., None]))


def _plain_read(s, cache, scale, out):
    case = s["case"]
    slot = s["rows"].long()
    number, token = slot // case["page"], slot % case["page"]
    out.copy_(_bytes(cache)[number, token].view(FP8).float() * scale[number, token // case["block"]][..., None])


def _plain_append8(s):
    q = _plain_rotate(_plain_norm(s["q"].float(), s["wq"]), s["rope"], s["positions"])
    k = _plain_rotate(_plain_norm(s["k"].float(), s["wk"]), s["rope"], s["positions"])
    s["q_out"].copy_(q)
    _plain_write(s, s["k_cache"], s["k_scale"], k)
    _plain_write(s, s["v_cache"], s["v_scale"], s["v"].float())
    _plain_read8(s)


def _plain_read8(s):
    _plain_read(s, s["k_cache"], s["k_scale"], s["k_out"])
    _plain_read(s, s["v_cache"], s["v_scale"], s["v_out"])


def _plain_attn8(s):
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
    inside = key % page
    block = inside // case["block"]
    k = _bytes(s["k_cache"])[at, inside].view(FP8).float().mul_(s["k_scale"][at, block][..., None])
    q = s["q"].float().view(pos.numel(), kvh, -1, case["dim"])
    score = torch.einsum("nhgd,nvhd->nhgv", q, k) * s["scale"]
    del k
    score = score.masked_fill(~live[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    vals = _bytes(s["v_cache"])[at, inside].view(FP8).float().mul_(s["v_scale"][at, block][..., None])
    out = torch.einsum("nhgv,nvhd->nhgd", p, vals) / total
    s["out"].copy_(out.view(s["out"].shape))
    s["lse"].copy_((top + torch.log(total)).view(s["lse"].shape))


def _plain_prompt(s):
    case = s["case"]
    kvh, d = case["kv_heads"], case["dim"]
    qp, kp = s["q_indptr"].long(), s["k_indptr"].long()
    nq, nk = qp[1:] - qp[:-1], kp[1:] - kp[:-1]
    i = torch.arange(s["most_q"], device=DEV)[None, :]
    j = torch.arange(s["most_k"], device=DEV)[None, :]
    rows = (qp[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    cols = (kp[:-1, None] + j).clamp_max(s["k"].shape[0] - 1)
    q = s["q"][rows].float().view(nq.numel(), s["most_q"], kvh, -1, d)
    k = s["k"][cols].float()
    v = s["v"][cols].float()
    score = torch.einsum("bihgd,bjhd->bhgij", q, k)
    score *= s["scale"]
    pos = (nk - nq)[:, None] + i
    seen = (j[:, None, :] <= pos[..., None]) & (j < nk[:, None])[:, None, :]
    if case["window"]:
        seen &= (j[:, None, :] > pos[..., None] - case["window"]) | (j < case["sinks"])[:, None, :]
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp_min(-3e38)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.einsum("bhgij,bjhd->bhgid", score, v) / total.clamp_min(1e-38)
    lse = (top + torch.log(total)).squeeze(-1)
    at = torch.arange(s["rows"], device=DEV)
    of = torch.searchsorted(qp[1:], at, right=True)
    inside = at - qp[of]
    s["out"][:s["rows"]] = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[of, inside].to(s["out"].dtype)
    s["lse"][:s["rows"]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[of, inside]


# ---------------------------------------------------------- the library's calls
def _own_calls(s):
    """The step's calls with their buffers, checked and marshalled once, as a decode loop with static buffers keeps them."""
    from speculative_decode_tree_gb300 import binding as B
    case = s["case"]
    if case["op"] == "prompt":
        plan = B.ddtree_prompt_attention_plan(case["batch"], s["q"].shape[0], s["k"].shape[0], case["heads"], case["kv_heads"],
                                              case["dim"], s["q"].dtype, window=case["window"], n_sinks=case["sinks"])
        workspace = torch.empty(B.ddtree_prompt_attention_workspace_size(plan), dtype=torch.uint8, device=DEV)
        return (B.BoundPromptAttention(plan, s["q"], s["k"], s["v"], s["q_indptr"], s["k_indptr"], s["scale"], s["out"],
                                       workspace, lse=s["lse"]),)
    cache = B.Draft8Cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], case["block"])
    if case["op"] == "attn8":
        plan = B.ddtree_draft8_attention_plan(case["batch"], case["heads"], cache, s["q"].dtype, window=case["window"],
                                              n_sinks=case["sinks"])
        workspace = torch.empty(B.ddtree_draft8_attention_workspace_size(plan), dtype=torch.uint8, device=DEV)
        return (B.BoundDraft8Attention(plan, s["q"], cache, s["table"], s["positions"], s["scale"], s["out"], workspace,
                                       token_rows=s["token_rows"], lse=s["lse"]),)
    read = B.BoundDraft8Read(cache, s["rows"], s["k_out"], s["v_out"], status=s["status"])
    if case["op"] == "read8":
        return (read,)
    r = s["rope"]
    rope = B.ddtree_rope_init(r["rot"], theta=r["theta"], interleaved=r["interleaved"],
                              scaling=B.DDTREE_ROPE_LINEAR if r["factor"] != 1.0 else B.DDTREE_ROPE_PLAIN, factor=r["factor"])
    return (B.BoundDraft8Append(cache, rope, s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], q_weight=s["wq"],
                                k_weight=s["wk"], eps=EPS, status=s["status"]), read)


PLAIN = {"append8": _plain_append8, "read8": _plain_read8, "attn8": _plain_attn8, "prompt": _plain_prompt}
OUTPUTS = {"append8": ("q_out", "k_out", "v_out"), "read8": ("k_out", "v_out"), "attn8": ("out", "lse"), "prompt": ("out", "lse")}


def run(state):
    if own:
        if "calls" not in state["kept"]:
            state["kept"]["calls"] = _own_calls(state)
        for call in state["kept"]["calls"]:
            call()
    else:
        PLAIN[state["case"]["op"]](state)
    return {k: state[k] for k in OUTPUTS[state["case"]["op"]]}


# ------------------------------------------------------- the definitions, 64 bits
def _turned(vec, rope, positions):
    """The rotation as a product of complex numbers, in 64 bits."""
    rot, half = rope["rot"], rope["rot"] // 2
    freq = torch.tensor([rope["theta"] ** (-2.0 * i / rot) / rope["factor"] for i in range(half)], dtype=torch.float64, device=DEV)
    angle = positions.double().unsqueeze(-1) * freq
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
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


def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _on_grid(x, scale):
    """The e4m3 number nearest to x / scale, ties to the even one, times the scale."""
    y = x / scale
    step = _two_to(torch.frexp(y)[1].clamp(-5, 9) - 4)  # y = m 2^e, m in [1/2, 1): four bits of it
    return torch.clamp(torch.round(y / step) * step, -TOP, TOP) * scale


def _values(cache, page, tok):
    """Codes of some rows in 64 bits."""
    return cache.view(torch.uint8)[page, tok].view(FP8).double()


def _exact_append8(s):
    case = s["case"]
    page, block = case["page"], case["block"]
    slots, rows = s["slots"].long(), s["rows"].long()
    key = lambda r: torch.div(r, page, rounding_mode="floor") * page + (r % page) - (r % page) % block  # noqa: E731
    # Blocks by the slot of their first token.
    ids, which = torch.unique(key(slots), return_inverse=True)
    found = torch.searchsorted(ids, key(rows)).clamp_max(ids.numel() - 1)
    inside = ids % page
    outs = []
    for cache, scale, x in ((s["k_cache"], s["k_scale"], _turned(_scaled(s["k"].double(), s["wk"]), s["rope"], s["positions"])),
                            (s["v_cache"], s["v_scale"], s["v"].double())):
        peak = torch.zeros(ids.numel(), case["kv_heads"], dtype=torch.float64, device=DEV)
        peak.scatter_reduce_(0, which[:, None].expand(-1, case["kv_heads"]), x.abs().amax(-1), "amax")
        old = scale[ids // page, inside // block].double()
        part, e = torch.frexp(peak / TOP)
        least = torch.where(peak > 0, _two_to((e - (part == 0.5).int()).clamp(LOW, HIGH)), torch.ones_like(peak))
        starts = torch.zeros(ids.numel(), dtype=torch.bool, device=DEV)
        starts[which[slots % page % block == 0]] = True
        new = torch.where(~starts[:, None] & (peak <= old * TOP), old, least)
        held = _values(cache, rows // page, rows % page) * scale[rows // page, rows % page // block].double()[..., None]
        full = torch.full((cache.shape[0] * page,), -1, dtype=torch.long, device=DEV)
        full[slots] = torch.arange(slots.numel(), device=DEV)
        mine = full[rows]
        value = torch.where((mine >= 0)[:, None, None], x[mine.clamp_min(0)], held)
        outs.append(_on_grid(value, new[found][..., None]))
    return {"q_out": _turned(_scaled(s["q"].double(), s["wq"]), s["rope"], s["positions"]), "k_out": outs[0], "v_out": outs[1]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append8":
        return _exact_append8(s)
    if case["op"] == "read8":
        where = s["rows"].long()
        page, tok = torch.div(where, case["page"], rounding_mode="floor"), where.remainder(case["page"])
        part = torch.div(tok, case["block"], rounding_mode="floor")
        return {o: _values(s[c], page, tok) * s[f][page, part].double().unsqueeze(-1)
                for o, c, f in (("k_out", "k_cache", "k_scale"), ("v_out", "v_cache", "v_scale"))}
    out, lse = s["out"].double(), s["lse"].double()
    group = case["heads"] // case["kv_heads"]
    if case["op"] == "attn8":
        for n, (pos, row) in enumerate(zip(s["positions"].tolist(), s["token_rows"].tolist())):
            since = max(0, pos - case["window"] + 1) if case["window"] else 0
            j = torch.cat([torch.arange(min(case["sinks"], since), device=DEV), torch.arange(since, pos + 1, device=DEV)])
            page, tok = s["table"][row, j // case["page"]].long(), j % case["page"]
            k = _values(s["k_cache"], page, tok) * s["k_scale"][page, tok // case["block"]].double().unsqueeze(-1)
            v = _values(s["v_cache"], page, tok) * s["v_scale"][page, tok // case["block"]].double().unsqueeze(-1)
            for g in range(case["kv_heads"]):
                heads = slice(g * group, (g + 1) * group)
                score = s["q"][n, heads].double() @ k[:, g].T * s["scale"]
                lse[n, heads] = torch.logsumexp(score, -1)
                out[n, heads] = torch.softmax(score, -1) @ v[:, g]
        return {"out": out, "lse": lse}
    qp, kp = s["q_indptr"].tolist(), s["k_indptr"].tolist()
    for b in range(case["batch"]):
        q, k, v = s["q"][qp[b]:qp[b + 1]], s["k"][kp[b]:kp[b + 1]], s["v"][kp[b]:kp[b + 1]]
        j = torch.arange(k.shape[0], device=DEV)
        for begin in range(0, q.shape[0], 4096):  # rows, a few at a time
            end = min(begin + 4096, q.shape[0])
            pos = torch.arange(begin, end, device=DEV).unsqueeze(1) + (k.shape[0] - q.shape[0])
            hidden = j > pos
            if case["window"]:
                hidden |= (j <= pos - case["window"]) & (j >= case["sinks"])
            for h in range(case["heads"]):
                score = (q[begin:end, h].double() @ k[:, h // group].double().T * s["scale"]).masked_fill(hidden, -math.inf)
                lse[qp[b] + begin:qp[b] + end, h] = torch.logsumexp(score, -1)
                out[qp[b] + begin:qp[b] + end, h] = torch.softmax(score, -1) @ v[:, h // group].double()
    return {"out": out, "lse": lse}
