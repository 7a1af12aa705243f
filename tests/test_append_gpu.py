"""The cache appends on the GPU against the float64 oracle.

Bound of a written value: half a step of its type for the one rounding
(finfo.eps / 2 of the value, 2^-25 where fp16 is subnormal), and for the 32-bit
work 64 * 2^-24 of the pair's length after the norm: the mean square's sum has
at most 21 steps (16 in a lane, 5 between lanes), rsqrtf and sincospif are good
to a few units, the angle's conversion to 32 bits to 2^-24 half turns (pi 2^-24
radians), and three products follow.  At position p both sides' angles carry
the 64-bit rounding of the frequency, p * 2^-52 radians each.
"""
import pytest
import torch

from oracle import append_oracle as A
from speculative_decode_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _bound(ref, lengths, positions, dtype, mscale):
    half = torch.finfo(dtype).eps / 2
    work = 64 * 2.0 ** -24 + positions.to(torch.float64).clamp_min(0) * 2.0 ** -51
    return ref.abs() * half + lengths * max(mscale, 1.0) * work[:, None, None] + (2.0 ** -25 if dtype == torch.float16 else 0)


def _close(got, ref, bound, what):
    got = got.detach().cpu().to(torch.float64)
    assert torch.isfinite(got).all(), what
    over = ((got - ref).abs() - bound).max()
    assert float(over) <= 0, f"{what}: {float(over):.3e} over the bound"


def _bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


ROPES = {"plain": dict(theta=10000.0), "linear": dict(theta=500000.0, scaling=A.LINEAR, factor=8.0),
         "yarn": dict(theta=10000.0, scaling=A.YARN, factor=40.0, original=4096)}


def _rope(rot, interleaved, kind):
    r = ROPES[kind]
    own = dict(theta=r["theta"], interleaved=interleaved, scaling=r.get("scaling", 0), factor=r.get("factor", 1.0),
               original_positions=r.get("original", 1))
    rope = B.ddtree_rope_init(rot, **own)
    return rope, A.frequencies(rot, r["theta"], r.get("scaling", 0), r.get("factor", 1.0), r.get("original", 1)), float(rope.mscale)


# ------------------------------------------------------------------ latent rows
def _mla(n, heads, interleaved, kind, *, seed=0, far=70000, wide=64, kv_wide=576, weight=True, heads_first=False,
         in_place=False, eps=1e-6, scale=1.0, slots=None, positions=None, spare=5):
    g = torch.Generator().manual_seed(seed)
    rope, freqs, mscale = _rope(64, interleaved, kind)
    kv = (torch.randn(n, kv_wide, generator=g) * scale).to(torch.bfloat16)
    shape = (heads, n, wide) if heads_first else (n, heads, wide)
    q = torch.randn(shape, generator=g).to(torch.bfloat16)
    w = (1 + 0.2 * torch.randn(512, generator=g)).to(torch.bfloat16) if weight else None
    pool = torch.randn(n + spare, 576, generator=g).to(torch.bfloat16)
    if positions is None:
        positions = torch.randint(0, far, (n,), generator=g).to(I32)
    if slots is None:
        slots = torch.randperm(n + spare, generator=g)[:n].to(I32)
    kv_d, q_d, pool_d = kv.cuda(), q.cuda(), pool.cuda()

    def view(t):
        t = t[..., wide - 64:]
        return t.transpose(0, 1) if heads_first else t
    out_d = q_d if in_place else torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    B.ddtree_mla_append(rope, kv_d[:, kv_wide - 576:], positions.cuda(), slots.cuda(), pool_d,
                        latent_weight=None if w is None else w.cuda(), eps=eps, q_rope=view(q_d) if heads else None,
                        q_out=view(out_d) if heads else None, status=status)
    torch.cuda.synchronize()
    kv_in = kv[:, kv_wide - 576:]
    ref_pool, ref_q = A.mla_append(kv_in, w, eps, view(q) if heads else None, positions, slots, pool, freqs, interleaved, mscale)
    written = [(i, int(s)) for i, s in enumerate(slots.tolist()) if 0 <= s < n + spare and int(positions[i]) >= 0]
    keep = torch.ones(n + spare, dtype=torch.bool)
    if written:
        tok, row = (torch.tensor(x) for x in zip(*written))
        keep[row] = False
        ref = ref_pool[row][:, None, :]
        length = torch.cat([ref[..., :512].abs(), A.pair_lengths(kv_in[tok][:, None, 512:], 32, interleaved)], -1)
        _close(pool_d.cpu()[row][:, None, :], ref, _bound(ref, length, positions[tok], torch.bfloat16, mscale), "pool rows")
    assert torch.equal(_bits(pool_d.cpu()[keep]), _bits(pool[keep])), "untouched rows"
    if heads:
        live = positions >= 0
        got = view(out_d).cpu()
        length = A.pair_lengths(view(q), 32, interleaved)
        _close(got[live], ref_q[live], _bound(ref_q, length, positions, torch.bfloat16, mscale)[live], "queries")
        before = view(q) if in_place else torch.full_like(view(q), 7.0)
        assert torch.equal(_bits(got[~live]), _bits(before[~live])), "padding queries"
        if wide > 64:
            rest = out_d.cpu()[..., :wide - 64]
            assert torch.equal(_bits(rest), _bits(q[..., :wide - 64] if in_place else torch.full_like(rest, 7.0)))
    return int(status)


@pytest.mark.parametrize("kind", ["plain", "linear", "yarn"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads", [(1, 8), (1, 0), (3, 1), (32, 7), (33, 9), (257, 16), (5, 128)])
def test_mla_rows_and_queries(n, heads, interleaved, kind):
    assert _mla(n, heads, interleaved, kind, seed=n + heads) == 0


@pytest.mark.parametrize("kw", [dict(wide=192), dict(wide=192, in_place=True), dict(in_place=True), dict(heads_first=True),
                                dict(heads_first=True, wide=128), dict(kv_wide=584), dict(weight=False), dict(eps=0.0),
                                dict(eps=1.0, scale=1e-3), dict(scale=300.0), dict(far=2 ** 31 - 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_mla_layouts_and_values(kw, interleaved):
    assert _mla(19, 10, interleaved, "yarn", **kw) == 0


def test_mla_zero_latents():
    g = torch.zeros(2, 576, dtype=torch.bfloat16, device="cuda")
    pool = torch.ones(2, 576, dtype=torch.bfloat16, device="cuda")
    B.ddtree_mla_append(_rope(64, True, "plain")[0], g, torch.tensor([3, 4], dtype=I32, device="cuda"),
                        torch.tensor([1, 0], dtype=I32, device="cuda"), pool,
                        latent_weight=torch.ones(512, dtype=torch.bfloat16, device="cuda"))
    assert bool((pool == 0).all())


def test_mla_padding_and_bad_slots():
    pos = torch.tensor([5, -1, 9, -1, 2 ** 31 - 1, 0], dtype=I32)
    assert _mla(6, 9, True, "plain", positions=pos, slots=torch.tensor([0, 1, -1, -1, 3, 2], dtype=I32)) == 0
    assert _mla(6, 9, False, "plain", positions=pos, slots=torch.tensor([0, 1, 11, 4, 3, 2], dtype=I32)) == B.DDTREE_ST_BAD_INDEX
    assert _mla(6, 9, False, "plain", positions=pos, slots=torch.tensor([0, 1, -2, 4, 3, 2], dtype=I32)) == B.DDTREE_ST_BAD_INDEX
    pos[1] = -2
    assert _mla(6, 9, False, "plain", positions=pos, slots=torch.tensor([0, 1, 5, 4, 3, 2], dtype=I32)) == B.DDTREE_ST_BAD_LENGTH


def test_mla_no_tokens_and_a_row_far_into_the_pool():
    rope = _rope(64, True, "plain")[0]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    ints = torch.empty(0, dtype=I32, device="cuda")
    pool = torch.ones(4, 576, **bf)
    B.ddtree_mla_append(rope, torch.empty(0, 576, **bf), ints, ints, pool)
    B.ddtree_mla_append(rope, torch.empty(0, 576, **bf), ints, ints, pool, q_rope=torch.empty(0, 8, 64, **bf),
                        q_out=torch.empty(0, 8, 64, **bf), latent_weight=torch.ones(512, **bf))
    cache = B.DraftCache(torch.ones(2, 4, 2, 64, **bf), torch.ones(2, 4, 2, 64, **bf))
    empty = [torch.empty(0, h, 64, **bf) for h in (4, 2, 2, 4)]
    B.ddtree_draft_append(cache, rope, *empty[:3], ints, ints, empty[3])
    torch.cuda.synchronize()
    assert bool((pool == 1).all()) and bool((cache.k == 1).all()) and bool((cache.v == 1).all())
    rows = 4_000_000  # byte offsets past 2^32
    pool = torch.zeros(rows, 576, dtype=torch.bfloat16, device="cuda")
    kv = torch.randn(2, 576, device="cuda").to(torch.bfloat16)
    pos = torch.zeros(2, dtype=I32, device="cuda")
    B.ddtree_mla_append(rope, kv, pos, torch.tensor([rows - 1, 1], dtype=I32, device="cuda"), pool)
    assert torch.equal(pool[rows - 1], kv[0]) and torch.equal(pool[1], kv[1]) and int((pool != 0).any(1).sum()) == 2


def test_mla_python_refusals():
    rope = _rope(64, True, "plain")[0]
    kv = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(4, dtype=I32, device="cuda")
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    for a, kw in (((rope, kv.cpu(), i, i, kv), {}), ((rope, kv.float(), i, i, kv), {}), ((rope, kv[:, :512], i, i, kv), {}),
                  ((rope, kv, i[:3], i, kv), {}), ((rope, kv, i, i.long(), kv), {}), ((rope, kv, i, i, kv[:, :575]), {}),
                  ((rope, kv, i, i, kv), dict(q_rope=q)), ((rope, kv, i, i, kv), dict(q_rope=q, q_out=q[:3])),
                  ((rope, kv, i, i, kv), dict(q_rope=q.transpose(1, 2), q_out=q)),
                  ((rope, kv, i, i, kv), dict(latent_weight=kv[0, :511]))):
        with pytest.raises((TypeError, ValueError)):
            B.ddtree_mla_append(*a, **kw)


# ---------------------------------------------------------------- drafter rows
def _draft(n, heads, kvh, dim, rot, interleaved, kind, dtype, *, seed=0, page=16, heads_first=False, norm=True, fused=True,
           in_place=False, slots=None, positions=None, far=70000, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    rope, freqs, mscale = _rope(rot, interleaved, kind)
    width = (heads + 2 * kvh) * dim
    qkv = (torch.randn(n, width, generator=g) * scale).to(dtype)

    def parts(t):
        q, k, v = t.split([heads * dim, kvh * dim, kvh * dim], 1)
        if not fused:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        return q.view(n, heads, dim), k.view(n, kvh, dim), v.view(n, kvh, dim)
    q, k, v = parts(qkv)
    qd, kd, vd = parts(qkv.cuda())
    wq, wk = ((1 + 0.2 * torch.randn(dim, generator=g)).to(dtype) if norm else None for _ in range(2))
    pages = -(-n // page) + 2
    shape = (pages, kvh, page, dim) if heads_first else (pages, page, kvh, dim)
    order = (lambda t: t.transpose(1, 2)) if heads_first else (lambda t: t)
    kc, vc = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
    kcd, vcd = kc.cuda(), vc.cuda()
    if positions is None:
        positions = torch.randint(0, far, (n,), generator=g).to(I32)
    if slots is None:
        slots = torch.randperm(pages * page, generator=g)[:n].to(I32)
    out = qd if in_place else torch.full((n, heads, dim), 7.0, dtype=dtype, device="cuda")
    before = out.detach().cpu().clone()
    status = torch.zeros(1, dtype=I32, device="cuda")
    cache = B.DraftCache(order(kcd), order(vcd))
    B.ddtree_draft_append(cache, rope, qd if heads else None, kd, vd, positions.cuda(), slots.cuda(), out if heads else None,
                          q_weight=None if wq is None else wq.cuda(), k_weight=None if wk is None else wk.cuda(),
                          status=status)
    torch.cuda.synchronize()
    total = pages * page
    good = torch.where((slots >= 0) & (slots < total), slots, torch.full_like(slots, -1))
    rq, rk, rv = A.draft_append(q, k, v, wq, wk, 1e-6, positions, good, order(kc), order(vc), freqs, interleaved, mscale)
    live = positions >= 0
    if heads:
        length = A.pair_lengths(A.norm(q, wq, 1e-6), rot // 2, interleaved)
        _close(out[live.cuda()], rq[live], _bound(rq, length, positions, dtype, mscale)[live], "queries")
        assert torch.equal(_bits(out.cpu()[~live]), _bits(before[~live])), "padding queries"
    # Keys: the rows that were written against the bound, all others and the values bit for bit.
    flat = lambda t: order(t).reshape(total, kvh, dim)  # noqa: E731
    got_k, got_v = flat(kcd.cpu()), flat(vcd.cpu())
    tok = torch.tensor([i for i in range(n) if good[i] >= 0 and live[i]], dtype=torch.long)
    row = good[tok].long()
    rk, rv = rk.reshape(total, kvh, dim), rv.reshape(total, kvh, dim)
    length = A.pair_lengths(A.norm(k[tok], wk, 1e-6), rot // 2, interleaved)
    if len(tok):
        _close(got_k[row], rk[row], _bound(rk[row], length, positions[tok], dtype, mscale), "keys")
    keep = torch.ones(total, dtype=torch.bool)
    keep[row] = False
    assert torch.equal(_bits(got_k[keep]), _bits(flat(kc)[keep])) and torch.equal(got_v.double(), rv)
    return int(status)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,kvh,dim,rot", [(1, 8, 2, 128, 128), (8, 32, 8, 128, 64), (3, 1, 1, 64, 16), (37, 7, 7, 64, 64),
                                                 (5, 0, 4, 256, 256), (2, 16, 1, 256, 48), (700, 5, 1, 64, 32)])
def test_draft_rows_and_queries(n, heads, kvh, dim, rot, interleaved, dtype):
    assert _draft(n, heads, kvh, dim, rot, interleaved, "yarn", dtype, seed=n + dim) == 0


@pytest.mark.parametrize("kw", [dict(heads_first=True), dict(page=1), dict(page=7, heads_first=True), dict(norm=False),
                                dict(fused=False), dict(in_place=True), dict(in_place=True, fused=False),
                                dict(far=2 ** 31 - 1), dict(scale=1e-4), dict(scale=50.0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_draft_layouts_and_values(kw, dtype):
    assert _draft(21, 12, 3, 128, 96, False, "linear", dtype, **kw) == 0


def test_draft_padding_and_bad_slots():
    pos = torch.tensor([5, -1, 9, -1, 2 ** 31 - 1, 0], dtype=I32)
    bf = torch.bfloat16
    assert _draft(6, 4, 2, 64, 64, True, "plain", bf, positions=pos, slots=torch.tensor([0, 1, -1, -1, 3, 2], dtype=I32)) == 0
    bad = torch.tensor([0, 1, 16 * 3, 4, 3, 2], dtype=I32)
    assert _draft(6, 4, 2, 64, 64, False, "plain", bf, positions=pos, slots=bad) == B.DDTREE_ST_BAD_INDEX
    pos[3] = -9
    assert _draft(6, 4, 2, 64, 64, False, "plain", bf, positions=pos) == B.DDTREE_ST_BAD_LENGTH


def test_draft_cache_refusals():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    for a, b in ((k.float(), k.float()), (k[0], k[0]), (k, k[:3]), (k, k.half()), (k.cpu(), k.cpu()),
                 (k, torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            B.DraftCache(a, b)


def test_appends_captured_and_replayed():
    rope, freqs, mscale = _rope(64, True, "yarn")
    n, h = 9, 3
    kv, q = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, h, 64, dtype=torch.bfloat16, device="cuda")
    pos, slots = (torch.zeros(n, dtype=I32, device="cuda") for _ in range(2))
    pool, out = torch.zeros(40, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(q)
    call = B.BoundMlaAppend(rope, kv, pos, slots, pool, q_rope=q, q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        kv.copy_(torch.randn(n, 576, generator=g)), q.copy_(torch.randn(n, h, 64, generator=g))
        pos.copy_(torch.randint(0, 5000, (n,), generator=g)), slots.copy_(torch.randperm(40, generator=g)[:n])
        graph.replay()
        got, gp = out.clone(), pool.clone()
        eager = torch.zeros_like(pool), torch.zeros_like(out)
        eager[0].copy_(pool)
        B.ddtree_mla_append(rope, kv, pos, slots, eager[0], q_rope=q, q_out=eager[1])
        assert torch.equal(got, eager[1]) and torch.equal(gp, eager[0])
