"""The 8-bit cache's writes and reads on the GPU against the float64 oracle.

Values are written as they came, so their codes and scales are the oracle's bit
for bit.  Keys pass 32-bit work first (64 * 2^-24 of a pair's length, as in the
16-bit append's tests) and then one rounding to e4m3: half a step of it, 2^-4 of
the number or 2^-10 scales where it is subnormal.  A key block's scale goes by
its largest element, known to 1e-5 of itself (64 * 2^-24 of a pair's length,
which is at most sqrt(2) times its larger element): it must be the scale of one
of the two ends of that range.
"""
import random

import pytest
import torch

from oracle import append_oracle as A
from oracle import draft8_oracle as O
from speculative_decode_tree_gb300 import binding as B
from test_append_gpu import _bound, _close, _rope

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _same(a, b):
    """Equal numbers, NaN where NaN is (scales that nobody wrote)."""
    return torch.equal(torch.nan_to_num(a, nan=-7.0), torch.nan_to_num(b, nan=-7.0))


class Case:
    def __init__(self, slots, heads, kvh, dim, *, block, page, pages, dtype=torch.bfloat16, interleaved=False, kind="plain", rot=None,
                 norm=True, heads_first=False, positions=None, seed=0, far=70000, in_place=False, wide=False, loud=(), scales=None):
        g = torch.Generator().manual_seed(seed)
        n = len(slots)
        self.slots, self.block, self.page, self.dim, self.dtype, self.interleaved = list(slots), block, page, dim, dtype, interleaved
        self.positions = torch.randint(0, far, (n,), generator=g).tolist() if positions is None else list(positions)
        shape = (pages, page, kvh, dim)
        raw = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
        self.codes = [torch.where(raw & 0x7F == 0x7F, raw - 1, raw), torch.where(raw.flip(0) & 0x7F == 0x7F, 0, raw.flip(0))]
        blocks = -(-page // block)
        self.scales = [torch.exp2(torch.randint(-9, -4, (pages, blocks, kvh), generator=g).float()) if scales is None else
                       torch.full((pages, blocks, kvh), scales) for _ in range(2)]
        self.q, self.k, self.v = (torch.randn(n, h, dim, generator=g).to(dtype) for h in (heads, kvh, kvh))
        for i in loud:
            self.k[i] *= 30
            self.v[i] *= 30
        self.wq, self.wk = ((1 + 0.2 * torch.randn(dim, generator=g)).to(dtype) if norm else None for _ in range(2))
        self.rope, self.freqs, self.mscale = _rope(rot or dim, interleaved, kind)
        self.heads, self.heads_first, self.in_place, self.wide = heads, heads_first, in_place, wide

    def device(self):
        def cache(c):
            return c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.heads_first else c.cuda()
        self.dev_codes = [cache(c) for c in self.codes]
        self.dev_scales = [s.cuda() for s in self.scales]
        self.cache = B.Draft8Cache(*self.dev_codes, *self.dev_scales, self.block)
        all_ = torch.cat([self.q, self.k, self.v], 1).cuda()
        h, kvh = self.heads, self.k.shape[1]
        parts = (all_[:, :h], all_[:, h:h + kvh], all_[:, h + kvh:])
        self.in_q, self.in_k, self.in_v = parts if self.wide else [p.contiguous() for p in parts]
        self.out = self.in_q if self.in_place else torch.full(self.q.shape, 7.0, dtype=self.dtype, device="cuda")
        self.status = torch.zeros(1, dtype=I32, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
        self.args = (self.cache, self.rope, self.in_q if h else None, self.in_k, self.in_v, i32(self.positions), i32(self.slots),
                     self.out if h else None)
        self.kw = dict(q_weight=None if self.wq is None else self.wq.cuda(), k_weight=None if self.wk is None else self.wk.cuda(),
                       status=self.status)

    def run(self):
        self.device()
        B.ddtree_draft8_append(*self.args, **self.kw)
        torch.cuda.synchronize()
        return int(self.status)

    def compare(self):
        pos = torch.tensor(self.positions)
        live = pos >= 0
        if self.heads:
            ref = A.rotate(A.norm(self.q, self.wq, 1e-6), pos, self.freqs, self.interleaved, self.mscale)
            length = A.pair_lengths(A.norm(self.q, self.wq, 1e-6), len(self.freqs), self.interleaved)
            got = self.out.cpu()
            if bool(live.any()):
                _close(got[live], ref[live], _bound(ref, length, pos, self.dtype, self.mscale)[live], "queries")
            before = self.q if self.in_place else torch.full_like(self.q, 7.0)
            assert torch.equal(got[~live].view(torch.int16), before[~live].view(torch.int16))
        # Values: bit for bit.
        codes, scales = self.codes[1].clone(), self.scales[1].double()
        O.write_rows(self.v.double(), codes, scales, self.block, self.positions, self.slots)
        assert _same(self.dev_scales[1].cpu().double(), scales), "value scales"
        assert torch.equal(self.dev_codes[1].cpu(), codes), "value codes"
        # Keys.
        x = A.rotate(A.norm(self.k, self.wk, 1e-6), pos, self.freqs, self.interleaved, self.mscale)
        length = A.pair_lengths(A.norm(self.k, self.wk, 1e-6), len(self.freqs), self.interleaved)
        ends = []
        for f in (1 - 1e-5, 1 + 1e-5):
            codes, scales = self.codes[0].clone(), self.scales[0].double()
            O.write_rows(x * f, codes, scales, self.block, self.positions, self.slots)
            ends.append((codes, scales))
        got_s, got_c = self.dev_scales[0].cpu().double(), self.dev_codes[0].cpu()
        which = got_s != ends[0][1]
        assert _same(torch.where(which, ends[1][1], ends[0][1]), got_s), "key scales"
        at = torch.arange(self.page) // self.block
        want = torch.where(which[:, at][..., None], ends[1][0], ends[0][0])
        mine = torch.zeros(self.codes[0].shape[:2], dtype=torch.bool)
        for n, s in enumerate(self.slots):
            if self.positions[n] >= 0 and 0 <= s < mine.numel():
                p, t = s // self.page, s % self.page
                mine[p, t] = True
                scale = got_s[p, t // self.block][:, None]
                work = length[n] * max(self.mscale, 1.0) * (64 * 2.0 ** -24 + max(self.positions[n], 0) * 2.0 ** -51)
                far = (O.values(got_c[p, t]) * scale - x[n]).abs() - (x[n].abs() * 2.0 ** -4).clamp_min(2.0 ** -10 * scale) - work
                assert float(far.max()) <= 0, f"key row {n}: {float(far.max()):.3e} over its bound"
        assert torch.equal(got_c[~mine], want[~mine]), "other rows"


def _check(*a, status=0, **kw):
    c = Case(*a, **kw)
    assert c.run() == status
    c.compare()
    return c


def _laid(n, page, pages, off, seed=0):
    """Slots of a run of tokens from place `off` on, over permuted pages."""
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    return [order[i // page] * page + i % page for i in range(off, off + n)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,block", [(64, 1), (64, 8), (64, 64), (64, 33), (128, 1), (128, 16), (128, 32), (128, 5), (256, 1), (256, 2), (256, 16), (256, 11)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_prompts(dim, block, dtype, interleaved):
    page = max(block, 48)
    n, pages = 211, 8
    _check(_laid(n, page, pages, block // 2), 6, 2, dim, block=block, page=page, pages=pages, dtype=dtype, interleaved=interleaved,
           seed=dim + block, rot=dim // 2)


@pytest.mark.parametrize("dim,block,page", [(64, 16, 16), (64, 64, 64), (128, 16, 64), (128, 16, 17), (128, 32, 48), (256, 8, 8), (256, 16, 1000), (64, 1, 1)])
@pytest.mark.parametrize("n", [1, 2, 9, 70])
def test_single_tokens_within_blocks(n, dim, block, page):
    blocks = -(-page // block)
    pages = -(-n // blocks) + 1
    r = random.Random(n)
    slots = []
    for of in r.sample(range(pages * blocks), n):
        size = min(block, page - of % blocks * block)
        slots.append(of // blocks * page + of % blocks * block + r.randrange(size))
    _check(slots, 4, 1, dim, block=block, page=page, pages=pages, seed=n, loud=range(0, n, 2))


@pytest.mark.parametrize("kw", [dict(heads_first=True), dict(wide=True), dict(in_place=True), dict(wide=True, in_place=True), dict(norm=False),
                                dict(kind="linear"), dict(kind="yarn", interleaved=True), dict(rot=16), dict(rot=16, interleaved=True),
                                dict(scales=0.0), dict(scales=float("nan")), dict(scales=-1.0), dict(scales=0.0173), dict(scales=2.0 ** -60),
                                dict(far=2 ** 31 - 1)])
@pytest.mark.parametrize("block", [1, 16])
def test_layouts_and_scales(kw, block):
    _check(_laid(37, 16, 5, 5) + [4 * 16 + 13], 5, 3, 128, block=block, page=16, pages=6, seed=3, loud=[37], **kw)


@pytest.mark.parametrize("heads,kvh", [(0, 1), (0, 5), (1, 1), (16, 16), (40, 8), (7, 7), (128, 2)])
def test_heads(heads, kvh):
    for block in (1, 8):
        _check(_laid(19, 24, 2, 3), heads, kvh, 64, block=block, page=24, pages=2, seed=heads)


def test_padding_and_bad_slots():
    slots = _laid(12, 16, 3, 3)
    slots[4] = -1
    pos = list(range(50, 62))
    pos[5] = -1  # between blocks: within one, its tokens would not follow one another
    for block in (1, 8):
        kw = dict(block=block, page=16, pages=3)
        _check(slots, 4, 2, 64, positions=pos, **kw)
        _check([48] + slots[1:], 4, 2, 64, positions=pos, status=B.DDTREE_ST_BAD_INDEX, **kw)
        _check([-2] + slots[1:], 4, 2, 64, positions=pos, status=B.DDTREE_ST_BAD_INDEX, **kw)
        _check([48] + slots[1:], 4, 2, 64, positions=[-1] + pos[1:], **kw)
        _check(slots, 4, 2, 64, positions=[-7] + pos[1:], status=B.DDTREE_ST_BAD_LENGTH, **kw)
        _check([-1] * 12, 4, 2, 64, positions=[-1] * 12, **kw)


@pytest.mark.parametrize("heads,kvh", [(0, 1), (0, 5), (0, 8), (32, 8)])
@pytest.mark.parametrize("n", [1, 12, 300, 2500])
@pytest.mark.parametrize("block", [1, 8, 16])
def test_bad_tokens_are_reported_with_and_without_queries(block, n, heads, kvh):
    # Few tokens are spread over CTAs by their heads, and without queries every CTA looks for runs alone.
    pages = -(-n // 16) + 1
    good = _laid(n, 16, pages, 0)
    last = n - 1
    for slots, pos, status in ((dict([(last, pages * 16)]), {}, B.DDTREE_ST_BAD_INDEX), (dict([(0, -2)]), {}, B.DDTREE_ST_BAD_INDEX),
                               ({}, dict([(last, -2)]), B.DDTREE_ST_BAD_LENGTH), ({}, dict([(0, -2 ** 31)]), B.DDTREE_ST_BAD_LENGTH),
                               (dict([(0, 2 ** 31 - 1)]), dict([(last, -9)]) if n > 1 else {},
                                B.DDTREE_ST_BAD_INDEX | (B.DDTREE_ST_BAD_LENGTH if n > 1 else 0)),
                               ({i: -5 for i in range(n)}, {}, B.DDTREE_ST_BAD_INDEX), ({i: -5 for i in range(n)}, {i: -1 for i in range(n)}, 0)):
        c = Case([slots.get(i, s) for i, s in enumerate(good)], heads, kvh, 128, block=block, page=16, pages=pages, seed=n,
                 positions=[pos.get(i, 40 + i) for i in range(n)])
        assert c.run() == status
        if n <= 12:
            c.compare()


def test_values_that_are_no_numbers():
    for block in (1, 16):
        c = Case(_laid(20, 16, 2, 0), 2, 2, 64, block=block, page=16, pages=2, norm=False, positions=[0] * 20, seed=5)
        c.v[3, 0, 5], c.v[3, 1, 6], c.v[4, 0, 7], c.v[5] = float("inf"), -float("inf"), float("nan"), float("nan")
        c.v[6], c.v[7, 0] = 0.0, 3e38
        c.v[8] *= 1e-25
        assert c.run() == 0
        codes, scales = c.codes[1].clone(), c.scales[1].double()
        O.write_rows(c.v.double(), codes, scales, block, c.positions, c.slots)
        assert torch.equal(c.dev_scales[1].cpu().double(), scales)
        got = c.dev_codes[1].cpu()
        nan = codes & 127 == 127
        assert torch.equal(got & 127 == 127, nan) and torch.equal(got[~nan], codes[~nan])


def test_blocks_over_several_calls_a_replay_and_another_stream():
    # A request's tokens one call at a time give what the oracle gives, in order.
    r = random.Random(3)
    slots = _laid(40, 16, 4, 0)
    c = Case(slots, 2, 2, 64, block=8, page=16, pages=4, norm=False, positions=[0] * 40, seed=6, loud=[r.randrange(40) for _ in range(9)])
    c.device()
    codes, scales = c.codes[1].clone(), c.scales[1].double()
    i, parts = 0, []
    while i < 40:
        parts.append((i, min(40, i + r.choice([1, 1, 2, 5, 9]))))
        i = parts[-1][1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a, b in parts:
        O.write_rows(c.v[a:b].double(), codes, scales, 8, [0] * (b - a), slots[a:b])
        B.ddtree_draft8_append(c.cache, c.rope, None, c.in_k[a:b], c.in_v[a:b], c.args[5][a:b], c.args[6][a:b], None, stream=side)
    side.synchronize()
    assert torch.equal(c.dev_codes[1].cpu(), codes) and torch.equal(c.dev_scales[1].cpu().double(), scales)
    # Captured, and replayed on a fresh cache: the same bits.
    calls = [B.BoundDraft8Append(c.cache, c.rope, None, c.in_k[a:b], c.in_v[a:b], c.args[5][a:b], c.args[6][a:b], None) for a, b in parts]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            call()
    for t, s in zip(c.dev_codes + c.dev_scales, c.codes + c.scales):
        t.copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.dev_codes[1].cpu(), codes) and torch.equal(c.dev_scales[1].cpu().double(), scales)


def test_no_tokens():
    c = Case(_laid(3, 16, 2, 0), 2, 2, 64, block=8, page=16, pages=2)
    c.device()
    e = lambda t: t[:0]  # noqa: E731
    B.ddtree_draft8_append(c.cache, c.rope, e(c.in_q), e(c.in_k), e(c.in_v), e(c.args[5]), e(c.args[6]), e(c.out))
    B.ddtree_draft8_read(c.cache, e(c.args[6]), e(c.in_k), e(c.in_v))
    torch.cuda.synchronize()
    assert torch.equal(c.dev_codes[0].cpu(), c.codes[0])


# ------------------------------------------------------------------ reads
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,block,page,kvh", [(64, 1, 1, 1), (64, 8, 48, 3), (128, 16, 16, 2), (128, 7, 17, 1), (256, 16, 64, 5), (256, 1, 3, 2)])
@pytest.mark.parametrize("heads_first", [False, True])
def test_reads(dim, block, page, kvh, dtype, heads_first):
    c = Case([0], 1, kvh, dim, block=block, page=page, pages=5, heads_first=heads_first, seed=dim)
    c.scales[1] = torch.rand_like(c.scales[1]) * 0.01 + 1e-3     # any number is a scale
    c.device()
    r = random.Random(1)
    slots = [r.randrange(5 * page) for _ in range(77)] + [0, 0, 5 * page - 1, -1]
    outs = [torch.full((81, kvh + 2, dim), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    st = torch.zeros(1, dtype=I32, device="cuda")
    B.ddtree_draft8_read(c.cache, torch.tensor(slots, dtype=I32, device="cuda"), outs[0][:, :kvh], outs[1][:, 1:kvh + 1], status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    keep = torch.full((81, kvh, dim), 7.0)
    for i in range(2):
        ref = O.read_rows(c.codes[i], c.scales[i], block, slots, keep)
        got = outs[i].cpu().double()
        mine = got[:, i:kvh + i]
        half = torch.finfo(dtype).eps / 2
        # The product in 32 bits and its rounding to 16.
        bound = ref.abs() * (half + 2.0 ** -24) + (2.0 ** -25 if dtype == torch.float16 else 0)
        assert bool(((mine - ref).abs() <= bound).all())
        if dtype == torch.bfloat16 and i == 0:
            assert torch.equal(mine, ref)
        rest = torch.cat([got[:, :i], got[:, kvh + i:]], 1)
        assert bool((rest == 7.0).all())


def test_reads_of_bad_slots_and_scales():
    c = Case([0], 1, 2, 64, block=8, page=16, pages=3, seed=1)
    c.scales[0][0, 0, 1], c.scales[1][2, 1, 0], c.scales[1][1, 0, 0], c.scales[0][1, 1, 1] = 0.0, float("nan"), -1.0, float("inf")
    c.device()

    def read(slots, k=True, v=True):
        outs = [torch.full((len(slots), 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        st = torch.zeros(1, dtype=I32, device="cuda")
        B.ddtree_draft8_read(c.cache, torch.tensor(slots, dtype=I32, device="cuda"), outs[0] if k else None, outs[1] if v else None, status=st)
        torch.cuda.synchronize()
        for i, on in enumerate((k, v)):
            ref = O.read_rows(c.codes[i], c.scales[i], 8, slots if on else [], torch.full((len(slots), 2, 64), 7.0))
            assert torch.equal(outs[i].cpu().double(), ref)
        return int(st)
    assert read([8, 9, 15]) == 0
    assert read([8, 48, -5, -1]) == B.DDTREE_ST_BAD_INDEX
    assert read(list(range(48))) == B.DDTREE_ST_BAD_SCALE
    assert read([40, 41], v=False) == 0 and read([40, 41], k=False) == B.DDTREE_ST_BAD_SCALE
    assert read([-1, 99, 0], v=False) == B.DDTREE_ST_BAD_INDEX | B.DDTREE_ST_BAD_SCALE


def test_rows_far_into_a_large_cache():
    # 2 x 4.3 GB: offsets pass 32 bits.
    pages, page, kvh, dim = 16900, 1000, 1, 256
    codes = [torch.zeros(pages, page, kvh, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages, 63, kvh, device="cuda") for _ in range(2)]
    cache = B.Draft8Cache(*codes, *scales, 16)
    rope = B.ddtree_rope_init(64, theta=1e4)
    k, v = (torch.randn(3, kvh, dim, device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = torch.tensor([pages * page - 8, pages * page - 7, 5], dtype=I32, device="cuda")
    zero = torch.zeros(3, dtype=I32, device="cuda")
    B.ddtree_draft8_append(cache, rope, None, k, v, zero, slots, None)
    out = torch.empty(3, kvh, dim, dtype=torch.bfloat16, device="cuda")
    B.ddtree_draft8_read(cache, slots, None, out)
    torch.cuda.synchronize()
    want = [torch.zeros(1, 16, kvh, dim, dtype=torch.uint8), torch.zeros(1, 16, kvh, dim, dtype=torch.uint8)]
    for rows, w, at in ((slice(0, 2), want[0], [0, 1]), (slice(2, 3), want[1], [5])):
        s = torch.zeros(1, 1, kvh, dtype=torch.float64)
        O.write_rows(v[rows].cpu().double(), w, s, 16, [0] * len(at), at)
        assert torch.equal(out[rows].cpu().double(), O.dequantised(w, s, 16)[0, at])
    assert int((codes[1] != 0).any(-1).sum()) == 3
