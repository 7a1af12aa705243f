"""The drafter's attention over its 8-bit cache on the GPU against the float64
oracle on the dequantised cache.

Bound of an output: half a step of its type for the final rounding; half a step
of fp16 (2^-11) of every weight p_j vscale_j: 2^-11 of sum |p v|; where a weight
is subnormal in fp16 2^-25, with 2^10 at least for the largest weight, so 2^-35 of
the largest scale times the number of keys times 448; and for the 32-bit work, as
in the 16-bit tests, two sums of D terms (codes times a query in fp16 are exact
products) and 64 units for the sums over keys, besides 8 units of the largest
|log2 vscale|, which the exponents carry.  lse has the same score error once.
"""
import math
import random

import pytest
import torch

from oracle import draft8_oracle as O
from speculative_decode_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
I32 = torch.int32
U = 2.0 ** -24


class Case:
    def __init__(self, positions, heads, kvh, dim, *, page=16, block=8, window=0, sinks=0, dtype=torch.bfloat16, heads_first=False,
                 seed=0, rows=None, scale=None, q_scale=1.0, freed=True, wide=False, any_scale=False, spread=5):
        g = torch.Generator().manual_seed(seed)
        r = random.Random(seed)
        n = len(positions)
        block = min(block, page)
        self.positions, self.window, self.sinks, self.page, self.block = list(positions), window, sinks, page, block
        self.dtype, self.dim, self.heads_first, self.wide = dtype, dim, heads_first, wide
        self.scale = dim ** -0.5 if scale is None else scale
        n_rows = n + 2 if rows is None else max(rows) + 1
        self.token_rows = r.sample(range(n_rows), n) if rows is None else list(rows)
        need = {}
        for p, row in zip(positions, self.token_rows):
            lo = max(0, p - window + 1) if window else 0
            used = {k for k in range(max(p, 0) // page + 1) if not freed or k >= lo // page or k * page < sinks}
            need[row] = need.get(row, set()) | (used if p >= 0 else set())
        pages = sum(len(x) for x in need.values()) + 3
        perm = list(range(pages))
        r.shuffle(perm)
        table = [[-1] * (max(max(positions), 0) // page + 2) for _ in range(n_rows)]
        for row, ks in need.items():
            for k in ks:
                table[row][k] = perm.pop()
        self.table = torch.tensor(table, dtype=I32)
        shape, blocks = (pages, page, kvh, dim), -(-page // block)
        self.codes = [O.codes_of((torch.randn(shape, generator=g) * 112).clamp(-448, 448)) for _ in range(2)]
        self.scales = [torch.exp2(torch.randint(-6 - spread, -6 + spread, (pages, blocks, kvh), generator=g).float()) if not any_scale else
                       torch.rand(pages, blocks, kvh, generator=g) * 0.02 + 1e-4 for _ in range(2)]
        q = (torch.randn(n, heads * (2 if wide else 1), dim, generator=g) * q_scale).to(dtype)
        self.q, self.q_dev = q[:, :heads], q.cuda()[:, :heads]
        self.out0, self.lse0 = torch.randn(n, heads, dim, generator=g).to(dtype), torch.randn(n, heads, generator=g)

    def device(self):
        def cache(c):
            return c.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.heads_first else c.cuda()
        self.cache = B.Draft8Cache(*[cache(c) for c in self.codes], *[s.cuda() for s in self.scales], self.block)
        n, h, d = self.q.shape
        self.plan = B.ddtree_draft8_attention_plan(n, h, self.cache, self.dtype, self.window, self.sinks)
        if self.wide:
            self.plan.q_stride = 2 * h * d
        self.ws = torch.full((B.ddtree_draft8_attention_workspace_size(self.plan),), 0xA5, dtype=torch.uint8, device="cuda")
        self.out, self.lse = self.out0.cuda(), self.lse0.cuda()
        self.args = (self.plan, self.q_dev, self.cache, self.table.cuda(), torch.tensor(self.positions, dtype=I32, device="cuda"),
                     self.scale, self.out, self.ws)
        self.kw = dict(token_rows=torch.tensor(self.token_rows, dtype=I32, device="cuda"), lse=self.lse)

    def run(self):
        self.device()
        B.ddtree_draft8_attention(*self.args, **self.kw)
        torch.cuda.synchronize()
        return B.ddtree_verify_mla_check(self.ws)

    def compare(self):
        ref, lse, mass, terms = O.attention(self.q, *self.codes, *self.scales, self.block, self.table, self.token_rows, self.positions,
                                            self.window, self.sinks, self.scale, self.out0, self.lse0)
        half = torch.finfo(self.dtype).eps / 2
        vs = self.scales[1].double()
        vs = vs[(vs >= 2.0 ** -64) & (vs <= 2.0 ** 96)]
        exponent = 8 * U * float(vs.log2().abs().max())
        score = self.dim * U * terms + exponent
        keys = max(max(self.positions), 0) + 1
        ob = ref.abs() * half + mass * (2.0 ** -11 + 2 * (2 * score + 64 * U)[..., None]) + keys * 448 * 2.0 ** -35 * float(vs.max()) + \
            (2.0 ** -25 if self.dtype == torch.float16 else 0)
        lb = score + 8 * U * lse.abs() + 64 * U
        out, got = self.out.cpu().double(), self.lse.cpu().double()
        assert torch.isfinite(out).all()
        over = ((out - ref).abs() - ob).max()
        assert float(over) <= 0, f"out {float(over):.3e} over its bound"
        none = torch.isinf(lse)
        assert torch.equal(torch.isinf(got), none)
        assert float(((got - lse).abs() - lb)[~none].max() if (~none).any() else 0) <= 0, "lse over its bound"
        for i, p in enumerate(self.positions):
            if p == -1:
                assert torch.equal(self.out[i].cpu(), self.out0[i]) and torch.equal(self.lse[i].cpu(), self.lse0[i])


def _check(*a, status=0, **kw):
    c = Case(*a, **kw)
    assert c.run() == status
    c.compare()
    return c


@pytest.mark.parametrize("pos", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 1023, 4096])
@pytest.mark.parametrize("dim,kvh", [(64, 3), (128, 1), (256, 2)])
def test_single_tokens_of_every_length(pos, dim, kvh):
    _check([pos], 4 * kvh, kvh, dim, page=1, seed=pos)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kvh", [(1, 1), (8, 2), (5, 1), (16, 16), (24, 1), (64, 1), (66, 2), (40, 1), (51, 3)])
def test_heads_and_types(heads, kvh, dim, dtype):
    _check([0, 1, 63, 64, 130, 777], heads, kvh, dim, dtype=dtype, seed=heads + dim)


@pytest.mark.parametrize("page,block", [(1, 1), (3, 2), (16, 16), (48, 32), (64, 1), (256, 64), (17, 5)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (64, 4), (100, 0), (100, 70), (1000, 33), (5000, 4), (7, 2 ** 31 - 1),
                                          (2 ** 31 - 1, 5)])
@pytest.mark.parametrize("heads_first", [False, True])
def test_windows_pages_and_orders(page, block, window, sinks, heads_first):
    _check([0, 3, 99, 640, 2049], 8, 2, 64, page=page, block=block, window=window, sinks=sinks, heads_first=heads_first,
           seed=page + window % 97)


@pytest.mark.parametrize("dim,block", [(128, 32), (256, 16), (128, 7)])
def test_pages_of_wider_heads(dim, block):
    _check([0, 3, 99, 640, 2049], 8, 2, dim, page=48, block=block, window=500, sinks=9, heads_first=True, seed=dim)
    _check([0, 3, 99, 640, 2049], 8, 2, dim, page=48, block=block, any_scale=True, seed=dim + 1)


def test_long_and_ragged():
    _check([30000, 5, 12345, 0, 777], 8, 2, 128, page=16, seed=1)
    _check([70001], 4, 1, 256, page=1, block=1, seed=2)
    _check([50000, 9], 12, 1, 64, page=64, block=64, seed=3)


def test_many_tokens():
    r = random.Random(4)
    _check([r.choice([0, 1, 40, r.randint(0, 300)]) for _ in range(301)], 4, 2, 64, page=16, seed=3)
    _check([r.randint(0, 20) for _ in range(4096)], 2, 1, 64, page=4, seed=4)


@pytest.mark.parametrize("kvh,dim", [(3, 64), (5, 128), (6, 64), (12, 128), (16, 64), (24, 64), (10, 256), (128, 64)])
def test_key_heads_that_shares_take_side_by_side(kvh, dim):
    _check([700, 3, -1, 129, 2500], 2 * kvh, kvh, dim, seed=kvh)
    _check([40] * 33, kvh, kvh, dim, page=8, seed=kvh + 1)


def test_one_long_request_among_many_short_ones():
    _check([9000] + [10, 60, 200, 127, 128] * 20, 8, 4, 64, seed=41)
    _check([30] * 70 + [6000, 100], 48, 8, 128, seed=42)
    _check([30] * 40 + [6000, 100], 40, 2, 256, seed=43)


def test_strided_outputs():
    c = Case([300, 5, 77], 8, 2, 64, seed=43)
    c.device()
    wide = torch.full((3, 11, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.plan.out_stride = 11 * 64
    B.ddtree_draft8_attention(*c.args[:6], wide[:, 2:10], c.ws, **c.kw)
    torch.cuda.synchronize()
    c.out = wide[:, 2:10].contiguous()
    c.compare()
    assert bool((wide[:, :2] == 7.0).all()) and bool((wide[:, 10:] == 7.0).all())


def test_padding_tokens_and_shared_requests():
    _check([-1, 100, -1, -1, 7, -1], 8, 2, 128, seed=5)
    _check([-1, -1], 8, 2, 128, seed=6)
    _check([100, 101, 102, 103, 40], 8, 2, 64, rows=[1, 1, 1, 1, 0], window=50, sinks=2, freed=False, seed=7)


@pytest.mark.parametrize("kw", [dict(wide=True), dict(q_scale=30.0), dict(q_scale=30.0, dtype=torch.float16), dict(scale=-0.2), dict(scale=0.0),
                                dict(q_scale=1e-4, dtype=torch.float16), dict(q_scale=1e30, scale=1e-31), dict(q_scale=1e-30, scale=1e29),
                                dict(spread=20, q_scale=1e-4), dict(any_scale=True), dict(q_scale=0.0)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_and_scales(kw, dim):
    _check([300, 500], 8, 2, dim, seed=8, **kw)


def test_value_blocks_of_very_different_scales():
    # One block's values are 2^40 times the others': its share of every output is what counts there; the sums see all keys.
    for dim in (64, 128, 256):
        c = Case([900], 8, 2, dim, seed=9)
        c.scales[1].fill_(2.0 ** -20)
        c.scales[1][int(c.table[c.token_rows[0], 20])] = 2.0 ** 20
        assert c.run() == 0
        c.compare()


def test_sums_see_value_blocks_2_to_the_100_apart():
    for dim in (64, 128, 256):
        c = Case([900, 20000], 8, 2, dim, seed=10)
        c.scales[1].fill_(2.0 ** -50)
        for n in range(2):
            c.scales[1][int(c.table[c.token_rows[n], 20])] = 2.0 ** 50
        assert c.run() == 0
        c.compare()


def test_one_large_score_among_many_keys_keeps_the_small_ones():
    c = Case([60000], 4, 1, 64, page=16, seed=13, scale=1.0)
    for codes, number in ((c.codes[0], 0.0), (c.codes[1], 1.0)):
        codes.copy_(O.codes_of(torch.full_like(codes, number, dtype=torch.float64)))
    for s in c.scales:
        s.fill_(1.0)
    c.q.zero_()
    c.q[:, :, 0] = 4.0
    c.q_dev.copy_(c.q)
    at = int(c.table[c.token_rows[0], 100 // 16])
    c.codes[0][at, 100 % 16, 0, 0] = int(O.codes_of(torch.tensor(4.0)))
    c.codes[1][at, 100 % 16, 0] = 0
    assert c.run() == 0
    c.compare()
    assert float(c.out.float().mean()) > 6e-3


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_largest_and_smallest_queries(dim):
    # Rows are moved into fp16's range by a power of two, from either end of bf16's.
    for q_scale, scale in ((4e37, 4e-40), (8e37, -2e-40), (1e-36, 1e35)):
        c = Case([700, 3, 64, 1], 12, 3, dim, seed=dim, q_scale=q_scale, scale=scale)
        c.q[0, 0, 5] = 3.3e38 if q_scale > 1 else 2.0 ** -126
        c.q_dev.copy_(c.q)
        assert c.run() == 0
        # 256 columns of 8e37 hold one number beyond bf16's range, an infinity: that row is none, and is compared as zero.
        odd = torch.isinf(c.q).any(-1)
        assert int(odd.sum()) == (dim == 256 and q_scale == 8e37) and bool(torch.isnan(c.out.cpu()[odd]).all())
        c.q[odd] = 0
        c.q_dev.copy_(c.q)
        assert c.run() == 0
        c.compare()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,heads", [(64, 8), (128, 8), (256, 8), (64, 24)])
@pytest.mark.parametrize("rising", [False, True])
def test_sums_over_very_many_keys(rising, dim, heads, dtype):
    # A plan of one SM, so that a share has a million keys.  Values of one sign, so that whatever a long sum loses adds
    # up.  Bound: half a step of the output; half a step of fp16 of every weight; the products, which cut sums off where
    # they do not fit into 32 bits, 2^-23 of the sum for every four of the 8,192 keys that a warp sums before they start
    # anew; 32-bit work as above.
    g = torch.Generator(device="cuda").manual_seed(dim)
    n, page, block = 1 << 22, 64, 16
    pages = n // page
    k = (torch.randn(pages, page, 1, dim, generator=g, device="cuda", dtype=torch.float16)).to(torch.float8_e4m3fn)
    v = (torch.rand(pages, page, 1, dim, generator=g, device="cuda", dtype=torch.float16) + 1).to(torch.float8_e4m3fn)
    scales = [torch.exp2(torch.randint(-1, 2, (pages, page // block, 1), generator=g, device="cuda").float()) for _ in range(2)]
    q = torch.randn(1, heads, dim, generator=g, device="cuda").to(dtype)
    order = torch.randperm(pages, generator=g, device="cuda")
    if rising:
        q[:, :, 0] = 1.0
        k.view(torch.uint8)[order, :, 0, 0] = torch.linspace(-400, 400, pages, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)[:, None]
    cache = B.Draft8Cache(k, v, *scales, block)
    plan = B.ddtree_draft8_attention_plan(1, heads, cache, dtype, num_sms=1)
    ws = torch.full((B.ddtree_draft8_attention_workspace_size(plan),), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse, outs = torch.empty_like(q), torch.empty(1, heads, device="cuda"), []
    for _ in range(2):
        B.ddtree_draft8_attention(plan, q, cache, order.to(I32)[None].contiguous(), torch.tensor([n - 1], dtype=I32, device="cuda"),
                                  dim ** -0.5, out, ws, lse=lse)
        assert B.ddtree_verify_mla_check(ws) == 0
        outs.append(out.clone())
    assert torch.equal(*outs)
    kf, vf = ((c[order, :, 0].float() * s[order].repeat_interleave(block, 1)).view(n, dim) for c, s in ((k, scales[0]), (v, scales[1])))
    half = torch.finfo(dtype).eps / 2
    for h in range(heads):
        s, terms, ref = [], 0.0, 0.0
        for part in kf.split(1 << 19):
            s.append((part.double() @ q[0, h].double()) * dim ** -0.5)
            terms = max(terms, float((part.double().abs() @ q[0, h].double().abs()).max()) * dim ** -0.5)
        s = torch.cat(s)
        ref_lse = torch.logsumexp(s, 0)
        for part, x in zip(vf.split(1 << 19), s.split(1 << 19)):
            ref = ref + torch.exp(x - ref_lse) @ part.double()
        score = dim * U * terms + 8 * U
        over = ((out[0, h].double() - ref).abs() - ref * (half + 2.0 ** -11 + 2048 * 2.0 ** -23 + 2 * (2 * score + 64 * U))).max()
        assert float(over) <= 0, f"out {float(over):.3e} over its bound"
        assert abs(float(lse[0, h]) - float(ref_lse)) <= score + 8 * U * abs(float(ref_lse)) + 64 * U


def test_bad_positions_rows_pages_and_scales():
    c = Case([100, 50, 20, 77], 8, 2, 64, seed=14)
    c.positions[0] = -5
    assert c.run() == B.DDTREE_ST_BAD_LENGTH
    c.compare()
    c = Case([100, 50, 20, 77], 8, 2, 64, seed=15)
    c.token_rows[1], c.token_rows[2] = -1, 99
    assert c.run() == B.DDTREE_ST_BAD_LENGTH
    c.compare()
    c = Case([100, 50, 20, 77], 8, 2, 64, seed=16)
    c.positions[3] = 16 * c.table.shape[1]
    assert c.run() == B.DDTREE_ST_BAD_LENGTH
    c.compare()
    c = Case([100, 50, 20, 77], 8, 2, 64, seed=17)
    c.table[c.token_rows[0], 2] = -1
    c.table[c.token_rows[1], 0] = c.codes[0].shape[0]
    c.table[c.token_rows[2], :] = -7      # nothing left to see
    assert c.run() == B.DDTREE_ST_BAD_INDEX
    c.compare()
    assert bool(torch.isinf(c.lse[2]).all()) and bool((c.out[2] == 0).all())
    for dim in (64, 128, 256):
        c = Case([100, 50, 20, 77], 8, 2, dim, seed=18)
        at = [int(c.table[c.token_rows[i], k]) for i, k in ((0, 3), (1, 0), (3, 1), (2, 0), (2, 1))]
        for page, which, b, h, value in ((at[0], 0, 1, 0, 0.0), (at[1], 1, 0, 1, math.nan), (at[2], 0, 0, 0, math.inf), (at[2], 1, 0, 1, -1.0)):
            c.scales[which][page, b, h] = value
        for page in at[3:]:
            c.scales[0][page] = 0.0
        for codes in c.codes:  # whatever lies in blocks without a scale
            codes[at[0], 8:, 0], codes[at[1], :8, 1] = 0x7F, 0xFF
            codes[at[3]], codes[at[4]] = 0x7F, 0x7F
        assert c.run() == B.DDTREE_ST_BAD_SCALE
        c.compare()
        assert bool(torch.isinf(c.lse[2]).all()) and bool((c.out[2] == 0).all())


def test_nothing_beyond_the_visible_keys_counts():
    # NaN codes and scales behind the token, before the window and in released pages change no bit.
    for dim in (64, 128, 256):
        base = Case([100, 37, 400], 8, 2, dim, window=64, sinks=3, freed=False, seed=18, block=1)
        assert base.run() == 0
        base.compare()
        c = Case([100, 37, 400], 8, 2, dim, window=64, sinks=3, freed=False, seed=18, block=1)
        keep = torch.zeros(c.codes[0].shape[:2], dtype=torch.bool)
        for p, row in zip(c.positions, c.token_rows):
            for j in range(p + 1):
                if j > p - 64 or j < 3:
                    keep[c.table[row, j // 16], j % 16] = True
        for codes, scales in zip(c.codes, c.scales):
            codes[~keep], scales[~keep] = 0x7F, float("nan")
        assert c.run() == 0
        assert torch.equal(c.out, base.out) and torch.equal(c.lse, base.lse)


def test_visible_nan_reaches_its_request_alone():
    c = Case([100, 37, 400], 8, 2, 128, seed=20)
    base = Case([100, 37, 400], 8, 2, 128, seed=20)
    assert base.run() == 0
    c.codes[1][int(c.table[c.token_rows[1], 1]), 3, 0, 7] = 0x7F
    c.codes[0][int(c.table[c.token_rows[0], 1]), 3, 1, 7] = 0x7F
    assert c.run() == 0
    nan = torch.isnan(c.out)
    assert bool(nan[1, :4, 7].all()) and int(nan[1].sum()) == 4 and bool(nan[0, 4:].all()) and not bool(nan[0, :4].any())
    assert torch.equal(c.out[2], base.out[2]) and torch.equal(c.lse[2], base.lse[2])


def test_equal_bits_on_other_streams_without_lse_and_in_a_replay():
    c = Case([5000, 12, 900], 16, 2, 128, page=16, seed=19)
    assert c.run() == 0
    c.compare()
    out, lse = c.out.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    c.out.zero_(), c.ws.fill_(0x3C)
    side.wait_stream(torch.cuda.current_stream())
    B.ddtree_draft8_attention(*c.args, **dict(c.kw, lse=None), stream=side)
    side.synchronize()
    assert torch.equal(c.out, out)
    bound = B.BoundDraft8Attention(*c.args, **c.kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bound()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    # Other lengths through the same graph: the table's rows hold what these need.
    c.positions = [17, 5, 700]
    c.args[4].copy_(torch.tensor(c.positions))
    g.replay()
    torch.cuda.synchronize()
    assert B.ddtree_verify_mla_check(c.ws) == 0
    c.compare()


def test_pages_far_into_a_large_cache():
    # 2 x 4.6 GB: offsets pass 32 bits.
    c = Case([300, 90], 8, 1, 256, page=16, block=16, seed=22)
    n, far = c.codes[0].shape[0], 1130000 - c.codes[0].shape[0]
    big = [torch.empty(1130000, 16, 1, 256, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(1130000, 1, 1, device="cuda") for _ in range(2)]
    for b, codes, s, own in zip(big, c.codes, scales, c.scales):
        b[far:].copy_(codes)
        s[far:].copy_(own)
    c.device()
    cache = B.Draft8Cache(*big, *scales, 16)
    assert big[0].numel() > 2 ** 32
    table = torch.where(c.table >= 0, c.table + far, c.table).cuda()
    B.ddtree_draft8_attention(c.plan, c.q_dev, cache, table, *c.args[4:], **c.kw)
    torch.cuda.synchronize()
    assert B.ddtree_verify_mla_check(c.ws) == 0
    c.compare()


def test_refusals():
    c = Case([5, 6], 8, 2, 64, seed=21)
    c.device()
    with pytest.raises(TypeError):
        B.ddtree_draft8_attention(c.plan, c.q_dev.half(), *c.args[2:], **c.kw)
    with pytest.raises(ValueError):
        B.ddtree_draft8_attention(*c.args[:7], c.ws[:-1], **c.kw)
    with pytest.raises(ValueError):
        B.ddtree_draft8_attention(c.plan, c.q_dev[:, :4], *c.args[2:], **c.kw)
    with pytest.raises(TypeError):
        B.ddtree_draft8_attention(c.plan, c.q_dev.cpu(), *c.args[2:], **c.kw)
    with pytest.raises(ValueError):
        B.Draft8Cache(c.cache.k, c.cache.v, c.cache.k_scale[:, :1], c.cache.v_scale, 8)
    with pytest.raises(ValueError):
        B.Draft8Cache(c.cache.k, c.cache.v.transpose(1, 2).contiguous().transpose(1, 2), c.cache.k_scale, c.cache.v_scale, 8)
