"""The drafter's attention on the GPU against the float64 oracle.

Bound of an output: half a step of its type (finfo.eps / 2 of the value, 2^-25
where fp16 is subnormal) for the final rounding; half a step of every
probability, which meets V in the cache's type: finfo.eps / 2 of sum |p v|; and
for the 32-bit work, relative to sum |p v| too, the errors of the scores, which
enter as exp: a product sum of D terms in at most D steps of 2^-24 of
sum |q k| scale each side of a difference, times two for numerator and
denominator, and some steps for the sums over keys (their rounding errors are
random, 64 units cover any tree of them met here).  lse has the same score error
once, the logarithm's and its own rounding.
"""
import random

import pytest
import torch

from oracle import draft_attention
from speculative_decode_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
I32 = torch.int32
U = 2.0 ** -24


def _bounds(ref, lse, mass, terms, dim, dtype):
    half = torch.finfo(dtype).eps / 2
    work = (2 * dim * U * terms + 64 * U)[..., None]
    out = ref.abs() * half + mass * (half + 2 * work) + (2.0 ** -25 if dtype == torch.float16 else 0)
    return out, dim * U * terms + 8 * U * lse.abs() + 64 * U


class Case:
    """Inputs of one call, on the CPU and on the device."""

    def __init__(self, positions, heads, kvh, dim, *, page=16, window=0, sinks=0, dtype=torch.bfloat16, heads_first=False,
                 seed=0, rows=None, scale=None, q_scale=1.0, freed=True, wide=False):
        g = torch.Generator().manual_seed(seed)
        r = random.Random(seed)
        n = len(positions)
        self.positions, self.window, self.sinks, self.page, self.dtype, self.dim = list(positions), window, sinks, page, dtype, dim
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
        stride = max(max(positions), 0) // page + 2
        table = [[-1] * stride for _ in range(n_rows)]
        for row, ks in need.items():
            for k in ks:
                table[row][k] = perm.pop()
        self.table = torch.tensor(table, dtype=I32)
        shape = (pages, kvh, page, dim) if heads_first else (pages, page, kvh, dim)
        self.k_raw, self.v_raw = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
        self.heads_first = heads_first
        q = (torch.randn(n, heads * (2 if wide else 1), dim, generator=g) * q_scale).to(dtype)
        self.q = q[:, :heads]
        self.out0 = torch.randn(n, heads, dim, generator=g).to(dtype)
        self.lse0 = torch.randn(n, heads, generator=g)
        self.q_dev = q.cuda()[:, :heads]
        self.wide = wide

    def order(self, t):
        return t.transpose(1, 2) if self.heads_first else t

    def device(self):
        self.k_dev, self.v_dev = self.k_raw.cuda(), self.v_raw.cuda()
        self.cache = B.DraftCache(self.order(self.k_dev), self.order(self.v_dev))
        n, h, d = self.q.shape
        self.plan = B.ddtree_draft_attention_plan(n, h, self.cache, self.window, self.sinks)
        if self.wide:
            self.plan.q_stride = 2 * h * d
        self.ws = torch.full((B.ddtree_draft_attention_workspace_size(self.plan),), 0xA5, dtype=torch.uint8, device="cuda")
        self.out, self.lse = self.out0.cuda(), self.lse0.cuda()
        self.args = (self.plan, self.q_dev, self.cache, self.table.cuda(), torch.tensor(self.positions, dtype=I32, device="cuda"),
                     self.scale, self.out, self.ws)
        self.kw = dict(token_rows=torch.tensor(self.token_rows, dtype=I32, device="cuda"), lse=self.lse)

    def run(self):
        self.device()
        B.ddtree_draft_attention(*self.args, **self.kw)
        torch.cuda.synchronize()
        return B.ddtree_verify_mla_check(self.ws)

    def compare(self):
        ref, lse, mass, terms = draft_attention(self.q, self.order(self.k_raw), self.order(self.v_raw), self.table, self.token_rows,
                                                self.positions, self.window, self.sinks, self.scale, self.out0, self.lse0)
        ob, lb = _bounds(ref, lse, mass, terms, self.dim, self.dtype)
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kvh", [(1, 1), (8, 2), (5, 1), (16, 16), (24, 1), (64, 1), (66, 2), (40, 1)])
def test_heads_and_types(heads, kvh, dim, dtype):
    _check([0, 1, 63, 64, 130, 777], heads, kvh, dim, dtype=dtype, seed=heads + dim)


@pytest.mark.parametrize("pos", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 1023, 4096])
@pytest.mark.parametrize("dim,kvh", [(64, 3), (128, 1), (256, 2)])
def test_single_tokens_of_every_length(pos, dim, kvh):
    _check([pos], 4 * kvh, kvh, dim, page=1, seed=pos)


@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (64, 4), (100, 0), (100, 70), (1000, 33), (5000, 4), (7, 2 ** 31 - 1),
                                          (2 ** 31 - 1, 5)])
@pytest.mark.parametrize("heads_first", [False, True])
def test_windows_pages_and_orders(page, window, sinks, heads_first):
    _check([0, 3, 99, 640, 2049], 8, 2, 64, page=page, window=window, sinks=sinks, heads_first=heads_first, seed=page + window % 97)


def test_long_and_ragged():
    _check([30000, 5, 12345, 0, 777], 8, 2, 128, page=16, seed=1)
    _check([70001], 4, 1, 256, page=1, seed=2)


def test_many_tokens():
    r = random.Random(4)
    _check([r.choice([0, 1, 40, r.randint(0, 300)]) for _ in range(301)], 4, 2, 64, page=16, seed=3)
    _check([r.randint(0, 20) for _ in range(4096)], 2, 1, 64, page=4, seed=4)


@pytest.mark.parametrize("kvh,dim", [(3, 64), (5, 128), (6, 64), (12, 128), (16, 64), (24, 64), (10, 256), (128, 64)])
def test_key_heads_that_shares_take_side_by_side(kvh, dim):
    _check([700, 3, -1, 129, 2500], 2 * kvh, kvh, dim, seed=kvh)
    _check([40] * 33, kvh, kvh, dim, page=8, seed=kvh + 1)


def test_one_long_request_among_many_short_ones():
    # More units than shares: the long request's units cross shares, the short ones' do not.
    _check([9000] + [10, 60, 200, 127, 128] * 20, 8, 4, 64, seed=41)
    _check([30] * 70 + [6000, 100], 48, 8, 128, seed=42)


def test_strided_outputs_and_caches_of_one_tensor():
    c = Case([300, 5, 77], 8, 2, 64, seed=43)
    c.device()
    both = torch.stack([c.k_dev, c.v_dev], 1)                   # [pages, 2, page, heads, dim]
    cache = B.DraftCache(both[:, 0], both[:, 1])
    wide = torch.full((3, 11, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = B.ddtree_draft_attention_plan(3, 8, cache)
    plan.out_stride = 11 * 64
    B.ddtree_draft_attention(plan, c.q_dev, cache, *c.args[3:6], wide[:, 2:10], c.ws, **c.kw)
    torch.cuda.synchronize()
    c.out = wide[:, 2:10].contiguous()
    c.compare()
    assert bool((wide[:, :2] == 7.0).all()) and bool((wide[:, 10:] == 7.0).all())


def test_padding_tokens_are_left_alone():
    _check([-1, 100, -1, -1, 7, -1], 8, 2, 128, seed=5)
    _check([-1, -1], 8, 2, 128, seed=6)


def test_tokens_that_share_a_request():
    _check([100, 101, 102, 103, 40], 8, 2, 64, rows=[1, 1, 1, 1, 0], window=50, sinks=2, freed=False, seed=7)


def test_strided_queries_and_peaky_scores():
    _check([300, 5], 8, 2, 128, wide=True, seed=8)
    _check([300, 500], 8, 2, 128, q_scale=30.0, seed=9)
    _check([300, 500], 8, 2, 128, q_scale=30.0, dtype=torch.float16, seed=10)
    _check([300, 500], 8, 2, 64, scale=-0.2, seed=11)
    _check([300, 500], 8, 2, 64, scale=0.0, seed=12)


def test_one_large_score_among_many_keys_keeps_the_small_ones():
    # One key scores 16 above 60,000 equal ones: their mass, 60000 e^-16, must not be lost to the type of the probabilities.
    for dtype in (torch.float16, torch.bfloat16):
        c = Case([60000], 4, 1, 64, page=16, dtype=dtype, seed=13, scale=1.0)
        c.q.zero_(), c.k_raw.zero_(), c.v_raw.fill_(1.0)
        c.q[:, :, 0] = 4.0
        c.q_dev.copy_(c.q)
        at = int(c.table[c.token_rows[0], 100 // 16])
        c.k_raw[at, 100 % 16, 0, 0] = 4.0
        c.v_raw[at, 100 % 16, 0] = 0.0
        assert c.run() == 0
        c.compare()
        assert float(c.out.float().mean()) > 6e-3


def test_bad_positions_rows_and_pages():
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
    c.table[c.token_rows[1], 0] = c.k_raw.shape[0]
    c.table[c.token_rows[2], :] = -7      # nothing left to see
    assert c.run() == B.DDTREE_ST_BAD_INDEX
    c.compare()
    assert bool(torch.isinf(c.lse[2]).all()) and bool((c.out[2] == 0).all())


def test_nothing_beyond_the_visible_keys_counts():
    # NaN and infinity behind the token, before the window and in released pages change no bit.
    base = Case([100, 37, 400], 8, 2, 64, window=64, sinks=3, freed=False, seed=18)
    assert base.run() == 0
    base.compare()
    c = Case([100, 37, 400], 8, 2, 64, window=64, sinks=3, freed=False, seed=18)
    c.k_raw.copy_(base.k_raw), c.v_raw.copy_(base.v_raw)
    keep = torch.zeros(c.k_raw.shape[:2], dtype=torch.bool)
    for p, row in zip(c.positions, c.token_rows):
        for j in range(p + 1):
            if j > p - 64 or j < 3:
                keep[c.table[row, j // 16], j % 16] = True
    c.k_raw[~keep], c.v_raw[~keep] = float("nan"), float("inf")
    assert c.run() == 0
    assert torch.equal(c.out, base.out) and torch.equal(c.lse, base.lse)


def test_equal_bits_on_other_streams_without_lse_and_in_a_replay():
    c = Case([5000, 12, 900], 16, 2, 128, page=16, seed=19)
    assert c.run() == 0
    c.compare()
    out, lse = c.out.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.out.zero_(), c.ws.fill_(0x3C)
    side.wait_stream(torch.cuda.current_stream())
    kw = dict(c.kw, lse=None)
    B.ddtree_draft_attention(*c.args, **kw, stream=side)
    side.synchronize()
    assert torch.equal(c.out, out)
    bound = B.BoundDraftAttention(*c.args, **c.kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bound()
    c.out.zero_(), c.lse.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    # Other lengths through the same graph, and a status that does not stick.
    c.args[4].copy_(torch.tensor([17, -5, 4999], dtype=I32))
    g.replay()
    # (the third token stands past the pages that its row holds: its table entries are -1)
    assert B.ddtree_verify_mla_check(c.ws) == B.DDTREE_ST_BAD_LENGTH | B.DDTREE_ST_BAD_INDEX
    c.args[4].copy_(torch.tensor([17, 3, 800], dtype=I32))
    g.replay()
    assert B.ddtree_verify_mla_check(c.ws) == 0
    c.positions = [17, 3, 800]
    c.compare()


def test_two_graphs_share_a_workspace():
    a, b = (Case([3000, 70], 8, 2, 64, seed=s) for s in (20, 21))
    a.device(), b.device()
    ws = torch.empty(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.ddtree_draft_attention(*c.args[:-1], ws, **c.kw)
        graphs.append(g)
    for g in (graphs[0], graphs[1], graphs[0], graphs[1]):
        g.replay()
    torch.cuda.synchronize()
    a.compare(), b.compare()


def test_offsets_past_32_bits():
    pages, page, kvh, dim = 40000, 64, 8, 128   # 2.6e9 elements each
    k = torch.zeros(pages, page, kvh, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    last = pages - 1
    k[last].normal_(), v[last].normal_(), k[1].normal_(), v[1].normal_()
    cache = B.DraftCache(k, v)
    plan = B.ddtree_draft_attention_plan(1, 16, cache)
    ws = torch.empty(B.ddtree_draft_attention_workspace_size(plan), dtype=torch.uint8, device="cuda")
    q = torch.randn(1, 16, dim, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(1, 16, device="cuda")
    table = torch.tensor([[1, last]], dtype=I32, device="cuda")
    B.ddtree_draft_attention(plan, q, cache, table, torch.tensor([100], dtype=I32, device="cuda"), 0.1, out, ws, lse=lse)
    pair = torch.tensor([[0, 1]], dtype=I32)
    kk, vv = (torch.stack([t[1], t[last]]).cpu() for t in (k, v))
    ref, rl, mass, terms = draft_attention(q.cpu(), kk, vv, pair, None, [100], 0, 0, 0.1, out.cpu(), lse.cpu())
    ob, lb = _bounds(ref, rl, mass, terms, dim, torch.bfloat16)
    assert bool(((out.cpu().double() - ref).abs() <= ob).all()) and bool(((lse.cpu().double() - rl).abs() <= lb).all())


def test_python_refusals():
    c = Case([10, 20], 8, 2, 64, seed=22)
    c.device()
    for i, bad in ((1, c.q_dev.float()), (1, c.q_dev[:1]), (1, c.q_dev.transpose(1, 2)), (3, c.args[3].long()), (3, c.args[3][0]),
                   (4, c.args[4][:1]), (6, c.out[:, :4]), (7, c.ws[:-1]), (7, c.ws.int())):
        a = list(c.args)
        a[i] = bad
        with pytest.raises((TypeError, ValueError)):
            B.ddtree_draft_attention(*a, **c.kw)


@pytest.mark.parametrize("heads,kvh,dim", [(8, 2, 64), (66, 2, 64), (40, 1, 128), (64, 1, 256)])
@pytest.mark.parametrize("entry", [-2, -2 ** 31, 2 ** 31 - 1])
def test_every_table_entry_outside_the_cache_is_reported(entry, heads, kvh, dim):
    c = Case([100, 50, 20], heads, kvh, dim, seed=45)
    c.table[c.token_rows[0], 2] = entry
    assert c.run() == B.DDTREE_ST_BAD_INDEX
    c.compare()


WIDE = [(d, t) for d in (64, 128, 256) for t in (torch.bfloat16, torch.float16)]


@pytest.mark.parametrize("dim,dtype", WIDE)
def test_wide_groups_over_many_tiles_a_share(dim, dtype):
    # 20 to 40 tiles a share: every ring of the kernel goes round more than once.
    n = {64: 50000, 128: 25000, 256: 15000}[dim]
    _check([n, n - 77, 3], 4 * 33, 4, dim, dtype=dtype, seed=46)


@pytest.mark.parametrize("dim,dtype", WIDE)
def test_wide_groups_of_many_short_requests(dim, dtype):
    r = random.Random(47)
    _check([r.choice([0, -1, 31, 32, 63, 64, 127, 128, r.randint(0, 300)]) for _ in range(331)], 66, 2, dim, dtype=dtype, seed=47)
    _check([3000] + [r.randint(0, 70) for _ in range(90)], 40, 1, dim, dtype=dtype, page=1, seed=48)


@pytest.mark.parametrize("dim,dtype", WIDE)
@pytest.mark.parametrize("page,window,sinks", [(1, 1, 0), (3, 100, 70), (16, 1000, 33), (64, 64, 4), (16, 7, 2 ** 31 - 1)])
def test_wide_groups_with_windows(page, window, sinks, dim, dtype):
    _check([0, 3, 99, 640, 2049], 40, 1, dim, dtype=dtype, page=page, window=window, sinks=sinks, heads_first=page == 16, seed=49)


@pytest.mark.parametrize("dim,dtype", WIDE)
@pytest.mark.parametrize("step", [0.05, -0.05, 0.004])
def test_wide_groups_whose_scores_rise_or_fall_along_the_keys(step, dim, dtype):
    c = Case([2500, 140], 33, 1, dim, dtype=dtype, page=16, freed=False, seed=50, scale=1.0)
    c.q.zero_(), c.k_raw.zero_()
    c.q[:, :, 0] = 4.0
    c.q_dev.copy_(c.q)
    for p, row in zip(c.positions, c.token_rows):
        for j in range(p + 1):
            c.k_raw[c.table[row, j // 16], j % 16, 0, 0] = step * j
    assert c.run() == 0
    c.compare()


@pytest.mark.parametrize("dim,dtype", WIDE)
def test_wide_groups_with_other_scales_strides_and_padding(dim, dtype):
    _check([300, -1, 500], 40, 1, dim, dtype=dtype, wide=True, seed=51)
    _check([300, 500], 66, 2, dim, dtype=dtype, q_scale=30.0, seed=52)
    _check([300, 500], 40, 1, dim, dtype=dtype, scale=-0.2, seed=53)
    _check([300, 500], 40, 1, dim, dtype=dtype, scale=0.0, seed=54)
    c = Case([100, 50, 20, 77], 40, 1, dim, dtype=dtype, seed=55)
    c.positions[3] = 16 * c.table.shape[1]
    c.table[c.token_rows[2], :] = -7      # nothing left to see
    assert c.run() == B.DDTREE_ST_BAD_INDEX | B.DDTREE_ST_BAD_LENGTH
    c.compare()
    assert bool((c.out[2:] == 0).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_wide_groups_see_nothing_else_and_replay_equal_bits(dim):
    base = Case([100, 37, 4000], 34, 1, dim, window=64, sinks=3, freed=False, seed=56)
    assert base.run() == 0
    base.compare()
    c = Case([100, 37, 4000], 34, 1, dim, window=64, sinks=3, freed=False, seed=56)
    keep = torch.zeros(c.k_raw.shape[:2], dtype=torch.bool)
    for p, row in zip(c.positions, c.token_rows):
        for j in range(p + 1):
            if j > p - 64 or j < 3:
                keep[c.table[row, j // 16], j % 16] = True
    c.k_raw[~keep], c.v_raw[~keep] = float("nan"), float("inf")
    assert c.run() == 0
    assert torch.equal(c.out, base.out) and torch.equal(c.lse, base.lse)
    bound = B.BoundDraftAttention(*c.args, **c.kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            bound()
    c.out.zero_(), c.lse.zero_(), c.ws.fill_(0x3C)
    g.replay(), g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, base.out) and torch.equal(c.lse, base.lse)
