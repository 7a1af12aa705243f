"""The attention over whole prompts on the GPU against the float64 oracle.

Bound of an output, as for the drafter's one-token attention: half a step of its
type for the final rounding (2^-25 where fp16 is subnormal), half a step of
every probability, which meets V in the inputs' type (of sum |p v|), and the
32-bit work: two sums of D terms, 64 units for the sums over keys.  Where fp16
probabilities (with their factor of 2^10) are subnormal they are 2^-25 of it off:
2^-35 of the largest |v| each.  lse has the scores' error once.
"""
import random

import pytest
import torch

from oracle import prompt_attention
from speculative_decode_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
I32 = torch.int32
U = 2.0 ** -24


class Case:
    """lens: queries of the sequences; ctx: keys before them (may be negative: more queries than keys)."""

    def __init__(self, lens, heads, kvh, dim, *, ctx=None, window=0, sinks=0, dtype=torch.bfloat16, seed=0, scale=None, q_scale=1.0,
                 packed=False, behind=3, before=0, same=False, lse=True):
        g = torch.Generator().manual_seed(seed)
        ctx = [0] * len(lens) if ctx is None else ctx
        self.qp, self.kp = [before], [before]
        for n, c in zip(lens, ctx):
            self.qp.append(self.qp[-1] + n)
            self.kp.append(self.kp[-1] + max(0, n + c))
        nq, nk = max(1, self.qp[-1] + behind), max(1, self.kp[-1] + behind)
        assert not packed or (nq == nk)
        self.q = (torch.randn(nq, heads, dim, generator=g) * q_scale).to(dtype)
        self.k, self.v = (torch.randn(nk, kvh, dim, generator=g).to(dtype) for _ in range(2))
        self.out0 = torch.randn(nq, heads, dim, generator=g).to(dtype)
        self.lse0 = torch.randn(nq, heads, generator=g)
        self.window, self.sinks, self.dtype, self.dim, self.packed, self.same = window, sinks, dtype, dim, packed, same
        self.scale = dim ** -0.5 if scale is None else scale
        self.want_lse = lse

    def device(self):
        h, kvh = self.q.shape[1], self.k.shape[1]
        if self.packed:
            all_ = torch.cat([self.q, self.k, self.v], 1).cuda()
            q, k, v = all_[:, :h], all_[:, h:h + kvh], all_[:, h + kvh:]
        else:
            q, k, v = self.q.cuda(), self.k.cuda(), self.v.cuda()
        self.plan = B.ddtree_prompt_attention_plan(len(self.qp) - 1, q.shape[0], k.shape[0], h, kvh, self.dim, self.dtype, self.window, self.sinks)
        self.ws = torch.full((B.ddtree_prompt_attention_workspace_size(self.plan),), 0xA5, dtype=torch.uint8, device="cuda")
        self.out, self.lse = self.out0.cuda(), self.lse0.cuda()
        self.q_indptr = torch.tensor(self.qp, dtype=I32, device="cuda")
        self.k_indptr = None if self.same else torch.tensor(self.kp, dtype=I32, device="cuda")
        self.args = (self.plan, q, k, v, self.q_indptr, self.k_indptr, self.scale, self.out, self.ws)
        self.kw = dict(lse=self.lse if self.want_lse else None)

    def run(self):
        self.device()
        B.ddtree_prompt_attention(*self.args, **self.kw)
        torch.cuda.synchronize()
        return B.ddtree_verify_mla_check(self.ws)

    def compare(self):
        ref, lse, mass, terms = prompt_attention(self.q, self.k, self.v, self.qp, self.kp, self.window, self.sinks, self.scale, self.out0, self.lse0)
        half = torch.finfo(self.dtype).eps / 2
        work = (2 * self.dim * U * terms + 64 * U)[..., None]
        keys = max(b - a for a, b in zip(self.kp, self.kp[1:]))
        finite = torch.isfinite(self.v.float())
        most = float(self.v.double()[finite].abs().max()) if bool(finite.any()) else 0.0
        ob = ref.abs() * half + mass * (half + 2 * work)
        if self.dtype == torch.float16:
            ob = ob + 2.0 ** -25 + keys * most * 2.0 ** -35
        lb = self.dim * U * terms + 8 * U * lse.abs() + 64 * U
        out, got = self.out.cpu().double(), self.lse.cpu().double()
        assert torch.equal(torch.isnan(out), torch.isnan(ref))
        good = torch.isfinite(ref)
        assert torch.equal(out[~good & ~torch.isnan(ref)], ref[~good & ~torch.isnan(ref)])
        over = ((out - ref).abs() - ob)[good]
        assert not over.numel() or float(over.max()) <= 0, f"out {float(over.max()):.3e} over its bound"
        if self.want_lse:
            none = ~torch.isfinite(lse)
            assert torch.equal(torch.nan_to_num(got[none], nan=7.0), torch.nan_to_num(lse[none], nan=7.0))
            over = ((got - lse).abs() - lb)[~none]
            assert not over.numel() or float(over.max()) <= 0, f"lse {float(over.max()):.3e} over its bound"
        else:
            assert torch.equal(got, self.lse0.double())
        rows = torch.ones(self.q.shape[0], dtype=torch.bool)
        rows[self.qp[0]:self.qp[-1]] = False
        assert torch.equal(self.out.cpu()[rows], self.out0[rows]) and torch.equal(self.lse.cpu()[rows], self.lse0[rows])


def _check(*a, status=0, **kw):
    c = Case(*a, **kw)
    assert c.run() == status
    c.compare()
    return c


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kvh", [(1, 1), (8, 2), (3, 1), (10, 2), (7, 7), (16, 1), (40, 1), (64, 1), (12, 4)])
def test_heads_and_types(heads, kvh, dim, dtype):
    _check([5, 1, 70, 200], heads, kvh, dim, dtype=dtype, seed=heads + dim)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513])
@pytest.mark.parametrize("dim,heads,kvh", [(64, 1, 1), (128, 4, 1), (256, 2, 1)])
def test_prompts_of_every_length(n, dim, heads, kvh):
    _check([n], heads, kvh, dim, seed=n, same=n % 2 == 0)


@pytest.mark.parametrize("lens", [[0], [0, 7, 0, 0, 130, 0], [1] * 70, [1, 2, 3, 250, 4], [0] * 33, [3, 0, 257, 0]])
def test_sequences(lens):
    _check(lens, 4, 2, 64, seed=len(lens))
    _check(lens, 4, 2, 128, seed=len(lens), before=5)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (100, 0), (100, 70), (200, 300), (128, 128), (5000, 4), (7, 2 ** 31 - 1), (2 ** 31 - 1, 5)])
@pytest.mark.parametrize("dim,heads,kvh", [(64, 8, 2), (128, 3, 1), (256, 2, 2)])
def test_windows_and_sinks(window, sinks, dim, heads, kvh):
    _check([700, 90, 3], heads, kvh, dim, window=window, sinks=sinks, seed=window % 97)
    _check([300, 90, 3], heads, kvh, dim, window=window, sinks=sinks, ctx=[500, 0, 1000], seed=sinks % 97)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_contexts(dim):
    _check([3, 64, 130, 1], 8, 2, dim, ctx=[1000, 1, 127, 0], seed=1)
    _check([3, 64, 130, 1], 8, 2, dim, ctx=[-1, -30, -130, -1], seed=2)     # queries that see nothing
    _check([3, 5], 8, 2, dim, ctx=[-3, -9], window=4, sinks=2, seed=3)


@pytest.mark.parametrize("window", [2 ** 24 - 1, 2 ** 24, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 2 ** 31 - 1])
def test_largest_windows_with_queries_that_see_nothing(window, sinks):
    for dim in (64, 128, 256):
        _check([200, 70], 4, 2, dim, ctx=[-60, -69], window=window, sinks=sinks, seed=dim)


@pytest.mark.parametrize("lens,ctx", [([3] * 900, None), ([1, 40, 0, 90] * 60, [0, 300, 5, -70] * 60), ([260, 700] * 20, [900, 0] * 20)])
@pytest.mark.parametrize("dim,heads,kvh", [(64, 16, 8), (128, 16, 8), (256, 8, 8)])
def test_many_items_for_each_cta(lens, ctx, dim, heads, kvh):
    _check(lens, heads, kvh, dim, ctx=ctx, window=600, sinks=2, seed=dim)


def test_one_short_chunk_behind_a_long_context_with_a_small_bound():
    # One product tile has no rows and waits for the next item all the while.
    c = Case([70], 8, 8, 64, ctx=[200000], seed=20, window=150000)
    c.device()
    c.plan.wait_limit_us = 200
    B.ddtree_prompt_attention(*c.args, **c.kw)
    torch.cuda.synchronize()
    assert B.ddtree_verify_mla_check(c.ws) == 0
    want = c.out.clone()
    c.plan.wait_limit_us = 0
    B.ddtree_prompt_attention(*c.args, **c.kw)
    assert torch.equal(c.out, want)


@pytest.mark.parametrize("kw", [dict(packed=True), dict(lse=False), dict(q_scale=30.0), dict(q_scale=30.0, dtype=torch.float16), dict(scale=-0.2),
                                dict(scale=0.0), dict(scale=-0.2, window=50, sinks=3), dict(before=9, behind=70), dict(behind=0)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_layouts_and_scores(kw, dim):
    _check([200, 77, 1], 6, 2, dim, seed=4, **kw)


def test_long_prompts():
    _check([3001], 2, 1, 128, seed=5)
    _check([2500], 2, 1, 64, seed=6, dtype=torch.float16)
    _check([1500, 700], 2, 2, 256, seed=7)


def test_rising_scores():
    # Every key outdoes those before it, so the maxima move all the way.
    for dim in (64, 128, 256):
        for dtype in (torch.bfloat16, torch.float16):
            c = Case([900], 2, 1, dim, seed=8, scale=1.0, dtype=dtype)
            c.q.zero_(), c.k.zero_()
            c.q[:, :, 0] = 1.0
            c.k[:, 0, 0] = torch.linspace(-60, 60, c.k.shape[0]).to(dtype)
            assert c.run() == 0
            c.compare()


def test_one_large_score_among_many_keys_keeps_the_small_ones():
    for dtype in (torch.float16, torch.bfloat16):
        c = Case([2], 4, 1, 64, ctx=[60000], dtype=dtype, seed=13, scale=1.0)
        c.q.zero_(), c.k.zero_(), c.v.fill_(1.0)
        c.q[:, :, 0] = 4.0
        c.k[100, 0, 0] = 4.0
        c.v[100] = 0.0
        assert c.run() == 0
        c.compare()
        assert float(c.out[:2].float().mean()) > 6e-3


@pytest.mark.parametrize("dim,heads,kvh", [(64, 4, 2), (128, 4, 2), (256, 2, 2)])
def test_what_a_row_does_not_see_has_no_part_in_it(dim, heads, kvh):
    # NaN and infinities in later keys, other sequences, rows of no sequence and before the window.
    for bad in (float("nan"), float("inf"), -float("inf")):
        c = Case([150, 40, 300], heads, kvh, dim, ctx=[0, 20, 0], window=64, sinks=3, seed=9, before=4)
        c.k[:4], c.v[:4], c.k[-3:], c.v[-3:], c.q[:4], c.q[-3:] = bad, bad, bad, bad, bad, bad
        c.v[c.kp[0] + 100, 1, 5] = bad              # seen by 64 rows of the first sequence
        c.k[c.kp[2] + 250, 0] = bad                 # and of the third
        assert c.run() == 0
        c.compare()
        assert not bool(torch.isnan(c.out[c.qp[1]:c.qp[2]]).any()) and bool(torch.isfinite(c.out[c.qp[0]:c.qp[0] + 100]).all())
        c = Case([130, 129], heads, kvh, dim, seed=10)
        c.v[129], c.k[129], c.q[130 + 128] = bad, bad, bad  # the last token of the first, the last row of the second
        assert c.run() == 0
        c.compare()
        assert bool(torch.isfinite(c.out[:129]).all()) and bool(torch.isfinite(c.out[130:258]).all())


@pytest.mark.parametrize("dim,heads,kvh", [(64, 4, 2), (128, 4, 2), (256, 2, 2)])
def test_old_context_that_was_not_read_back(dim, heads, kvh):
    # Between the sinks and the first row's window anything may lie; 130 sinks end inside a key tile.
    for sinks, n in ((3, 90), (130, 300)):
        for bad in (float("nan"), float("inf")):
            c = Case([n, 7], heads, kvh, dim, ctx=[1000, 700], window=64, sinks=sinks, seed=sinks)
            for b in range(2):
                first = c.kp[b + 1] - (c.qp[b + 1] - c.qp[b]) - 64 + 1
                c.k[c.kp[b] + sinks:first], c.v[c.kp[b] + sinks:first] = bad, bad
            assert c.run() == 0
            c.compare()
            assert bool(torch.isfinite(c.out[c.qp[0]:c.qp[-1]]).all())


def test_more_rows_done_again_than_one_round_takes():
    # 8,000 items of which every second one has a NaN in a value that its rows see.
    c = Case([2] * 1000, 8, 8, 64, seed=19, same=True)
    c.v[0:2000:2, ::2, 1] = float("nan")
    assert c.run() == 0
    c.compare()


def test_rows_far_apart():
    # Keys and values 4 MB apart: offsets pass 32 bits; with a NaN the rows go one by one.
    for bad in (False, True):
        c = Case([40, 1100], 2, 1, 64, seed=15)
        if bad:
            c.v[c.kp[2] - 1, 0, 3] = float("nan")
        c.device()
        n, step = c.k.shape[0], 1 << 21
        far = torch.empty(n * step, dtype=torch.bfloat16, device="cuda")
        k, v = (torch.as_strided(far, (n, 1, 64), (step, 64, 1), at) for at in (0, 4096))
        k.copy_(c.k), v.copy_(c.v)
        B.ddtree_prompt_attention(c.plan, c.args[1], k, v, *c.args[4:], **c.kw)
        torch.cuda.synchronize()
        assert B.ddtree_verify_mla_check(c.ws) == 0
        c.compare()


def test_two_streams_with_a_workspace_each():
    cases = [Case([700, 30, 5], 8, 2, 128, seed=16 + i) for i in range(2)] + [Case([90] * 9, 4, 2, 64, seed=18)]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.device()
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(cases, streams):
            B.ddtree_prompt_attention(*c.args, **c.kw, stream=s)
    torch.cuda.synchronize()
    for c in cases:
        assert B.ddtree_verify_mla_check(c.ws) == 0
        c.compare()


def test_bad_sequences_write_nothing():
    base = Case([30, 50], 4, 2, 64, seed=11)
    for which, values in (("qp", [0, 40, 30]), ("qp", [-1, 30, 80]), ("qp", [0, 30, 84]), ("kp", [0, 90, 80]), ("kp", [0, 30, 90]), ("kp", [-5, 30, 80]),
                          ("qp", [0, 2 ** 31 - 1, -2 ** 31])):
        c = Case([30, 50], 4, 2, 64, seed=11)
        c.device()
        (c.q_indptr if which == "qp" else c.k_indptr).copy_(torch.tensor(values, dtype=I32))
        B.ddtree_prompt_attention(*c.args, **c.kw)
        assert B.ddtree_verify_mla_check(c.ws) == B.DDTREE_ST_BAD_LENGTH
        assert torch.equal(c.out.cpu(), c.out0) and torch.equal(c.lse.cpu(), c.lse0)
    assert base.run() == 0
    base.compare()


def test_equal_bits_on_another_stream_and_in_a_replay_with_other_lengths():
    c = Case([500, 12, 90], 16, 2, 128, seed=12)
    assert c.run() == 0
    c.compare()
    out, lse = c.out.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    c.out.copy_(c.out0), c.ws.fill_(0x3C)
    side.wait_stream(torch.cuda.current_stream())
    B.ddtree_prompt_attention(*c.args, stream=side)
    side.synchronize()
    assert torch.equal(c.out, out)
    bound = B.BoundPromptAttention(*c.args, **c.kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bound()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    for lens in ([1, 600, 1], [0, 0, 3], [602, 0, 0]):
        c.qp = [0, lens[0], lens[0] + lens[1], sum(lens)]
        c.kp = [3, 3 + lens[0], 3 + lens[0] + lens[1], 3 + sum(lens)] if sum(lens) < 600 else c.qp
        c.q_indptr.copy_(torch.tensor(c.qp))
        c.k_indptr.copy_(torch.tensor(c.kp))
        c.out.copy_(c.out0), c.lse.copy_(c.lse0)
        g.replay()
        torch.cuda.synchronize()
        assert B.ddtree_verify_mla_check(c.ws) == 0
        c.compare()


def test_random_shapes():
    r = random.Random(14)
    for i in range(25):
        kvh = r.choice([1, 2, 3])
        lens = [r.choice([0, 1, r.randint(1, 40), r.randint(1, 400)]) for _ in range(r.randint(1, 6))]
        ctx = [r.choice([0, 0, r.randint(0, 300)]) for _ in lens]
        _check(lens, kvh * r.choice([1, 2, 4, 5, 8]), kvh, r.choice([64, 128, 256]), ctx=ctx, window=r.choice([0, 0, 1, 33, 128, 200]),
               sinks=r.choice([0, 1, 40, 130]), dtype=r.choice([torch.bfloat16, torch.float16]), seed=i, before=r.choice([0, 3]))


def test_refusals():
    c = Case([5, 6], 8, 2, 64, seed=21)
    c.device()
    plan, q, k, v = c.args[:4]
    for bad, err in (((plan, q.half(), *c.args[2:]), TypeError), ((plan, q[:, :4], *c.args[2:]), ValueError), ((plan, q.cpu(), *c.args[2:]), TypeError),
                     ((plan, q, k[:-1], *c.args[3:]), ValueError), ((plan, q, k, v, c.q_indptr[:-1], *c.args[5:]), ValueError),
                     ((*c.args[:8], c.ws[:-1]), ValueError), ((plan, q.transpose(0, 1).contiguous().transpose(0, 1), *c.args[2:]), ValueError)):
        with pytest.raises(err):
            B.ddtree_prompt_attention(*bad, **c.kw)
    with pytest.raises(B.DDTreeError):
        B.ddtree_prompt_attention(plan, q, k, v, c.q_indptr, c.k_indptr, float("inf"), c.out, c.ws)
    with pytest.raises(B.DDTreeError):
        B.ddtree_prompt_attention(plan, q, k, v, c.q_indptr, c.k_indptr, 1.0, q, c.ws)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,ctx", [([3] * 90, 700), ([200] * 40, 0), ([1, 60, 129, 250] * 12, 300)])
def test_rising_scores_of_short_sequences(lens, ctx, dim, dtype):
    # Short sequences take two threads for a row, each with half of its keys and half of its columns of O: where the
    # maximum rises at every key tile, both halves have to be scaled before a product goes on top of them.  More items
    # than two for each SM, many times over: equal bits each time.
    c = Case(lens, 8, 4, dim, ctx=[ctx] * len(lens), seed=22, scale=1.0, dtype=dtype)
    c.q[:, :, 0] = 1.0
    c.q[:, :, 1:] *= 0.01
    for a, b in zip(c.kp, c.kp[1:]):
        c.k[a:b, :, 0] = torch.linspace(-60, 60, b - a).to(dtype)[:, None]
    assert c.run() == 0
    c.compare()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(50):
        c.out.copy_(c.out0), c.lse.copy_(c.lse0)
        B.ddtree_prompt_attention(*c.args, **c.kw)
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    assert B.ddtree_verify_mla_check(c.ws) == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,tokens,heads,log_keys", [(64, 2, 8, 20), (128, 2, 8, 20), (256, 2, 8, 20), (64, 300, 4, 19), (128, 300, 4, 19)])
@pytest.mark.parametrize("rising,window", [(False, 0), (True, 0), (False, 300000)])
def test_sums_over_very_many_keys(dim, tokens, heads, log_keys, rising, window, dtype):
    # Values of one sign, so that whatever a long sum loses adds up.  Bound: half a step of the output; half a step of
    # every probability; and in the tensor cores, which cut sums off where they do not fit into 32 bits, 2^-23 of the sum
    # for every four keys of the 16,384 that one sum goes over.  lse: 64 units for sums that are halves of halves.
    g = torch.Generator(device="cuda").manual_seed(dim + tokens)
    n, sinks = 1 << log_keys, 5000 if window else 0
    q, k = (torch.randn(*s, generator=g, device="cuda").to(dtype) for s in ((tokens, heads, dim), (n, 1, dim)))
    v = (torch.rand(n, 1, dim, generator=g, device="cuda") + 1).to(dtype)
    if rising:
        q[:, :, 0] = 1.0
        k[:, 0, 0] = (torch.linspace(-40, 40, n, device="cuda")).to(dtype)
    plan = B.ddtree_prompt_attention_plan(1, tokens, n, heads, 1, dim, dtype, window, sinks)
    ws = torch.full((B.ddtree_prompt_attention_workspace_size(plan),), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(tokens, heads, device="cuda")
    indptr = [torch.tensor([0, m], dtype=I32, device="cuda") for m in (tokens, n)]
    B.ddtree_prompt_attention(plan, q, k, v, *indptr, dim ** -0.5, out, ws, lse=lse)
    assert B.ddtree_verify_mla_check(ws) == 0
    half, kd, vd = torch.finfo(dtype).eps / 2, k[:, 0].double(), v[:, 0].double()
    j = torch.arange(n, device="cuda")[None, :]
    for first in range(0, tokens, 50):
        rows = slice(first, min(tokens, first + 50))
        p = torch.arange(n - tokens + first, n - tokens + rows.stop, device="cuda")[:, None]
        seen = j <= p
        if window:
            seen &= (j > p - window) | (j < sinks)
        for h in range(heads):
            s = (q[rows, h].double() @ kd.T) * dim ** -0.5
            terms = (q[rows, h].double().abs() @ kd.abs().T).amax(-1) * dim ** -0.5
            s.masked_fill_(~seen, -float("inf"))
            ref_lse = torch.logsumexp(s, -1)
            ref = torch.exp(s - ref_lse[:, None]) @ vd
            bound = ref * (half + half + 4096 * 2.0 ** -23 + (2 * dim * U * terms + 64 * U)[:, None] * 2)
            over = ((out[rows, h].double() - ref).abs() - bound).max()
            assert float(over) <= 0, f"out {float(over):.3e} over its bound"
            over = ((lse[rows, h].double() - ref_lse).abs() - (dim * U * terms + 8 * U * ref_lse.abs() + 64 * U)).max()
            assert float(over) <= 0, f"lse {float(over):.3e} over its bound"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("flat", [True, False])
def test_sums_over_many_keys_row_by_row(flat, dim, dtype):
    # The last value is no number, so the rows before it are done again one by one: constant values (no powers of two)
    # and, where flat, equal weights.  Bound: half a step of the output, and of 32-bit sums that go over 32 + 724 + 12 terms.
    n, heads = 1 << 18, 4
    g = torch.Generator(device="cuda").manual_seed(dim)
    q = torch.zeros(2, heads, dim, device="cuda", dtype=dtype) if flat else torch.randn(2, heads, dim, generator=g, device="cuda").to(dtype)
    k = torch.randn(n, 1, dim, generator=g, device="cuda").to(dtype)
    value = (1 + torch.arange(dim, device="cuda") / dim).to(dtype)
    v = value.expand(n, 1, dim).contiguous()
    v[n - 1] = float("nan")
    plan = B.ddtree_prompt_attention_plan(1, 2, n, heads, 1, dim, dtype)
    ws = torch.full((B.ddtree_prompt_attention_workspace_size(plan),), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, heads, device="cuda")
    B.ddtree_prompt_attention(plan, q, k, v, torch.tensor([0, 2], dtype=I32, device="cuda"), torch.tensor([0, n], dtype=I32, device="cuda"),
                              dim ** -0.5, out, ws, lse=lse)
    assert B.ddtree_verify_mla_check(ws) == 0
    half = torch.finfo(dtype).eps / 2
    assert bool(torch.isnan(out[1]).all())
    # Numerator and denominator each lose at most 768 half steps of 32 bits, and 64 more for the exponentials.
    over = ((out[0].double() / value.double() - 1).abs() - half - 2 * (768 + 64) * U).max()
    assert float(over) <= 0, f"{float(over):.3e} over its bound"
    s = (q[0].double() @ k[:n - 1, 0].double().T) * dim ** -0.5
    terms = (q[0].double().abs() @ k[:n - 1, 0].double().abs().T).amax(-1) * dim ** -0.5
    ref = torch.logsumexp(s, -1)
    over = ((lse[0].double() - ref).abs() - (dim * U * terms + 8 * U * ref.abs() + (768 + 64) * U)).max()
    assert float(over) <= 0, f"lse {float(over):.3e} over its bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("values", [False, True])
def test_rows_whose_scores_are_all_minus_infinity(values, dim, dtype):
    # exp(-inf) / 0 is no number; a row that sees no key at all is zero (queries before the first key).
    for lens, ctx in (([30, 5], [-2, 0]), ([700], [-3])):
        c = Case(lens, 4, 2, dim, ctx=ctx, dtype=dtype, seed=33)
        c.q[:, :, 0] = -1.0
        c.k[c.kp[0]:c.kp[0] + 9, 0, 0] = float("inf")   # the first rows see nothing but such keys
        c.k[c.kp[0]:c.kp[0] + 9, 0, 1:] = 0.5
        if values:
            c.v[c.kp[0] + 12, 0, 3] = float("nan")      # row by row
        assert c.run() == 0
        c.compare()
        first = c.qp[0] - ctx[0]
        assert bool(torch.isnan(c.out[first:first + 9, :2]).all()) and bool((c.out[c.qp[0]:first] == 0).all())
        assert bool(torch.isneginf(c.lse[c.qp[0]:first]).all()) and bool(torch.isfinite(c.lse[first + 9:c.qp[1]]).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens", [[700, 90], [40] * 30])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_keys_and_queries_that_are_no_numbers_cost_no_second_pass(dim, lens, bad):
    # Rows that see such a key are none, whatever the values are; only values that some rows of an item do not see
    # have their items done again (a bit in the words behind the status block).
    def marked(c):
        words = c.ws[256:256 + 4 * c.plan.max_items].view(I32)
        return int((words < 0).sum())
    c = Case(lens, 8, 2, dim, seed=30)
    c.k[c.kp[0], 0, 3], c.k[c.kp[1] + 20, 1], c.q[c.qp[1] + 5] = bad, bad, bad
    assert c.run() == 0
    c.compare()
    assert marked(c) == 0
    c = Case(lens, 8, 2, dim, seed=31)
    c.v[c.kp[0] + 7, 0, 3] = bad
    assert c.run() == 0
    c.compare()
    assert marked(c) > 0
