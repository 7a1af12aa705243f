"""The drafter's attention with few shares: plans for one to three SMs give every
share many tiles and several units of small inputs, so that stages, queries,
offsets and the running maximum go from tile to tile and from unit to unit in
each of the kernel's forms, and share counts that key heads do not divide."""
import random

import pytest
import torch

from speculative_decode_tree_gb300 import binding as B
from test_draft_attn_gpu import Case

pytestmark = pytest.mark.gpu
I32 = torch.int32
BF, HF = torch.bfloat16, torch.float16

# (columns, query heads of a key head): 16 rows in registers, 32 rows in registers, tensor memory.
NARROW = [(64, 8), (128, 4), (256, 16)]
MIDDLE = [(64, 17), (64, 24), (64, 32)]
WIDE = [(64, 33), (128, 17), (256, 64)]
FORMS = [(d, g, t) for d, g in NARROW + MIDDLE + WIDE for t in (BF, HF)]


class FewShares(Case):
    def __init__(self, sms, *a, **kw):
        super().__init__(*a, **kw)
        self.sms = sms

    def device(self):
        super().device()
        q_stride = self.plan.q_stride
        n, h, _ = self.q.shape
        self.plan = B.ddtree_draft_attention_plan(n, h, self.cache, self.window, self.sinks, num_sms=self.sms)
        self.plan.q_stride = q_stride
        self.ws = torch.full((B.ddtree_draft_attention_workspace_size(self.plan),), 0xA5, dtype=torch.uint8, device="cuda")
        self.args = (self.plan,) + self.args[1:7] + (self.ws,)


def _check(sms, *a, status=0, **kw):
    c = FewShares(sms, *a, **kw)
    assert c.run() == status
    c.compare()
    return c


@pytest.mark.parametrize("dim,group,dtype", FORMS)
@pytest.mark.parametrize("sms,kvh", [(1, 3), (3, 4)])
def test_many_tiles_a_share(sms, kvh, dim, group, dtype):
    _check(sms, [3000, 1, 777, -1, 1500], group * kvh, kvh, dim, dtype=dtype, seed=dim + group + sms)


@pytest.mark.parametrize("dim,group,dtype", FORMS)
def test_many_units_a_share(dim, group, dtype):
    r = random.Random(dim + group)
    _check(1, [r.choice([-1, 0, 31, 63, 64, 127, 128, r.randint(0, 300)]) for _ in range(67)], 2 * group, 2, dim, dtype=dtype,
           page=r.choice([1, 16, 48]), seed=dim * group)


@pytest.mark.parametrize("dim,group,dtype", FORMS)
@pytest.mark.parametrize("page,window,sinks", [(3, 100, 70), (16, 1000, 33)])
def test_windows(page, window, sinks, dim, group, dtype):
    _check(1, [0, 3, 99, -1, 640, 2049], group, 1, dim, dtype=dtype, page=page, window=window, sinks=sinks, heads_first=page == 16,
           seed=81)


@pytest.mark.parametrize("dim,group,dtype", FORMS)
def test_scores_that_rise_along_the_keys(dim, group, dtype):
    c = FewShares(1, [2000, 140, 700], group, 1, dim, dtype=dtype, page=16, freed=False, seed=82, scale=1.0)
    c.q.zero_(), c.k_raw.zero_()
    c.q[:, :, 0] = 4.0
    c.q_dev.copy_(c.q)
    for p, row in zip(c.positions, c.token_rows):
        for j in range(p + 1):
            c.k_raw[c.table[row, j // 16], j % 16, 0, 0] = 0.05 * j
    assert c.run() == 0
    c.compare()


@pytest.mark.parametrize("dim,group,dtype", FORMS)
def test_bad_data_among_good(dim, group, dtype):
    c = FewShares(2, [500, 50, 900, 77, 20], 2 * group, 2, dim, dtype=dtype, seed=83)
    c.positions[1] = -5
    c.table[c.token_rows[2], 7] = c.k_raw.shape[0]
    c.table[c.token_rows[4], :] = -7
    assert c.run() == B.DDTREE_ST_BAD_LENGTH | B.DDTREE_ST_BAD_INDEX
    c.compare()


@pytest.mark.parametrize("dim,group,dtype", FORMS)
def test_replays_with_other_lengths(dim, group, dtype):
    c = FewShares(2, [1500, 12, 900, 64], 2 * group, 2, dim, dtype=dtype, page=16, freed=False, seed=84, wide=True)
    assert c.run() == 0
    c.compare()
    out, lse = c.out.clone(), c.lse.clone()
    bound = B.BoundDraftAttention(*c.args, **c.kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bound()
        bound()
    c.out.zero_(), c.lse.zero_(), c.ws.fill_(0x3C)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    c.positions = [700, 0, 63, -1]
    c.args[4].copy_(torch.tensor(c.positions, dtype=I32))
    c.out.copy_(c.out0), c.lse.copy_(c.lse0)
    g.replay()
    assert B.ddtree_verify_mla_check(c.ws) == 0
    c.compare()
