"""Pins of the drafter-attention oracle, and the entry points' host-side
refusals and plans (no GPU)."""
import ctypes
import math

import pytest
import torch

from oracle import draft_attention, visible_keys
from speculative_decode_tree_gb300 import binding as B
from test_append_oracle import BAD_CACHES, ODD, OFF, P, Q, _cache


@pytest.fixture(scope="module")
def lib():
    from speculative_decode_tree_gb300.build import build
    build()
    return B.library()


def test_visible_keys():
    assert visible_keys(5, 0, 3) == [0, 1, 2, 3, 4, 5]
    assert visible_keys(5, 2, 0) == [4, 5] and visible_keys(5, 2, 2) == [0, 1, 4, 5]
    assert visible_keys(5, 1, 9) == [0, 1, 2, 3, 4, 5] and visible_keys(0, 4, 2) == [0]


@pytest.mark.parametrize("window,sinks", [(0, 0), (4, 0), (5, 2), (100, 3), (3, 50)])
def test_equals_dense_masked_attention(window, sinks):
    g = torch.Generator().manual_seed(3)
    L, H, KV, D, page = 23, 6, 2, 8, 5
    k, v = (torch.randn(L, KV, D, generator=g, dtype=torch.float64) for _ in range(2))
    q = torch.randn(1, H, D, generator=g, dtype=torch.float64)
    order = torch.randperm(7, generator=g)
    table = torch.full((3, 6), -1)
    table[2, :5] = order[:5]
    kc, vc = torch.zeros(7, page, KV, D, dtype=torch.float64), torch.zeros(7, page, KV, D, dtype=torch.float64)
    for j in range(L):
        kc[table[2, j // page], j % page], vc[table[2, j // page], j % page] = k[j], v[j]
    out, lse, mass, _ = draft_attention(q, kc, vc, table, [2], [L - 1], window, sinks, 0.3, torch.zeros(1, H, D), torch.zeros(1, H))
    mask = torch.tensor([j in visible_keys(L - 1, window, sinks) for j in range(L)])
    ref = torch.nn.functional.scaled_dot_product_attention(
        q[0][:, None, :], k.transpose(0, 1).repeat_interleave(3, 0), v.transpose(0, 1).repeat_interleave(3, 0),
        attn_mask=mask[None, None, :].expand(H, 1, L), scale=0.3)[:, 0]
    assert torch.allclose(out[0], ref, atol=1e-12) and bool((mass[0] + 1e-12 >= out[0].abs()).all())
    s = 0.3 * torch.einsum("hd,lhd->hl", q[0], k.repeat_interleave(3, 1)).masked_fill(~mask, -math.inf)
    assert torch.allclose(lse[0], torch.logsumexp(s, -1))


def test_plans(lib):
    c = _cache(n_kv_heads=2, page_stride=16 * 128, token_stride=128)
    plan = B.DraftPlan()

    def make(n=4, h=8, cache=c, window=0, sinks=0, sms=152):
        return lib.ddtree_draft_attention_plan(n, h, ctypes.addressof(cache) if cache else None, window, sinks, sms, ctypes.addressof(plan))
    for h, tile in ((2, 16), (32, 16), (34, 32), (64, 32), (66, 64), (128, 64)):
        assert make(h=h) == 0 and plan.row_tile == tile and plan.n_heads == h
        assert B.ddtree_draft_attention_workspace_size(plan) == plan.workspace_bytes and plan.workspace_bytes % 256 == 0
    for dim in (128, 256):
        wide = _cache(n_kv_heads=2, head_dim=dim, head_stride=dim, token_stride=2 * dim, page_stride=32 * dim)
        for h, tile in ((32, 16), (34, 64), (128, 64)):
            assert make(h=h, cache=wide) == 0 and plan.row_tile == tile
    assert make(n=4096) == 0 and make(sinks=2 ** 31 - 1, window=1) == 0
    for bad in (dict(n=0), dict(n=4097), dict(h=0), dict(h=7), dict(h=130), dict(cache=None), dict(window=-1), dict(sinks=-1),
                dict(sms=-1), dict(sms=4097)):
        assert make(**bad) == B.DDTREE_EINVAL, bad
    for bad in BAD_CACHES:
        assert make(cache=_cache(**bad)) == B.DDTREE_EINVAL, bad
    assert lib.ddtree_draft_attention_workspace_size(None) == 0


def test_call_refusals(lib):
    c = _cache()
    plan = B.DraftPlan()
    assert lib.ddtree_draft_attention_plan(4, 8, ctypes.addressof(c), 0, 0, 152, ctypes.addressof(plan)) == 0
    ok = dict(plan=ctypes.addressof(plan), q=P, cache=ctypes.addressof(c), table=P, rows=4, stride=8, trows=None, pos=P, scale=0.1,
              out=Q, lse=P, ws=P, wsb=plan.workspace_bytes)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.ddtree_draft_attention(*[a[k] for k in ok], None)
    for bad in (dict(plan=None), dict(q=None), dict(q=OFF), dict(cache=None), dict(table=None), dict(table=ODD), dict(rows=0),
                dict(rows=3), dict(stride=0), dict(trows=ODD), dict(pos=None), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(out=None), dict(out=OFF), dict(out=P), dict(lse=ODD), dict(ws=None), dict(ws=OFF)):
        assert call(**bad) == B.DDTREE_EINVAL, bad
    assert call(wsb=plan.workspace_bytes - 1) == B.DDTREE_EWORKSPACE
    for kw in (dict(head_dim=128, head_stride=128, token_stride=256), dict(n_kv_heads=4), dict(page_size=8), dict(dtype=1)):
        other = _cache(**kw)
        assert call(cache=ctypes.addressof(other)) == B.DDTREE_EINVAL, kw
    for field, value in (("row_tile", 32), ("tile_keys", 8), ("n_shares", 0), ("workspace_bytes", 0), ("q_stride", 504), ("q_stride", 516),
                         ("out_stride", 8), ("n_heads", 7), ("window", -1)):
        p = B.DraftPlan.from_buffer_copy(plan)
        setattr(p, field, value)
        assert call(plan=ctypes.addressof(p)) == B.DDTREE_EINVAL, field
