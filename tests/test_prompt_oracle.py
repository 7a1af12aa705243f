"""Pins of the prompt oracle and refusals of the entry point (no GPU)."""
import ctypes
import math

import pytest
import torch

from oracle import draft_attention, prompt_attention
from oracle.prompt_oracle import visible
from speculative_decode_tree_gb300 import binding as B
from test_append_oracle import ODD, OFF, P, Q


def _inputs(lens, ctx, heads, kvh, dim=8, seed=0):
    g = torch.Generator().manual_seed(seed)
    qp, kp = [0], [0]
    for n, c in zip(lens, ctx):
        qp.append(qp[-1] + n)
        kp.append(kp[-1] + n + c)
    q, k, v = (torch.randn(r, h, dim, generator=g, dtype=torch.float64) for r, h in ((qp[-1], heads), (kp[-1], kvh), (kp[-1], kvh)))
    return q, k, v, qp, kp


def test_whole_prompts_equal_causal_sdpa():
    q, k, v, qp, kp = _inputs([7, 1, 4], [0, 0, 0], 4, 2)
    out, _, _, _ = prompt_attention(q, k, v, qp, kp, 0, 0, 0.3, torch.zeros_like(q), torch.zeros(12, 4))
    for b in range(3):
        s = slice(qp[b], qp[b + 1])
        ref = torch.nn.functional.scaled_dot_product_attention(q[s].transpose(0, 1), k[s].transpose(0, 1).repeat_interleave(2, 0),
                                                               v[s].transpose(0, 1).repeat_interleave(2, 0), is_causal=True, scale=0.3)
        assert torch.allclose(out[s].transpose(0, 1), ref, atol=1e-12)


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (3, 2), (1, 5)])
def test_rows_are_those_of_the_one_token_attention(window, sinks):
    q, k, v, qp, kp = _inputs([5, 3], [4, 0], 2, 1, seed=1)
    out, lse, mass, terms = prompt_attention(q, k, v, qp, kp, window, sinks, 0.3, torch.zeros_like(q), torch.zeros(8, 2))
    for b in range(2):
        page = kp[b + 1] - kp[b]
        n = qp[b + 1] - qp[b]
        table = torch.zeros(n, 1, dtype=torch.int32)
        s = slice(qp[b], qp[b + 1])
        ref = draft_attention(q[s], k[None, kp[b]:kp[b + 1]], v[None, kp[b]:kp[b + 1]], table, None, list(range(page - n, page)), window, sinks,
                              0.3, torch.zeros(n, 2, 8), torch.zeros(n, 2))
        for x, y in zip((out, lse, mass, terms), ref):
            assert torch.allclose(x[s], y, atol=1e-12)


def test_more_queries_than_keys_and_values_that_are_no_numbers():
    assert visible(3, 1, 0, 0).tolist() == [[False], [False], [True]]
    q, k, v, qp, kp = _inputs([3], [0], 1, 1, seed=2)
    out, lse, _, _ = prompt_attention(q, k[:1], v[:1], [0, 3], [0, 1], 0, 0, 0.3, torch.ones_like(q), torch.ones(3, 1))
    assert out[:2].abs().max() == 0 and lse[:2].eq(-math.inf).all() and torch.allclose(out[2, 0], v[0, 0])
    v[1, 0, 2] = math.nan
    out, _, _, _ = prompt_attention(q, k, v, qp, kp, 0, 0, 0.3, torch.ones_like(q), torch.ones(3, 1))
    assert torch.isnan(out).nonzero().tolist() == [[1, 0, 2], [2, 0, 2]]


@pytest.fixture(scope="module")
def lib():
    from speculative_decode_tree_gb300.build import build
    build()
    return B.library()


def test_plan_and_refusals(lib):
    ok = dict(batch=3, q=100, k=120, h=8, kvh=2, dim=64, dtype=torch.bfloat16, window=0, n_sinks=0)

    def make(**kw):
        a = dict(ok, **kw)
        return B.ddtree_prompt_attention_plan(*[a[n] for n in list(ok)[:7]], window=a["window"], n_sinks=a["n_sinks"])
    for bad in (dict(batch=0), dict(batch=1025), dict(q=0), dict(k=0), dict(q=(1 << 24) + 1), dict(k=(1 << 24) + 1), dict(h=7), dict(h=0), dict(kvh=0),
                dict(h=130, kvh=2), dict(h=129, kvh=129), dict(dim=96), dict(window=-1), dict(n_sinks=-1)):
        with pytest.raises(B.DDTreeError) as e:
            make(**bad)
        assert e.value.code == B.DDTREE_EINVAL, bad
    with pytest.raises(TypeError):
        make(dtype=torch.float32)
    plan = make()
    assert 1 <= plan.tile_tokens <= 64 and plan.max_items == (100 // plan.tile_tokens + 3) * 2
    assert plan.workspace_bytes % 256 == 0 and plan.workspace_bytes >= 256 + 4 * plan.max_items
    assert lib.ddtree_prompt_attention_workspace_size(None) == 0
    far = ctypes.c_void_p(1 << 14)
    good = dict(plan=ctypes.addressof(plan), q=P, k=P, v=P, qi=P, ki=None, scale=0.1, out=Q, lse=None, ws=far, wsb=plan.workspace_bytes)

    def call(**kw):
        a = dict(good, **kw)
        return lib.ddtree_prompt_attention(*[a[n] for n in good], None)
    for bad in (dict(plan=None), dict(q=None), dict(q=OFF), dict(k=None), dict(k=OFF), dict(v=None), dict(v=OFF), dict(qi=None), dict(qi=ODD),
                dict(ki=ODD), dict(scale=float("nan")), dict(scale=3e38), dict(out=None), dict(out=OFF), dict(out=P), dict(lse=ODD), dict(ws=None),
                dict(ws=OFF)):
        assert call(**bad) == B.DDTREE_EINVAL, bad
    assert call(wsb=plan.workspace_bytes - 1) == B.DDTREE_EWORKSPACE
    for field, value in (("tile_tokens", 1), ("max_items", 5), ("workspace_bytes", 256), ("q_stride", 504), ("q_stride", 516), ("k_stride", 120),
                         ("v_stride", 1 << 33), ("out_stride", 8), ("wait_limit_us", -1), ("batch", 4)):
        kept = getattr(plan, field)
        setattr(plan, field, value)
        assert call() == B.DDTREE_EINVAL, field
        setattr(plan, field, kept)


def test_workspace_of_long_sums(lib):
    # Room for sums that go on beyond 16,384 keys, in plans of more than 32,768, and none where no row sees as many.
    def extra(q, k, h, kvh, dim, window=0, n_sinks=0, batch=1):
        p = B.ddtree_prompt_attention_plan(batch, q, k, h, kvh, dim, torch.bfloat16, window, n_sinks)
        return p.workspace_bytes - 256 - (4 * p.max_items + 255) // 256 * 256
    for dim in (64, 128, 256):
        assert extra(5000, 32768, 8, 2, dim) == 0 and extra(5000, 1 << 24, 8, 2, dim, window=30000, n_sinks=2000) == 0
        rows = 128 * (1 if dim == 256 else 2)
        assert extra(100000, 32769, 8, 2, dim) == extra(100000, 1 << 24, 8, 2, dim, 2 ** 31 - 1, 2 ** 31 - 1) == 160 * rows * dim * 4
        assert extra(100, 1 << 24, 8, 2, dim, window=4096, n_sinks=30000, batch=3) == (100 // 32 + 3) * 2 * 128 * dim * 4
