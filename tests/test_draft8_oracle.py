"""Pins of the 8-bit oracle and refusals of the 8-bit entry points (no GPU)."""
import ctypes

import pytest
import torch

from oracle import draft8_oracle as O
from speculative_decode_tree_gb300 import binding as B
from test_append_oracle import ODD, OFF, P, Q


def test_table_and_rounding_against_torchs_type():
    every = torch.arange(256, dtype=torch.uint8)
    theirs = every.view(torch.float8_e4m3fn).to(torch.float64)
    assert torch.equal(torch.nan_to_num(O.TABLE, nan=999.0), torch.nan_to_num(theirs, nan=999.0))
    good = every[~torch.isnan(O.TABLE)]
    assert torch.equal(O.codes_of(O.values(good)), good)
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(5000, generator=g) * 10.0 ** torch.randint(-4, 3, (5000,), generator=g), (O.TABLE[:126] + O.TABLE[1:127]).float() / 2,
                   torch.tensor([0.0, -0.0, 448.0, -448.0, 2.0 ** -10, 2.0 ** -11])]).clamp(-448, 448)
    assert torch.equal(O.codes_of(x), x.to(torch.float8_e4m3fn).view(torch.uint8))


def test_beyond_the_range():
    x = torch.tensor([449.0, 1e30, -1e30, float("inf"), -float("inf"), float("nan")])
    assert O.codes_of(x).tolist()[:5] == [126, 126, 254, 126, 254] and O.codes_of(x).tolist()[5] & 127 == 127


@pytest.mark.parametrize("top,scale", [(0.0, 1.0), (448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8), (1e-30, 2.0 ** -64), (1e38, 2.0 ** 96)])
def test_scales(top, scale):
    assert O.scale_for(top) == scale


def test_blocks_start_grow_and_keep():
    codes, scales = torch.zeros(1, 4, 1, 2, dtype=torch.uint8), torch.zeros(1, 2, 1, dtype=torch.float64)
    one = lambda *v: torch.tensor(v, dtype=torch.float64).view(1, 1, 2)  # noqa: E731
    O.write_rows(one(1.75, -1.0), codes, scales, 2, [0], [0])
    assert float(scales[0, 0, 0]) == 2.0 ** -8 and O.dequantised(codes, scales, 2)[0, 0, 0].tolist() == [1.75, -1.0]
    O.write_rows(one(0.5, 0.0), codes, scales, 2, [0], [1])        # fits: the scale stays
    assert float(scales[0, 0, 0]) == 2.0 ** -8
    O.write_rows(one(7.0, 0.0), codes, scales, 2, [0], [1])        # grows, the first row moves along
    assert float(scales[0, 0, 0]) == 2.0 ** -6 and O.dequantised(codes, scales, 2)[0, :2, 0].tolist() == [[1.75, -1.0], [7.0, 0.0]]
    O.write_rows(one(0.5, 0.0), codes, scales, 2, [0], [0])        # the first token again: afresh
    assert float(scales[0, 0, 0]) == 2.0 ** -9
    O.write_rows(one(0.5, 0.0), codes, scales, 2, [0, -1], [3])    # a block without a scale counts as new
    assert float(scales[0, 1, 0]) == 2.0 ** -9 and O.read_rows(codes, scales, 2, [3, -1], torch.full((2, 1, 2), 7.0)).tolist() == [[[0.5, 0.0]], [[7.0, 7.0]]]


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 2)])
def test_attention_equals_sdpa_over_the_values(window, sinks):
    g = torch.Generator().manual_seed(window)
    pages, page, kvh, d, block = 6, 4, 2, 8, 3
    k, v = (torch.randint(0, 120, (pages, page, kvh, d), generator=g).to(torch.uint8) for _ in range(2))
    ks, vs = (2.0 ** torch.randint(-3, 3, (pages, 2, kvh), generator=g).double() for _ in range(2))
    vs[4, 0, 1] = float("nan")  # tokens 0 to 2 of page 4, of one key head
    q, table = torch.randn(2, 4, d, generator=g), torch.tensor([[3, 1, 4], [0, 5, 2]], dtype=torch.int32)
    out, lse, _, _ = O.attention(q, k, v, ks, vs, block, table, [1, 0], [6, 9], window, sinks, 0.1, torch.zeros(2, 4, d), torch.zeros(2, 4))
    at = torch.arange(page) // block
    kx, vx = ((k if c is ks else v).view(torch.float8_e4m3fn).double() * c[:, at][..., None] for c in (ks, vs))
    for n, (row, pos) in enumerate(((1, 6), (0, 9))):
        kk, vv = (c[table[row].long()].reshape(3 * page, kvh, d) for c in (kx, vx))
        j = torch.arange(3 * page)
        seen = (j <= pos) & ((j > pos - window) | (j < sinks) | (window == 0))
        for h in range(4):
            here = seen & ~torch.isnan(vv[:, h // 2, 0])
            assert bool((here != seen).any()) == (row == 0 and h // 2 == 1)
            ref = torch.nn.functional.scaled_dot_product_attention(q[n, h].double()[None], kk[here, h // 2], vv[here, h // 2], scale=0.1)[0]
            assert torch.allclose(out[n, h], ref, rtol=1e-12)
            assert torch.allclose(lse[n, h], torch.logsumexp(0.1 * kk[here, h // 2] @ q[n, h].double(), 0), rtol=1e-12)


@pytest.fixture(scope="module")
def lib():
    from speculative_decode_tree_gb300.build import build
    build()
    return B.library()


def cache8(**kw):
    d = dict(k=1 << 12, v=1 << 13, k_scale=1 << 14, v_scale=1 << 15, n_pages=10, page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64,
             page_size=16, n_kv_heads=2, head_dim=64, block_tokens=8)
    d.update(kw)
    return B._Cache8Struct(*[d[f] for f, _ in B._Cache8Struct._fields_])


BAD_CACHES = [dict(k=None), dict(v=(1 << 12) + 8), dict(k_scale=None), dict(v_scale=(1 << 12) + 2), dict(n_pages=0),
              dict(n_pages=(1 << 31) // 16), dict(page_stride=24), dict(token_stride=0), dict(head_stride=48), dict(head_stride=72),
              dict(page_size=0), dict(page_size=65537), dict(n_kv_heads=0), dict(n_kv_heads=129), dict(head_dim=96),
              dict(block_tokens=0), dict(block_tokens=17), dict(page_size=128, block_tokens=65)]


def test_append_refusals(lib):
    rope = B.ddtree_rope_init(64, theta=1e4)
    big = B.ddtree_rope_init(128, theta=1e4)
    odd = B.ddtree_rope_init(24, theta=1e4)
    cache = cache8()
    ok = dict(n=4, h=8, dtype=0, cache=ctypes.addressof(cache), rope=ctypes.addressof(rope), q=P, qs=512, k=P, ks=128, v=P, vs=128, wq=P,
              wk=None, eps=1e-6, pos=P, slots=P, o=Q, os=512, status=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.ddtree_draft8_append(*[a[k] for k in ok], None)
    for bad in (dict(n=-1), dict(n=(1 << 24) + 1), dict(h=513), dict(dtype=2), dict(cache=None), dict(rope=None),
                dict(rope=ctypes.addressof(big)), dict(rope=ctypes.addressof(odd)), dict(q=None), dict(q=OFF), dict(qs=504), dict(k=None),
                dict(ks=120), dict(v=OFF), dict(vs=132), dict(wq=OFF), dict(wk=OFF), dict(eps=-1.0), dict(eps=float("nan")), dict(pos=None),
                dict(slots=ODD), dict(o=None), dict(os=0), dict(o=P, os=1024), dict(status=ODD)):
        assert call(**bad) == B.DDTREE_EINVAL, bad
    for bad in BAD_CACHES:
        c = cache8(**bad)
        assert call(cache=ctypes.addressof(c)) == B.DDTREE_EINVAL, bad
    assert lib.ddtree_draft8_append(0, 8, 0, ctypes.addressof(cache), ctypes.addressof(rope), None, 0, None, 0, None, 0, None, None, 0.0, None,
                                    None, None, 0, None, None) in (B.DDTREE_OK, B.DDTREE_EUNSUPPORTED)


def test_read_refusals(lib):
    cache = cache8()
    ok = dict(n=4, dtype=0, cache=ctypes.addressof(cache), slots=P, k=P, ks=128, v=Q, vs=128, status=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.ddtree_draft8_read(*[a[k] for k in ok], None)
    for bad in (dict(n=-1), dict(n=(1 << 24) + 1), dict(dtype=2), dict(cache=None), dict(slots=None), dict(slots=ODD), dict(k=None, v=None),
                dict(k=OFF), dict(v=OFF), dict(ks=120), dict(vs=132), dict(k=Q), dict(status=ODD)):
        assert call(**bad) == B.DDTREE_EINVAL, bad
    for bad in BAD_CACHES:
        c = cache8(**bad)
        assert call(cache=ctypes.addressof(c)) == B.DDTREE_EINVAL, bad
    assert lib.ddtree_draft8_read(0, 0, ctypes.addressof(cache), None, None, 0, None, 0, None, None) in (B.DDTREE_OK, B.DDTREE_EUNSUPPORTED)


def test_host_tensors_are_refused():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.uint8)
    s = torch.zeros(4, 2, 2)
    with pytest.raises(TypeError):
        B.Draft8Cache(k.float(), k.float(), s, s, 8)
    if not torch.cuda.is_available():
        with pytest.raises((TypeError, RuntimeError, AssertionError)):
            B.Draft8Cache(k, k, s, s, 8)


def test_attention_plan_and_refusals(lib):
    cache, plan = cache8(), B.Draft8Plan()
    make = lambda n=4, h=8, c=cache, dtype=0, w=0, s=0, sms=152: lib.ddtree_draft8_attention_plan(  # noqa: E731
        n, h, ctypes.addressof(c), dtype, w, s, sms, ctypes.addressof(plan))
    for kw in (dict(n=0), dict(n=4097), dict(h=7), dict(h=130), dict(h=0), dict(dtype=2), dict(w=-1), dict(s=-1), dict(sms=-1), dict(sms=4097)):
        assert make(**kw) == B.DDTREE_EINVAL, kw
    for bad in BAD_CACHES:
        assert make(c=cache8(**bad)) == B.DDTREE_EINVAL, bad
    assert make(h=128) == 0 and plan.row_tiles == 4
    assert make() == 0 and plan.row_tiles == 1 and plan.n_shares % 152 == 0 and plan.n_shares > 0
    assert B.ddtree_draft8_attention_workspace_size(plan) == plan.workspace_bytes > 0 and plan.workspace_bytes % 256 == 0
    ok = dict(plan=ctypes.addressof(plan), q=P, cache=ctypes.addressof(cache), table=P, rows=4, stride=8, of=None, pos=P, scale=0.1, out=Q,
              lse=None, ws=P, wsb=plan.workspace_bytes)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.ddtree_draft8_attention(*[a[k] for k in ok], None)
    for bad in (dict(plan=None), dict(q=None), dict(q=OFF), dict(cache=None), dict(table=None), dict(table=ODD), dict(rows=0), dict(rows=3),
                dict(stride=0), dict(of=ODD), dict(pos=None), dict(pos=ODD), dict(scale=float("nan")), dict(scale=3e38), dict(out=None),
                dict(out=OFF), dict(out=P), dict(lse=ODD), dict(ws=None), dict(ws=OFF)):
        assert call(**bad) == B.DDTREE_EINVAL, bad
    assert call(wsb=plan.workspace_bytes - 1) == B.DDTREE_EWORKSPACE
    for other in (dict(head_dim=128, page_stride=4096, token_stride=256, head_stride=128), dict(page_size=8), dict(block_tokens=4), dict(n_kv_heads=4)):
        assert call(cache=ctypes.addressof(cache8(**other))) == B.DDTREE_EINVAL, other
    for field, value in (("row_tiles", 2), ("tile_keys", 64), ("n_shares", 0), ("workspace_bytes", 256), ("q_stride", 8), ("out_stride", 516)):
        kept = getattr(plan, field)
        setattr(plan, field, value)
        assert call() == B.DDTREE_EINVAL, field
        setattr(plan, field, kept)
