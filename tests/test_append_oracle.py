"""Pins of the append oracle, the rotation's host set-up, and the entry points'
host-side refusals (no GPU)."""
import ctypes
import math

import pytest
import torch

from oracle import append_oracle as A
from speculative_decode_tree_gb300 import binding as B


@pytest.fixture(scope="module")
def lib():
    from speculative_decode_tree_gb300.build import build
    build()
    return B.library()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_pins(interleaved):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 3, 24, generator=g, dtype=torch.float64)
    f = A.frequencies(16, 10000.0)
    zero = torch.zeros(5, dtype=torch.int32)
    assert torch.equal(A.rotate(x, zero, f, interleaved), x)
    pos = torch.tensor([0, 1, 7, 1000, 99999], dtype=torch.int32)
    y = A.rotate(x, pos, f, interleaved)
    assert torch.allclose(A.pair_lengths(y, 8, interleaved), A.pair_lengths(x, 8, interleaved))
    assert torch.equal(y[..., 16:], x[..., 16:])
    # A rotation by p and one by q give a product that depends on p - q alone.
    a, b = x[:1].expand(5, 3, 24), x[1:2].expand(5, 3, 24)
    dots = [(A.rotate(a, pos + s, f, interleaved) * A.rotate(b, pos + s + 11, f, interleaved)).sum(-1) for s in (0, 5)]
    assert torch.allclose(dots[0], dots[1]) and torch.allclose(dots[0][0], dots[0][4])


def test_a_worked_pair():
    x = torch.tensor([[[1.0, 0.0]]])
    y = A.rotate(x, torch.tensor([2]), A.frequencies(2, 10000.0), True)
    assert torch.allclose(y, torch.tensor([[[math.cos(2.0), math.sin(2.0)]]], dtype=torch.float64))


@pytest.mark.parametrize("rot,theta,scaling,factor,original", [
    (64, 10000.0, A.PLAIN, 1.0, 1), (128, 500000.0, A.LINEAR, 8.0, 1), (64, 10000.0, A.YARN, 40.0, 4096),
    (256, 1e6, A.YARN, 4.0, 32768), (16, 10000.0, A.YARN, 16.0, 8), (2, 10.0, A.PLAIN, 1.0, 1)])
def test_rope_init_matches_the_frequencies(lib, rot, theta, scaling, factor, original):
    r = B.ddtree_rope_init(rot, theta=theta, scaling=scaling, factor=factor, original_positions=original)
    want = A.frequencies(rot, theta, scaling, factor, original)
    got = torch.tensor([t / 2.0 ** 64 * 2 * math.pi for t in r.turns[:rot // 2]], dtype=torch.float64)
    # The fraction of a turn is cut below 2^-64: at most 2 pi 2^-64 radians, whatever the frequency (a slow pair's
    # relative error is larger for it: 2.8e-7 radians are 8e11 units).  Both sides take pow, a few products and a ramp
    # in 64 bits besides: some 2^-52 each, theta^x's exponent magnified by ln theta.
    assert bool(((got - want).abs() <= 2 * math.pi * 2.0 ** -64 + 1e-13 * want).all())
    assert list(r.turns[rot // 2:]) == [0] * (128 - rot // 2)
    assert r.mscale == pytest.approx(0.1 * math.log(factor) + 1 if scaling == A.YARN else 1.0, rel=1e-7)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(theta=1.0), dict(theta=float("nan")),
                                dict(theta=float("inf")), dict(scaling=3), dict(scaling=1, factor=0.5),
                                dict(scaling=1, factor=float("inf")), dict(scaling=2, factor=2.0, original_positions=0),
                                dict(scaling=2, factor=2.0, beta_slow=0.0), dict(scaling=2, factor=2.0, beta_fast=1.0),
                                dict(mscale=-1.0), dict(mscale=float("nan"))])
def test_rope_init_refusals(lib, kw):
    with pytest.raises(B.DDTreeError) as e:
        B.ddtree_rope_init(kw.pop("rot_dim", 64), **{"theta": 10000.0, **kw})
    assert e.value.code == B.DDTREE_EINVAL


P, Q, ODD, OFF = (ctypes.c_void_p(x) for x in (1 << 12, 1 << 13, (1 << 12) + 2, (1 << 12) + 8))


def test_mla_append_refusals(lib):
    rope = B.ddtree_rope_init(64, theta=1e4)
    small = B.ddtree_rope_init(32, theta=1e4)
    ok = dict(n=4, h=8, rope=ctypes.addressof(rope), kv=P, kvs=576, w=P, eps=1e-6, q=P, qt=512, qh=64, pos=P, slots=P, pool=P,
              rows=100, o=Q, ot=512, oh=64, status=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.ddtree_mla_append(*[a[k] for k in ok], None)
    for bad in (dict(n=-1), dict(n=(1 << 24) + 1), dict(h=-1), dict(h=129), dict(rope=None), dict(rope=ctypes.addressof(small)),
                dict(kv=None), dict(kv=OFF), dict(kvs=568), dict(kvs=580), dict(w=OFF), dict(eps=-1.0),
                dict(eps=float("nan")), dict(q=None), dict(q=OFF), dict(qt=63), dict(qh=65), dict(pos=None), dict(pos=ODD),
                dict(slots=None), dict(slots=ODD), dict(pool=None), dict(pool=OFF), dict(rows=0), dict(rows=1 << 31),
                dict(o=None), dict(o=OFF), dict(ot=0), dict(oh=12), dict(o=P, ot=1024), dict(status=ODD)):
        assert call(**bad) == B.DDTREE_EINVAL, bad


def _cache(**kw):
    d = dict(k=1 << 12, v=1 << 13, n_pages=10, page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64, page_size=16,
             n_kv_heads=2, head_dim=64, dtype=0)
    d.update(kw)
    return B._CacheStruct(*[d[f] for f, _ in B._CacheStruct._fields_])


BAD_CACHES = [dict(k=None), dict(v=(1 << 12) + 8), dict(n_pages=0), dict(n_pages=(1 << 31) // 16), dict(page_stride=12),
              dict(token_stride=0), dict(head_stride=32), dict(page_size=0), dict(page_size=65537), dict(n_kv_heads=0),
              dict(n_kv_heads=129), dict(head_dim=96), dict(dtype=2)]


def test_no_tokens_need_no_pointers(lib):
    rope, cache = B.ddtree_rope_init(64, theta=1e4), _cache()
    rc = lib.ddtree_mla_append(0, 8, ctypes.addressof(rope), None, 0, None, 0.0, None, 0, 0, None, None, P, 9, None, 0, 0, None, None)
    assert rc in (B.DDTREE_OK, B.DDTREE_EUNSUPPORTED)  # without a device there is nothing to run on
    rc = lib.ddtree_draft_append(0, 8, ctypes.addressof(cache), ctypes.addressof(rope), None, 0, None, 0, None, 0, None, None, 0.0,
                                 None, None, None, 0, None, None)
    assert rc in (B.DDTREE_OK, B.DDTREE_EUNSUPPORTED)
    assert lib.ddtree_mla_append(0, 8, ctypes.addressof(rope), None, 0, None, 0.0, None, 0, 0, None, None, None, 9, None, 0, 0, None,
                                 None) == B.DDTREE_EINVAL


def test_draft_append_refusals(lib):
    rope = B.ddtree_rope_init(64, theta=1e4)
    big = B.ddtree_rope_init(128, theta=1e4)
    odd = B.ddtree_rope_init(24, theta=1e4)
    cache = _cache()
    ok = dict(n=4, h=8, cache=ctypes.addressof(cache), rope=ctypes.addressof(rope), q=P, qs=512, k=P, ks=128, v=P, vs=128, wq=P,
              wk=None, eps=1e-6, pos=P, slots=P, o=Q, os=512, status=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.ddtree_draft_append(*[a[k] for k in ok], None)
    for bad in (dict(n=-1), dict(n=(1 << 24) + 1), dict(h=513), dict(cache=None), dict(rope=None), dict(rope=ctypes.addressof(big)),
                dict(rope=ctypes.addressof(odd)), dict(q=None), dict(q=OFF), dict(qs=504), dict(k=None), dict(ks=120), dict(v=OFF),
                dict(vs=132), dict(wq=OFF), dict(wk=OFF), dict(eps=-1.0), dict(pos=None), dict(slots=ODD), dict(o=None),
                dict(os=0), dict(o=P, os=1024), dict(status=ODD)):
        assert call(**bad) == B.DDTREE_EINVAL, bad
    for bad in BAD_CACHES:
        c = _cache(**bad)
        assert call(cache=ctypes.addressof(c)) == B.DDTREE_EINVAL, bad
