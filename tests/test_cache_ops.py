"""The cache operators' host side: the rotary table and every refusal that
needs no GPU (CPU only).  Pointers here are made up: a refused call launches
nothing and reads nothing through them."""
import ctypes
import math

import pytest
import torch

import varlen_gqa_split_b200 as vg

OK, INVALID, UNSUPPORTED, NULL, ALIGNMENT, BAD_PLAN = 0, -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def L():
    from varlen_gqa_split_b200 import build
    build.build()
    return vg.lib()


def _create(L, D=8, n=4, axes=2, freq=None, axis=None, layout=0, scale=1.0):
    h = ctypes.c_void_p()
    f = (ctypes.c_double * max(n, 1))(*(freq if freq is not None else [1.0] * n))
    a = (ctypes.c_int32 * max(n, 1))(*(axis if axis is not None else [0] * n))
    return L.attn_rope_create(ctypes.byref(h), D, n, axes, f, a, layout, scale), h


@pytest.mark.parametrize("kw", [dict(D=1, n=1), dict(D=258, n=4), dict(n=0), dict(D=7, n=4), dict(axes=0),
                                dict(axes=9), dict(layout=2), dict(layout=-1), dict(scale=math.inf),
                                dict(scale=math.nan), dict(freq=[1.0, math.nan, 1.0, 1.0]),
                                dict(freq=[math.inf, 1.0, 1.0, 1.0]), dict(axis=[0, 1, 2, 0]),
                                dict(axis=[0, -1, 0, 0])])
def test_rope_create_refusals(L, kw):
    rc, h = _create(L, **kw)
    assert rc == INVALID and not h.value


def test_rope_create_nulls_and_destroy(L):
    f, a = (ctypes.c_double * 4)(), (ctypes.c_int32 * 4)()
    h = ctypes.c_void_p()
    assert L.attn_rope_create(None, 8, 4, 1, f, a, 0, 1.0) == NULL
    assert L.attn_rope_create(ctypes.byref(h), 8, 4, 1, None, a, 0, 1.0) == NULL
    assert L.attn_rope_create(ctypes.byref(h), 8, 4, 1, f, None, 0, 1.0) == NULL
    rc, h = _create(L, D=256, n=128, axes=8)
    assert rc == OK and h.value
    L.attn_rope_destroy(h)
    L.attn_rope_destroy(h)                                   # already gone, unknown, NULL: ignored
    L.attn_rope_destroy(0x1234)
    L.attn_rope_destroy(None)
    assert _apply(L, h) == BAD_PLAN and _apply(L, 0x1234) == BAD_PLAN


def _apply(L, h, dtype=0, x=0x10000, xs=16, T=4, H=2, pos=0x900000, ps=4, grad=0, out=0x20000, os_=16):
    return L.attn_rope_apply(h, dtype, x, xs, T, H, pos, ps, grad, out, os_, None)


def test_rope_apply_refusals(L):
    rc, h = _create(L)                                       # D = 8, two axes
    assert rc == OK
    assert _apply(L, None) == NULL
    for name in ("x", "pos", "out"):
        assert _apply(L, h, **{name: None}) == NULL
    assert _apply(L, h, dtype=3) == UNSUPPORTED
    assert _apply(L, h, dtype=-1) == UNSUPPORTED
    assert _apply(L, h, T=-1) == INVALID
    assert _apply(L, h, T=1 << 31, ps=1 << 31) == INVALID
    assert _apply(L, h, H=0) == INVALID
    assert _apply(L, h, xs=15) == INVALID                    # less than a token's heads
    assert _apply(L, h, os_=15) == INVALID
    assert _apply(L, h, ps=3) == INVALID                     # axes overlap
    assert _apply(L, h, x=0x10001) == ALIGNMENT
    assert _apply(L, h, dtype=2, out=0x20002) == ALIGNMENT
    assert _apply(L, h, pos=0x900002) == ALIGNMENT
    # overlaps other than x itself: shifted by a row, by half a row, another stride
    assert _apply(L, h, out=0x10000 + 32) == INVALID
    assert _apply(L, h, out=0x10000 + 16) == INVALID
    assert _apply(L, h, out=0x10000, os_=24) == INVALID
    assert _apply(L, h, x=0x10000, xs=40, out=0x10000 + 2 * 16 - 2, os_=40) == INVALID
    assert _apply(L, h, T=0) == OK                           # nothing to do, nothing launched
    L.attn_rope_destroy(h)


def test_plan_entry_points_refuse_unknown_plans(L):
    p = 0x10000
    cache = (1024, 256, 16, 4, p, 8)
    for plan in (None, 0x1234):
        assert L.attn_append_paged(plan, None, p, 256, p, 256, p, 256, 4, p, 4, p, p, p, *cache, p, p, None) == BAD_PLAN
        assert L.attn_key_weights(plan, p, 4, p, 256, 8, p, p, p, 1.0, p, p, 64, None, None, None) == BAD_PLAN
        assert L.attn_key_weights_paged(plan, p, 4, p, *cache, p, p, p, 1.0, p, p, 64, None, None, None) == BAD_PLAN
        assert L.attn_evict_paged(plan, p, p, p, p, 0, 0, p, p, 64, p, p, *cache, p, p, None) == BAD_PLAN


def test_rope_table_and_binding_checks(L):
    freqs, axes = vg.rope_table(8, (2, 3, 3), base=1e4)
    assert axes == [0, 0, 1, 1, 1, 2, 2, 2]
    assert freqs == [1e4 ** (-i / 8) for i in range(8)]
    freqs, axes = vg.rope_table(6, (2, 4), base=100.0, restart=True)
    assert freqs == [100.0 ** (-i / 2) for i in range(2)] + [100.0 ** (-i / 4) for i in range(4)]
    with pytest.raises(ValueError):
        vg.rope_table(8, (2, 3))
    with pytest.raises(ValueError):
        vg.Rope(16, [1.0] * 8, [0] * 7)
    with pytest.raises(ValueError):
        vg.Rope(16, [1.0] * 8, layout="thirds")
    with pytest.raises(vg.AttnError):
        vg.Rope(16, [1.0] * 9)
    r = vg.Rope(16, *vg.rope_table(8, (4, 4)))
    assert r.n_axes == 2
    r.close()
    with pytest.raises(vg.AttnError):
        r.apply(torch.zeros(1, 1, 16), torch.zeros(2, 1, dtype=torch.int32))
