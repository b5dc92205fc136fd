"""The 4-bit latent cache's and its pages' entry points on the host: status codes before any HIP call, and the
binding's refusals.  No GPU."""

import ctypes
import os

import pytest
import torch

from gated_delta_rule_04_amd import kda, mla
from oracle import mla_fp4 as orc4

OK, NULL, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5
P = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x1008)

pytestmark = pytest.mark.skipif(not os.path.exists(kda.LIB_PATH), reason="libkda.so not built")


def test_row_bytes():
    for R in (128, 256, 512):
        for Dr in (0, 64):
            assert kda.lib().kda_mla_fp4_row_bytes(R, Dr) == orc4.row_bytes(R, Dr) == mla.fp4_row_bytes(R, Dr)
    assert len({orc4.row_bytes(R, Dr) for R in (128, 512) for Dr in (0, 64)}) == 4
    for R, Dr in ((64, 0), (512, 32), (-128, 0), (384, 64)):
        assert kda.lib().kda_mla_fp4_row_bytes(R, Dr) == 0
        with pytest.raises(ValueError):
            mla.fp4_row_bytes(R, Dr)


def test_append_validation():
    def call(c=P, w=None, eps=1e-6, rope=P, num_pos=8, pos=P, slots=P, cache=P, pages=4, page=16, q_pe=P, q=P, T=3, H=2,
             R=512, Dr=64, dt=1):
        return kda.lib().kda_mla_cache_append_fp4(c, w, eps, rope, num_pos, 0, pos, slots, cache, pages, page, q_pe, q, T,
                                                  H, R, Dr, dt, None)

    assert call(dt=9) == DTYPE and call(dt=0) == UNSUPPORTED and call(dt=2) == UNSUPPORTED
    assert call(T=-1) == SHAPE and call(pages=-1) == SHAPE and call(page=0) == SHAPE
    assert call(eps=-1.0) == SHAPE and call(eps=float("nan")) == SHAPE
    assert call(pages=1 << 20, page=1 << 12) == SHAPE and call(H=0) == SHAPE and call(num_pos=0) == SHAPE
    for R, Dr in ((64, 64), (512, 32), (384, 0), (-128, 0)):
        assert call(R=R, Dr=Dr) == UNSUPPORTED
    for miss in ("c", "pos", "slots", "cache", "q"):
        assert call(**{miss: None}) == NULL, miss
    for odd in ("c", "w", "rope", "cache", "q_pe", "q"):
        assert call(**{odd: ODD}) == UNSUPPORTED, odd
    assert call(T=0, c=None, slots=None, cache=None) == OK


def test_gather_validation():
    def call(cache=P, table=P, cu=P, starts=None, rows=P, N=2, T=9, R=512, Dr=64, pages=4, page=16, per=3, dt=1):
        return kda.lib().kda_mla_cache_gather_fp4(cache, table, cu, starts, rows, N, T, R, Dr, pages, page, per, dt, None)

    assert call(dt=9) == DTYPE and call(dt=0) == UNSUPPORTED
    assert call(N=-1) == SHAPE and call(N=65537) == SHAPE and call(T=-1) == SHAPE and call(page=0) == SHAPE
    assert call(pages=-1) == SHAPE and call(per=-1) == SHAPE and call(pages=1 << 20, page=1 << 12) == SHAPE
    assert call(per=1 << 20, page=1 << 12) == SHAPE and call(T=(1 << 25) + 1) == SHAPE
    for R, Dr in ((64, 64), (512, 32), (384, 0)):
        assert call(R=R, Dr=Dr) == UNSUPPORTED
    for miss in ("cache", "table", "cu", "rows"):
        assert call(**{miss: None}) == NULL, miss
    assert call(cache=ODD) == UNSUPPORTED and call(rows=ODD) == UNSUPPORTED
    assert call(T=0, rows=None) == OK and call(N=0, cu=None) == OK


def test_paged_validation():
    def call(q=P, cache=P, table=P, lens=P, cu=None, o=P, lse=P, N=2, Tq=2, H=4, R=512, Dr=64, pages=8, page=16, per=4,
             scale=0.1, dt=1, ws=P, wsb=None):
        L = kda.lib()
        if wsb is None:
            wsb = L.kda_mla_paged_fp4_workspace_bytes(N, Tq, H, R, Dr, page, per, dt)
        return L.kda_mla_paged_attn_fp4(q, cache, table, lens, cu, o, lse, N, Tq, H, R, Dr, pages, page, per, scale, dt, ws,
                                        wsb, None)

    assert call(dt=9) == DTYPE and call(dt=0) == UNSUPPORTED and call(dt=2) == UNSUPPORTED
    assert call(N=-1) == SHAPE and call(H=0) == SHAPE and call(H=1025) == SHAPE and call(page=0) == SHAPE
    assert call(pages=-1) == SHAPE and call(per=-1) == SHAPE and call(Tq=3) == SHAPE and call(N=65537, Tq=65537) == SHAPE
    assert call(pages=1 << 20, page=1 << 12) == SHAPE and call(per=1 << 20, page=1 << 12) == SHAPE
    assert call(Tq=1 << 24, H=4, cu=P) == SHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=scale) == SHAPE
    for R, Dr in ((64, 64), (512, 32), (384, 0)):
        assert call(R=R, Dr=Dr) == UNSUPPORTED
    for miss in ("q", "cache", "table", "lens", "o"):
        assert call(**{miss: None}) == NULL, miss
    for odd in ("q", "cache", "o", "lse"):
        assert call(**{odd: ODD}) == UNSUPPORTED, odd
    need = kda.lib().kda_mla_paged_fp4_workspace_bytes(2, 2, 4, 512, 64, 16, 4, 1)
    if need:
        assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
        assert call(ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert call(N=0, Tq=0, q=None, cache=None, table=None, lens=None, o=None) == OK and call(cu=P, Tq=0, q=None) == OK
    assert kda.lib().kda_mla_paged_fp4_workspace_bytes(2, 2, 4, 100, 0, 16, 4, 1) == 0


def test_plan_and_release_validation():
    L = kda.lib()

    def plan(new=P, lens=P, table=P, free=P, count=P, F=5, cu=P, pos=P, slots=P, kv=P, out=P, left=P, N=2, T=9, page=16,
             per=3, ws=P, wsb=None):
        wsb = L.kda_mla_cache_plan_workspace_bytes(N) if wsb is None else wsb
        return L.kda_mla_cache_plan(new, lens, table, free, count, F, cu, pos, slots, kv, out, left, N, T, page, per, ws, wsb,
                                    None)

    def release(done=P, lens=P, table=P, free=P, count=P, F=5, out=P, left=P, N=2, page=16, per=3, ws=P, wsb=None):
        wsb = L.kda_mla_cache_release_workspace_bytes(N) if wsb is None else wsb
        return L.kda_mla_cache_release(done, lens, table, free, count, F, out, left, N, page, per, ws, wsb, None)

    for call, names in ((plan, ("new", "lens", "table", "free", "count", "cu", "pos", "slots", "kv", "out", "left")),
                        (release, ("done", "lens", "table", "free", "count", "out", "left"))):
        assert call(N=-1) == SHAPE and call(N=65537) == SHAPE and call(page=0) == SHAPE and call(per=-1) == SHAPE
        assert call(F=-1) == SHAPE and call(per=1 << 20, page=1 << 12) == SHAPE
        for miss in names:
            assert call(**{miss: None}) == NULL, miss
        assert call(ws=None) == WORKSPACE and call(wsb=7) == WORKSPACE and call(ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert plan(T=-1) == SHAPE and plan(T=(1 << 27) + 1) == SHAPE
    assert L.kda_mla_cache_plan_workspace_bytes(65537) == 0 and L.kda_mla_cache_release_workspace_bytes(-1) == 0


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


I32, U8 = torch.int32, torch.uint8


def test_binding_refusals():
    c, pos, slots, cache = z(5, 576), z(5, dtype=I32), z(5, dtype=I32), z(4, 16, 400, dtype=U8)
    with pytest.raises(ValueError, match="GPU"):
        mla.cache_append_fp4(c, pos, slots, cache, 512)
    with pytest.raises(ValueError):
        mla.cache_append_fp4(c, pos, slots, z(4, 16, 576, dtype=U8), 512)
    with pytest.raises(TypeError):
        mla.cache_append_fp4(c, pos, slots, z(4, 16, 400), 512)
    with pytest.raises(ValueError):
        mla.cache_append_fp4(c, pos, slots, cache, 500)
    with pytest.raises(ValueError):
        mla.cache_append_fp4(c, pos, slots[:4], cache, 512)
    q, table, lens = z(3, 2, 576), z(3, 2, dtype=I32), z(3, dtype=I32)
    with pytest.raises(ValueError, match="GPU"):
        mla.paged_attn_fp4(q, cache, table, lens, 512, 0.1)
    with pytest.raises(ValueError):
        mla.paged_attn_fp4(q, z(4, 16, 272, dtype=U8), table, lens, 512, 0.1)
    with pytest.raises(TypeError):
        mla.paged_attn_fp4(q, z(4, 16, 400), table, lens, 512, 0.1)
    with pytest.raises(ValueError):
        mla.paged_attn_fp4(z(2, 2, 576), cache, table, lens, 512, 0.1)
    cu = z(4, dtype=I32)
    with pytest.raises(ValueError, match="GPU"):
        mla.cache_gather_fp4(cache, table, cu, 7, 512)
    with pytest.raises(ValueError):
        mla.cache_gather_fp4(cache, table, cu, 7, 256)
    with pytest.raises(ValueError):
        mla.cache_gather_fp4(cache, table, cu[:3], 7, 512)
    with pytest.raises(ValueError):
        mla.cache_gather_fp4(cache, table, cu, -1, 512)
    with pytest.raises(TypeError):
        mla.cache_gather_fp4(cache, table, cu.long(), 7, 512)
    with pytest.raises(ValueError):
        mla.cache_gather_fp4(cache, table, cu, 7, 512, out=z(7, 512))
    free, count = z(9, dtype=I32), z(1, dtype=I32)
    with pytest.raises(ValueError, match="GPU"):
        mla.cache_plan(lens, lens, table, free, count, 16, 5)
    with pytest.raises(ValueError):
        mla.cache_plan(lens[:2], lens, table, free, count, 16, 5)
    with pytest.raises(TypeError):
        mla.cache_plan(lens.long(), lens, table, free, count, 16, 5)
    with pytest.raises(ValueError):
        mla.cache_plan(lens, lens, table, free, count, 16, -5)
    with pytest.raises(ValueError):
        mla.cache_plan(lens, lens, table, free, z(2, dtype=I32), 16, 5)
    with pytest.raises(ValueError):
        mla.cache_plan(lens, lens, table, free, count, 16, 5, out={"slots": z(4, dtype=I32)})
    with pytest.raises(ValueError, match="GPU"):
        mla.cache_release(z(3, dtype=torch.bool), lens, table, free, count, 16)
    with pytest.raises(TypeError):
        mla.cache_release(lens, lens, table, free, count, 16)
