"""The latent-attention entry points on the host: status codes before any HIP
call, and the binding's refusals.  No GPU."""

import ctypes
import os

import pytest
import torch

from gated_delta_rule_04_amd import kda, mla

OK, NULL, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5
P = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x1008)

needs_lib = pytest.mark.skipif(not os.path.exists(kda.LIB_PATH), reason="libkda.so not built")


@needs_lib
def test_append_validation():
    def call(c=P, w=None, eps=1e-6, rope=P, num_pos=8, pos=P, slots=P, cache=P, pages=4, page=16, q_pe=P, q=P, T=3, H=2,
             R=512, Dr=64, dt=1):
        return kda.lib().kda_mla_cache_append(c, w, eps, rope, num_pos, 0, pos, slots, cache, pages, page, q_pe, q, T, H,
                                              R, Dr, dt, None)

    assert call(dt=9) == DTYPE and call(dt=0) == UNSUPPORTED and call(dt=2) == UNSUPPORTED
    assert call(T=-1) == SHAPE and call(pages=-1) == SHAPE and call(page=0) == SHAPE
    assert call(eps=-1.0) == SHAPE and call(eps=float("nan")) == SHAPE
    assert call(pages=1 << 20, page=1 << 12) == SHAPE       # slots must fit an int
    assert call(H=0) == SHAPE and call(H=1025) == SHAPE and call(num_pos=0) == SHAPE
    for R, Dr in ((64, 64), (512, 32), (384, 0), (-128, 0)):
        assert call(R=R, Dr=Dr) == UNSUPPORTED
    assert call(Dr=0) == UNSUPPORTED and call(Dr=0, rope=None) == UNSUPPORTED   # nothing to rotate
    for miss in ("c", "pos", "slots", "cache", "q"):
        assert call(**{miss: None}) == NULL, miss
    for odd in ("c", "w", "rope", "cache", "q_pe", "q"):
        assert call(**{odd: ODD}) == UNSUPPORTED, odd
    assert call(T=(1 << 27) + 1) == SHAPE and call(T=1 << 27, H=64) == SHAPE     # threads of a launch fit 32 bits
    assert call(T=0, c=None, slots=None, cache=None) == OK


def paged(q=P, cache=P, table=P, lens=P, cu=None, o=P, lse=P, N=2, Tq=2, H=4, R=512, Dr=64, pages=8, page=16, per=4,
          scale=0.1, dt=1, ws=P, wsb=None):
    L = kda.lib()
    if wsb is None:
        wsb = L.kda_mla_paged_workspace_bytes(N, Tq, H, R, Dr, page, per, dt)
    return L.kda_mla_paged_attn(q, cache, table, lens, cu, o, lse, N, Tq, H, R, Dr, pages, page, per, scale, dt, ws, wsb,
                                None)


@needs_lib
def test_paged_validation():
    assert paged(dt=9) == DTYPE and paged(dt=0) == UNSUPPORTED and paged(dt=2) == UNSUPPORTED
    assert paged(N=-1) == SHAPE and paged(H=0) == SHAPE and paged(H=1025) == SHAPE and paged(page=0) == SHAPE
    assert paged(pages=-1) == SHAPE and paged(per=-1) == SHAPE
    assert paged(Tq=3) == SHAPE                              # one token a sequence without cu_seqlens
    assert paged(N=65537, Tq=65537) == SHAPE
    assert paged(pages=1 << 20, page=1 << 12) == SHAPE and paged(per=1 << 20, page=1 << 12) == SHAPE
    assert paged(Tq=1 << 24, H=4, cu=P) == SHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert paged(scale=scale) == SHAPE
    for R, Dr in ((64, 64), (512, 32), (384, 0)):
        assert paged(R=R, Dr=Dr) == UNSUPPORTED
    for miss in ("q", "cache", "table", "lens", "o"):
        assert paged(**{miss: None}) == NULL, miss
    for odd in ("q", "cache", "o", "lse"):
        assert paged(**{odd: ODD}) == UNSUPPORTED, odd
    assert paged(N=0, Tq=0, q=None, cache=None, table=None, lens=None, o=None) == OK
    assert paged(cu=P, Tq=0, q=None) == OK
    assert kda.lib().kda_mla_paged_workspace_bytes(2, 2, 4, 100, 0, 16, 4, 1) == 0


def _attn(fn, **kw):
    a = dict(q=P, kv=P, k_pe=P, o=P, lse=P, dout=P, dq=P, dkv=P, dk_pe=P, cu=None, N=2, B=2, T=64, H=3, Dn=128, Dr=64,
             Dv=128, scale=0.1, dt=1, ws=P, wsb=None)
    a.update(kw)
    L = kda.lib()
    sizes = [a[n] for n in ("N", "B", "T", "H", "Dn", "Dr", "Dv")]
    if fn == "fwd":
        return L.kda_mla_attn_fwd(a["q"], a["kv"], a["k_pe"], a["o"], a["lse"], a["cu"], *sizes, a["scale"], a["dt"], None)
    if a["wsb"] is None:
        a["wsb"] = L.kda_mla_attn_bwd_workspace_bytes(*sizes[1:], a["N"], a["dt"])
    return L.kda_mla_attn_bwd(*(a[n] for n in ("q", "kv", "k_pe", "o", "lse", "dout", "dq", "dkv", "dk_pe", "cu")), *sizes,
                              a["scale"], a["dt"], a["ws"], a["wsb"], None)


@needs_lib
@pytest.mark.parametrize("fn", ["fwd", "bwd"])
def test_expanded_validation(fn):
    call = lambda **kw: _attn(fn, **kw)  # noqa: E731
    assert call(dt=9) == DTYPE and call(dt=0) == UNSUPPORTED and call(dt=2) == UNSUPPORTED
    assert call(B=-1) == SHAPE and call(T=-1) == SHAPE and call(H=0) == SHAPE and call(H=1025) == SHAPE
    assert call(N=1) == SHAPE and call(cu=P) == SHAPE        # without documents N = B; with them B = 1
    assert call(B=1 << 16, N=1 << 16, T=1 << 16) == SHAPE
    assert call(B=1, N=1 << 23, cu=P) == SHAPE and call(B=1, N=1, T=1 << 27, H=64) == SHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=scale) == SHAPE
    for Dn, Dr, Dv in ((96, 0, 96), (128, 32, 128), (128, 64, 64)):
        assert call(Dn=Dn, Dr=Dr, Dv=Dv) == UNSUPPORTED
    for miss in ("q", "kv", "k_pe", "o") + (("lse", "dout", "dq", "dkv", "dk_pe") if fn == "bwd" else ()):
        assert call(**{miss: None}) == NULL, miss
    for odd in ("q", "kv", "k_pe", "o", "lse") + (("dout", "dq", "dkv", "dk_pe") if fn == "bwd" else ()):
        assert call(**{odd: ODD}) == UNSUPPORTED, odd
    assert call(T=0, q=None) == OK and call(B=0, N=0, q=None) == OK


@needs_lib
def test_backward_workspace():
    L = kda.lib()
    need = L.kda_mla_attn_bwd_workspace_bytes(2, 64, 3, 128, 64, 128, 2, 1)
    assert need >= 2 * 64 * 3 * (1 + 64) * 4
    assert _attn("bwd", wsb=need - 1) == WORKSPACE and _attn("bwd", ws=None) == WORKSPACE
    assert _attn("bwd", ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert L.kda_mla_attn_bwd_workspace_bytes(2, 64, 3, 100, 64, 100, 2, 1) == 0


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


I32 = torch.int32


@needs_lib
def test_binding_refusals():
    q, kv, pe = z(1, 8, 2, 192), z(1, 8, 2, 256), z(1, 8, 64)
    o, lse = z(1, 8, 2, 128), z(1, 8, 2, dtype=torch.float32)
    with pytest.raises(ValueError, match="GPU"):
        mla.attn_fwd(q, kv, pe)
    with pytest.raises(ValueError):
        mla.attn_fwd(q, z(1, 7, 2, 256), pe)
    with pytest.raises(ValueError):
        mla.attn_fwd(q, kv, z(1, 7, 64))
    with pytest.raises(ValueError):
        mla.attn_fwd(q, z(1, 8, 2, 128), pe)                 # no value channels
    with pytest.raises(TypeError):
        mla.attn_fwd(q, kv.float(), pe)
    with pytest.raises(TypeError):
        mla.attn_fwd(q, kv, pe, lse=z(1, 8, 2))
    with pytest.raises(TypeError):
        mla.attn_fwd(q, kv, pe, cu_seqlens=torch.tensor([0, 8]))
    with pytest.raises(ValueError):
        mla.attn_bwd(q, kv, pe, o, lse, z(1, 8, 2, 64))
    with pytest.raises(ValueError):
        mla.attn_bwd(q, kv, pe, o, lse[:, :7], o)
    pq, cache, table, lens = z(3, 2, 576), z(4, 16, 576), z(3, 2, dtype=I32), z(3, dtype=I32)
    with pytest.raises(ValueError, match="GPU"):
        mla.paged_attn(pq, cache, table, lens, 512, 0.1)
    with pytest.raises(ValueError):
        mla.paged_attn(z(2, 2, 576), cache, table, lens, 512, 0.1)
    with pytest.raises(ValueError):
        mla.paged_attn(pq, cache, table, lens, 512, 0.1, cu_seqlens=z(3, dtype=I32))
    with pytest.raises(ValueError):
        mla.paged_attn(pq, z(4, 16, 512), table, lens, 512, 0.1)
    with pytest.raises(TypeError):
        mla.paged_attn(pq, cache, table.long(), lens, 512, 0.1)
    c, pos, slots = z(5, 576), z(5, dtype=I32), z(5, dtype=I32)
    with pytest.raises(ValueError, match="GPU"):
        mla.cache_append(c, pos, slots, cache, 512)
    with pytest.raises(ValueError):
        mla.cache_append(c, None, slots, cache, 512, rope=z(9, 64, dtype=torch.float32))
    with pytest.raises(ValueError):
        mla.cache_append(c, pos, slots, cache, 512, q_pe=z(5, 2, 64))
    with pytest.raises(ValueError):
        mla.cache_append(c, pos, slots[:4], cache, 512)
    with pytest.raises(TypeError):
        mla.cache_append(c, pos, slots, cache, 512, norm_weight=z(512))
    with pytest.raises(TypeError):
        mla.cache_append(c, pos.long(), slots, cache, 512)
