"""Latent attention (ctypes binding of the kda_mla_* calls of libkda.so): the
mixer between the KDA layers of the hybrid models.  Argument marshalling only,
as in ``kda``; there is no fallback.

    cache_append(c_kv, positions, slots, cache, latent_dim, rope=..., norm_weight=..., q_pe=..., q=...)
    o, lse = paged_attn(q, cache, block_table, seq_lens, latent_dim, scale, cu_seqlens=None)
    o, lse = attn_fwd(q, kv, k_pe, scale=None, cu_seqlens=None)
    grads = attn_bwd(q, kv, k_pe, o, lse, do, scale=None, cu_seqlens=None)   # dq, dkv, dk_pe

Shapes (see include/kda.h).  Absorbed (serving): a cache row is [latent of R
channels ; rotary key of Dr channels]; c_kv [T, R + Dr]; cache [num_pages,
page_size, R + Dr]; q [Tq, H, R + Dr]; o [Tq, H, R].  Expanded (training):
q [B, T, H, Dn + Dr]; kv [B, T, H, Dn + Dv], each head's key part and value;
k_pe [B, T, Dr] shared by the heads (None: Dr = 0); o [B, T, H, Dv].  bfloat16;
lse float32.  Calls run on the current stream of the tensors' device.
"""

import contextlib
import ctypes
import math

import torch

from .kda import KDA_BF16, KDA_F16, KDA_F32, KdaError, _check_dev, _expect, _num_seqs, _ptr, lib

__all__ = ["cache_append", "paged_attn", "paged_workspace_bytes", "attn_fwd", "attn_bwd", "attn_bwd_workspace_bytes"]

_DT = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32, torch.float16: KDA_F16}


def _same(first, *ts, dtype=None, name):
    """Raise unless every given tensor has `dtype` (first's dtype by default)."""
    want = first.dtype if dtype is None else dtype
    for t in ts:
        if t is not None and t.dtype != want:
            raise TypeError("%s must be %s" % (name, str(want).replace("torch.", "")))


def _dt(t):
    if t.dtype not in _DT:
        raise TypeError("unsupported dtype %s (bfloat16)" % t.dtype)
    return _DT[t.dtype]


def _check(*ts):
    """Contiguous GPU tensors of one device."""
    _check_dev(*ts)
    devs = {t.device for t in ts if t is not None}
    if len(devs) > 1:
        raise ValueError("tensors must be on one device, got %s" % sorted(str(d) for d in devs))


@contextlib.contextmanager
def _on(t):
    """t's device made current; yields its current stream."""
    with torch.cuda.device(t.device):
        yield ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _nbytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def cache_append(c_kv, positions, slots, cache, latent_dim, rope=None, norm_weight=None, eps=1e-6, interleaved=False,
                 q_pe=None, q=None):
    """Writes new tokens' rows into the paged latent cache, in place: the first
    latent_dim channels of c_kv [T, R + Dr] RMS-normalised (norm_weight [R]
    float32; None: as they are), the others rotated by the token's position
    (rope [num_pos, Dr] float32: cos, then sin; None: as they are).  slots
    int32 [T]: page * page_size + offset, outside the cache for a token that
    is not kept.  With q_pe [T, H, Dr], q [T, H, R + Dr] gets the rotated
    queries in its last Dr channels.  Returns cache."""
    if c_kv.dim() != 2 or cache.dim() != 3:
        raise ValueError("c_kv must be [T, R + Dr] and cache [num_pages, page_size, R + Dr]")
    T, D = c_kv.shape
    R = int(latent_dim)
    Dr = D - R
    _expect(cache, (cache.shape[0], cache.shape[1], D), "cache")
    _expect(slots, (T,), "slots")
    _expect(positions, (T,), "positions")
    _expect(norm_weight, (R,), "norm_weight")
    if rope is not None:
        if positions is None:
            raise ValueError("rope needs positions")
        if rope.dim() != 2:
            raise ValueError("rope must be [num_pos, Dr]")
        _expect(rope, (rope.shape[0], Dr), "rope")
    if (q_pe is None) != (q is None):
        raise ValueError("q_pe and q go together")
    H = 1
    if q_pe is not None:
        if q_pe.dim() != 3:
            raise ValueError("q_pe must be [T, H, Dr]")
        H = q_pe.shape[1]
        _expect(q_pe, (T, H, Dr), "q_pe")
        _expect(q, (T, H, D), "q")
    _same(c_kv, cache, q_pe, q, name="cache, q_pe and q (c_kv's dtype)")
    _same(c_kv, norm_weight, rope, dtype=torch.float32, name="norm_weight and rope")
    _same(c_kv, positions, slots, dtype=torch.int32, name="positions and slots")
    _check(c_kv, positions, slots, cache, rope, norm_weight, q_pe, q)
    with _on(c_kv) as stream:
        st = lib().kda_mla_cache_append(_ptr(c_kv), _ptr(norm_weight), float(eps), _ptr(rope),
                                        0 if rope is None else rope.shape[0], int(bool(interleaved)),
                                        _ptr(positions), _ptr(slots), _ptr(cache), cache.shape[0], cache.shape[1],
                                        _ptr(q_pe), _ptr(q), T, H, R, Dr, _dt(c_kv), stream)
    if st != 0:
        raise KdaError(st, "kda_mla_cache_append")
    return cache


def paged_workspace_bytes(N, Tq, H, R, Dr, page_size, max_pages, dtype=torch.bfloat16):
    """Bytes of device workspace paged_attn needs."""
    return int(lib().kda_mla_paged_workspace_bytes(N, Tq, H, R, Dr, page_size, max_pages, _DT[dtype]))


def paged_attn(q, cache, block_table, seq_lens, latent_dim, scale, cu_seqlens=None, out=None, lse=None,
               workspace=None):
    """Absorbed latent attention of new tokens over the paged cache.  Without
    cu_seqlens every sequence has one new token (q [N, H, R + Dr]); with it,
    sequence n's are rows cu[n] .. cu[n+1]-1 of q [Tq, H, R + Dr], the last of
    its seq_lens[n] cache rows.  Returns (o [Tq, H, R], lse [Tq, H])."""
    if q.dim() != 3 or cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [Tq, H, R + Dr], cache [num_pages, page_size, R + Dr], block_table [N, max_pages]")
    Tq, H, D = q.shape
    N, max_pages = block_table.shape
    num_pages, page_size, _ = cache.shape
    R = int(latent_dim)
    _expect(cache, (num_pages, page_size, D), "cache")
    _expect(seq_lens, (N,), "seq_lens")
    if cu_seqlens is None:
        _expect(q, (N, H, D), "q (one token a sequence)")
    else:
        _expect(cu_seqlens, (N + 1,), "cu_seqlens")
    _expect(out, (Tq, H, R), "out")
    _expect(lse, (Tq, H), "lse")
    _same(q, cache, out, name="cache and out (q's dtype)")
    _same(q, block_table, seq_lens, cu_seqlens, dtype=torch.int32, name="block_table, seq_lens and cu_seqlens")
    _same(q, lse, dtype=torch.float32, name="lse")
    dt = _dt(q)
    _check(q, cache, block_table, seq_lens, cu_seqlens, out, lse, workspace)
    with _on(q) as stream:
        o = out if out is not None else torch.empty((Tq, H, max(R, 0)), dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((Tq, H), dtype=torch.float32, device=q.device)
        ws = workspace
        if ws is None:
            need = paged_workspace_bytes(N, Tq, H, R, D - R, page_size, max_pages, q.dtype)
            ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        st = lib().kda_mla_paged_attn(_ptr(q), _ptr(cache), _ptr(block_table), _ptr(seq_lens), _ptr(cu_seqlens),
                                      _ptr(o), _ptr(lse), N, Tq, H, R, D - R, num_pages, page_size, max_pages,
                                      float(scale), dt, _ptr(ws), _nbytes(ws), stream)
    if st != 0:
        raise KdaError(st, "kda_mla_paged_attn")
    return o, lse


def _expanded_shapes(q, kv, k_pe):
    """Sizes (B, T, H, Dn, Dr, Dv), after checking that kv and k_pe agree with q."""
    if q.dim() != 4 or kv.dim() != 4:
        raise ValueError("q must be [B, T, H, Dn + Dr] and kv [B, T, H, Dn + Dv]")
    B, T, H, Dq = q.shape
    Dr = 0
    if k_pe is not None:
        if k_pe.dim() != 3:
            raise ValueError("k_pe must be [B, T, Dr]")
        Dr = k_pe.shape[-1]
        _expect(k_pe, (B, T, Dr), "k_pe")
    Dn = Dq - Dr
    _expect(kv, (B, T, H, kv.shape[-1]), "kv")
    Dv = kv.shape[-1] - Dn
    if Dn <= 0 or Dv <= 0:
        raise ValueError("q, kv and k_pe widths do not fit: q [.., Dn + Dr], kv [.., Dn + Dv], k_pe [.., Dr]")
    return B, T, H, Dn, Dr, Dv


def attn_fwd(q, kv, k_pe=None, scale=None, cu_seqlens=None, out=None, lse=None):
    """Expanded latent attention, causal.  scale defaults to (Dn + Dr)^-0.5.
    Returns (o [B, T, H, Dv], lse [B, T, H])."""
    B, T, H, Dn, Dr, Dv = _expanded_shapes(q, kv, k_pe)
    N = _num_seqs(B, cu_seqlens)
    _expect(out, (B, T, H, Dv), "out")
    _expect(lse, (B, T, H), "lse")
    _same(q, kv, k_pe, out, name="kv, k_pe and out (q's dtype)")
    _same(q, lse, dtype=torch.float32, name="lse")
    dt = _dt(q)
    _check(q, kv, k_pe, cu_seqlens, out, lse)
    scale = 1.0 / math.sqrt(Dn + Dr) if scale is None else float(scale)
    with _on(q) as stream:
        o = out if out is not None else torch.empty((B, T, H, Dv), dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
        st = lib().kda_mla_attn_fwd(_ptr(q), _ptr(kv), _ptr(k_pe), _ptr(o), _ptr(lse), _ptr(cu_seqlens), N, B, T, H,
                                    Dn, Dr, Dv, scale, dt, stream)
    if st != 0:
        raise KdaError(st, "kda_mla_attn_fwd")
    return o, lse


def attn_bwd_workspace_bytes(B, T, H, Dn, Dr, Dv, num_seqs, dtype=torch.bfloat16):
    """Bytes of device workspace attn_bwd needs."""
    return int(lib().kda_mla_attn_bwd_workspace_bytes(B, T, H, Dn, Dr, Dv, num_seqs, _DT[dtype]))


def attn_bwd(q, kv, k_pe, o, lse, do, scale=None, cu_seqlens=None, workspace=None, out=None):
    """Gradients of <do, o> for attn_fwd(q, kv, k_pe, scale, cu_seqlens), whose
    o and lse are passed back.  Returns a dict with dq, dkv and dk_pe (None
    without k_pe); `out` takes preallocated ones."""
    B, T, H, Dn, Dr, Dv = _expanded_shapes(q, kv, k_pe)
    N = _num_seqs(B, cu_seqlens)
    _expect(o, (B, T, H, Dv), "o")
    _expect(do, (B, T, H, Dv), "do")
    _expect(lse, (B, T, H), "lse")
    _same(q, kv, k_pe, o, do, name="kv, k_pe, o and do (q's dtype)")
    _same(q, lse, dtype=torch.float32, name="lse")
    dt = _dt(q)
    _check(q, kv, k_pe, o, lse, do, cu_seqlens, workspace)
    scale = 1.0 / math.sqrt(Dn + Dr) if scale is None else float(scale)
    shapes = {"dq": (B, T, H, Dn + Dr), "dkv": (B, T, H, Dn + Dv), "dk_pe": (B, T, Dr) if Dr else None}
    with _on(q) as stream:
        gr = {}
        for n, shape in shapes.items():
            t = None if out is None or shape is None else out.get(n)
            _expect(t, shape, n)
            _same(q, t, name=n)
            gr[n] = t if t is not None or shape is None else torch.empty(shape, dtype=q.dtype, device=q.device)
        _check(q, *gr.values())
        ws = workspace
        if ws is None:
            ws = torch.empty(max(attn_bwd_workspace_bytes(B, T, H, Dn, Dr, Dv, N, q.dtype), 1), dtype=torch.uint8,
                             device=q.device)
        st = lib().kda_mla_attn_bwd(_ptr(q), _ptr(kv), _ptr(k_pe), _ptr(o), _ptr(lse), _ptr(do), _ptr(gr["dq"]),
                                    _ptr(gr["dkv"]), _ptr(gr["dk_pe"]), _ptr(cu_seqlens), N, B, T, H, Dn, Dr, Dv,
                                    scale, dt, _ptr(ws), _nbytes(ws), stream)
    if st != 0:
        raise KdaError(st, "kda_mla_attn_bwd")
    return gr
