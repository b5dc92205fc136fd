"""Latent attention (ctypes binding of the kda_mla_* calls of libkda.so): the
mixer between the KDA layers of the hybrid models.  Argument marshalling only,
as in ``kda``; there is no fallback.

    cache_append(c_kv, positions, slots, cache, latent_dim, rope=..., norm_weight=..., q_pe=..., q=...)
    o, lse = paged_attn(q, cache, block_table, seq_lens, latent_dim, scale, cu_seqlens=None)
    o, lse = attn_fwd(q, kv, k_pe, scale=None, cu_seqlens=None)
    grads = attn_bwd(q, kv, k_pe, o, lse, do, scale=None, cu_seqlens=None)   # dq, dkv, dk_pe

Pages on the device, and the cache in 4 bits:

    step = cache_plan(new_lens, seq_lens, block_table, free_pages, free_count, page_size, num_tokens)
    left = cache_release(finished, seq_lens, block_table, free_pages, free_count, page_size)
    cache_append_fp4(...), o, lse = paged_attn_fp4(...)   # as above, cache uint8 [.., fp4_row_bytes(R, Dr)]
    rows = cache_gather_fp4(cache, block_table, cu_seqlens, num_tokens, latent_dim, starts=None)

Shapes (see include/kda.h).  Absorbed (serving): a cache row is [latent of R
channels ; rotary key of Dr channels]; c_kv [T, R + Dr]; cache [num_pages,
page_size, R + Dr]; q [Tq, H, R + Dr]; o [Tq, H, R].  Expanded (training):
q [B, T, H, Dn + Dr]; kv [B, T, H, Dn + Dv], each head's key part and value;
k_pe [B, T, Dr] shared by the heads (None: Dr = 0); o [B, T, H, Dv].  bfloat16;
lse float32.  Calls run on the current stream of the tensors' device.
"""

import functools
import math

import torch

from .kda import KDA_BF16, KDA_F16, KDA_F32, KdaError, _num_seqs, lib

__all__ = ["cache_append", "paged_attn", "paged_workspace_bytes", "attn_fwd", "attn_bwd", "attn_bwd_workspace_bytes",
           "cache_plan", "cache_release", "fp4_row_bytes", "cache_append_fp4", "cache_gather_fp4", "paged_attn_fp4",
           "paged_fp4_workspace_bytes"]

_DT = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32, torch.float16: KDA_F16}


def _raw_stream(index):
    """torch.cuda.current_stream(index).cuda_stream, without making a Stream object (2 us of a 10 us call)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _dt(t):
    if t.dtype not in _DT:
        raise TypeError("unsupported dtype %s (bfloat16)" % t.dtype)
    return _DT[t.dtype]


def _check(first, *tensors):
    """Each of (tensor or None, name, shape, dtype) as said, contiguous and on
    `first`'s device, which is a GPU: the kernels size every access from the
    first tensors' sizes.  A shape of None is not compared."""
    for t, name, shape, dtype in tensors:
        if t is None:
            continue
        if shape is not None and t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        if t.dtype != dtype:
            raise TypeError("%s must be %s" % (name, str(dtype).replace("torch.", "")))
    dev = first.device
    if not first.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not first.is_contiguous():
        raise ValueError("tensors must be contiguous")
    for t, name, _, _ in tensors:
        if t is not None:
            if t.device != dev:
                raise ValueError("tensors must be on one device: %s is on %s" % (name, t.device))
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous: %s" % name)
    return dev


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name, dev, *args):
    """Library call `name` on dev's current stream, with dev current."""
    fn = getattr(lib(), name)
    if torch.cuda.current_device() == dev.index:
        st = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev.index))
    if st != 0:
        raise KdaError(st, name)


def _workspace(workspace, need, dev):
    """The caller's workspace (any contiguous tensor of dev), or one of `need` bytes; with its size."""
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous and on the tensors' device")
        return workspace, workspace.numel() * workspace.element_size()
    return (torch.empty(need, dtype=torch.uint8, device=dev) if need else None), need


@functools.lru_cache(maxsize=64)
def fp4_row_bytes(latent_dim, rope_dim):
    """Bytes of a row of the 4-bit cache."""
    n = int(lib().kda_mla_fp4_row_bytes(latent_dim, rope_dim))
    if n == 0:
        raise ValueError("no 4-bit cache of %d + %d channels (128, 256 or 512 and 0 or 64)" % (latent_dim, rope_dim))
    return n


def _append(name, fp4, c_kv, positions, slots, cache, latent_dim, rope, norm_weight, eps, interleaved, q_pe, q):
    if c_kv.dim() != 2 or cache.dim() != 3:
        raise ValueError("c_kv must be [T, R + Dr] and cache [num_pages, page_size, R + Dr]")
    T, D = c_kv.shape
    R = int(latent_dim)
    Dr = D - R
    row = fp4_row_bytes(R, Dr) if fp4 else D
    H = 1
    if rope is not None:
        if positions is None:
            raise ValueError("rope needs positions")
        if rope.dim() != 2:
            raise ValueError("rope must be [num_pos, Dr]")
    if (q_pe is None) != (q is None):
        raise ValueError("q_pe and q go together")
    if q_pe is not None:
        if q_pe.dim() != 3:
            raise ValueError("q_pe must be [T, H, Dr]")
        H = q_pe.shape[1]
    dt, f32, i32 = c_kv.dtype, torch.float32, torch.int32
    dev = _check(c_kv, (cache, "cache", (cache.shape[0], cache.shape[1], row), torch.uint8 if fp4 else dt),
                 (slots, "slots", (T,), i32), (positions, "positions", (T,), i32),
                 (norm_weight, "norm_weight", (R,), f32),
                 (rope, "rope", None if rope is None else (rope.shape[0], Dr), f32), (q_pe, "q_pe", (T, H, Dr), dt),
                 (q, "q", (T, H, D), dt))
    _call(name, dev, _ptr(c_kv), _ptr(norm_weight), float(eps), _ptr(rope),
          0 if rope is None else rope.shape[0], int(bool(interleaved)), _ptr(positions), _ptr(slots), _ptr(cache),
          cache.shape[0], cache.shape[1], _ptr(q_pe), _ptr(q), T, H, R, Dr, _dt(c_kv))
    return cache


def cache_append(c_kv, positions, slots, cache, latent_dim, rope=None, norm_weight=None, eps=1e-6, interleaved=False,
                 q_pe=None, q=None):
    """Writes new tokens' rows into the paged latent cache, in place: the first
    latent_dim channels of c_kv [T, R + Dr] RMS-normalised (norm_weight [R]
    float32; None: as they are), the others rotated by the token's position
    (rope [num_pos, Dr] float32: cos, then sin; None: as they are).  slots
    int32 [T]: page * page_size + offset, outside the cache for a token that
    is not kept.  With q_pe [T, H, Dr], q [T, H, R + Dr] gets the rotated
    queries in its last Dr channels.  Returns cache."""
    return _append("kda_mla_cache_append", False, c_kv, positions, slots, cache, latent_dim, rope, norm_weight, eps,
                   interleaved, q_pe, q)


def cache_append_fp4(c_kv, positions, slots, cache, latent_dim, rope=None, norm_weight=None, eps=1e-6,
                     interleaved=False, q_pe=None, q=None):
    """cache_append into a 4-bit cache, uint8 [num_pages, page_size, fp4_row_bytes(R, Dr)]: the latent in 4 bits with
    a power-of-two scale for every 32 channels (include/kda.h), the rotary key in bfloat16.  Returns cache."""
    return _append("kda_mla_cache_append_fp4", True, c_kv, positions, slots, cache, latent_dim, rope, norm_weight, eps,
                   interleaved, q_pe, q)


@functools.lru_cache(maxsize=256)
def paged_workspace_bytes(N, Tq, H, R, Dr, page_size, max_pages, dtype=torch.bfloat16):
    """Bytes of device workspace paged_attn needs."""
    return int(lib().kda_mla_paged_workspace_bytes(N, Tq, H, R, Dr, page_size, max_pages, _DT[dtype]))


def _paged(name, fp4, need, q, cache, block_table, seq_lens, latent_dim, scale, cu_seqlens, out, lse, workspace):
    if q.dim() != 3 or cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q must be [Tq, H, R + Dr], cache [num_pages, page_size, row], block_table [N, max_pages]")
    Tq, H, D = q.shape
    N, max_pages = block_table.shape
    num_pages, page_size, _ = cache.shape
    R = int(latent_dim)
    row = fp4_row_bytes(R, D - R) if fp4 else D
    if cu_seqlens is None and N != Tq:
        raise ValueError("q must be [N, H, R + Dr], one token a sequence, without cu_seqlens")
    dt, i32 = q.dtype, torch.int32
    dev = _check(q, (cache, "cache", (num_pages, page_size, row), torch.uint8 if fp4 else dt),
                 (block_table, "block_table", None, i32), (seq_lens, "seq_lens", (N,), i32),
                 (cu_seqlens, "cu_seqlens", (N + 1,), i32), (out, "out", (Tq, H, R), dt),
                 (lse, "lse", (Tq, H), torch.float32))
    code = _dt(q)
    if not 0 <= R <= D:
        raise ValueError("latent_dim must be within q's width")
    if out is None:
        out = q.new_empty((Tq, H, R))
    if lse is None:
        lse = torch.empty((Tq, H), dtype=torch.float32, device=dev)
    ws, nbytes = _workspace(workspace, 0 if workspace is not None else
                            need(N, Tq, H, R, D - R, page_size, max_pages, dt), dev)
    _call(name, dev, _ptr(q), _ptr(cache), _ptr(block_table), _ptr(seq_lens), _ptr(cu_seqlens),
          _ptr(out), _ptr(lse), N, Tq, H, R, D - R, num_pages, page_size, max_pages, float(scale), code, _ptr(ws),
          nbytes)
    return out, lse


def paged_attn(q, cache, block_table, seq_lens, latent_dim, scale, cu_seqlens=None, out=None, lse=None,
               workspace=None):
    """Absorbed latent attention of new tokens over the paged cache.  Without
    cu_seqlens every sequence has one new token (q [N, H, R + Dr]); with it,
    sequence n's are rows cu[n] .. cu[n+1]-1 of q [Tq, H, R + Dr], the last of
    its seq_lens[n] cache rows.  Returns (o [Tq, H, R], lse [Tq, H])."""
    return _paged("kda_mla_paged_attn", False, paged_workspace_bytes, q, cache, block_table, seq_lens, latent_dim,
                  scale, cu_seqlens, out, lse, workspace)


@functools.lru_cache(maxsize=256)
def paged_fp4_workspace_bytes(N, Tq, H, R, Dr, page_size, max_pages, dtype=torch.bfloat16):
    """Bytes of device workspace paged_attn_fp4 needs."""
    return int(lib().kda_mla_paged_fp4_workspace_bytes(N, Tq, H, R, Dr, page_size, max_pages, _DT[dtype]))


def paged_attn_fp4(q, cache, block_table, seq_lens, latent_dim, scale, cu_seqlens=None, out=None, lse=None,
                   workspace=None):
    """paged_attn over a 4-bit cache (cache_append_fp4), on the values that its rows stand for."""
    return _paged("kda_mla_paged_attn_fp4", True, paged_fp4_workspace_bytes, q, cache, block_table, seq_lens,
                  latent_dim, scale, cu_seqlens, out, lse, workspace)


def cache_gather_fp4(cache, block_table, cu_seqlens, num_tokens, latent_dim, starts=None, out=None):
    """Rows of a 4-bit cache as bfloat16 [num_tokens, R + Dr], sequence after sequence: row cu_seqlens[n] + i is row
    starts[n] + i (None: i) of sequence n; one that is not in the cache is zeros.  Rows in front of the first sequence
    and behind the last are left as they were.  Dr follows from the cache's row bytes."""
    if cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("cache must be [num_pages, page_size, row], block_table [N, max_pages]")
    num_pages, page_size, row = cache.shape
    N, max_pages = block_table.shape
    R, T = int(latent_dim), int(num_tokens)
    Dr = next((d for d in (0, 64) if fp4_row_bytes(R, d) == row), None)
    if Dr is None:
        raise ValueError("no 4-bit cache of latent_dim %d has rows of %d bytes" % (R, row))
    if T < 0:
        raise ValueError("num_tokens must not be negative")
    i32 = torch.int32
    dev = _check(cache, (cache, "cache", None, torch.uint8), (block_table, "block_table", None, i32),
                 (cu_seqlens, "cu_seqlens", (N + 1,), i32), (starts, "starts", (N,), i32),
                 (out, "out", (T, R + Dr), torch.bfloat16))
    if out is None:
        out = torch.empty((T, R + Dr), dtype=torch.bfloat16, device=dev)
    _call("kda_mla_cache_gather_fp4", dev, _ptr(cache), _ptr(block_table), _ptr(cu_seqlens), _ptr(starts), _ptr(out),
          N, T, R, Dr, num_pages, page_size, max_pages, KDA_BF16)
    return out


def _outputs(out, sizes, workspace, need, dev):
    """The given int32 outputs, and new ones in the place of those that are not, and the workspace with its size.  What
    is new is one allocation (7 of them took 9 us of a 20 us call)."""
    out = out or {}
    unknown = set(out) - set(sizes)
    if unknown:
        raise ValueError("unknown outputs: %s" % ", ".join(sorted(unknown)))
    new = [n for n in sizes if out.get(n) is None]
    if workspace is not None:
        workspace, nbytes = _workspace(workspace, 0, dev)
        ws = ()
    else:
        nbytes, ws = need, (need // 4,)
    parts = ()
    if ws or new:
        lengths = [*ws, *(sizes[n] for n in new)]
        parts = torch.empty(sum(lengths), dtype=torch.int32, device=dev).split(lengths)
        if ws:
            workspace, parts = parts[0], parts[1:]
    got = dict(zip(new, parts))
    return {n: got[n] if n in got else out[n] for n in sizes}, workspace, nbytes


def cache_plan(new_lens, seq_lens, block_table, free_pages, free_count, page_size, num_tokens, out=None,
               workspace=None):
    """Pages for a step's new tokens, from lengths on the GPU (all tensors int32): sequence n has seq_lens[n] rows in
    the cache and new_lens[n] new tokens; pages come from the end of the stack free_pages[:free_count] and are written
    into block_table [N, max_pages].  Sequences are served in order; one whose tokens do not fit its table's row or the
    num_tokens rows of the batch, or whose pages are not there, is refused.  Returns a dict:

        cu_seqlens [N + 1]       for the calls that take the new tokens
        positions, slots [num_tokens]  0 and -1 for tokens of refused sequences and behind the last one
        kv_lens [N]              rows with the new ones, the attention's seq_lens; -1 for a refused sequence
        seq_lens [N], free_count [1]   the state after the step

    `out` takes preallocated ones; {"seq_lens": seq_lens, "free_count": free_count} updates the state in place, as a
    captured step does."""
    if block_table.dim() != 2 or new_lens.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("new_lens must be [N], block_table [N, max_pages], free_pages [num_free]")
    N, max_pages = block_table.shape
    T = int(num_tokens)
    if T < 0:
        raise ValueError("num_tokens must not be negative")
    i32 = torch.int32
    sizes = {"cu_seqlens": N + 1, "positions": T, "slots": T, "kv_lens": N, "seq_lens": N, "free_count": 1}
    dev = _check(block_table, (block_table, "block_table", None, i32), (new_lens, "new_lens", (N,), i32),
                 (seq_lens, "seq_lens", (N,), i32), (free_pages, "free_pages", None, i32),
                 (free_count, "free_count", (1,), i32),
                 *((t, "out[%r]" % n, (sizes[n],), i32) for n, t in (out or {}).items() if n in sizes))
    o, ws, nbytes = _outputs(out, sizes, workspace, _plan_bytes("plan", N), dev)
    _call("kda_mla_cache_plan", dev, _ptr(new_lens), _ptr(seq_lens), _ptr(block_table), _ptr(free_pages),
          _ptr(free_count), free_pages.numel(), _ptr(o["cu_seqlens"]), _ptr(o["positions"]), _ptr(o["slots"]),
          _ptr(o["kv_lens"]), _ptr(o["seq_lens"]), _ptr(o["free_count"]), N, T, int(page_size), max_pages, _ptr(ws),
          nbytes)
    return o


@functools.lru_cache(maxsize=64)
def _plan_bytes(call, N):
    return int(getattr(lib(), "kda_mla_cache_%s_workspace_bytes" % call)(N))


def cache_release(finished, seq_lens, block_table, free_pages, free_count, page_size, out=None, workspace=None):
    """The pages of the sequences with finished[n] (bool [N]) back to the end of the stack free_pages[:free_count], in
    place.  Returns a dict: seq_lens [N], 0 for these, and free_count [1]; `out` as for cache_plan."""
    if block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("block_table must be [N, max_pages], free_pages [num_free]")
    N, max_pages = block_table.shape
    i32 = torch.int32
    sizes = {"seq_lens": N, "free_count": 1}
    dev = _check(block_table, (block_table, "block_table", None, i32), (finished, "finished", (N,), torch.bool),
                 (seq_lens, "seq_lens", (N,), i32), (free_pages, "free_pages", None, i32),
                 (free_count, "free_count", (1,), i32),
                 *((t, "out[%r]" % n, (sizes[n],), i32) for n, t in (out or {}).items() if n in sizes))
    o, ws, nbytes = _outputs(out, sizes, workspace, _plan_bytes("release", N), dev)
    _call("kda_mla_cache_release", dev, _ptr(finished), _ptr(seq_lens), _ptr(block_table), _ptr(free_pages),
          _ptr(free_count), free_pages.numel(), _ptr(o["seq_lens"]), _ptr(o["free_count"]), N, int(page_size),
          max_pages, _ptr(ws), nbytes)
    return o


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
    Dn = Dq - Dr
    Dv = kv.shape[-1] - Dn
    if Dn <= 0 or Dv <= 0:
        raise ValueError("q, kv and k_pe widths do not fit: q [.., Dn + Dr], kv [.., Dn + Dv], k_pe [.., Dr]")
    return B, T, H, Dn, Dr, Dv


def attn_fwd(q, kv, k_pe=None, scale=None, cu_seqlens=None, out=None, lse=None):
    """Expanded latent attention, causal.  scale defaults to (Dn + Dr)^-0.5.
    Returns (o [B, T, H, Dv], lse [B, T, H])."""
    B, T, H, Dn, Dr, Dv = _expanded_shapes(q, kv, k_pe)
    N = _num_seqs(B, cu_seqlens)
    dt = q.dtype
    dev = _check(q, (kv, "kv", (B, T, H, Dn + Dv), dt), (k_pe, "k_pe", (B, T, Dr), dt),
                 (cu_seqlens, "cu_seqlens", None, torch.int32), (out, "out", (B, T, H, Dv), dt),
                 (lse, "lse", (B, T, H), torch.float32))
    code = _dt(q)
    if out is None:
        out = q.new_empty((B, T, H, Dv))
    if lse is None:
        lse = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    _call("kda_mla_attn_fwd", dev, _ptr(q), _ptr(kv), _ptr(k_pe), _ptr(out), _ptr(lse), _ptr(cu_seqlens), N, B, T, H,
          Dn, Dr, Dv, 1.0 / math.sqrt(Dn + Dr) if scale is None else float(scale), code)
    return out, lse


@functools.lru_cache(maxsize=256)
def attn_bwd_workspace_bytes(B, T, H, Dn, Dr, Dv, num_seqs, dtype=torch.bfloat16):
    """Bytes of device workspace attn_bwd needs."""
    return int(lib().kda_mla_attn_bwd_workspace_bytes(B, T, H, Dn, Dr, Dv, num_seqs, _DT[dtype]))


def attn_bwd(q, kv, k_pe, o, lse, do, scale=None, cu_seqlens=None, workspace=None, out=None):
    """Gradients of <do, o> for attn_fwd(q, kv, k_pe, scale, cu_seqlens), whose
    o and lse are passed back.  Returns a dict with dq, dkv and dk_pe (None
    without k_pe); `out` takes preallocated ones."""
    B, T, H, Dn, Dr, Dv = _expanded_shapes(q, kv, k_pe)
    N = _num_seqs(B, cu_seqlens)
    dt = q.dtype
    shapes = {"dq": (B, T, H, Dn + Dr), "dkv": (B, T, H, Dn + Dv), "dk_pe": (B, T, Dr)}
    gr = {n: None if out is None else out.get(n) for n in shapes}
    dev = _check(q, (kv, "kv", (B, T, H, Dn + Dv), dt), (k_pe, "k_pe", (B, T, Dr), dt), (o, "o", (B, T, H, Dv), dt),
                 (do, "do", (B, T, H, Dv), dt), (lse, "lse", (B, T, H), torch.float32),
                 (cu_seqlens, "cu_seqlens", None, torch.int32), *((gr[n], n, shapes[n], dt) for n in gr))
    code = _dt(q)
    for n in gr:
        if gr[n] is None and (n != "dk_pe" or Dr):
            gr[n] = q.new_empty(shapes[n])
    ws, nbytes = _workspace(workspace, 0 if workspace is not None else
                            attn_bwd_workspace_bytes(B, T, H, Dn, Dr, Dv, N, dt), dev)
    _call("kda_mla_attn_bwd", dev, _ptr(q), _ptr(kv), _ptr(k_pe), _ptr(o), _ptr(lse), _ptr(do), _ptr(gr["dq"]),
          _ptr(gr["dkv"]), _ptr(gr["dk_pe"]), _ptr(cu_seqlens), N, B, T, H, Dn, Dr, Dv,
          1.0 / math.sqrt(Dn + Dr) if scale is None else float(scale), code, _ptr(ws), nbytes)
    return gr
