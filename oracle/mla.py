"""CPU fp64 oracle of latent attention (test infrastructure only: used by
tests/, never by the product path).

Source: the miniKimiK3 card ("Architecture") and the Kimi-K3-Tiny-L13 card
name latent attention as the mixer between the KDA layers; no page gives its
formula.  Reading: one latent vector c_t of R channels and one rotary key r_t
of Dr channels a token, shared by all heads.

    expanded   k_t,h = [kv_t,h[:Dn] ; r_t],  v_t,h = kv_t,h[Dn:],
               o_i,h = sum_{j<=i} p_ij v_j,h,  p = softmax_j(scale q_i,h . k_j,h)
    absorbed   k_j = cache row j = [c_j ; r_j],  v_j = c_j
    rotation   pairs (x_a, x_b) -> (x_a cos - x_b sin, x_b cos + x_a sin)

Beside the values, ``attention`` and ``attention_backward`` give, for each
output, how far a computation may be off that rounds to bfloat16 where the
library says it does.  With e = 2^-8 (half a bfloat16 step, relative), u =
2^-24 (half a float32 step) and float32 sums of n products off by at most
n u sum|.|:

    s         ds_ij = (D + 16) u scale sum_c |q_c||k_c|   (its sum, scaling and
              the arguments of exp and log, a few roundings of |s| each)
    p         relative 2 ds + 64 u (exp and the row's sum, lse), and e where it
              is rounded as an operand
    o         (e + ep) sum_j p |v| + n u sum_j p |v| + e |o|
    delta     sum_j p (ep |dp| + err_dp) + n u sum_j p |dp| (summed so in float32)
    dS        p (err_dp + err_delta) + |dS| (ep + e)
    dq, dk, dv  the operands' errors carried through the sums, + e |result|
"""

import numpy as np

E = 2.0 ** -8
U = 2.0 ** -24


def _f64(a):
    return np.asarray(a.detach().cpu().double().numpy() if hasattr(a, "detach") else a, dtype=np.float64)


def rotate(x, cos, sin, interleaved=False):
    """x [..., Dr]; cos, sin [..., Dr / 2]."""
    x = _f64(x)
    y = np.empty_like(x)
    half = x.shape[-1] // 2
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, half), slice(half, None))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def append(c, R, rope=None, positions=None, norm_weight=None, eps=1e-6, interleaved=False, q_pe=None):
    """The rows [T, R + Dr] that the tokens' cache rows get, and the rotated
    queries [T, H, Dr] (None without q_pe), unrounded."""
    c = _f64(c).copy()
    if norm_weight is not None:
        lat = c[:, :R]
        c[:, :R] = lat / np.sqrt((lat * lat).mean(-1, keepdims=True) + eps) * _f64(norm_weight)
    q = None if q_pe is None else _f64(q_pe).copy()
    if rope is not None:
        tab = _f64(rope)
        row = tab[np.clip(np.asarray(positions), 0, tab.shape[0] - 1)]
        half = row.shape[-1] // 2
        cos, sin = row[:, :half], row[:, half:]
        c[:, R:] = rotate(c[:, R:], cos, sin, interleaved)
        if q is not None:
            q = rotate(q, cos[:, None], sin[:, None], interleaved)
    return c, q


def attend(q, k, v, first, scale):
    """One head: queries [n, D]; row i sees keys 0 .. first + i.  Returns o,
    lse, and the bounds on their errors (module docstring)."""
    n, D = q.shape
    m = k.shape[0]
    if m == 0:
        z = np.zeros((n, v.shape[1]))
        return z, np.full(n, -np.inf), z, np.zeros(n)
    s = q @ k.T * scale
    ds = (D + 16) * U * (np.abs(q) @ np.abs(k).T) * scale
    ok = np.arange(m)[None, :] <= np.arange(n)[:, None] + first
    s = np.where(ok, s, -np.inf)
    ds = np.where(ok, ds, 0.0)
    top = s.max(-1, keepdims=True)
    some = np.isfinite(top)
    e = np.where(ok, np.exp(s - np.where(some, top, 0.0)), 0.0)
    l = e.sum(-1, keepdims=True)
    p = e / np.where(l == 0, 1.0, l)
    with np.errstate(divide="ignore"):
        lse = np.where(some, np.where(some, top, 0.0) + np.log(l), -np.inf)[:, 0]
    o = p @ v
    worst = ds.max(-1, keepdims=True)
    mag = p @ np.abs(v)
    err = (E + 2 * worst + (64 + m) * U) * mag + E * np.abs(o)
    return o, lse, err, worst[:, 0] + (64 + m) * U + 4 * U * np.abs(np.where(np.isfinite(lse), lse, 0.0))


def documents(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(c) for c in np.asarray(cu)]
    return [(0, cu[n], cu[n + 1]) for n in range(len(cu) - 1)]


def _head(q, kv, k_pe, Dn, b, x, h):
    k = kv[b, x, h, :Dn]
    if k_pe is not None:
        k = np.concatenate([k, k_pe[b, x]], -1)
    return q[b, x, h], k, kv[b, x, h, Dn:]


def attention(q, kv, k_pe=None, scale=None, cu_seqlens=None):
    """Expanded form.  Returns o [B, T, H, Dv], lse [B, T, H] and the bounds on
    their errors (NaN for tokens behind the last document)."""
    q, kv = _f64(q), _f64(kv)
    k_pe = None if k_pe is None else _f64(k_pe)
    B, T, H, D = q.shape
    Dn = D - (0 if k_pe is None else k_pe.shape[-1])
    scale = D ** -0.5 if scale is None else scale
    o = np.full((B, T, H, kv.shape[-1] - Dn), np.nan)
    lse = np.full((B, T, H), np.nan)
    err, err_l = o.copy(), lse.copy()
    for b, s, e in documents(B, T, cu_seqlens):
        x = slice(s, e)
        for h in range(H):
            qq, k, v = _head(q, kv, k_pe, Dn, b, x, h)
            o[b, x, h], lse[b, x, h], err[b, x, h], err_l[b, x, h] = attend(qq, k, v, 0, scale)
    return o, lse, err, err_l


def attention_backward(q, kv, k_pe, do, scale=None, cu_seqlens=None):
    """Gradients of <do, o>.  Returns two dicts, dq, dkv, dk_pe and the bounds
    on their errors."""
    q, kv, do = _f64(q), _f64(kv), _f64(do)
    k_pe = None if k_pe is None else _f64(k_pe)
    B, T, H, D = q.shape
    Dr = 0 if k_pe is None else k_pe.shape[-1]
    Dn = D - Dr
    scale = D ** -0.5 if scale is None else scale
    g = dict(dq=np.full(q.shape, np.nan), dkv=np.full(kv.shape, np.nan))
    if Dr:
        g["dk_pe"] = np.full(k_pe.shape, np.nan)
    err = {n: a.copy() for n, a in g.items()}
    A = np.abs
    for b, st, en in documents(B, T, cu_seqlens):
        x = slice(st, en)
        n = en - st
        if Dr:
            g["dk_pe"][b, x] = 0.0
            err["dk_pe"][b, x] = 0.0
        for h in range(H):
            qq, k, v = _head(q, kv, k_pe, Dn, b, x, h)
            d = do[b, x, h]
            if n == 0:
                continue
            o, lse, _, err_l = attend(qq, k, v, 0, scale)
            ok = np.tril(np.ones((n, n), bool))
            p = np.where(ok, np.exp(np.where(ok, qq @ k.T * scale, -np.inf) - lse[:, None]), 0.0)
            dp = d @ v.T
            delta = (d * o).sum(-1, keepdims=True)
            ds = p * (dp - delta)
            # bounds
            es = (D + 16) * U * (A(qq) @ A(k).T) * scale
            ep = es + err_l[:, None] + 64 * U
            Dv = v.shape[1]
            e_dp = (Dv + 4) * U * (A(d) @ A(v).T)
            nU = (n + 8) * U
            e_delta = (p * (ep * A(dp) + (1 + ep) * e_dp + nU * A(dp))).sum(-1, keepdims=True)
            e_ds = p * (e_dp + e_delta) * (1 + ep) + A(ds) * (ep + E)
            e_p = p * (ep + E)
            dq, dk, dv = ds @ k * scale, ds.T @ qq * scale, p.T @ d
            e_dq = (e_ds @ A(k) + nU * (A(ds) @ A(k))) * scale + E * A(dq)
            e_dk = (e_ds.T @ A(qq) + nU * (A(ds).T @ A(qq))) * scale
            e_dv = e_p.T @ A(d) + nU * (p.T @ A(d)) + E * A(dv)
            g["dq"][b, x, h], err["dq"][b, x, h] = dq, e_dq
            g["dkv"][b, x, h, :Dn], err["dkv"][b, x, h, :Dn] = dk[:, :Dn], e_dk[:, :Dn] + E * A(dk[:, :Dn])
            g["dkv"][b, x, h, Dn:], err["dkv"][b, x, h, Dn:] = dv, e_dv
            if Dr:
                g["dk_pe"][b, x] += dk[:, Dn:]
                err["dk_pe"][b, x] += e_dk[:, Dn:] + H * U * A(dk[:, Dn:])
        if Dr:
            err["dk_pe"][b, x] += E * A(g["dk_pe"][b, x])
    return g, err


def paged_rows(cache, table, length):
    """The cache rows of one sequence: [length, D] and which are there."""
    cache = _f64(cache)
    pages, ps, D = cache.shape
    j = np.arange(length)
    page = np.asarray(table)[j // ps] if length else np.zeros(0, int)
    there = (page >= 0) & (page < pages)
    rows = np.zeros((length, D))
    rows[there] = cache[page[there], (j % ps)[there]]
    return rows, there


def paged_attention(q, cache, block_table, seq_lens, R, scale, cu_seqlens=None):
    """Absorbed form.  Returns o [Tq, H, R], lse [Tq, H] and the bounds on
    their errors (NaN for rows behind the last sequence)."""
    q = _f64(q)
    Tq, H, D = q.shape
    table, lens = np.asarray(block_table), np.asarray(seq_lens)
    N = table.shape[0]
    cu = np.arange(N + 1) if cu_seqlens is None else np.asarray(cu_seqlens)
    o = np.full((Tq, H, R), np.nan)
    lse = np.full((Tq, H), np.nan)
    err, err_l = o.copy(), lse.copy()
    cap = table.shape[1] * (cache.shape[1])
    for n in range(N):
        L = int(min(max(lens[n], 0), cap))
        rows, there = paged_rows(cache, table[n], L)
        # the rows that are there, and how many of them each new token sees
        before = np.concatenate([[0], np.cumsum(there)])
        for i in range(cu[n], cu[n + 1]):
            sees = int(before[min(max(L - (cu[n + 1] - cu[n]) + (i - cu[n]) + 1, 0), L)])
            k = rows[there][:sees]
            for h in range(H):
                r = attend(q[i, h][None], k, k[:, :R], sees, scale)
                o[i, h], lse[i, h], err[i, h], err_l[i, h] = (a[0] for a in r)
    return o, lse, err, err_l
