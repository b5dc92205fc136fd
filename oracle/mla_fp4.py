"""CPU float64 oracle of the paged 4-bit latent cache and of its pages (test
infrastructure only: used by tests/, never by the product path).

A latent block of 32 channels is held as 4-bit codes (sign, two bits of
exponent, one of fraction: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one exponent E, the
smallest with max|y| <= 7 * 2^E, held to [-125, 125] (MXFP4 of the OCP
Microscaling Formats specification 1.0, which leaves the choice of E open).  A
scale byte (E + 127) from 253 on stands for NaN: 6 * 2^126 would pass bfloat16's
range.  A channel gets the nearest code, the even one of two equally near, and 6
above 6.
"""

import numpy as np

from .mla import _f64, append

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def row_bytes(R, Dr):
    return -(-(R // 2 + 2 * Dr + R // 32) // 16) * 16


def quantise(y):
    """Codes [.., R] and scale bytes [.., R / 32] of latents y [.., R]."""
    y = _f64(y)
    b = y.reshape(y.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    m, x = np.frexp(np.abs(b).max(-1))
    e = np.where(m == 0, -125, np.clip(x - np.where(m <= 7 / 8, 3, 2), -125, 125))
    v = np.ldexp(b, -e[..., None])
    # the codes are multiples of 0.5 up to 2, of 1 up to 4, of 2 up to 6, and the even codes the even multiples
    a = np.minimum(np.abs(v), 6.0)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    near = np.searchsorted(MAGNITUDES, np.rint(a / step) * step)
    codes = near + 8 * np.signbit(v)
    codes[bad] = 0
    return codes.reshape(y.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales):
    """What codes [.., R] and scale bytes [.., R / 32] stand for."""
    s = np.where(scales >= 253, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0) * np.repeat(s, 32, -1)


def pack(codes, pe_bits, scales):
    """Cache rows [.., row_bytes] from codes, the rotary keys' bf16 bits (uint16 [.., Dr]) and scales."""
    R, Dr = codes.shape[-1], pe_bits.shape[-1]
    row = np.zeros(codes.shape[:-1] + (row_bytes(R, Dr),), np.uint8)
    row[..., :R // 2] = codes[..., 0::2] | codes[..., 1::2] << 4
    row[..., R // 2:R // 2 + 2 * Dr] = pe_bits.astype("<u2").view(np.uint8).reshape(pe_bits.shape[:-1] + (2 * Dr,))
    row[..., R // 2 + 2 * Dr:R // 2 + 2 * Dr + R // 32] = scales
    return row


def unpack(rows, R, Dr):
    """float64 [.., R + Dr] that cache rows stand for."""
    rows = np.ascontiguousarray(rows)
    codes = np.stack([rows[..., :R // 2] & 15, rows[..., :R // 2] >> 4], -1).reshape(rows.shape[:-1] + (R,))
    lat = values(codes, rows[..., R // 2 + 2 * Dr:R // 2 + 2 * Dr + R // 32])
    bits = np.ascontiguousarray(rows[..., R // 2:R // 2 + 2 * Dr]).view("<u2").astype(np.uint32) << 16
    return np.concatenate([lat, bits.view(np.float32).astype(np.float64)], -1)


def append_rows(c, R, **kw):
    """Codes, scales and unrounded rotary keys of the tokens' rows, and the rotated queries (arguments of
    oracle.mla.append)."""
    rows, q = append(c, R, **kw)
    codes, scales = quantise(rows[:, :R])
    return codes, scales, rows[:, R:], q


def plan(new_lens, seq_lens, table, free_pages, free_count, page_size, T):
    """One sequence after the other.  Returns cu_seqlens, positions, slots, kv_lens, seq_lens, free_count and the
    table (a copy)."""
    table = np.array(table, np.int64)
    N, per = table.shape
    P = page_size
    stack = [int(p) for p in free_pages[:min(max(int(free_count), 0), len(free_pages))]]
    free = len(stack)
    cu, kv, after = [0], [], []
    pos, slots = np.zeros(T, np.int64), np.full(T, -1, np.int64)
    tokens = asked = 0
    for n in range(N):
        s, a = min(max(int(seq_lens[n]), 0), per * P), max(int(new_lens[n]), 0)
        begin, tokens = tokens, tokens + a
        ok = a == 0 or (s + a <= per * P and tokens <= T)
        need = -(-(s + a) // P) - -(-s // P) if ok else 0
        asked += need
        if need and asked > free:
            ok = False
        if ok and need:
            for i in range(need):
                table[n, -(-s // P) + i] = stack.pop()
        cu.append(min(tokens, T))
        kv.append(s + a if ok else -1)
        after.append(s + a if ok else s)
        for i in range(a if ok else 0):
            page = int(table[n, (s + i) // P])
            row = page * P + (s + i) % P
            pos[begin + i] = s + i
            slots[begin + i] = row if page >= 0 and row <= 2 ** 31 - 1 else -1
    return dict(cu_seqlens=cu, positions=pos, slots=slots, kv_lens=kv, seq_lens=after, free_count=[len(stack)],
                block_table=table)


def release(finished, seq_lens, table, free_pages, free_count, page_size):
    """Returns free_pages (a copy), seq_lens and free_count."""
    N, per = np.asarray(table).shape
    free = np.array(free_pages, np.int64)
    count = min(max(int(free_count), 0), len(free))
    after = []
    for n in range(N):
        s = min(max(int(seq_lens[n]), 0), per * page_size)
        after.append(0 if finished[n] else s)
        for i in range(-(-s // page_size) if finished[n] else 0):
            if count < len(free):
                free[count] = table[n][i]
                count += 1
    return dict(free_pages=free, seq_lens=after, free_count=[count])
