"""Paged caches in which every page is seen: inputs of the absorbed latent attention's tests.

Each page carries a positive mark in one of the latent's upper channels, where the queries are zero.  A mark does not
change a score; the outputs' upper channels are weighted sums of marks alone, all of one sign, so that their bounds are
about 1% of their values, and a page, tile or part whose values are lost (or taken twice) moves some channel by far
more, however long the cache is.
"""

import numpy as np
import torch


def marked(seed, lens, page, H, R, Dr, q_lens=None, pool=0, rise=None):
    """q, cache (bfloat16, CPU), table, lens, cu.  Sequences draw their pages from a pool that they share (`pool` more
    pages than the longest needs); `rise` scales the scores along each sequence from rise[0] to rise[1]."""
    r = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    lens = np.asarray(lens, np.int32)
    per = max(1, -(-int(lens.max()) // page))
    pages = per + pool
    half = R // 2
    cache = torch.randn((pages, page, R + Dr), generator=g)
    if rise is not None:
        cache *= torch.linspace(rise[0], rise[1], pages)[:, None, None]
    cache[:, :, half:R] = 0
    p = torch.arange(pages)
    cache[p, :, half + p % half] = (4 + (p * 37 % 64) / 16.0)[:, None]
    table = np.stack([r.permutation(pages)[:per] for _ in lens])
    if rise is not None:
        table.sort(-1)
    cu = None if q_lens is None else np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = torch.randn((len(lens) if cu is None else int(cu[-1]), H, R + Dr), generator=g)
    q[..., half:R] = 0
    return q.to(torch.bfloat16), cache.to(torch.bfloat16), table.astype(np.int32), lens, cu


def run_length(lens, q_lens, H, R, page, per):
    """Rows of a block and (block, 64-row tile) units of a workgroup's run, as the kernel cuts the work."""
    lens = np.minimum(np.maximum(np.asarray(lens, np.int64), 0), page * per)
    q_lens = np.ones(len(lens), np.int64) if q_lens is None else np.asarray(q_lens, np.int64)
    rows = int(q_lens.sum()) * H
    mean = -(-rows // len(lens))
    height = 32 if mean <= 32 else 64 if mean <= 64 else 128
    units = int((-(-q_lens * H // height) * np.maximum(-(-lens // 64), 1)).sum())
    groups = min((rows // height + len(lens)) * max(-(-page * per // 64), 1), 512 if R == 128 else 256)
    return height, -(-units // groups)
