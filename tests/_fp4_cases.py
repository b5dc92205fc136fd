"""Inputs of the 4-bit latent cache's tests: the bf16 cases' caches in 4 bits, and what they stand for."""

import numpy as np
import torch

from oracle import mla_fp4 as orc4


def in_fp4(cache, R):
    """A bf16 cache [num_pages, page_size, R + Dr] as 4-bit rows (uint8, CPU) and the float64 values that they stand for.
    A latent that is NaN in a row becomes a NaN scale."""
    c = cache.double().numpy()
    codes, scales = orc4.quantise(c[..., :R])
    bits = cache[..., R:].contiguous().view(torch.int16).numpy().astype(np.uint16)
    rows = orc4.pack(codes, bits, scales)
    return torch.from_numpy(rows), orc4.unpack(rows, R, cache.shape[-1] - R)


def lengths(seed, N, hi, zero=0.2):
    r = np.random.default_rng(seed)
    x = r.integers(0, hi + 1, N)
    x[r.random(N) < zero] = 0
    return x.astype(np.int32)


def pages(seed, N, per, page, spare=5):
    """seq_lens, block_table (entries that are not owned hold anything), free_pages (longer than what is free), free_count."""
    r = np.random.default_rng(seed)
    lens = lengths(seed + 1, N, per * page)
    order = r.permutation(N * per + spare).astype(np.int32)
    table = order[:N * per].reshape(N, per).copy()
    owned = np.arange(per) < -(-lens // page)[:, None]
    free = np.concatenate([table[~owned], order[N * per:]])
    table[~owned] = r.integers(-9, 1 << 30, int((~owned).sum()))
    stack = np.full(len(order), -77, np.int32)
    stack[:len(free)] = free
    return lens, table, stack, np.array([len(free)], np.int32)
