"""Pins of the latent-attention oracle: closed forms, finite differences, the
absorbed form against the expanded one, and that its error bounds are neither
zero nor wide."""

import numpy as np
import pytest
import torch

from oracle import mla as orc

from ._paged_cases import marked


def _rng(seed):
    return np.random.default_rng(seed)


def test_equal_scores_give_running_means():
    r = _rng(0)
    kv = r.standard_normal((1, 9, 2, 6))
    o, lse, _, _ = orc.attention(np.zeros((1, 9, 2, 3)), kv)
    n = np.arange(1, 10)
    np.testing.assert_allclose(o, np.cumsum(kv[..., 3:], 1) / n[None, :, None, None], atol=1e-14)
    np.testing.assert_allclose(lse[0, :, 0], np.log(n), atol=1e-14)


def test_a_large_score_selects_its_value():
    kv = _rng(1).standard_normal((1, 5, 1, 8))
    kv[..., :4] = 0
    kv[0, 2, 0, :4] = 1
    o, _, _, _ = orc.attention(np.full((1, 5, 1, 4), 50.0), kv, scale=1.0)
    np.testing.assert_allclose(o[0, 2:, 0], np.repeat(kv[0, 2, :, 4:], 3, 0), atol=1e-12)


def test_documents_are_separate_sequences():
    r = _rng(2)
    q, kv, pe = r.standard_normal((1, 11, 2, 6)), r.standard_normal((1, 11, 2, 8)), r.standard_normal((1, 11, 2))
    o, lse, _, _ = orc.attention(q, kv, pe, cu_seqlens=[0, 4, 4, 10])
    for s, e in ((0, 4), (4, 10)):
        one, l1, _, _ = orc.attention(q[:, s:e], kv[:, s:e], pe[:, s:e])
        np.testing.assert_array_equal(o[:, s:e], one)
        np.testing.assert_array_equal(lse[:, s:e], l1)
    assert np.isnan(o[:, 10:]).all()


@pytest.mark.parametrize("Dr", [0, 2])
def test_backward_is_the_derivative(Dr):
    r = _rng(3)
    B, T, H, Dn = 1, 7, 2, 3
    x = dict(q=r.standard_normal((B, T, H, Dn + Dr)), kv=r.standard_normal((B, T, H, Dn + 4)))
    if Dr:
        x["k_pe"] = r.standard_normal((B, T, Dr))
    do = r.standard_normal((B, T, H, 4))
    cu = [0, 3, 7]
    loss = lambda y: float((orc.attention(y["q"], y["kv"], y.get("k_pe"), cu_seqlens=cu)[0] * do).sum())  # noqa: E731
    g, err = orc.attention_backward(x["q"], x["kv"], x.get("k_pe"), do, cu_seqlens=cu)
    h = 1e-6
    for n, gn in (("q", "dq"), ("kv", "dkv"), ("k_pe", "dk_pe")):
        if n not in x:
            continue
        for i in r.integers(0, x[n].size, 12):
            up, down = ({k: v.copy() for k, v in x.items()} for _ in range(2))
            up[n].reshape(-1)[i] += h
            down[n].reshape(-1)[i] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - g[gn].reshape(-1)[i]) < 1e-7
        assert (err[gn] > 0).all() and np.isfinite(err[gn]).all()


def test_absorbed_equals_expanded():
    """With k = W_k c and v = W_v c the two forms agree."""
    r = _rng(4)
    T, H, R, Dr, Dn, Dv, ps = 13, 3, 8, 2, 4, 5, 4
    c, pe, q = r.standard_normal((T, R)), r.standard_normal((T, Dr)), r.standard_normal((T, H, Dn + Dr))
    wk, wv = r.standard_normal((H, Dn, R)), r.standard_normal((H, Dv, R))
    kv = np.concatenate([np.einsum("hdr,tr->thd", wk, c), np.einsum("hdr,tr->thd", wv, c)], -1)
    scale = 0.3
    o, lse, _, _ = orc.attention(q[None], kv[None], pe[None], scale=scale)
    table = np.array([[2, 0, 3, 1]])
    cache = np.zeros((4, ps, R + Dr))
    rows = np.concatenate([c, pe], -1)
    for t in range(T):
        cache[table[0, t // ps], t % ps] = rows[t]
    qa = np.concatenate([np.einsum("hdr,thd->thr", wk, q[..., :Dn]), q[..., Dn:]], -1)
    for first in (0, 6, 12):  # the last T - first tokens as new ones
        oa, la, _, _ = orc.paged_attention(qa[first:], cache, table, [T], R, scale, cu_seqlens=[0, T - first])
        np.testing.assert_allclose(np.einsum("hdr,thr->thd", wv, oa), o[0, first:], atol=1e-12)
        np.testing.assert_allclose(la, lse[0, first:], atol=1e-12)


def test_paged_rows_that_see_nothing_and_missing_pages():
    r = _rng(5)
    cache = r.standard_normal((3, 2, 6))
    q = r.standard_normal((4, 1, 6))
    o, lse, _, _ = orc.paged_attention(q, cache, [[0, 7, 2]], [1], 4, 1.0, cu_seqlens=[0, 3])
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all()   # one row in the cache, three new tokens
    np.testing.assert_allclose(o[2, 0], cache[0, 0, :4])
    assert np.isnan(o[3]).all()
    a, _, _, _ = orc.paged_attention(q[:1], cache, [[0, 7, 2]], [6], 4, 1.0)
    b, _, _, _ = orc.paged_attention(q[:1], cache, [[0, 2, 2]], [4], 4, 1.0)
    np.testing.assert_array_equal(a, b)                        # page 7 is not there


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_angles(interleaved):
    r = _rng(6)
    Dr, P = 8, 40
    ang = np.arange(P)[:, None] * 10.0 ** -np.arange(Dr // 2)
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    c = r.standard_normal((2, 3 + Dr))
    rot = lambda i, p: orc.append(c[i:i + 1], 3, rope, [p], interleaved=interleaved)[0][0, 3:]  # noqa: E731
    np.testing.assert_allclose(np.linalg.norm(rot(0, 7)), np.linalg.norm(c[0, 3:]))
    np.testing.assert_allclose(rot(0, 12) @ rot(1, 5), rot(0, 30) @ rot(1, 23))
    np.testing.assert_array_equal(rot(0, -3), c[0, 3:])
    np.testing.assert_array_equal(rot(0, P + 9), rot(0, P - 1))
    row, _ = orc.append(c, 3, norm_weight=np.array([1.0, 2.0, 3.0]), eps=0.0)
    np.testing.assert_allclose((row[:, :3] / [1, 2, 3]) ** 2 @ np.ones(3), 3.0)
    np.testing.assert_array_equal(row[:, 3:], c[:, 3:])


def _bf16(x):
    return torch.tensor(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("mul", [4, 8])
def test_bounds_tell_a_delta_of_the_rounded_output(mul):
    """Rows that attend to few keys: the float32 sum of p dp keeps dq inside the bounds, <do, o> of the rounded o does
    not (a planted mistake)."""
    g = torch.Generator().manual_seed(3)
    T, D, Dv = 400, 192, 128
    q, k, v, do = (_bf16(torch.randn((T, n), generator=g) * c) for n, c in ((D, mul), (D, 1), (Dv, 1), (Dv, 1)))
    kv = np.concatenate([k, v], -1)[None, :, None]
    want, err = orc.attention_backward(q[None, :, None], kv, None, do[None, :, None])
    want, err = want["dq"][0, :, 0], err["dq"][0, :, 0]
    f = np.float32
    scale = f(D ** -0.5)
    s = np.where(np.tril(np.ones((T, T), bool)), q.astype(f) @ k.astype(f).T * scale, f(-np.inf))
    top = s.max(-1, keepdims=True)
    e = np.exp(s - top)
    lse = top + np.log(e.sum(-1, keepdims=True))
    p, dp = np.exp(s - lse), do.astype(f) @ v.astype(f).T
    o = _bf16(_bf16(e).astype(f) @ v.astype(f) / e.sum(-1, keepdims=True))

    def worst(delta):
        ds = _bf16(p * (dp - delta)).astype(f)
        return (np.abs(_bf16(ds @ k.astype(f) * scale) - want) / err)[128:].max()

    assert worst((p * dp).sum(-1, keepdims=True)) < 1
    assert worst((o.astype(f) * do.astype(f)).sum(-1, keepdims=True)) > 2


def test_bounds_tell_every_lost_part_of_a_long_cache():
    """A cache of 20,000 rows attended in parts of 64 rows and joined: any part's sums lost, or taken twice, are
    outside the bounds (planted mistakes); the join of all is inside."""
    R, page, L, H = 128, 64, 20000, 2
    q, cache, table, lens, _ = marked(9, [L], page, H, R, 0, pool=3)
    want, _, err, _ = orc.paged_attention(q, cache, table, lens, R, 0.1)
    k = orc.paged_rows(cache, table[0], L)[0]
    for h in range(H):
        s = k @ q[0, h].double().numpy() * 0.1
        w = np.exp(s - s.max())
        p = _bf16(w)  # weights are rounded as operands
        parts = np.stack([p[j:j + 64] @ k[j:j + 64] for j in range(0, L, 64)]) / w.sum()
        off = np.abs(_bf16(parts.sum(0)) - want[0, h])
        assert (off <= err[0, h]).all()
        assert (off[R // 2:] <= 0.02 * want[0, h, R // 2:]).all()
        for part in parts:
            for wrong in (parts.sum(0) - part, parts.sum(0) + part):
                assert (np.abs(wrong - want[0, h]) > 2 * err[0, h]).any()
