"""The 4-bit cache's oracle against its definition, by brute force.  CPU."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import mla_fp4 as orc

CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest(v):
    """Code of a value by exact fractions: nearest magnitude, even code of two, 6 above 6."""
    a = min(abs(Fraction(v)), Fraction(6))
    return min(range(8), key=lambda c: (abs(a - Fraction(CODES[c])), c % 2))


def test_codes_and_exponents_by_brute_force():
    r = np.random.default_rng(1)
    y = r.standard_normal((40, 64)) * np.exp2(r.integers(-20, 20, (40, 1)).astype(float))
    y[0, :32], y[1, 3] = 0.0, 7.0 * 2.0 ** 30
    y[2, :32] = np.linspace(-6, 6, 32) * 0.25
    codes, scales = orc.quantise(y)
    for row, cs, ss in zip(y.reshape(-1, 2, 32), codes.reshape(-1, 2, 32), scales):
        for b, c, s in zip(row, cs, ss):
            top = max(abs(Fraction(x)) for x in b)
            e = -125
            while top > 7 * Fraction(2) ** e:
                e += 1
            assert s == e + 127
            for x, k in zip(b, c):
                assert k & 7 == _nearest(Fraction(x) / Fraction(2) ** e)
                assert k >> 3 == np.signbit(x)


@pytest.mark.parametrize("tie,want", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (7.0, 7)])
def test_ties_go_to_the_even_code(tie, want):
    y = np.zeros((1, 32))
    y[0, 0], y[0, 1], y[0, 2] = 6.0, tie, -tie
    codes, scales = orc.quantise(y * 8.0)
    assert scales[0, 0] == 127 + 3 and list(codes[0, :3]) == [7, want, want + 8]


def test_limits_and_values_that_are_not_finite():
    y = np.zeros((1, 160))
    y[0, 5], y[0, 40], y[0, 70], y[0, 100] = 1e300, 1e-300, np.inf, np.nan
    codes, scales = orc.quantise(y)
    assert list(scales[0]) == [252, 2, 255, 255, 2]
    assert codes[0, 5] == 7 and not codes[0, 32:].any()
    v = orc.values(codes, scales)[0]
    assert v[5] == 6 * 2.0 ** 125 and np.isnan(v[64:128]).all() and not v[128:].any()


def test_rows_round_trip_and_are_fixed_points():
    r = np.random.default_rng(2)
    for R, Dr in ((128, 0), (128, 64), (256, 64), (512, 0)):
        codes, scales = orc.quantise(r.standard_normal((5, R)))
        pe = r.integers(0, 1 << 15, (5, Dr)).astype(np.uint16) & 0x7f00
        rows = orc.pack(codes, pe, scales)
        assert rows.shape[1] % 16 == 0 and rows.shape[1] - (R // 2 + 2 * Dr + R // 32) < 16
        v = orc.unpack(rows, R, Dr)
        again = orc.values(*orc.quantise(v[:, :R]))
        assert np.array_equal(v[:, :R], orc.values(codes, scales)) and v.shape == (5, R + Dr)
        # a value that a row can hold is kept: its block may take a smaller exponent, which has it too
        assert np.array_equal(v[:, :R], again)


def test_error_is_within_half_a_step():
    """A code is off by at most half the step around it, a channel by at most 1/7 of its block's largest."""
    r = np.random.default_rng(3)
    y = r.standard_normal((300, 32))
    v = orc.values(*orc.quantise(y))
    top = np.abs(y).max(-1, keepdims=True)
    assert (np.abs(v - y) <= top / 3.5 * 1.0 + 1e-12).all()
    assert np.sqrt(((v - y) ** 2).sum() / (y ** 2).sum()) < 0.12


def test_plan_and_release_keep_every_page_once():
    """Steps of a serving loop: every page is always in exactly one table or in the list, and slots never repeat."""
    r = np.random.default_rng(4)
    N, per, P, pages = 7, 5, 4, 24
    table, lens = np.full((N, per), -1), np.zeros(N, int)
    free, count = r.permutation(pages), pages
    for step in range(200):
        new = r.integers(0, 6, N)
        T = int(new.sum()) - int(r.integers(0, 2)) if new.sum() else 0
        p = orc.plan(new, lens, table, free, count, P, max(T, 0))
        table, lens, count = p["block_table"], np.array(p["seq_lens"]), p["free_count"][0]
        kept = p["slots"][p["slots"] >= 0]
        assert len(set(kept)) == len(kept)
        owned = [table[n, i] for n in range(N) for i in range(-(-lens[n] // P))]
        assert sorted(owned + list(free[:count])) == list(range(pages))
        for n in range(N):
            if p["kv_lens"][n] >= 0:
                assert p["kv_lens"][n] == lens[n]
        done = r.random(N) < 0.2
        q = orc.release(done, lens, table, free, count, P)
        free, lens, count = q["free_pages"], np.array(q["seq_lens"]), q["free_count"][0]
        assert not lens[done].any()


def test_plan_refuses_in_order():
    table = np.full((4, 3), -1)
    # capacity 12: the first does not fit its row, the second takes both pages, the third has none left, the fourth fits
    # the page it has
    table[3, 0] = 9
    p = orc.plan([13, 8, 1, 2], [0, 0, 0, 1], table, np.array([5, 6]), 2, 4, 30)
    assert p["kv_lens"] == [-1, 8, -1, 3] and p["free_count"] == [0] and p["seq_lens"] == [0, 8, 0, 3]
    assert p["cu_seqlens"] == [0, 13, 21, 22, 24] and list(p["block_table"][1]) == [6, 5, -1]
    assert list(p["slots"][13:24]) == [24, 25, 26, 27, 20, 21, 22, 23, -1, 37, 38]
    p = orc.plan([3, 2], [0, 0], np.full((2, 3), -1), np.array([5, 6]), 2, 4, 4)  # the second's tokens end behind T
    assert p["kv_lens"] == [3, -1] and p["cu_seqlens"] == [0, 3, 4] and p["free_count"] == [1]


def test_scales_past_the_largest_are_nan():
    codes = np.tile(np.arange(16, dtype=np.uint8), (5, 2))
    v = orc.values(codes, np.array([[0], [252], [253], [254], [255]], np.uint8))
    assert np.isfinite(v[:2]).all() and v[0, 7] == 6 * 2.0 ** -127 and v[1, 15] == -6 * 2.0 ** 125
    assert np.isnan(v[2:]).all()
