"""Latent attention on the GPU against the CPU fp64 oracle.

Tolerances: elementwise, the oracle's own bounds (oracle/mla.py): half a bf16
step for the output and for each operand the kernels round to bf16 (the
softmax weights, and dS in the backward), half a float32 step an addition for
the float32 sums.  A rotated or normalised value: half a bf16 step, plus 16
float32 half steps of its terms.  Inputs are drawn once per case; nothing is
re-drawn.
"""

import numpy as np
import pytest
import torch

from gated_delta_rule_04_amd import mla
from oracle import mla as orc

from ._paged_cases import marked, run_length

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
CANARY = 77.0


def _randn(seed, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(BF16)


def _i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32))


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _within(name, got, ref, err):
    got = got.detach().cpu().double().numpy()
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), name
    ok = ~inf & ~np.isnan(ref)
    assert np.isfinite(got[ok]).all(), name + ": non-finite values"
    d = np.abs(got[ok] - ref[ok])
    over = d / np.maximum(err[ok], 1e-30)
    print("BOUND %-28s max-abs %.3e, of its bound at most %.2f" % (name, d.max(initial=0), over.max(initial=0)), flush=True)
    assert (d <= err[ok] + 1e-30).all(), "%s: %.3e off, %.2f times the bound" % (name, d.max(), over.max())


HEADS = [(64, 0), (64, 64), (128, 0), (128, 64)]


def _expanded(seed, B, T, H, Dn, Dr, scale=1.0):
    return (_randn(seed, B, T, H, Dn + Dr, scale=scale), _randn(seed + 1, B, T, H, 2 * Dn),
            _randn(seed + 2, B, T, Dr) if Dr else None, _randn(seed + 3, B, T, H, Dn))


def _check_expanded(tag, q, kv, pe, do, cu=None, scale=None):
    dq, dkv, dpe, ddo = _cuda(q, kv, pe, do)
    dcu = None if cu is None else _i32(cu).cuda()
    B, T, H, _ = q.shape
    o = torch.full(tuple(do.shape), CANARY, dtype=BF16, device="cuda")
    lse = torch.full((B, T, H), CANARY, device="cuda")
    mla.attn_fwd(dq, dkv, dpe, scale=scale, cu_seqlens=dcu, out=o, lse=lse)
    r = orc.attention(q, kv, pe, scale=scale, cu_seqlens=cu)
    _within(tag + " o", o, r[0], r[2])
    _within(tag + " lse", lse, r[1], r[3])
    need = mla.attn_bwd_workspace_bytes(B, T, H, do.shape[-1], 0 if pe is None else pe.shape[-1], do.shape[-1],
                                        B if cu is None else len(cu) - 1)
    ws = torch.full((max(need, 1) + 256,), 255, dtype=torch.uint8, device="cuda")  # NaN bits
    out = {"dq": torch.full_like(dq, CANARY), "dkv": torch.full_like(dkv, CANARY)}
    if pe is not None:
        out["dk_pe"] = torch.full_like(dpe, CANARY)
    mla.attn_bwd(dq, dkv, dpe, o, lse, ddo, scale=scale, cu_seqlens=dcu, workspace=ws[:need], out=out)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 255).all())
    g, err = orc.attention_backward(q, kv, pe, do, scale=scale, cu_seqlens=cu)
    for n in g:
        _within(tag + " " + n, out[n], g[n], err[n])
    if cu is not None and cu[-1] < T:  # rows behind the last document stay as they were
        for t in (o, lse, *out.values()):
            assert bool((t[:, cu[-1]:] == CANARY).all()), tag
    return o, lse, out


@pytest.mark.parametrize("Dn,Dr", HEADS)
@pytest.mark.parametrize("T", [1, 2, 31, 33, 64, 65, 127, 129, 200, 321])
def test_expanded_lengths(Dn, Dr, T):
    print("CASE expanded", Dn, Dr, T, flush=True)
    _check_expanded("T%d" % T, *_expanded(T, 2 if T < 200 else 1, T, 3, Dn, Dr))


@pytest.mark.parametrize("Dn,Dr", HEADS)
@pytest.mark.parametrize("cu", [[0, 1, 1, 70, 71, 200], [0, 0, 130, 130], [0, 64, 128, 256, 300], [0, 5], [0, 0]])
def test_expanded_documents(Dn, Dr, cu):
    print("CASE documents", Dn, Dr, cu, flush=True)
    T = cu[-1] + (9 if Dn == 64 else 0)
    if T:
        _check_expanded("docs", *_expanded(7, 1, T, 2, Dn, Dr), cu=cu)


def test_expanded_many_short_documents():
    r = np.random.default_rng(3)
    cu = np.concatenate([[0], np.cumsum(r.integers(0, 9, 150))]).tolist()
    _check_expanded("short docs", *_expanded(8, 1, cu[-1] + 3, 2, 64, 64), cu=cu)


@pytest.mark.parametrize("scale", [0.02, 1.5])
def test_expanded_scales_and_large_scores(scale):
    """Scores of hundreds, and ones that rise along the keys: the running maximum moves at every tile."""
    q, kv, pe, do = _expanded(11, 1, 300, 2, 128, 64, scale=4.0)
    kv = (kv.float() * torch.linspace(0.1, 3.0, 300)[None, :, None, None]).to(BF16)
    _check_expanded("large", q, kv, pe, do, scale=scale)


@pytest.mark.parametrize("Dn,Dr", HEADS)
@pytest.mark.parametrize("mul", [4, 8])
def test_expanded_rows_that_attend_to_few_keys(Dn, Dr, mul):
    """Sharp rows far into a document: their dS is small beside any common error of delta."""
    print("CASE sharp", Dn, Dr, mul, flush=True)
    _check_expanded("sharp", *_expanded(61, 1, 400, 2, Dn, Dr, scale=mul))
    _check_expanded("sharp docs", *_expanded(62, 1, 500, 1, Dn, Dr, scale=mul), cu=[0, 190, 191, 480])


def test_expanded_odd_heads_and_batch():
    _check_expanded("H1", *_expanded(21, 1, 150, 1, 128, 64))
    _check_expanded("H13 B5", *_expanded(22, 5, 70, 13, 64, 0))


@pytest.mark.parametrize("Dn,Dr", HEADS)
def test_expanded_heads_by_eights_and_many_tiles(Dn, Dr):
    """Heads (times batch rows) that are a multiple of 8, several tiles each: a launch order of its own."""
    print("CASE eights", Dn, Dr, flush=True)
    _check_expanded("H8", *_expanded(25, 1, 300, 8, Dn, Dr))
    _check_expanded("B3 H8", *_expanded(26, 3, 300, 8, Dn, Dr))
    _check_expanded("H16 docs", *_expanded(27, 1, 420, 16, Dn, Dr), cu=[0, 140, 140, 141, 410])


def test_expanded_most_heads():
    _check_expanded("H 1024", *_expanded(24, 1, 40, 1024, 64, 0))


def test_expanded_offsets_past_32_bits():
    """Packed documents whose q, kv, o and gradients pass 2^31 elements: the last ones are as when they are alone."""
    H, Dn, Dr, doc, last = 96, 128, 64, 230, 610
    n = (1 << 31) // (H * Dn * doc) + 1  # documents ahead, so that o passes 2^31 elements too
    cu = np.concatenate([np.arange(n + 1) * doc, n * doc + np.array([77, 77, last])])
    T = int(cu[-1])
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF16)  # noqa: E731
    q, kv, pe, do = rnd(1, T, H, Dn + Dr), rnd(1, T, H, 2 * Dn), rnd(1, T, Dr), rnd(1, T, H, Dn)
    assert do.numel() > 1 << 31

    def run(args, cu):
        cu = _i32(cu).cuda()
        o, lse = mla.attn_fwd(*args[:3], cu_seqlens=cu)
        return [o, lse, *mla.attn_bwd(*args[:3], o, lse, args[3], cu_seqlens=cu).values()]

    end = [t[:, n * doc:].clone() for t in (q, kv, pe, do)]
    for a, b in zip(run((q, kv, pe, do), cu), run(end, cu[n:] - n * doc)):
        assert torch.equal(a[:, n * doc:], b) and bool(torch.isfinite(b.float()).all())


def test_calls_without_a_log_sum_exp():
    """lse is optional in the library: the outputs are the same bits without it."""
    ptr = lambda t: t.data_ptr()  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    q, kv, pe, _ = _cuda(*_expanded(71, 1, 200, 3, 128, 64))
    o, _ = mla.attn_fwd(q, kv, pe)
    got = torch.empty_like(o)
    assert mla.lib().kda_mla_attn_fwd(ptr(q), ptr(kv), ptr(pe), ptr(got), None, None, 1, 1, 200, 3, 128, 64, 128,
                                      192 ** -0.5, mla.KDA_BF16, stream) == 0
    assert torch.equal(o, got)
    q, cache, table, lens, _ = _paged(72, [300, 20000], 64, 5, 128, 64)
    q, cache, table, lens = _cuda(q, cache, _i32(table), _i32(lens))
    o, _ = mla.paged_attn(q, cache, table, lens, 128, 0.1)
    need = mla.paged_workspace_bytes(2, 2, 5, 128, 64, 64, table.shape[1])
    got, ws = torch.empty_like(o), torch.empty(need, dtype=torch.uint8, device="cuda")
    assert mla.lib().kda_mla_paged_attn(ptr(q), ptr(cache), ptr(table), ptr(lens), None, ptr(got), None, 2, 2, 5, 128, 64,
                                        cache.shape[0], 64, table.shape[1], 0.1, mla.KDA_BF16, ptr(ws), need, stream) == 0
    assert torch.equal(o, got)


def test_expanded_other_documents_do_not_matter():
    cu, T = [0, 90, 170, 300], 300
    q, kv, pe, do = _expanded(31, 1, T, 2, 128, 64)
    dcu = _i32(cu).cuda()

    def run(q, kv, pe, do):
        args = _cuda(q, kv, pe)
        o, lse = mla.attn_fwd(*args, cu_seqlens=dcu)
        return [o, lse, *mla.attn_bwd(*args, o, lse, do.cuda(), cu_seqlens=dcu).values()]

    clean = run(q, kv, pe, do)
    for t in (q, kv, pe, do):
        t[:, 90:170] = float("nan")
    t = q[:, 100]
    t[:] = float("inf")
    for a, b in zip(clean, run(q, kv, pe, do)):
        assert torch.equal(a[:, :90], b[:, :90]) and torch.equal(a[:, 170:], b[:, 170:])
        assert bool(torch.isnan(b[:, 90:170].float()).any())


def test_expanded_repeats_bitwise_and_empty():
    q, kv, pe, do = _cuda(*_expanded(41, 2, 300, 3, 128, 64))
    runs = []
    for _ in range(2):
        o, lse = mla.attn_fwd(q, kv, pe)
        runs.append([o, lse, *mla.attn_bwd(q, kv, pe, o, lse, do).values()])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    for shape in ((0, 5), (2, 0)):
        e = [torch.empty(shape + (3, 192), dtype=BF16, device="cuda"), torch.empty(shape + (3, 256), dtype=BF16, device="cuda"),
             torch.empty(shape + (64,), dtype=BF16, device="cuda")]
        o, lse = mla.attn_fwd(*e)
        g = mla.attn_bwd(*e, o, lse, o)
        assert o.shape == shape + (3, 128) and g["dq"].shape == e[0].shape


# ---------------------------------------------------------------------------
# absorbed form over the paged cache
# ---------------------------------------------------------------------------
def _paged(seed, lens, page, H, R, Dr, q_lens=None, spare=2, pad=0):
    """Inputs on the CPU.  Everything in the cache that no sequence owns is NaN."""
    r = np.random.default_rng(seed)
    N, D = len(lens), R + Dr
    per = max(1, max(-(-int(n) // page) for n in lens)) + 1
    pages = N * per + spare
    table = r.permutation(pages)[:N * per].reshape(N, per).astype(np.int32)
    cache = torch.full((pages, page, D), float("nan"), dtype=BF16)
    rows = _randn(seed, int(sum(lens)), D)
    at = 0
    for n, L in enumerate(lens):
        j = np.arange(L)
        cache[torch.as_tensor(table[n][j // page]).long(), torch.as_tensor(j % page)] = rows[at:at + L]
        at += L
    cu = None if q_lens is None else np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    Tq = N if q_lens is None else int(cu[-1])
    q = _randn(seed + 1, Tq + pad, H, D)
    return q, cache, table, np.asarray(lens, np.int32), cu


def _check_paged(tag, q, cache, table, lens, cu, R, scale=None):
    scale = (128 + q.shape[-1] - R) ** -0.5 if scale is None else scale
    Tq, H, D = q.shape
    dev = _cuda(q, cache, _i32(table), _i32(lens), None if cu is None else _i32(cu))
    o = torch.full((Tq, H, R), CANARY, dtype=BF16, device="cuda")
    lse = torch.full((Tq, H), CANARY, device="cuda")
    need = mla.paged_workspace_bytes(len(lens), Tq, H, R, D - R, cache.shape[1], table.shape[1])
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    mla.paged_attn(*dev[:4], R, scale, cu_seqlens=dev[4], out=o, lse=lse, workspace=ws[:need] if need else None)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 255).all())
    r = orc.paged_attention(q, cache, table, lens, R, scale, cu_seqlens=cu)
    _within(tag + " o", o, r[0], r[2])
    _within(tag + " lse", lse, r[1], r[3])
    if cu is not None and cu[-1] < Tq:
        assert bool((o[cu[-1]:] == CANARY).all()) and bool((lse[cu[-1]:] == CANARY).all())
    return o, lse


LATENT = [(128, 0), (128, 64), (256, 0), (256, 64), (512, 0), (512, 64)]


@pytest.mark.parametrize("R,Dr", LATENT)
@pytest.mark.parametrize("page", [1, 16, 24, 64, 100])
def test_paged_single_tokens(R, Dr, page):
    print("CASE paged", R, Dr, page, flush=True)
    _check_paged("page %d" % page, *_paged(page, [1, 63, 64, 65, 0, 300], page, 5, R, Dr), R)


@pytest.mark.parametrize("H", [1, 8, 16, 31, 32, 33, 64, 65, 96, 100, 128, 129])
@pytest.mark.parametrize("R,Dr", [(128, 0), (512, 64)])
def test_paged_heads(H, R, Dr):
    print("CASE heads", H, R, flush=True)
    _check_paged("H %d" % H, *_paged(H, [70, 131], 16, H, R, Dr), R)


@pytest.mark.parametrize("R,Dr", LATENT)
def test_paged_chunks(R, Dr):
    """New tokens that end a longer cache, fill it, outnumber it (rows that see nothing), or are none; padding behind."""
    print("CASE chunks", R, Dr, flush=True)
    _check_paged("chunks", *_paged(5, [200, 70, 9, 40, 0], 24, 3, R, Dr, q_lens=[50, 70, 20, 0, 6], pad=11), R)


def test_paged_chunk_spans_many_row_blocks():
    _check_paged("long chunk", *_paged(6, [150, 260], 64, 12, 512, 64, q_lens=[150, 33]), 512)


def test_paged_long_cache_is_split():
    _check_paged("long", *_paged(9, [20000], 64, 8, 128, 64), 128)
    _check_paged("long ragged", *_paged(10, [9000, 3, 0, 2500], 64, 4, 512, 64), 512)


def _check_all_rows(tag, q, cache, table, lens, cu, R, scale, run=None):
    """Every row of a large call against float64 on the GPU, within the bounds of oracle.mla.attend."""
    if run is not None:  # the shapes give each workgroup at least this many tiles in a row
        assert run_length(lens, None if cu is None else np.diff(cu), q.shape[1], R, cache.shape[1], table.shape[1])[1] >= run
    Tq, H, D = q.shape
    dq, dc, dt, dl = _cuda(q, cache, _i32(table), _i32(lens))
    o, lse = mla.paged_attn(dq, dc, dt, dl, R, scale, cu_seqlens=None if cu is None else _i32(cu).cuda())
    torch.cuda.synchronize()
    print("DONE", tag, flush=True)
    starts = np.arange(len(lens) + 1) if cu is None else cu
    worst = [0.0, 0.0]
    for n, L in enumerate(lens):
        b, e, L = int(starts[n]), int(starts[n + 1]), int(L)
        if e == b:
            continue
        j = torch.arange(L, device="cuda")
        page = dt[n].long()[j // cache.shape[1]]
        there = (page >= 0) & (page < cache.shape[0])
        k = dc[page.clamp(0, cache.shape[0] - 1), j % cache.shape[1]].double() * there[:, None]
        qq = dq[b:e].double().reshape(-1, D)
        tok = torch.arange(e - b, device="cuda").repeat_interleave(H)
        sees = there & (j <= (L - (e - b) + tok)[:, None])
        s = (qq @ k.T * scale).masked_fill(~sees, -float("inf"))
        es = ((D + 16) * orc.U * scale * (qq.abs() @ k.abs().T)).masked_fill(~sees, 0.0)
        lse64 = torch.logsumexp(s, -1) if L else torch.full((len(qq),), -float("inf"), device="cuda").double()
        empty = torch.isinf(lse64)
        p = torch.exp(s - lse64.masked_fill(empty, 0.0)[:, None])
        want, mag = p @ k[:, :R], p @ k[:, :R].abs()
        w = es.amax(-1, keepdim=True) if L else es.sum(-1, keepdim=True)
        err = (orc.E + 2 * w + (64 + L) * orc.U) * mag + orc.E * want.abs()
        err_l = w[:, 0] + (64 + L) * orc.U + 4 * orc.U * lse64.masked_fill(empty, 0.0).abs()
        got, got_l = o[b:e].double().reshape(-1, R), lse[b:e].double().reshape(-1)
        assert bool((got_l[empty] == -float("inf")).all()) and bool((got[empty] == 0).all()), (tag, n)
        off, off_l = (got - want).abs(), (got_l - lse64)[~empty].abs()
        assert bool((off <= err + 1e-30).all()) and bool((off_l <= err_l[~empty]).all()), (tag, n, float((off / (err + 1e-30)).max()))
        worst = [max(worst[0], float((off / (err + 1e-30)).max())), max([worst[1], *(off_l / err_l[~empty]).tolist()])]
    print("BOUND %-28s of its bound at most %.2f, lse %.2f" % (tag, *worst), flush=True)


def _many(R, seed, hi=6000):
    """Lengths whose tiles are more than 32 times the workgroups', short and empty sequences among them."""
    lens = np.random.default_rng(seed).integers(1, hi + 1, 420 if R == 128 else 220)
    lens[3::17] = lens[3::17] % 200
    lens[5], lens[40] = 0, hi
    return lens


@pytest.mark.parametrize("R,Dr", LATENT)
@pytest.mark.parametrize("H,page", [(5, 16), (40, 64), (96, 100)])
def test_paged_long_runs_of_tiles(R, Dr, H, page):
    """Runs of more than 32 tiles a workgroup, over the ends of sequences, in blocks of 32, 64 and 128 rows."""
    print("CASE runs", R, Dr, H, page, flush=True)
    lens = _many(R, H)
    _check_all_rows("runs H%d R%d" % (H, R), *marked(H + R, lens, page, H, R, Dr, pool=9), R, 0.1, run=33)


@pytest.mark.parametrize("H", [5, 40, 96])
def test_paged_long_runs_with_missing_pages(H):
    print("CASE runs, missing", H, flush=True)
    q, cache, table, lens, cu = marked(71 + H, _many(512, H + 1), 24, H, 512, 64, pool=9)
    r = np.random.default_rng(H)
    gone = r.random(table.shape) < 0.03
    table[gone] = r.choice([-1, cache.shape[0], 1 << 30], int(gone.sum()))
    _check_all_rows("missing H%d" % H, q, cache, table, lens, cu, 512, 0.1, run=33)


@pytest.mark.parametrize("R,Dr,H", [(512, 64, 5), (512, 0, 40), (512, 64, 96), (256, 64, 12), (128, 0, 8)])
def test_paged_long_runs_of_rising_scores(R, Dr, H):
    print("CASE runs, rising", R, Dr, H, flush=True)
    _check_all_rows("rising H%d R%d" % (H, R), *marked(81 + H, _many(R, H + 2), 64, H, R, Dr, pool=9, rise=(0.05, 4.0)), R,
                    0.3, run=33)


@pytest.mark.parametrize("R,Dr", LATENT)
def test_paged_long_runs_of_chunks(R, Dr):
    """Several row blocks a sequence, each a run of tiles or more."""
    print("CASE runs, chunks", R, Dr, flush=True)
    r = np.random.default_rng(R + Dr)
    N = 48 if R == 128 else 24
    q_lens = r.integers(0, 90, N)
    lens = np.maximum(r.integers(1500, 6000, N), q_lens)
    lens[2], lens[7] = q_lens[2], q_lens[7] // 2  # a first chunk, and one with rows that see nothing
    _check_all_rows("chunks R%d" % R, *marked(91 + R, lens, 24, 16, R, Dr, q_lens=q_lens, pool=9), R, 0.1, run=17)


@pytest.mark.parametrize("R,Dr,H,lens", [(128, 0, 8, [20000]), (512, 64, 12, [131072]), (256, 0, 64, [70000, 900]),
                                         (512, 64, 96, [30000, 0, 41000])])
def test_paged_every_part_of_a_long_cache(R, Dr, H, lens):
    print("CASE parts", R, H, lens, flush=True)
    _check_all_rows("parts R%d" % R, *marked(101 + H, lens, 64, H, R, Dr, pool=3), R, 0.1)


def test_paged_scores_that_rise_and_large_ones():
    q, cache, table, lens, cu = _paged(12, [700], 16, 16, 256, 64)
    up = torch.linspace(0.05, 4.0, 700)
    for j in range(700):
        cache[table[0][j // 16], j % 16] = (cache[table[0][j // 16], j % 16].float() * up[j]).to(BF16)
    _check_paged("rising", q, cache, table, lens, cu, 256, scale=0.7)


def test_paged_missing_pages_are_left_out():
    q, cache, table, lens, cu = _paged(13, [200, 130, 64], 16, 9, 128, 64)
    table[0][[0, 3, 7]] = [-1, 1 << 30, cache.shape[0]]
    table[1][:] = -5                       # nothing is there: a row that sees nothing
    _check_paged("missing", q, cache, table, lens, cu, 128)


def test_paged_lengths_are_clamped_and_pages_shared():
    q, cache, table, lens, cu = _paged(14, [48, 48], 16, 4, 128, 0)
    table = table[:, :3].copy()
    table[1] = table[0]                    # a shared prefix
    _check_paged("clamped", q, cache, table, np.array([1 << 30, -7], np.int32), cu, 128)


def test_paged_rows_of_other_sequences_do_not_matter():
    q, cache, table, lens, cu = _paged(15, [100, 90, 300], 16, 8, 512, 64)
    args = lambda: (*_cuda(q, cache, _i32(table), _i32(lens)), 512, 0.07)  # noqa: E731
    o, lse = mla.paged_attn(*args())
    for j in range(90):
        cache[table[1][j // 16], j % 16] = float("nan")
    o2, lse2 = mla.paged_attn(*args())
    keep = torch.tensor([0, 2], device="cuda")
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert bool(torch.isnan(o2[1].float()).all())


def test_paged_many_sequences():
    """More sequences than threads of a workgroup: single tokens, and chunks with empty ones among them."""
    r = np.random.default_rng(23)
    lens = r.integers(0, 90, 700).tolist()
    _check_paged("700 single", *_paged(23, lens, 16, 2, 128, 64), 128)
    _check_paged("700 chunks", *_paged(24, lens, 16, 2, 128, 0, q_lens=r.integers(0, 4, 700).tolist(), pad=3), 128)


@pytest.mark.parametrize("R,Dr,H", [(128, 64, 1), (512, 0, 80)])
def test_paged_most_sequences(R, Dr, H):
    """65,536 sequences of one cache row or none (with 80 heads of 512 channels, offsets of q and o past 2^31): a row
    that sees one row gives its latent, exactly."""
    print("CASE most sequences", R, H, flush=True)
    N, pages, page = 1 << 16, 300, 4
    g = torch.Generator(device="cuda").manual_seed(R)
    cache = torch.randn((pages, page, R + Dr), generator=g, device="cuda").to(BF16)
    table = torch.randint(0, pages, (N, 2), generator=g, device="cuda", dtype=torch.int32)
    lens = (torch.rand(N, generator=g, device="cuda") < 0.8).to(torch.int32)
    q = torch.randn((N, H, R + Dr), generator=g, device="cuda", dtype=BF16)
    o, lse = mla.paged_attn(q, cache, table, lens, R, 0.05)
    for b in range(0, N, 4096):
        x = slice(b, b + 4096)
        one = lens[x, None, None] == 1
        row = cache[table[x, 0].long(), 0]
        assert torch.equal(o[x], torch.where(one, row[:, None, :R], torch.zeros((), dtype=BF16, device="cuda")).expand(-1, H, -1))
        s = (q[x].float() * row[:, None].float()).sum(-1) * 0.05
        mag = (q[x].float() * row[:, None].float()).abs().sum(-1) * 0.05
        off = (lse[x] - s).abs() - (2 * (R + Dr + 16) * orc.U * mag + 64 * orc.U)  # two float32 sums
        assert bool((torch.where(one[..., 0], off, -torch.ones_like(off)) <= 0).all())
        assert bool(torch.isneginf(lse[x][lens[x] == 0]).all())


def test_paged_most_heads():
    _check_paged("H 1024", *_paged(25, [130], 64, 1024, 256, 0), 256)


def test_paged_no_pages_and_no_rows():
    q = _randn(26, 3, 4, 192).cuda()
    empty = torch.empty((0, 16, 192), dtype=BF16, device="cuda")
    for per in (0, 2):  # a table that names pages of an empty cache, and none
        table = torch.zeros((3, per), dtype=torch.int32, device="cuda")
        o, lse = mla.paged_attn(q, empty, table, _i32([0, 5, 9]).cuda(), 128, 0.1)
        assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    o, lse = mla.paged_attn(q[:0], empty, table[:0], _i32([]).cuda(), 128, 0.1)
    assert o.shape == (0, 4, 128)


def test_two_calls_at_once_on_two_streams():
    args = []
    for i in range(2):
        q, cache, table, lens, cu = _paged(27 + i, [3000, 500], 64, 12, 512, 64)
        args.append(_cuda(q, cache, _i32(table), _i32(lens)))
    want = [mla.paged_attn(*a, 512, 0.07) for a in args]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in args], []
    for _ in range(3):
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(mla.paged_attn(*a, 512, 0.07))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_paged_offsets_past_32_bits():
    """Pages whose rows lie past 2^31 elements and 2^32 bytes of the cache."""
    page, D = 64, 576
    pages = (1 << 32) // (page * D * 2) + 40
    cache = torch.empty((pages, page, D), dtype=BF16, device="cuda")
    table = np.array([[pages - 1, 3, pages - 7]], np.int32)
    small = _randn(16, 3, page, D)
    for i, p in enumerate(table[0]):
        cache[int(p)] = small[i].cuda()
    q = _randn(17, 1, 12, D)
    o, lse = mla.paged_attn(q.cuda(), cache, _i32(table).cuda(), _i32([150]).cuda(), 512, 0.07)
    r = orc.paged_attention(q, small, np.array([[0, 1, 2]]), [150], 512, 0.07)
    _within("far o", o, r[0], r[2])
    c, w = _randn(18, 2, D), torch.ones(512)
    mla.cache_append(c.cuda(), None, _i32([(pages - 1) * page + 63, (pages - 2) * page]).cuda(), cache, 512,
                     norm_weight=w.cuda())
    row, _ = orc.append(c, 512, norm_weight=w)
    for i, got in enumerate((cache[pages - 1, 63], cache[pages - 2, 0])):
        _within("far row", got, row[i], orc.E * np.abs(row[i]) + 16 * orc.U * np.abs(row[i]))


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("R,Dr", LATENT)
@pytest.mark.parametrize("T", [1, 7, 130])
def test_append(R, Dr, T):
    print("CASE append", R, Dr, T, flush=True)
    r = np.random.default_rng(T)
    P, page, H, n_pos = 9, 24, 5, 300
    ang = np.arange(n_pos)[:, None] * 100.0 ** (-np.arange(Dr // 2) / max(Dr // 2, 1))
    rope = torch.tensor(np.concatenate([np.cos(ang), np.sin(ang)], 1), dtype=torch.float32)
    c, q_pe, q0 = _randn(T, T, R + Dr), _randn(T + 1, T, H, Dr), _randn(T + 2, T, H, R + Dr)
    w = 1 + 0.3 * torch.randn(R, generator=torch.Generator().manual_seed(T))
    pos = r.integers(-5, n_pos + 5, T).astype(np.int32)
    slots = r.permutation(P * page)[:T].astype(np.int32)
    slots[::4] = r.choice([-1, P * page, 1 << 30], len(slots[::4]))
    for inter, use_w, use_rope in ((False, True, Dr > 0), (True, False, Dr > 0), (False, True, False)):
        cache0 = _randn(T + 3, P, page, R + Dr)
        cache, q = cache0.cuda(), q0.cuda()
        got = mla.cache_append(c.cuda(), _i32(pos).cuda(), _i32(slots).cuda(), cache, R,
                               rope=rope.cuda() if use_rope else None, norm_weight=w.cuda() if use_w else None,
                               eps=1e-5, interleaved=inter, q_pe=q_pe.cuda() if Dr else None, q=q if Dr else None)
        assert got is cache
        row, qr = orc.append(c, R, rope if use_rope else None, pos, w if use_w else None, 1e-5, inter, q_pe if Dr else None)
        mag, qmag = np.abs(row), np.abs(q_pe.double().numpy()).max() * np.ones(q_pe.shape) if Dr else None
        mag[:, R:] = np.abs(c.double().numpy()[:, R:]).max(initial=0)
        flat = cache.cpu().view(P * page, -1)
        kept = (slots >= 0) & (slots < P * page)
        _within("row", flat[torch.as_tensor(slots[kept]).long()], row[kept], (orc.E * np.abs(row) + 16 * orc.U * mag)[kept])
        others = np.setdiff1d(np.arange(P * page), slots[kept])
        assert torch.equal(flat[torch.as_tensor(others)], cache0.view(P * page, -1)[torch.as_tensor(others)])
        if Dr:
            assert torch.equal(q.cpu()[..., :R], q0[..., :R])
            _within("q", q[..., R:], qr, orc.E * np.abs(qr) + 16 * orc.U * qmag)
        else:
            assert torch.equal(q.cpu(), q0)


def test_append_without_rotation_copies_any_bits():
    c = _randn(3, 4, 576)
    c[0, :40] = float("inf")
    c[1, 500:] = float("nan")
    c[2, 570] = float("-inf")
    cache = torch.zeros((1, 8, 576), dtype=BF16, device="cuda")
    mla.cache_append(c.cuda(), None, _i32([1, 3, 5, 7]).cuda(), cache, 512)
    assert torch.equal(cache[0, 1::2].cpu().view(torch.int16), c.view(torch.int16))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_prefill_then_decode_equals_the_expanded_form():
    """A layer as it is served: a chunk of tokens appended and attended, then single tokens; against the expanded
    form on the same projections.  The inputs of both are rounded to bf16 on the way (the absorbed queries, the
    expanded keys and values), so the comparison is to the two forms' relative size: each rounding is at most 2^-8 of
    its value, scores are about one, so the softmax weights are off by about 3 2^-8 (q', rows, k) and a value by
    about 2 2^-8: under 8 2^-8 in relative L2."""
    g = torch.Generator().manual_seed(5)
    H, Dn, Dr, Dv, R, page = 8, 128, 64, 128, 512, 16
    lens, steps, n_pos = [70, 33], 4, 128
    T = max(lens) + steps
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    wk, wv = rnd(H, Dn, R) * R ** -0.5, rnd(H, Dv, R) * R ** -0.5
    ang = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(Dr // 2) / (Dr // 2))
    rope = torch.tensor(np.concatenate([np.cos(ang), np.sin(ang)], 1), dtype=torch.float32).cuda()
    c = rnd(2, T, R + Dr).to(BF16)
    q = rnd(2, T, H, Dn + Dr).to(BF16)
    weight = (1 + 0.1 * rnd(R)).cuda()
    scale = (Dn + Dr) ** -0.5
    # expanded, from the same definitions on the CPU
    pos = np.tile(np.arange(T), 2)
    rows, qr = orc.append(c.reshape(2 * T, -1), R, rope, pos, weight, q_pe=q[..., Dn:].reshape(2 * T, H, Dr))
    lat = torch.tensor(rows[:, :R]).float()
    kv = torch.cat([torch.einsum("hdr,tr->thd", wk, lat), torch.einsum("hdr,tr->thd", wv, lat)], -1)
    kv = kv.view(2, T, H, -1).to(BF16).cuda()
    qe = torch.cat([q[..., :Dn].float(), torch.tensor(qr).float().view(2, T, H, Dr)], -1).to(BF16).cuda()
    pe = torch.tensor(rows[:, R:]).float().to(BF16).view(2, T, Dr).cuda()
    want, _ = mla.attn_fwd(qe, kv, pe, scale=scale)
    # absorbed, through the cache
    cache = torch.full((14, page, R + Dr), float("nan"), dtype=BF16, device="cuda")
    table = torch.randperm(14, generator=g)[:2 * 6].view(2, 6).to(torch.int32)
    slot = lambda n, t: int(table[n, t // page]) * page + t % page  # noqa: E731
    table_d, qa_k = table.cuda(), torch.einsum("hdr,bthd->bthr", wk, q[..., :Dn].float()).to(BF16)
    err, ref = 0.0, 0.0

    def feed(spans):
        nonlocal err, ref
        at = [(n, t) for n, (s, e) in enumerate(spans) for t in range(s, e)]
        n_i, t_i = torch.tensor([a[0] for a in at]), torch.tensor([a[1] for a in at])
        qa = torch.zeros((len(at), H, R + Dr), dtype=BF16)
        qa[..., :R] = qa_k[n_i, t_i]
        qa = qa.cuda()
        mla.cache_append(c[n_i, t_i].cuda(), t_i.to(torch.int32).cuda(), _i32([slot(*a) for a in at]).cuda(), cache, R,
                         rope=rope, norm_weight=weight, q_pe=q[n_i, t_i][..., Dn:].contiguous().cuda(), q=qa)
        single = all(e - s == 1 for s, e in spans)
        cu = None if single else _i32(np.concatenate([[0], np.cumsum([e - s for s, e in spans])])).cuda()
        o, _ = mla.paged_attn(qa, cache, table_d, _i32([e for _, e in spans]).cuda(), R, scale, cu_seqlens=cu)
        got = torch.einsum("hdr,thr->thd", wv, o.float().cpu())
        exp = want[n_i.cuda(), t_i.cuda()].float().cpu()
        err += float((got - exp).square().sum())
        ref += float(exp.square().sum())

    feed([(0, lens[0]), (0, lens[1])])
    for s in range(steps):
        feed([(lens[0] + s, lens[0] + s + 1), (lens[1] + s, lens[1] + s + 1)])
    rel = (err / ref) ** 0.5
    print("TOGETHER rel-L2 %.3e" % rel, flush=True)
    assert rel <= 8 * 2.0 ** -8


def test_calls_in_a_graph_and_on_another_stream():
    q, kv, pe, do = _cuda(*_expanded(51, 1, 333, 3, 128, 64))
    cu = _i32([0, 100, 100, 333]).cuda()
    pq, cache, table, lens, pcu = _paged(52, [300, 90], 16, 6, 512, 64, q_lens=[20, 1])
    pargs = _cuda(pq, cache, _i32(table), _i32(lens), _i32(pcu))
    c, slots = _randn(53, 21, 576).cuda(), _i32(np.arange(21) + 16 * int(table[0][0])).cuda()[:21]
    slots = _i32([int(table[0][j // 16]) * 16 + j % 16 for j in range(21)]).cuda()
    cache0 = pargs[1].clone()

    def work():
        o, lse = mla.attn_fwd(q, kv, pe, cu_seqlens=cu)
        gr = mla.attn_bwd(q, kv, pe, o, lse, do, cu_seqlens=cu)
        mla.cache_append(c, None, slots, pargs[1], 512)
        po, pl = mla.paged_attn(*pargs[:4], 512, 0.07, cu_seqlens=pargs[4])
        return [o, lse, *gr.values(), po, pl]

    eager = [t.clone() for t in work()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = work()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = work()
    for _ in range(3):
        pargs[1].copy_(cache0)
        for t in outs:
            t.fill_(3.0)
        work()  # eager work between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, outs))
