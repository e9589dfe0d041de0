"""GPU tests of the softmax-attention operators at their edges against the fp64 definitions:
queries that stand before cached rows, pages that no row of the call is on, sums that are not
numbers, scales that are tiny or not positive, and every way of shaping scores at every head
size."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from attn_util import (assert_out, bf16, cache_norm, host_cache, i32, make_cache, make_table, row_norm, score_error,
                       spread_positions, up, upload_cache)
from test_gpu_attn_split import _unsplit

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _qkv(rng, T, H, H_kv, d):
    return [bf16(rng.normal(size=(T, h, d))) for h in (H, H_kv, H_kv)]


def _slopes(H):
    return (2.0 ** -np.arange(1, H + 1)).astype(np.float32)


def _same_kind(got, ref):
    """NaN where the definition has NaN and nowhere else."""
    assert np.array_equal(np.isnan(got), np.isnan(ref))


# ------------------------------------------------------------------ queries before cached rows
@pytest.mark.parametrize("d,page,opt", [(64, 16, {}), (128, 64, dict(slopes=True)), (128, 32, dict(softcap=9.0)),
                                        (256, 128, dict(slopes=True, softcap=20.0))])
@pytest.mark.parametrize("split", [False, True])
def test_window_hides_cached_rows_ahead_of_the_query(gdn_lib, d, page, opt, split):
    """start below cache_len: cached rows further ahead than the window are hidden, those
    that only some of the tokens see among them, and their NaNs stay away."""
    print(f"[case] extend, start below cache_len, d={d} page={page} {opt} split={split}", flush=True)
    rng = np.random.default_rng(d + page)
    lens, H, H_kv = [70, 5, 33, 2], 4, 2
    if split:
        lens, old, start, w = [7, 3], [2500, 1700], [100, 1200], 900
    else:
        old, start, w = [400, 131, 300, 90], [0, 60, 290, 500], 45
    c = make_cache(rng, sum(-(-o // page) for o in old), H_kv, page, d)
    table = make_table(rng, old, page, c["k"].shape[0])
    knorm = cache_norm(c)
    for n, (o, s, L) in enumerate(zip(old, start, lens)):
        for r in range(o):
            if r - (s + L - 1) >= w and r % 7 == 0:    # hidden from all of the sequence's tokens
                c["kv"[r % 2]][table[n, r // page], :, r % page, r % d] = 0x7f
    edge = start[0] + w + 1                             # seen by tokens 2 and later only
    c["v"][table[0, edge // page], 0, edge % page, 3] = 0xff
    q, k, v = _qkv(rng, sum(lens), H, H_kv, d)
    kw = dict(window=w, softcap=opt.get("softcap", 0.0))
    slopes = _slopes(H) if opt.get("slopes") else None
    with np.errstate(invalid="ignore"):
        ref, mag = oa.attn_extend(q, k, v, _cu(lens), 0.1, cache=c, table=table, cache_len=old, start=start, slopes=slopes, **kw)
    assert np.isnan(ref).sum() == 2 * (lens[0] - 2)     # two heads of the group, one column
    args = [up(x, BF16) for x in (q, k, v)] + [i32(_cu(lens))]
    kw.update(scale=0.1, cache=upload_cache(gdn_lib, c), block_table=i32(table), cache_len=i32(old), start=i32(start),
              slopes=up(slopes))
    if split:
        assert gdn_lib.attn_extend_workspace_size(*args, **kw) > 0
    got = gdn_lib.attn_extend(*args, **kw).float().cpu().numpy()
    _same_kind(got, ref)
    ds = score_error(q, max(row_norm(k), knorm), 0.1, opt.get("softcap", 0.0), 0.5 if opt.get("slopes") else 0.0, max(old))
    assert_out(got, ref, np.nan_to_num(mag), ds, "extend")


# ------------------------------------------------------------------ pages that hold nothing of the call
def _poison_unowned(c, table, value):
    """Codes and scales of the pages that no sequence owns, as in memory that was never written."""
    free = np.setdiff1d(np.arange(c["k"].shape[0]), table[table >= 0])
    for a in ("k", "v"):
        c[a][free], c[a + "_scale"][free] = 0x7f, value
    assert 0 in free


def _table_without_page_0(rng, counts, page, pages):
    t = make_table(rng, counts, page, pages - 1)
    return np.where(t >= 0, t + 1, t)


@pytest.mark.parametrize("value", [math.nan, math.inf, 2.0 ** 127])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 32), (256, 32), (64, 64), (128, 128)])
def test_extend_scales_of_other_pages_do_not_leak(gdn_lib, d, page, value):
    print(f"[case] extend, foreign scales {value}, d={d} page={page}", flush=True)
    rng = np.random.default_rng(d + page)
    lens, old, H, H_kv = [5, 70, 3], [70, 200, 17], 4, 2
    c = make_cache(rng, 60, H_kv, page, d)
    table = _table_without_page_0(rng, old, page, 60)
    table[1, 1] = -1                                    # a page that is not there
    knorm = cache_norm(c)
    _poison_unowned(c, table, value)
    q, k, v = _qkv(rng, sum(lens), H, H_kv, d)
    for w in (0, 50):
        ref, mag = oa.attn_extend(q, k, v, _cu(lens), 0.1, cache=c, table=table, cache_len=old, window=w)
        got = gdn_lib.attn_extend(*(up(x, BF16) for x in (q, k, v)), i32(_cu(lens)), scale=0.1, cache=upload_cache(gdn_lib, c),
                                  block_table=i32(table), cache_len=i32(old), window=w).float().cpu().numpy()
        assert_out(got, ref, mag, score_error(q, max(row_norm(k), knorm), 0.1), f"window {w}")


@pytest.mark.parametrize("value", [math.nan, math.inf, 2.0 ** 127])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (256, 16), (128, 128)])
def test_decode_scales_of_other_pages_do_not_leak(gdn_lib, d, page, value):
    print(f"[case] decode, foreign scales {value}, d={d} page={page}", flush=True)
    rng = np.random.default_rng(d + page)
    lens, H, H_kv = [70, 200, 17, 1], 4, 2
    c = make_cache(rng, 60, H_kv, page, d)
    table = _table_without_page_0(rng, lens, page, 60)
    table[1, 1] = 0 if page == 128 else -1
    if page == 128:
        table[1, 1] = 99
    knorm = cache_norm(c)
    _poison_unowned(c, table, value)
    q = bf16(rng.normal(size=(len(lens), H, d)))
    ref, mag, _ = oa.attn_decode(q, c, table, lens, 0.1)
    got = gdn_lib.attn_decode(up(q, BF16), upload_cache(gdn_lib, c), i32(table), i32(lens), scale=0.1).float().cpu().numpy()
    assert_out(got, ref, mag, score_error(q, knorm, 0.1), "decode")


@pytest.mark.parametrize("pos", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (256, 16)])
def test_pages_outside_of_the_window_may_hold_any_scale(gdn_lib, d, page, pos):
    """Pages none of whose rows is seen: their codes and scales reach nothing."""
    print(f"[case] hidden pages, d={d} page={page} pos={pos}", flush=True)
    rng = np.random.default_rng(d + page)
    lens, H, H_kv, w = [300, 100, 290], 4, 2, 75
    c = make_cache(rng, 80, H_kv, page, d, track=pos)
    table = make_table(rng, lens, page, 80)
    if pos:
        last = spread_positions(rng, c, table, lens)
        q_pos, start = last, [x + 1 for x in last]
    else:
        q_pos, start = None, None
    knorm = cache_norm(c)
    for n, L in enumerate(lens):
        for j in range(-(-L // page)):
            rows = np.arange(j * page, min(L, (j + 1) * page))
            at = c["pos"][table[n, j]].max() if pos else rows.max()
            if (q_pos[n] if pos else L - 1) - at >= w:  # for every head
                c["v"][table[n, j], :, 5:9] = 0x7f
                c["k_scale"][table[n, j]] = c["v_scale"][table[n, j]] = math.nan
    q = bf16(rng.normal(size=(len(lens), H, d)))
    g = upload_cache(gdn_lib, c)
    assert np.isnan(c["v_scale"]).any()
    ref, mag, _ = oa.attn_decode(q, c, table, lens, 0.1, window=w, q_pos=q_pos)
    ds = score_error(q, knorm, 0.1)
    got = gdn_lib.attn_decode(up(q, BF16), g, i32(table), i32(lens), scale=0.1, window=w, q_pos=i32(q_pos)).float().cpu().numpy()
    assert_out(got, ref, mag, ds, "decode")
    q, k, v = _qkv(rng, 9, H, H_kv, d)
    ref, mag = oa.attn_extend(q, k, v, [0, 3, 7, 9], 0.1, cache=c, table=table, cache_len=lens, start=start, window=w)
    got = gdn_lib.attn_extend(*(up(x, BF16) for x in (q, k, v)), i32([0, 3, 7, 9]), scale=0.1, cache=g, block_table=i32(table),
                              cache_len=i32(lens), start=i32(start), window=w).float().cpu().numpy()
    assert_out(got, ref, mag, score_error(q, max(row_norm(k), knorm), 0.1), "extend")


# ------------------------------------------------------------------ sums that are not numbers
@pytest.mark.parametrize("long", [False, True])
def test_a_nan_sum_leaves_the_weights_of_hidden_rows(gdn_lib, long):
    """A NaN key that one head sees: the weights of the rows that its window hides stay."""
    print(f"[case] decode accumulating, NaN sum, long={long}", flush=True)
    rng = np.random.default_rng(31)
    lens, H, H_kv, d, page, w = [1700 if long else 300, 90], 4, 2, 64, 16, 60
    c = make_cache(rng, 120, H_kv, page, d, track=True)
    table = make_table(rng, lens, page, 120)
    q_pos = spread_positions(rng, c, table, lens)
    seen = [i for i in range(lens[0]) if abs(q_pos[0] - c["pos"][table[0, i // page], 0, i % page]) < w]
    assert 3 < len(seen) < lens[0]
    c["k"][table[0, seen[2] // page], 0, seen[2] % page, 1] = 0x7f
    q = bf16(rng.normal(size=(2, H, d)))
    with np.errstate(invalid="ignore"):
        ref, _, want = oa.attn_decode(q, c, table, lens, 0.1, window=w, q_pos=q_pos)
    assert np.isnan(want).sum() == len(seen)
    g = upload_cache(gdn_lib, c)
    out = gdn_lib.attn_decode(up(q, BF16), g, i32(table), i32(lens), scale=0.1, window=w, q_pos=i32(q_pos), accumulate=True)
    _same_kind(out.float().cpu().numpy(), ref)
    got = host_cache(g)["weight"]
    _same_kind(got, want)
    same = want == c["weight"]                          # rows that are not seen, or of no sequence
    assert same.any() and np.array_equal(got[same], c["weight"][same])


# ------------------------------------------------------------------ scales
@pytest.mark.parametrize("scale", [1e-39, 2e-38, 0.0, -0.1])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_that_are_tiny_or_not_positive(gdn_lib, scale, d):
    print(f"[case] extend scale={scale} d={d}", flush=True)
    rng = np.random.default_rng(d)
    T, H = 1100, 2
    q, k, v = _qkv(rng, T, H, 1, d)
    ref, mag = oa.attn_extend(q, k, v, [0, T], scale)
    args = [up(x, BF16) for x in (q, k, v)] + [i32([0, T])]
    assert gdn_lib.attn_extend_workspace_size(*args, scale=scale) > 0
    ds = score_error(q, row_norm(k), abs(scale))
    assert_out(gdn_lib.attn_extend(*args, scale=scale).float().cpu().numpy(), ref, mag, ds, "split")
    out = torch.empty_like(args[0])
    _unsplit(gdn_lib, *args, scale=scale, out=out)
    assert_out(out.float().cpu().numpy(), ref, mag, ds, "whole")


@pytest.mark.parametrize("size", [3e3, 3e4, 1e5])
@pytest.mark.parametrize("cached", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_of_any_size(gdn_lib, d, cached, size):
    """Queries and keys whose scores reach 1e8, 1e10 and 1e12: the key of the largest score is the output,
    wherever no other comes near it."""
    print(f"[case] extend, large scores, d={d} cached={cached} size={size}", flush=True)
    rng = np.random.default_rng(d)
    lens, H, page = ([40, 9], 2, 32) if cached else ([1200], 2, 32)
    q, k, v = _qkv(rng, sum(lens), H, 1, d)
    q, k = bf16(q * size), bf16(k * size)
    args, kw = [up(x, BF16) for x in (q, k, v)] + [i32(_cu(lens))], dict(scale=0.5)
    keys, values = [], []
    old = [900, 70] if cached else [0]
    if cached:
        c = make_cache(rng, 40, 1, page, d)
        c["k_scale"] *= 2.0 ** round(math.log2(size))
        table = make_table(rng, old, page, 40)
        kw.update(cache=upload_cache(gdn_lib, c), block_table=i32(table), cache_len=i32(old))
    for n, (a, b) in enumerate(zip(_cu(lens), _cu(lens)[1:])):
        ck, cv = oa.cached_rows(c, table[n], old[n], 0)[:2] if cached else (np.zeros((0, d)), np.zeros((0, d)))
        keys.append(np.concatenate([ck, k[a:b, 0]]))
        values.append(np.concatenate([cv, v[a:b, 0]]))
    assert gdn_lib.attn_extend_workspace_size(*args, **kw) > 0
    whole = torch.empty_like(args[0])
    _unsplit(gdn_lib, *args, out=whole, **kw)
    got = [x.float().cpu().numpy() for x in (whole, gdn_lib.attn_extend(*args, **kw))]
    want, seen = [], []
    for n, a in enumerate(_cu(lens)[:-1]):
        for i in range(lens[n]):
            for h in range(H):
                s = 0.5 * (keys[n][:old[n] + i + 1] @ q[a + i, h].astype(np.float64))
                order = np.argsort(-s)
                # (an fp32 score is off by (d + 4) 2^-24 |q| |k| at most)
                off = 0.5 * (d + 4) * 2.0 ** -24 * np.linalg.norm(q[a + i, h].astype(np.float64)) * np.linalg.norm(keys[n], axis=1).max()
                if len(s) > 1 and s[order[0]] - s[order[1]] < 2 * off + 1000:
                    continue
                want.append(values[n][order[0]])
                seen.append([x[a + i, h] for x in got])
    assert len(want) > 0.8 * sum(lens) * H
    want = np.stack(want)
    for j, name in enumerate(("whole", "split")):        # (one weight, rounded to bf16, and the output's rounding)
        assert_out(np.stack([x[j] for x in seen]), want, np.abs(want), 0.0, name)


# ------------------------------------------------------------------ the largest cached values
@pytest.mark.parametrize("pos", [False, True])
def test_a_cached_value_past_the_largest_float_reaches_who_sees_it(gdn_lib, pos):
    """Values near bf16's largest may round to 2^128 in the cache: infinite for the rows that
    see them, whether or not a window hides them from others."""
    print(f"[case] extend, cached 2^128, pos={pos}", flush=True)
    rng = np.random.default_rng(41)
    lens, old, H, d, page, w = [60], [100], 2, 64, 16, 80
    c = make_cache(rng, 8, 1, page, d, track=pos)
    if pos:
        c["pos"][:] = 0
    table = make_table(rng, old, page, 8)
    if pos:
        for r in range(100):
            c["pos"][table[0, r // page], 0, r % page] = r
    at, row = table[0, 50 // page], 50 % page
    c["v"][at], c["v_scale"][at] = 0, 2.0 ** 120
    c["v"][at, 0, row, 9] = 0x78                        # 256
    q, k, v = _qkv(rng, lens[0], H, 1, d)
    ref, mag = oa.attn_extend(q, k, v, [0, 60], 0.1, cache=c, table=table, cache_len=old, window=w)
    got = gdn_lib.attn_extend(*(up(x, BF16) for x in (q, k, v)), i32([0, 60]), scale=0.1, cache=upload_cache(gdn_lib, c),
                              block_table=i32(table), cache_len=i32(old), window=w).float().cpu().numpy()
    sees = np.abs(100 + np.arange(60) - 50) < w
    assert sees.any() and not sees.all()
    assert (got[sees, :, 9] == math.inf).all()
    got[sees, :, 9] = ref[sees, :, 9] = mag[sees, :, 9] = 0.0
    assert_out(got, ref, mag, score_error(q, max(row_norm(k), cache_norm(c)), 0.1), "beside it")


# ------------------------------------------------------------------ every way of shaping scores
SHAPES = {"raw": {}, "negative scale": dict(scale=-0.1), "bias": dict(slopes=True), "cap": dict(softcap=4.0),
          "cap, negative scale": dict(softcap=4.0, scale=-0.1), "cap and bias": dict(softcap=4.0, slopes=True)}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cached", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_extend_shapes_of_scores(gdn_lib, d, cached, shape):
    print(f"[case] extend d={d} cached={cached} {shape}", flush=True)
    rng = np.random.default_rng(d)
    opt, lens, old, H, H_kv, page = SHAPES[shape], [197, 40, 1], [150, 0, 77], 6, 2, 32
    q, k, v = _qkv(rng, sum(lens), H, H_kv, d)
    scale, softcap, slopes = opt.get("scale", 0.1), opt.get("softcap", 0.0), _slopes(H) if opt.get("slopes") else None
    kw, gkw, knorm = {}, {}, row_norm(k)
    if cached:
        c = make_cache(rng, 12, H_kv, page, d)
        table = make_table(rng, old, page, 12)
        knorm = max(knorm, cache_norm(c))
        kw, gkw = dict(cache=c, table=table, cache_len=old), dict(cache=upload_cache(gdn_lib, c), block_table=i32(table),
                                                                  cache_len=i32(old))
    ref, mag = oa.attn_extend(q, k, v, _cu(lens), scale, softcap=softcap, slopes=slopes, **kw)
    got = gdn_lib.attn_extend(*(up(x, BF16) for x in (q, k, v)), i32(_cu(lens)), scale=scale, softcap=softcap, slopes=up(slopes),
                              **gkw).float().cpu().numpy()
    assert_out(got, ref, mag, score_error(q, knorm, abs(scale), softcap, 0.5 if opt.get("slopes") else 0.0, 400), shape)


# ------------------------------------------------------------------ the hint of the cached rows
def test_extend_hints_change_the_split_only(gdn_lib):
    print("[case] extend, max_cached", flush=True)
    rng = np.random.default_rng(51)
    lens, old, H, H_kv, d, page = [3, 9, 1], [1700, 40, 0], 4, 2, 128, 32
    c = make_cache(rng, 60, H_kv, page, d)
    table = make_table(rng, old, page, 60, width=200)
    q, k, v = _qkv(rng, sum(lens), H, H_kv, d)
    ref, mag = oa.attn_extend(q, k, v, _cu(lens), 0.1, cache=c, table=table, cache_len=old)
    args = [up(x, BF16) for x in (q, k, v)] + [i32(_cu(lens))]
    kw = dict(scale=0.1, cache=upload_cache(gdn_lib, c), block_table=i32(table), cache_len=i32(old))
    need = []
    for hint in (0, 1700, 1, 2 ** 31 - 1):             # (also where it is too small)
        need.append(gdn_lib.attn_extend_workspace_size(*args, max_cached=hint, **kw))
        got = gdn_lib.attn_extend(*args, max_cached=hint, **kw).float().cpu().numpy()
        assert_out(got, ref, mag, score_error(q, max(row_norm(k), cache_norm(c)), 0.1), f"hint {hint}")
    assert need[0] == need[3] > need[1] > need[2] == 0
