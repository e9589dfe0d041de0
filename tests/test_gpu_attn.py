"""GPU tests of the softmax-attention operators against the fp64 definitions."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from attn_util import (BF, assert_out, assert_same_cache, bf16, cache_norm, host_cache, i32, make_cache, make_table,
                       row_norm, score_error, spread_positions, up, upload_cache)

pytestmark = pytest.mark.gpu
POISON = -7.0


def _qkv(rng, T, H, H_kv, d):
    return bf16(rng.normal(size=(T, H, d))), bf16(rng.normal(size=(T, H_kv, d))), bf16(rng.normal(size=(T, H_kv, d)))


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)])


# ------------------------------------------------------------------ store
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_store(gdn_lib, d, page):
    print(f"[case] store d={d} page={page}", flush=True)
    rng = np.random.default_rng(d + page)
    H, lens, old = 3, [1, 0, page, 2 * page + 3, 5, 4], [0, 3, page - 1, 7, -1, page]
    counts = [max(a, 0) + b for a, b in zip(old, lens)]
    c = make_cache(rng, sum(-(-x // page) for x in counts) + 2, H, page, d, track=True)
    table = make_table(rng, counts, page, c["k"].shape[0])
    table[5, 1] = c["k"].shape[0] + 5                  # the last sequence's new page is out of range
    _, k, v = _qkv(rng, sum(lens), 1, H, d)
    k *= bf16(2.0 ** rng.integers(-6, 6, (sum(lens), H, 1)))
    k[3, 0, 5], k[4, 1, 0], v[6, 2, 1], v[0, 0, 0] = math.nan, math.inf, -math.inf, 3e38
    v[-1], k[-2] = 0.0, 1e-30
    start = [100 * n for n in range(len(lens))]
    ref = oa.kv_store(c, k, v, _cu(lens), old, table, start)
    g = upload_cache(gdn_lib, c)
    gdn_lib.kv_store(up(k, torch.bfloat16), up(v, torch.bfloat16), i32(_cu(lens)), g, i32(table), i32(old), start=i32(start))
    got = host_cache(g)
    for a in ("k", "v"):                               # any NaN code is NaN
        got[a], ref[a] = (np.where(x & 0x7f == 0x7f, 0x7f, x) for x in (got[a], ref[a]))
    assert_same_cache(got, ref, "store")


def test_store_one_token_each_strided_and_untracked(gdn_lib):
    print("[case] store one token each, strided rows", flush=True)
    rng = np.random.default_rng(5)
    N, H, d, page = 9, 2, 128, 16
    old = [0, 1, 15, 16, 17, 40, -1, 3, 8]
    c = make_cache(rng, 40, H, page, d)
    table = make_table(rng, [max(o, 0) + 1 for o in old], page, 40, width=4)
    qkv = bf16(rng.normal(0, 30, (N, 8 * H * d)))
    t = up(qkv, torch.bfloat16)
    k, v = t[:, 8:8 + H * d].unflatten(1, (H, d)), t[:, 4 * H * d:5 * H * d].unflatten(1, (H, d))
    ref = oa.kv_store(c, qkv[:, 8:8 + H * d].reshape(N, H, d), qkv[:, 4 * H * d:5 * H * d].reshape(N, H, d), None, old, table)
    g = upload_cache(gdn_lib, c)
    gdn_lib.kv_store(k, v, None, g, i32(table), i32(old))
    assert_same_cache(host_cache(g), ref, "store one")


# ------------------------------------------------------------------ extend
EXT = [
    # lens, H, H_kv, d, options
    ([1], 1, 1, 64, {}),
    ([1, 2, 0, 3], 4, 2, 64, {}),
    ([63, 64, 65], 2, 1, 128, {}),
    ([130, 7], 6, 2, 128, {}),                       # groups of 3 heads
    ([33], 14, 2, 256, {}),                          # groups of 7
    ([200], 2, 2, 256, {}),
    ([150], 40, 1, 64, {}),                          # a group of 40 heads: tiles of 3.2 tokens
    ([129, 64], 4, 4, 64, dict(causal=False)),
    ([140, 20], 4, 1, 128, dict(softcap=5.0)),
    ([140, 20], 4, 1, 128, dict(slopes=True)),
    ([300], 2, 1, 64, dict(window=1)),
    ([300, 65], 2, 1, 64, dict(window=50)),
    ([300, 10], 2, 1, 128, dict(visible=True)),
    ([300, 10], 2, 1, 128, dict(visible=True, window=70, softcap=20.0, slopes=True)),
    ([290, 64, 70], 4, 2, 128, dict(doc=True)),
    ([290, 64, 70], 4, 2, 64, dict(doc=True, window=40, causal=False, slopes=True)),
]


def _ext_options(rng, lens, H, opt):
    kw, ref = {}, {}
    for key in ("causal", "softcap", "window"):
        if key in opt:
            kw[key] = ref[key] = opt[key]
    if opt.get("slopes"):
        s = (2.0 ** -np.arange(1, H + 1)).astype(np.float32)
        kw["slopes"], ref["slopes"] = up(s), s
    if opt.get("visible"):
        vis = [min(100, n) for n in lens]
        kw["visible"], ref["visible"] = i32(vis), vis
    if opt.get("doc"):
        doc = np.concatenate([np.sort(rng.integers(-1, 4, n)) if i % 2 == 0 else rng.integers(-1, 3, n)
                              for i, n in enumerate(lens)])
        kw["doc"], ref["doc"] = i32(doc), doc
    return kw, ref


@pytest.mark.parametrize("lens,H,H_kv,d,opt", EXT)
def test_extend(gdn_lib, lens, H, H_kv, d, opt):
    print(f"[case] extend {lens} H={H}/{H_kv} d={d} {opt}", flush=True)
    rng = np.random.default_rng(sum(lens) + H + d)
    T = sum(lens)
    q, k, v = _qkv(rng, T + 3, H, H_kv, d)             # three padding tokens behind the last sequence
    kw, rkw = _ext_options(rng, lens + [3], H, opt)
    k[T:], v[T:] = math.nan, math.inf
    scale = d ** -0.5
    ref, mag = oa.attn_extend(q[:T], k[:T], v[:T], _cu(lens), scale, **{a: b[:T] if a == "doc" else b for a, b in rkw.items()})
    out = torch.full((T + 3, H, d), POISON, dtype=torch.bfloat16, device="cuda")
    gdn_lib.attn_extend(up(q, torch.bfloat16), up(k, torch.bfloat16), up(v, torch.bfloat16), i32(_cu(lens)), scale=scale,
                        out=out, **{a: (b[:len(lens)] if a == "visible" else b) for a, b in kw.items()})
    got = out.float().cpu().numpy()
    assert (got[T:] == POISON).all()
    ds = score_error(q[:T], row_norm(k[:T]), scale, opt.get("softcap", 0.0), 0.5 if opt.get("slopes") else 0.0, max(lens))
    assert_out(got[:T], ref, mag, ds, "extend")


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,opt", [(64, {}), (128, dict(softcap=10.0, slopes=True)), (256, {}),
                                   (128, dict(window=45, slopes=True, pos=True)), (64, dict(window=20)),
                                   (128, dict(visible=True))])
def test_extend_over_cache(gdn_lib, page, d, opt):
    print(f"[case] extend over cache page={page} d={d} {opt}", flush=True)
    rng = np.random.default_rng(page + d)
    lens, old, H, H_kv = [3, 70, 1, 5, 9], [100, 64, 0, -1, 129], 4, 2
    c = make_cache(rng, 40, H_kv, page, d, track=opt.get("pos", False))
    table = make_table(rng, old, page, 40)
    start = None
    if opt.get("pos"):
        start = [x + 1 for x in spread_positions(rng, c, table, old)]
    table[4, min(3, table.shape[1] - 1)] = -1          # a page that is not there: its rows are not seen
    for a in ("k", "v"):                               # the rows behind the held ones hold NaN
        for n, o in enumerate(old):
            if o > 0 and o % page and table[n, o // page] >= 0:
                c[a][table[n, o // page], :, o % page:] = 0x7f
    q, k, v = _qkv(rng, sum(lens), H, H_kv, d)
    kw, rkw = _ext_options(rng, lens, H, opt)
    scale = d ** -0.5
    ref, mag = oa.attn_extend(q, k, v, _cu(lens), scale, cache=c, table=table, cache_len=old, start=start, **rkw)
    out = torch.full(q.shape, POISON, dtype=torch.bfloat16, device="cuda")
    g = upload_cache(gdn_lib, c)
    gdn_lib.attn_extend(up(q, torch.bfloat16), up(k, torch.bfloat16), up(v, torch.bfloat16), i32(_cu(lens)), scale=scale,
                        cache=g, block_table=i32(table), cache_len=i32(old), start=i32(start), out=out, **kw)
    got = out.float().cpu().numpy()
    assert (got[np.isnan(ref)] == POISON).all()
    ds = score_error(q, max(row_norm(k), cache_norm(c)), scale, opt.get("softcap", 0.0), 0.5 if opt.get("slopes") else 0.0, 600)
    assert_out(got, ref, mag, ds, "extend over cache")
    assert_same_cache(host_cache(g), c, "read only")


@pytest.mark.parametrize("opt", [{}, dict(doc=True), dict(window=30), dict(visible=True)])
def test_extend_hidden_values_do_not_leak(gdn_lib, opt):
    """NaN and infinite keys and values reach only the rows that see them."""
    print(f"[case] extend hidden values {opt}", flush=True)
    rng = np.random.default_rng(9)
    lens, H, H_kv, d = [200, 90], 4, 2, 128
    q, k, v = _qkv(rng, 290, H, H_kv, d)
    v[150, 0, 7], v[151, 1], k[120, 0], v[260] = math.nan, math.inf, math.nan, -math.inf
    kw, rkw = _ext_options(rng, lens, H, opt)
    with np.errstate(invalid="ignore"):
        ref, mag = oa.attn_extend(q, k, v, _cu(lens), 0.1, **rkw)
    got = gdn_lib.attn_extend(up(q, torch.bfloat16), up(k, torch.bfloat16), up(v, torch.bfloat16), i32(_cu(lens)),
                              scale=0.1, **kw).float().cpu().numpy()
    assert np.isnan(ref).any() and np.isfinite(ref).any()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    fin = np.isfinite(ref)
    tol = (BF * (np.abs(ref) + mag) + 1e-3 * mag) * 1.01
    assert (np.abs(got[fin] - ref[fin]) <= tol[fin]).all()


# ------------------------------------------------------------------ decode
DEC = [
    # kv_len, H, H_kv, d, page, options
    ([1], 1, 1, 64, 16, {}),
    ([0, 1, -1, 15, 16, 17], 4, 2, 64, 16, {}),
    ([63, 64, 65, 300], 8, 1, 128, 32, {}),
    ([257, 1000], 14, 2, 256, 64, {}),
    ([1500, 3], 4, 2, 128, 128, {}),
    ([700], 20, 1, 64, 64, {}),                      # more than 16 heads in a group
    ([700, 90], 7, 7, 128, 16, dict(softcap=4.0)),
    ([700, 90], 8, 2, 128, 64, dict(slopes=True)),
    ([700, 90, 1300], 8, 2, 64, 32, dict(window=64)),
    ([700, 90, 1300], 8, 2, 256, 16, dict(window=200, slopes=True, track=True, softcap=30.0)),
    ([700, 0, 90, -1, 1300], 8, 2, 128, 64, dict(track=True)),
    ([700, 90], 40, 2, 64, 128, dict(track=True, softcap=9.0)),
    ([2100, 64, 5], 6, 2, 128, 64, dict(window=100, track=True, nopos=True)),
]


@pytest.mark.parametrize("lens,H,H_kv,d,page,opt", DEC)
def test_decode(gdn_lib, lens, H, H_kv, d, page, opt):
    print(f"[case] decode {lens} H={H}/{H_kv} d={d} page={page} {opt}", flush=True)
    rng = np.random.default_rng(sum(lens) + H + d)
    N, pages = len(lens), sum(-(-max(x, 0) // page) for x in lens) + 3
    c = make_cache(rng, pages, H_kv, page, d, track=opt.get("track", False))
    table = make_table(rng, lens, page, pages, width=max(-(-max(lens) // page), 1) + 2)
    q_pos = None
    if opt.get("track") and not opt.get("nopos"):
        q_pos = [x + 2 for x in spread_positions(rng, c, table, lens)]
    elif opt.get("nopos"):
        c["pos"] = None
    if len(lens) > 1 and lens[-1] > page:
        table[-1, 1] = pages + 1                       # a page that is not there
    for a in ("k", "v"):
        for n, o in enumerate(lens):
            if o > 0 and o % page and table[n, o // page] >= 0 and table[n, o // page] < pages:
                c[a][table[n, o // page], :, o % page:] = 0xff
    q = bf16(rng.normal(size=(N, H, d)))
    scale, kw, rkw = d ** -0.5, {}, {}
    for key in ("softcap", "window"):
        if key in opt:
            kw[key] = rkw[key] = opt[key]
    if opt.get("slopes"):
        s = (2.0 ** -np.arange(1, H + 1)).astype(np.float32)
        kw["slopes"], rkw["slopes"] = up(s), s
    ref, mag, w = oa.attn_decode(q, c, table, lens, scale, q_pos=q_pos, **rkw)
    ds = score_error(q, cache_norm(c), scale, opt.get("softcap", 0.0), 0.5 if opt.get("slopes") else 0.0, 3000)
    for hint in (0, max(max(lens), 1), 1):             # the hint changes the splits only
        g = upload_cache(gdn_lib, c)
        out = torch.full(q.shape, POISON, dtype=torch.bfloat16, device="cuda")
        gdn_lib.attn_decode(up(q, torch.bfloat16), g, i32(table), i32(lens), scale=scale, q_pos=i32(q_pos), out=out,
                            accumulate=opt.get("track", False), max_kvlen=hint, **kw)
        got = out.float().cpu().numpy()
        assert (got[np.isnan(ref)] == POISON).all()
        assert_out(got, ref, mag, ds, f"decode hint {hint}")
        after = host_cache(g)
        if opt.get("track"):
            add = w - c["weight"]
            tol = add * (2 * ds + 2.0 ** -18) + 2.0 ** -23 * w
            bad = np.abs(after["weight"] - w) > tol
            assert not bad.any(), f"weights off by {np.abs(after['weight'] - w)[bad].max():.2e}"
        c2 = dict(c, weight=None)
        assert_same_cache(after, c2, "read only")


def test_decode_nan_in_seen_rows_shows(gdn_lib):
    print("[case] decode NaN", flush=True)
    rng = np.random.default_rng(11)
    c = make_cache(rng, 20, 2, 16, 64)
    table = make_table(rng, [100, 100], 16, 20)
    c["v"][table[0, 2], 0, 3, 9], c["k"][table[1, 1], 1, 0, 0] = 0x7f, 0x7f
    q = bf16(rng.normal(size=(2, 4, 64)))
    with np.errstate(invalid="ignore"):
        ref, _, _ = oa.attn_decode(q, c, table, [100, 100], 0.1)
    got = gdn_lib.attn_decode(up(q, torch.bfloat16), upload_cache(gdn_lib, c), i32(table), i32([100, 100]),
                              scale=0.1).float().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.isnan(ref).sum() == 2 + 2 * 64


# ------------------------------------------------------------------ evict
@pytest.mark.parametrize("lens,budget,recent,H,d,page", [
    ([40], 10, 0, 1, 64, 16), ([40, 10, -1, 100], 17, 5, 2, 64, 16), ([300, 299, 0], 150, 150, 2, 128, 32),
    ([1000, 64, 65], 64, 10, 3, 256, 64), ([4500], 2000, 100, 1, 64, 128), ([130], 129, 1, 2, 128, 64),
    ([500], 1, 1, 1, 64, 16), ([33], 1000, 4, 1, 64, 16)])
def test_evict(gdn_lib, lens, budget, recent, H, d, page):
    print(f"[case] evict {lens} budget={budget} recent={recent} H={H} d={d} page={page}", flush=True)
    rng = np.random.default_rng(sum(lens) + budget)
    pages = sum(-(-max(x, 0) // page) for x in lens) + 2
    c = make_cache(rng, pages, H, page, d, track=True)
    table = make_table(rng, lens, page, pages, width=-(-max(lens) // page) + 1)
    spread_positions(rng, c, table, lens)
    c["weight"] = np.round(c["weight"] * 20) / 4       # many ties
    c["weight"][:, :, 3] = math.nan
    c["weight"][:, :, 5] = 0.0
    c["weight"][:, 0, 6] = -0.0
    c["weight"][:, :, 7], c["weight"][:, :, 9], c["weight"][:, :, 11] = -2.5, math.inf, -math.inf
    ref, new = oa.kv_evict(c, table, lens, budget, recent)
    g, n32 = upload_cache(gdn_lib, c), i32(lens)
    got_new = gdn_lib.kv_evict(g, i32(table), n32, budget, recent=recent, new_len=n32)
    assert got_new.tolist() == new.tolist()
    assert_same_cache(host_cache(g), ref, "evict")


def test_evict_leaves_a_sequence_with_a_bad_page(gdn_lib):
    print("[case] evict bad page", flush=True)
    rng = np.random.default_rng(3)
    c = make_cache(rng, 20, 2, 16, 64, track=True)
    table = make_table(rng, [100, 90], 16, 20)
    spread_positions(rng, c, table, [100, 90])
    table[0, 6] = 20
    ref, new = oa.kv_evict(c, table, [100, 90], 40, 4)
    assert new.tolist() == [100, 40]
    g = upload_cache(gdn_lib, c)
    assert gdn_lib.kv_evict(g, i32(table), i32([100, 90]), 40, recent=4).tolist() == [100, 40]
    assert_same_cache(host_cache(g), ref, "evict")


@pytest.mark.parametrize("pos", [False, True])
def test_extend_over_cache_hidden_values_do_not_leak(gdn_lib, pos):
    """NaN codes in cached rows that a window hides from some of the new tokens."""
    print(f"[case] extend over cache, hidden NaN, pos={pos}", flush=True)
    rng = np.random.default_rng(21)
    lens, old, H, H_kv, d, page = [70, 33], [200, 131], 4, 2, 128, 32
    c = make_cache(rng, 14, H_kv, page, d, track=pos)
    table = make_table(rng, old, page, 14)
    start = [x + 1 for x in spread_positions(rng, c, table, old)] if pos else None
    c["v"][table[0, 4], 0, 7, 3], c["v"][table[0, 5], 1, 9], c["k"][table[0, 5], 0, 11, 0] = 0x7f, 0xff, 0x7f
    c["v"][table[1, 3], :, 30, 100] = 0x7f
    q, k, v = _qkv(rng, sum(lens), H, H_kv, d)
    window = 110 if pos else 60
    with np.errstate(invalid="ignore"):
        ref, mag = oa.attn_extend(q, k, v, _cu(lens), 0.1, cache=c, table=table, cache_len=old, start=start, window=window)
    got = gdn_lib.attn_extend(up(q, torch.bfloat16), up(k, torch.bfloat16), up(v, torch.bfloat16), i32(_cu(lens)), scale=0.1,
                              cache=upload_cache(gdn_lib, c), block_table=i32(table), cache_len=i32(old), start=i32(start),
                              window=window).float().cpu().numpy()
    nan = np.isnan(ref)
    assert nan.any() and not nan.all() and np.array_equal(np.isnan(got), nan)
    tol = (BF * (np.abs(ref) + mag) + 1e-3 * mag) * 1.01
    assert (np.abs(got[~nan] - ref[~nan]) <= tol[~nan]).all()


@pytest.mark.parametrize("pos", [False, True])
def test_decode_hidden_values_do_not_leak(gdn_lib, pos):
    """NaN codes in rows outside of the window leave the output as it is."""
    print(f"[case] decode, hidden NaN, pos={pos}", flush=True)
    rng = np.random.default_rng(22)
    c = make_cache(rng, 20, 2, 32, 64, track=pos)
    table = make_table(rng, [300, 64], 32, 20)
    q_pos = spread_positions(rng, c, table, [300, 64]) if pos else None
    for a in ("k", "v"):
        c[a][table[0, 0], :, 5], c[a][table[0, 6], 1, 0, 7] = 0x7f, 0xff
    q = bf16(rng.normal(size=(2, 4, 64)))
    ref, mag, _ = oa.attn_decode(q, c, table, [300, 64], 0.1, window=100, q_pos=q_pos)
    got = gdn_lib.attn_decode(up(q, torch.bfloat16), upload_cache(gdn_lib, c), i32(table), i32([300, 64]), scale=0.1, window=100,
                              q_pos=i32(q_pos)).float().cpu().numpy()
    assert np.isfinite(ref).all()
    assert_out(got, ref, mag, score_error(q, cache_norm(c), 0.1), "decode")
