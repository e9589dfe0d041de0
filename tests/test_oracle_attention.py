"""Pins of oracle/attention.py: the e4m3 format against torch's own conversion, the
attention against a dense softmax written another way, the store and the eviction against
hand-checkable cases."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa


def test_e4m3_table_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    t = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(oa.E4M3))
    assert np.array_equal(t[~np.isnan(t)], oa.E4M3[~np.isnan(t)])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, 100, 4000), rng.normal(0, 2.0 ** -7, 4000), oa.E4M3[:0x7f],
                        (oa.E4M3[:0x7e] + oa.E4M3[1:0x7f]) / 2, [448.0, -448.0, 0.0, -0.0]]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oa.e4m3_encode(x), want)
    assert (oa.e4m3_encode([math.nan, math.inf, -math.inf]) & 0x7f == 0x7f).all()


@pytest.mark.parametrize("top,scale", [(448.0, 1.0), (449.0, 2.0), (0.0, 2.0 ** -64), (1.75, 2.0 ** -8),
                                       (1.7578125, 2.0 ** -7), (1.0, 2.0 ** -8), (2.0 ** -90, 2.0 ** -64)])
def test_page_scale(top, scale):
    assert oa.page_scale([top, -top / 2, math.nan, math.inf]) == scale


def _cache(pages, H, page, d, rng, track=True):
    c = dict(k=oa.e4m3_encode(rng.normal(0, 20, (pages, H, page, d))), v=oa.e4m3_encode(rng.normal(0, 20, (pages, H, page, d))),
             k_scale=2.0 ** rng.integers(-7, -4, (pages, H)).astype(float), v_scale=2.0 ** rng.integers(-7, -4, (pages, H)).astype(float),
             pos=None, weight=None)
    if track:
        c["pos"] = np.tile(np.arange(page), (pages, H, 1))
        c["weight"] = rng.random((pages, H, page))
    return c


def test_attention_is_the_dense_softmax():
    rng = np.random.default_rng(1)
    q, k, v = (rng.normal(size=(7, 2, 8)) for _ in range(3))
    out, mag = oa.attn_extend(q, k, v, [0, 7], 0.3)
    for h in range(2):
        s = torch.from_numpy(0.3 * q[:, h] @ k[:, h].T).masked_fill(torch.ones(7, 7).triu(1).bool(), -math.inf)
        assert np.allclose(out[:, h], (s.softmax(1) @ torch.from_numpy(v[:, h])).numpy(), atol=1e-12)
    # a prefix mask of everything is no mask, a window of 1 is the token itself
    full, _ = oa.attn_extend(q, k, v, [0, 7], 0.3, causal=False)
    assert np.allclose(oa.attn_extend(q, k, v, [0, 7], 0.3, visible=[7])[0], full)
    assert np.allclose(oa.attn_extend(q, k, v, [0, 7], 0.3, window=1)[0], v)
    # two documents are two sequences; a negative id sees nothing
    doc = np.array([4, 4, 4, 1, 1, -1, -1])
    got = oa.attn_extend(q, k, v, [0, 7], 0.3, doc=doc)[0]
    assert np.allclose(got[:5], oa.attn_extend(q[:5], k[:5], v[:5], [0, 3, 5], 0.3)[0])
    assert (got[5:] == 0).all()
    # a NaN value reaches only the rows that see it
    v2 = v.copy()
    v2[4] = math.nan
    got = oa.attn_extend(q, k, v2, [0, 7], 0.3)[0]
    assert np.isfinite(got[:4]).all() and np.isnan(got[4:]).all()
    # a large cap does nothing, a bias moves the weight towards the near
    assert np.allclose(oa.attn_extend(q, k, v, [0, 7], 0.3, softcap=1e6)[0], out, atol=1e-6)
    near = oa.attn_extend(q, k, v, [0, 7], 0.3, slopes=[50.0, 50.0])[0]
    assert np.allclose(near, v, atol=1e-6)


def test_cached_prefix_is_the_same_attention():
    """Splitting a sequence into a cached prefix and new tokens changes nothing, when the
    new rows hold what the cache would."""
    rng = np.random.default_rng(2)
    c = _cache(6, 1, 16, 8, rng, track=False)
    table = np.array([[3, 0, 5]])
    k, v, _, _, _ = oa.cached_rows(c, table[0], 40, 0)
    q = rng.normal(size=(40, 2, 8))
    whole, _ = oa.attn_extend(q, k[:, None], v[:, None], [0, 40], 0.5, slopes=[0.1, 0.2], window=20)
    part, _ = oa.attn_extend(q[25:], k[25:, None], v[25:, None], [0, 15], 0.5, slopes=[0.1, 0.2], window=20, cache=c,
                             table=table, cache_len=[25])
    assert np.allclose(part, whole[25:])
    dec, _, _ = oa.attn_decode(q[39:], c, table, [40], 0.5, slopes=[0.1, 0.2], window=20)
    assert np.allclose(dec[0], whole[39])


def test_decode_weights_sum_to_the_heads_and_bad_pages_hold_nothing():
    rng = np.random.default_rng(3)
    c = _cache(6, 2, 16, 8, rng)
    q = rng.normal(size=(2, 6, 8))
    _, _, w = oa.attn_decode(q, c, np.array([[1, 2, 9], [4, -1, 0]]), [37, 40], 0.5)
    add = (w - c["weight"]).sum((1, 2))
    assert np.allclose(add[[1, 2]].sum(), 6) and np.allclose(add[[4, 0]].sum(), 6) and add[3] == add[5] == 0
    out, _, _ = oa.attn_decode(q, c, np.array([[-1], [99]]), [5, 0], 0.5)
    assert (out == 0).all()


def test_store_grows_the_scale_and_rounds_again():
    c = _cache(2, 1, 16, 8, np.random.default_rng(4))
    k = np.zeros((3, 1, 8))
    k[0], k[1], k[2] = 1.0, 3.0, 1000.0
    one = oa.kv_store(c, k[:2], k[:2], [0, 2], [0], np.array([[1]]))
    assert one["k_scale"][1, 0] == 2.0 ** -7 and (oa.E4M3[one["k"][1, 0, 1]] * 2.0 ** -7 == 3.0).all()
    two = oa.kv_store(one, k[2:], k[2:], None, [2], np.array([[1]]), start=[70])
    assert two["k_scale"][1, 0] == 4.0 and (oa.E4M3[two["k"][1, 0, :3, 0]] * 4 == [1.0, 3.0, 1024.0]).all()
    assert two["pos"][1, 0, :3].tolist() == [0, 1, 70] and (two["weight"][1, 0, :3] == 0).all()
    assert np.array_equal(two["k"][1, 0, 3:], c["k"][1, 0, 3:]) and np.array_equal(two["k"][0], c["k"][0])
    skipped = oa.kv_store(c, k[:1], k[:1], None, [-1], np.array([[1]]))
    assert all(np.array_equal(skipped[a], c[a]) for a in c)


def test_evict_keeps_newest_then_heaviest():
    c = _cache(2, 1, 16, 8, np.random.default_rng(5))
    table = np.array([[0, 1]])
    c["k_scale"][:], c["v_scale"][:] = 0.5, 0.5
    c["pos"][:, 0] = np.arange(32).reshape(2, 16)
    c["weight"][:] = 0
    c["weight"][0, 0, [3, 5]] = [2.0, 1.0]
    c["weight"][1, 0, 0] = 1.0                         # row 16 ties with row 5: row 5 is first
    c["weight"][0, 0, 0] = math.nan
    got, new = oa.kv_evict(c, table, [20], 5, recent=2)
    assert new.tolist() == [5] and sorted(got["pos"][0, 0, :5].tolist()) == [3, 5, 16, 18, 19]
    # rows 0, 1, 2, 4 are dropped and filled in order by 5, 16, 18, 19
    assert got["pos"][0, 0, :5].tolist() == [5, 16, 18, 3, 19]
    assert np.array_equal(got["k"][0, 0, 1], c["k"][1, 0, 0]) and np.array_equal(got["k"][0, 0, 5:], c["k"][0, 0, 5:])
    same, new = oa.kv_evict(c, table, [5], 5)
    assert new.tolist() == [5] and all(np.array_equal(same[a], c[a], equal_nan=a == "weight") for a in c)


def test_planted_mistakes_are_seen():
    """The comparisons the kernels are held to tell these apart."""
    rng = np.random.default_rng(6)
    q, k, v = (rng.normal(size=(20, 1, 8)) for _ in range(3))
    ref, mag = oa.attn_extend(q, k, v, [0, 20], 0.5)
    for kw in (dict(window=19), dict(visible=[2]), dict(softcap=3.0), dict(slopes=[0.05]), dict(causal=False)):
        other, _ = oa.attn_extend(q, k, v, [0, 20], 0.5, **kw)
        assert (np.abs(other - ref) > 2.0 ** -8 * (np.abs(ref) + mag) * 1.01).any(), kw
