"""GPU tests of attn_extend with its keys split over workgroups (few rows, many keys)
against the fp64 definition."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from attn_util import (assert_out, bf16, cache_norm, i32, make_cache, make_table, row_norm, score_error,
                       spread_positions, up, upload_cache)

pytestmark = pytest.mark.gpu
POISON = -7.0
BF16 = torch.bfloat16


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _unsplit(gdn, *args, **kw):
    """The same call without a workspace."""
    from hybrid_model_linear_amd import attention
    opt = dict(scale=None, causal=True, softcap=0.0, slopes=None, window=0, doc=None, visible=None, cache=None,
               block_table=None, cache_len=None, start=None)
    opt.update(kw)
    a, i = attention._extend_args(*args, **opt)
    attention._run("gdn_attn_extend", gdn.load().gdn_attn_extend, a, i)


DENSE = [
    ([2200, 3], 2, 1, 64, {}),
    ([3, 1900], 4, 4, 128, {}),
    ([1100], 14, 2, 256, {}),                        # groups of 7
    ([1300], 2, 2, 128, dict(visible=True, softcap=5.0)),
    ([1300, 900], 2, 1, 256, dict(window=700, slopes=True)),
    ([1025, 700], 4, 1, 64, dict(causal=False, slopes=True, softcap=20.0)),
    ([1300, 1030], 2, 2, 128, dict(doc=True)),
    ([1500], 2, 1, 64, dict(doc=True, causal=False)),
]


@pytest.mark.parametrize("lens,H,H_kv,d,opt", DENSE)
def test_new_tokens(gdn_lib, lens, H, H_kv, d, opt):
    print(f"[case] split extend {lens} H={H}/{H_kv} d={d} {opt}", flush=True)
    rng = np.random.default_rng(sum(lens) + H + d)
    T = sum(lens)
    q, k, v = (bf16(rng.normal(size=(T + 3, h, d))) for h in (H, H_kv, H_kv))
    k[T:], v[T:] = math.nan, math.inf                 # three padding tokens behind the last sequence
    kw, rkw = {a: opt[a] for a in ("causal", "softcap", "window") if a in opt}, {}
    rkw.update(kw)
    if opt.get("slopes"):
        rkw["slopes"] = (2.0 ** -np.arange(1, H + 1)).astype(np.float32)
        kw["slopes"] = up(rkw["slopes"])
    if opt.get("visible"):
        rkw["visible"] = [min(600, n) for n in lens]
        kw["visible"] = i32(rkw["visible"])
    if opt.get("doc"):                                 # one sequence of runs, one of scattered ids; some rows see nothing
        doc = np.concatenate([np.sort(rng.integers(-1, 3, n)) if i % 2 == 0 else rng.integers(-1, 3, n)
                              for i, n in enumerate(lens)] + [[0, 1, 2]])
        rkw["doc"], kw["doc"] = doc[:T], i32(doc)
    scale = d ** -0.5
    ref, mag = oa.attn_extend(q[:T], k[:T], v[:T], _cu(lens), scale, **rkw)
    ds = score_error(q[:T], row_norm(k[:T]), scale, opt.get("softcap", 0.0), 0.5 if opt.get("slopes") else 0.0, max(lens))
    args = [up(x, BF16) for x in (q, k, v)] + [i32(_cu(lens))]
    assert gdn_lib.attn_extend_workspace_size(*args, scale=scale, **kw) > 0
    for name, call in (("split", gdn_lib.attn_extend), ("whole", lambda *a, **b: _unsplit(gdn_lib, *a, **b))):
        out = torch.full((T + 3, H, d), POISON, dtype=BF16, device="cuda")
        call(*args, scale=scale, out=out, **kw)
        got = out.float().cpu().numpy()
        assert (got[T:] == POISON).all()
        assert_out(got[:T], ref, mag, ds, name)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("d,opt", [(64, {}), (128, dict(softcap=10.0, slopes=True)), (256, dict(slopes=True)), (256, {}),
                                   (128, dict(window=800, slopes=True, pos=True)), (64, dict(window=900))])
def test_cached_rows(gdn_lib, page, d, opt):
    print(f"[case] split extend over cache page={page} d={d} {opt}", flush=True)
    rng = np.random.default_rng(page + d)
    lens, old, H, H_kv = [3, 70, 1, 5, 9], [1500, 640, 0, -1, 2101], 4, 2
    pages = sum(-(-max(o, 0) // page) for o in old) + 2
    c = make_cache(rng, pages, H_kv, page, d, track=opt.get("pos", False))
    table = make_table(rng, old, page, pages)
    start = None
    if opt.get("pos"):
        start = [x + 1 for x in spread_positions(rng, c, table, old)]
    table[4, 3] = -1                                   # a page that is not there
    for a in ("k", "v"):                               # the rows behind the held ones hold NaN
        for n, o in enumerate(old):
            if o > 0 and o % page and table[n, o // page] >= 0:
                c[a][table[n, o // page], :, o % page:] = 0x7f
    q, k, v = (bf16(rng.normal(size=(sum(lens), h, d))) for h in (H, H_kv, H_kv))
    kw = {a: opt[a] for a in ("softcap", "window") if a in opt}
    rkw = dict(kw)
    if opt.get("slopes"):
        rkw["slopes"] = (2.0 ** -np.arange(1, H + 1)).astype(np.float32)
        kw["slopes"] = up(rkw["slopes"])
    scale = d ** -0.5
    ref, mag = oa.attn_extend(q, k, v, _cu(lens), scale, cache=c, table=table, cache_len=old, start=start, **rkw)
    g = upload_cache(gdn_lib, c)
    args = [up(x, BF16) for x in (q, k, v)] + [i32(_cu(lens))]
    kw.update(scale=scale, cache=g, block_table=i32(table), cache_len=i32(old), start=i32(start))
    assert gdn_lib.attn_extend_workspace_size(*args, **kw) > 0
    rows = np.ones(sum(lens), bool)
    rows[_cu(lens)[3]:_cu(lens)[4]] = False            # the sequence with cache_len < 0 is left as it is
    dist = 3 * (max(old) + max(lens))
    ds = score_error(q, max(row_norm(k), cache_norm(c)), scale, opt.get("softcap", 0.0), 0.5 if opt.get("slopes") else 0.0, dist)
    for name, call in (("split", gdn_lib.attn_extend), ("whole", lambda *a, **b: _unsplit(gdn_lib, *a, **b))):
        out = torch.full(q.shape, POISON, dtype=BF16, device="cuda")
        call(*args, out=out, **kw)
        got = out.float().cpu().numpy()
        assert (got[~rows] == POISON).all()
        assert_out(got[rows], ref[rows], mag[rows], ds, name)


def test_hidden_and_seen_values_that_are_not_finite(gdn_lib):
    print("[case] split extend, NaN and infinity", flush=True)
    rng = np.random.default_rng(9)
    T, H, d = 1200, 2, 64
    q, k, v = (bf16(rng.normal(size=(T, h, d))) for h in (H, 1, 1))
    k[700, 0, 3] = math.nan                            # seen by tokens 700 and later
    v[900, 0, 5] = math.inf                            # by tokens 900 and later
    ref, mag = oa.attn_extend(np.nan_to_num(q), k, v, [0, T], d ** -0.5)
    got = gdn_lib.attn_extend(*(up(x, BF16) for x in (q, k, v)), i32([0, T])).float().cpu().numpy()
    assert np.isfinite(got[:700]).all() and np.isnan(got[700:]).all()
    assert_out(got[:700], ref[:700], mag[:700], score_error(q, row_norm(k), d ** -0.5), "before the NaN")
    k[700, 0, 3] = 0.0
    ref, mag = oa.attn_extend(q, k, v, [0, T], d ** -0.5)
    got = gdn_lib.attn_extend(*(up(x, BF16) for x in (q, k, v)), i32([0, T])).float().cpu().numpy()
    assert (got[900:, :, 5] == math.inf).all()
    got[900:, :, 5] = ref[900:, :, 5] = 0.0
    assert_out(got, ref, mag if mag.ndim < 3 else np.nan_to_num(mag, posinf=0.0), score_error(q, row_norm(k), d ** -0.5), "beside the infinity")


def test_captured_with_the_callers_workspace_on_another_stream(gdn_lib):
    print("[case] split extend captured", flush=True)
    rng = np.random.default_rng(4)
    T, H, d = 1100, 4, 128
    x = [up(bf16(rng.normal(size=(T, h, d))), BF16) for h in (H, 2, 2)]
    cu = i32([0, T])
    want = gdn_lib.attn_extend(*x, cu)
    need = gdn_lib.attn_extend_workspace_size(*x, cu)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="inconsistent sizes"):
        gdn_lib.attn_extend(*x, cu, workspace=ws[:need - 256])
    out, side, graph = torch.empty_like(x[0]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn_lib.attn_extend(*x, cu, workspace=ws, out=out)
        with torch.cuda.graph(graph, stream=side):
            gdn_lib.attn_extend(*x, cu, workspace=ws, out=out)
    torch.cuda.synchronize()
    for _ in range(3):
        out.fill_(POISON)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
