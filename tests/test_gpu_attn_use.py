"""GPU tests of the softmax-attention operators as they are used: the layer call over
prefill, chunks, decode steps and evictions against the fp64 definitions; strided views, large
batches and caches, other streams, graph capture, repeated calls."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import attention as oa
from attn_util import (assert_out, assert_same_cache, bf16, cache_norm, host_cache, i32, make_cache, make_table, row_norm,
                       score_error, spread_positions, up, upload_cache)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def test_forward_attn_through_prefill_chunk_decode_and_eviction(gdn_lib):
    """One layer over a batch of three sequences (the third a padding row in decode): two
    prefill chunks, decode steps that accumulate weights, an eviction, decode steps with the
    positions that are left; capped scores, distance bias and a window."""
    print("[case] forward_attn", flush=True)
    rng = np.random.default_rng(1)
    H, H_kv, d, page, pages = 6, 2, 128, 16, 40
    slopes = (2.0 ** -np.arange(1, H + 1)).astype(np.float32)
    layer = SimpleNamespace(num_heads=H, num_kv_heads=H_kv, head_dim=d, layer_id=3, scaling=0.09, logit_cap=15.0,
                            sliding_window_size=90, alibi_slopes=up(slopes))
    ref_kw = dict(softcap=15.0, slopes=slopes, window=90)
    g = gdn_lib.kv_cache(pages, H_kv, d, page, track=True)
    c = host_cache(g)
    table = np.arange(pages - 1)[:36].reshape(3, 12)[:, ::-1].copy()
    held, pos = np.array([0, 0, 0]), np.array([0, 0, 0])

    def batch(mode, **kw):
        return SimpleNamespace(forward_mode=mode, kv_pool={3: g}, block_table=i32(table), cache_len=i32(held),
                               positions=i32(pos), **kw)

    def check(out, ref, mag, q, knew, what):
        ds = score_error(q, max(row_norm(knew), cache_norm(c)), 0.09, 15.0, 0.5, 200)
        assert_out(out.float().cpu().numpy().reshape(ref.shape), ref, mag, ds, what)

    def tokens(n):
        x = bf16(rng.normal(size=(n, H + 2 * H_kv, d)))
        t = up(x, BF).view(n, -1)                       # one fused projection: strided views
        return (x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]), (t[:, :H * d], t[:, H * d:(H + H_kv) * d], t[:, (H + H_kv) * d:])

    for lens in ([30, 7, 16], [21, 40, 1]):
        (q, k, v), t = tokens(sum(lens))
        out = gdn_lib.forward_attn(layer, batch("extend", cu_seqlens=i32(_cu(lens))), *t)
        ref, mag = oa.attn_extend(q, k, v, _cu(lens), 0.09, cache=c, table=table, cache_len=held, start=pos, **ref_kw)
        check(out, ref, mag, q, k, "extend")
        c = oa.kv_store(c, k, v, _cu(lens), held, table, pos)
        assert_same_cache(host_cache(g), c, "store")
        held, pos = held + lens, pos + lens
    # target verify leaves the cache as it is
    (q, k, v), t = tokens(6)
    out = gdn_lib.forward_attn(layer, batch("target_verify", cu_seqlens=i32([0, 2, 4, 6])), *t)
    ref, mag = oa.attn_extend(q, k, v, [0, 2, 4, 6], 0.09, cache=c, table=table, cache_len=held, start=pos, **ref_kw)
    check(out, ref, mag, q, k, "verify")
    assert_same_cache(host_cache(g), c, "verify")
    held[2] = -1                                        # sequence 2 has ended: a padding row
    for step in range(12):
        (q, k, v), t = tokens(3)
        out = gdn_lib.forward_attn(layer, batch("decode", accumulate_weights=True), *t)
        c = oa.kv_store(c, k, v, None, held, table, pos)
        held[:2] += 1
        ref, mag, w = oa.attn_decode(q, c, table, held, 0.09, q_pos=pos, **ref_kw)
        live = ~np.isnan(ref[:, 0, 0])
        assert live.tolist() == [True, True, False]
        got = host_cache(g)
        assert_same_cache(got, dict(c, weight=None), "decode store")
        ds = score_error(q, cache_norm(c), 0.09, 15.0, 0.5, 200)
        assert (np.abs(got["weight"] - w) <= (w - c["weight"]) * (2 * ds + 2.0 ** -18) + 2.0 ** -23 * w).all()
        check(out[:2], ref[:2], mag[:2], q, k, f"decode {step}")
        c["weight"] = got["weight"]                     # (the accumulated sums as the kernels hold them)
        pos[:2] += 1
        if step == 6:
            c, new = oa.kv_evict(c, table, held, 25, 8)
            t32 = i32(held)
            gdn_lib.kv_evict(g, i32(table), t32, 25, recent=8, new_len=t32)
            assert t32.tolist() == new.tolist() == [25, 25, -1]
            assert_same_cache(host_cache(g), c, "evict")
            held = new.copy()


def test_decode_of_many_ragged_sequences(gdn_lib):
    """More sequences and heads than one round of workgroups: taken longest first, equal
    lengths, empty and padding rows among them."""
    print("[case] decode 300 sequences", flush=True)
    rng = np.random.default_rng(2)
    N, H, H_kv, d, page = 300, 4, 2, 64, 16
    lens = np.where(rng.random(N) < 0.3, 33, rng.integers(-1, 60, N))
    c = make_cache(rng, sum(-(-max(x, 0) // page) for x in lens), H_kv, page, d)
    table = make_table(rng, lens, page, c["k"].shape[0])
    q = bf16(rng.normal(size=(N, H, d)))
    ref, mag, _ = oa.attn_decode(q, c, table, lens, 0.125)
    out = torch.full((N, H, d), -7.0, dtype=BF, device="cuda")
    gdn_lib.attn_decode(up(q, BF), upload_cache(gdn_lib, c), i32(table), i32(lens), scale=0.125, out=out)
    got = out.float().cpu().numpy()
    assert (got[lens < 0] == -7.0).all() and (got[lens == 0] == 0).all()
    assert_out(got, ref, mag, score_error(q, cache_norm(c), 0.125), "decode 300")
    # the same with more sequences than are ordered
    reps = 2
    out2 = gdn_lib.attn_decode(up(np.tile(q, (reps, 1, 1)), BF), upload_cache(gdn_lib, c), i32(np.tile(table, (reps, 1))),
                               i32(np.tile(lens, reps)), scale=0.125, out=torch.full((reps * N, H, d), -7.0, dtype=BF, device="cuda"))
    assert torch.equal(out2.view(reps, N, H, d)[1], out) and torch.equal(out2[:N], out)


def test_decode_long_context_in_many_splits(gdn_lib):
    print("[case] decode 40000", flush=True)
    rng = np.random.default_rng(3)
    c = make_cache(rng, 315, 1, 128, 64, track=True)
    table = make_table(rng, [40000, 130], 128, 315)
    last = spread_positions(rng, c, table, [40000, 130])
    q = bf16(rng.normal(size=(2, 3, 64)))
    ref, mag, w = oa.attn_decode(q, c, table, [40000, 130], 0.2, q_pos=last)
    g = upload_cache(gdn_lib, c)
    out = gdn_lib.attn_decode(up(q, BF), g, i32(table), i32([40000, 130]), scale=0.2, q_pos=i32(last), accumulate=True)
    ds = score_error(q, cache_norm(c), 0.2)
    assert_out(out.float().cpu().numpy(), ref, mag, ds, "decode 40000")
    # (the normaliser sums 40000 weights in fp32, a few hundred to a lane)
    got = host_cache(g)["weight"]
    assert (np.abs(got - w) <= (w - c["weight"]) * (2 * ds + 2.0 ** -14) + 2.0 ** -23 * w).all()


@pytest.mark.parametrize("op", ["decode", "extend", "store", "evict"])
def test_pages_past_4_gib(gdn_lib, op):
    """Pages whose bytes lie past 32-bit offsets: the same as in a small cache."""
    print(f"[case] pages past 4 GiB: {op}", flush=True)
    rng = np.random.default_rng(4)
    H, page, d, N = 8, 64, 128, 2
    small = make_cache(rng, 8, H, page, d, track=True)
    tab = np.array([[5, 0, 3], [1, 7, 2]])
    spread_positions(rng, small, tab, [190, 150])
    pages = 70000                                       # 64 KiB each: 4.3 GiB of keys, as many of values
    far = np.array([69999, 3, 69000, 65536, 40000, 66000, 12, 68001])
    big = gdn_lib.kv_cache(pages, H, d, page, track=True)
    ids = torch.from_numpy(far).cuda()
    s = upload_cache(gdn_lib, small)
    for a in ("k", "v"):
        getattr(big, a).view(torch.uint8)[ids] = getattr(s, a).view(torch.uint8)
    for a in ("k_scale", "v_scale", "pos", "weight"):
        getattr(big, a)[ids] = getattr(s, a)
    q, k = up(rng.normal(size=(9, 16, d)), BF), up(rng.normal(size=(9, H, d)), BF)
    got = []
    for c, t in ((s, tab), (big, far[tab])):
        t = i32(t)
        if op == "decode":
            got.append([gdn_lib.attn_decode(q[:N], c, t, i32([190, 150]), accumulate=True)])
        elif op == "extend":
            got.append([gdn_lib.attn_extend(q, k, k, i32([0, 5, 9]), cache=c, block_table=t, cache_len=i32([190, 150]))])
        elif op == "store":
            gdn_lib.kv_store(k, k, i32([0, 2, 9]), c, t, i32([190, 126]))
            got.append([])
        else:
            got.append([gdn_lib.kv_evict(c, t, i32([190, 150]), 80, recent=10)])
    for a in ("k", "v"):
        got[0].append(getattr(s, a).view(torch.uint8))
        got[1].append(getattr(big, a).view(torch.uint8)[ids])
    for a in ("k_scale", "v_scale", "pos", "weight"):
        got[0].append(getattr(s, a))
        got[1].append(getattr(big, a)[ids])
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert big.k.view(torch.uint8)[100].sum() == 0


def _steps(gdn, c, table, held, pos, q, k, v, ws):
    """A decode step that accumulates, then an eviction: all in place, nothing allocated by
    the caller but the outputs."""
    gdn.kv_store(k, v, None, c, table, held, start=pos)
    held += 1
    o = gdn.attn_decode(q, c, table, held, q_pos=pos, accumulate=True, softcap=20.0, workspace=ws[0])
    gdn.kv_evict(c, table, held, 120, recent=20, new_len=held, workspace=ws[1])
    pos += 1
    return o


def _use_state(gdn, rng):
    N, H, H_kv, d, page = 5, 8, 2, 64, 16
    c = make_cache(rng, 60, H_kv, page, d, track=True)
    table = make_table(rng, [150] * N, page, 60, width=80)   # a wide table: the decode is split
    lens = [100, 125, 0, 119, 140]
    pos = spread_positions(rng, c, table, [150] * N)
    return dict(c=upload_cache(gdn, c), table=i32(table), held=i32(lens), pos=i32([p + 1 for p in pos]),
                q=up(rng.normal(size=(N, H, d)), BF), k=up(rng.normal(size=(N, H_kv, d)), BF), v=up(rng.normal(size=(N, H_kv, d)), BF))


def _clone(gdn, s):
    c = s["c"]
    k, v = (x.view(torch.uint8).clone().view(torch.float8_e4m3fn) for x in (c.k, c.v))
    return dict({a: x.clone() for a, x in s.items() if a != "c"},
                c=gdn.KVCache(k, v, c.k_scale.clone(), c.v_scale.clone(), c.pos.clone(), c.weight.clone()))


def _same(a, b):
    for x in ("k", "v"):
        assert torch.equal(getattr(a["c"], x).view(torch.uint8), getattr(b["c"], x).view(torch.uint8)), x
    for x in ("k_scale", "v_scale", "pos", "weight"):
        assert torch.equal(getattr(a["c"], x), getattr(b["c"], x)), x
    assert torch.equal(a["held"], b["held"])


def test_captured_steps_replay_like_eager_ones(gdn_lib):
    """Store, decode and eviction in two graphs that share a caller's workspaces, replayed
    in turn with new inputs, eager work and synchronisations between."""
    print("[case] graph capture", flush=True)
    gdn, rng = gdn_lib, np.random.default_rng(5)
    s = _use_state(gdn, rng)
    ws = [torch.empty(gdn.attn_decode_workspace_size(s["q"], s["c"], s["table"], s["held"], accumulate=True), dtype=torch.uint8,
                      device="cuda"),
          torch.empty(gdn.kv_evict_workspace_size(s["c"], s["table"], s["held"], 120, recent=20), dtype=torch.uint8, device="cuda")]
    e = _clone(gdn, s)
    warm = _clone(gdn, s)
    _steps(gdn, **warm, ws=ws)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = _steps(gdn, **s, ws=ws)
        graphs.append((gr, o))
    _same(s, e)                                         # capturing ran nothing
    for step in range(6):
        for x in ("q", "k", "v"):
            new = torch.randn_like(s[x])
            s[x].copy_(new)
            e[x].copy_(new)
        gr, o = graphs[step % 2]
        gr.replay()
        want = _steps(gdn, **e, ws=[None, None])        # eager, with its own workspaces
        if step % 3 == 0:
            torch.cuda.synchronize()
        assert torch.equal(o, want), f"replay {step}"
        _same(s, e)


def test_calls_on_other_streams(gdn_lib):
    print("[case] streams", flush=True)
    gdn, rng = gdn_lib, np.random.default_rng(6)
    s = _use_state(gdn, rng)
    e = _clone(gdn, s)
    a, b = _clone(gdn, s), _clone(gdn, s)
    want = _steps(gdn, **e, ws=[None, None])
    torch.cuda.synchronize()
    outs = []
    for x in (a, b):                                    # two in flight, each with its own state and workspaces
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            outs.append(_steps(gdn, **x, ws=[None, None]))
    torch.cuda.synchronize()
    for x, o in zip((a, b), outs):
        assert torch.equal(o, want)
        _same(x, e)


def test_extend_views_repeated_and_split_batches(gdn_lib):
    """Strided views of one projection, the same bits again, and each sequence by itself."""
    print("[case] extend views", flush=True)
    rng = np.random.default_rng(7)
    lens, H, H_kv, d = [70, 1, 200, 33], 6, 2, 128
    T = sum(lens)
    x = up(rng.normal(size=(T, (H + 2 * H_kv) * d + 64)), BF)
    q, k, v = (x[:, a:b].unflatten(1, (-1, d)) for a, b in ((0, H * d), (H * d, (H + H_kv) * d), ((H + H_kv) * d, (H + 2 * H_kv) * d)))
    out = gdn_lib.attn_extend(q, k, v, i32(_cu(lens)), softcap=8.0)
    assert torch.equal(out, gdn_lib.attn_extend(q.contiguous(), k.contiguous(), v.contiguous(), i32(_cu(lens)), softcap=8.0))
    wide = torch.zeros(T, H + 1, d, dtype=BF, device="cuda")
    gdn_lib.attn_extend(q, k, v, i32(_cu(lens)), softcap=8.0, out=wide[:, 1:])
    assert torch.equal(wide[:, 1:], out) and (wide[:, 0] == 0).all()
    for n in range(len(lens)):
        a, b = _cu(lens)[n], _cu(lens)[n + 1]
        assert torch.equal(gdn_lib.attn_extend(q[a:b], k[a:b], v[a:b], i32([0, b - a]), softcap=8.0), out[a:b])


def test_extend_long_documents(gdn_lib):
    """More documents and tiles than one block of tile flags."""
    print("[case] extend long documents", flush=True)
    rng = np.random.default_rng(8)
    L, H, d = 6000, 1, 64
    doc = np.repeat(np.arange(60), 100)
    doc[3000:3500], doc[5990:] = 7, -1                  # a document that comes back, padding at the end
    q, k, v = (bf16(rng.normal(size=(L, 1, d))) for _ in range(3))
    got = gdn_lib.attn_extend(*(up(x, BF) for x in (q, k, v)), i32([0, L]), doc=i32(doc), scale=0.125).float().cpu().numpy()
    ref, mag = np.zeros((L, 1, d)), np.zeros((L, 1, d))
    for i in range(L):
        if doc[i] >= 0:
            j = np.flatnonzero(doc[:i + 1] == doc[i])
            ref[i, 0], _, mag[i, 0] = oa.attend(q[i, 0].astype(float), k[j, 0].astype(float), v[j, 0].astype(float),
                                                np.ones(len(j), bool), i - j, 0.125)
    assert (got[5990:] == 0).all()
    assert_out(got, ref, mag, score_error(q, row_norm(k), 0.125), "documents")


def test_empty_calls_launch_nothing(gdn_lib):
    print("[case] empty calls", flush=True)
    z = torch.zeros(0, 4, 64, dtype=BF, device="cuda")
    kv = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    c = gdn_lib.kv_cache(2, 2, 64, 16, track=True)
    tab = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    none = i32([])
    assert gdn_lib.attn_extend(z, kv, kv, i32([0])).shape == (0, 4, 64)
    assert gdn_lib.attn_extend(z, kv, kv, i32([0, 0, 0])).shape == (0, 4, 64)
    assert gdn_lib.attn_decode(z, c, tab, none).shape == (0, 4, 64)
    assert gdn_lib.kv_evict(c, tab, none, 5).shape == (0,)
    gdn_lib.kv_store(kv, kv, None, c, tab, none)
    gdn_lib.kv_store(kv, kv, i32([0, 0]), c, torch.zeros(1, 3, dtype=torch.int32, device="cuda"), i32([4]))
    torch.cuda.synchronize()
    assert c.k.view(torch.uint8).sum() == 0


def test_the_widest_window_hides_nothing(gdn_lib):
    print("[case] window 2^31 - 1", flush=True)
    rng = np.random.default_rng(12)
    lens, H, H_kv, d, page, w = [150, 9], 4, 2, 64, 16, 2 ** 31 - 1
    x = [up(bf16(rng.normal(size=(sum(lens), h, d))), torch.bfloat16) for h in (H, H_kv, H_kv)]
    cu, old = i32([0, 150, 159]), [200, 40]
    c = make_cache(rng, 20, H_kv, page, d, track=True)
    table = make_table(rng, old, page, 20)
    c["pos"][:] = rng.integers(0, 1000, c["pos"].shape)
    for causal in (True, False):
        assert torch.equal(gdn_lib.attn_extend(*x, cu, causal=causal, window=w), gdn_lib.attn_extend(*x, cu, causal=causal))
    for track in (True, False):
        g = upload_cache(gdn_lib, dict(c, pos=c["pos"] if track else None))
        kw = dict(cache=g, block_table=i32(table), cache_len=i32(old))
        assert torch.equal(gdn_lib.attn_extend(*x, cu, window=w, **kw), gdn_lib.attn_extend(*x, cu, **kw))
        q = x[0][:2]
        assert torch.equal(gdn_lib.attn_decode(q, g, i32(table), i32(old), window=w), gdn_lib.attn_decode(q, g, i32(table), i32(old)))
