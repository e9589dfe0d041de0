"""GPU tests of the step operators as they are used: sequences cut into segments, streams and
captured steps, large buffers, and a step of a small hybrid model that runs them together with
the framework's layers."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import attention as oa, step as os_
from attn_util import assert_out, cache_norm, row_norm, score_error
from test_gpu_step import BF, F8, F32, call_scan, check_norm, check_scan, host, i32, rounded, scan_case, up

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ segments
LENS, INIT = [600, 0, 33, 32, 1, 700, 31, 900, 64], [1, 0, 0, 1, 1, 0, 1, 1, 1]


@pytest.mark.parametrize("S,G,dtype", [(16, 1, BF), (8, 2, F32), (64, 1, F32), (128, 1, BF), (32, 1, BF)])
@pytest.mark.parametrize("hint", [0, 100, 300, 900, 1 << 30])
def test_scan_in_segments(gdn_lib, S, G, dtype, hint):
    """Ragged sequences, some in one segment and some in many, with hints that are missing, too
    small, right and too large; the caller's workspace, dirty; the pool written and kept."""
    print("[case] segments", S, G, dtype, hint, flush=True)
    rng = np.random.default_rng(S + G)
    for keep in (False, True):
        c, g = scan_case(rng, LENS, 24 * G, S, G, dtype, skip=(6,), pad=3)
        kw = dict(has_init=i32(INIT), max_seqlen=hint, keep_pool=keep)
        args = [g[k] for k in ("x", "dt", "A", "B", "C", "cu", "slot", "pool")]
        need = gdn_lib.selective_scan_workspace_size(*args, D=g["D"], z=g["z"], dt_bias=g["dt_bias"], **kw)
        # (too small a hint: nothing to gain from cutting)
        assert (need > 0) == (hint != 100), need
        ws = torch.full((need + 1024,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN
        out = torch.full((sum(LENS) + 3, 24 * G), 7.0, dtype=dtype, device="cuda")
        call_scan(gdn_lib, g, out=out, workspace=ws[:need] if need else None, **kw)
        check_scan(c, out, g["pool"], dtype, f"segments, keep {keep}", has_init=INIT, keep=keep, untouched=7.0)
        assert (ws[need:] == 0xFF).all(), "past the workspace"


def test_scan_without_tokens(gdn_lib):
    """T = 0: every slot keeps its state, or is cleared."""
    print("[case] no tokens", flush=True)
    rng = np.random.default_rng(9)
    c, g = scan_case(rng, [0, 0, 0], 40, 16, 1, BF)
    before = g["pool"].clone()
    assert call_scan(gdn_lib, g, has_init=i32([1, 0, 1])).shape == (0, 40)
    cleared = int(c["slot"][1])
    assert (g["pool"][cleared] == 0).all()
    before[cleared] = 0
    assert torch.equal(g["pool"], before)


def test_scan_segments_with_growing_states(gdn_lib):
    """Positive factors that overflow over a segment leave states of 0 as they are."""
    print("[case] growing", flush=True)
    rng = np.random.default_rng(10)
    c, g = scan_case(rng, [1200], 64, 16, 1, F32, z=False, skipw=False)
    for t in (g["x"], g["pool"]):
        t.zero_()
    g["A"].fill_(3.0)
    g["dt"].fill_(2.0)
    out = call_scan(gdn_lib, g, max_seqlen=1200)
    assert (out == 0).all() and (g["pool"] == 0).all()


def test_scan_workspace_refusals_and_without_one(gdn_lib):
    print("[case] workspace", flush=True)
    rng = np.random.default_rng(1)
    c, g = scan_case(rng, [1500], 40, 16, 1, BF)
    need = gdn_lib.selective_scan_workspace_size(*(g[k] for k in ("x", "dt", "A", "B", "C", "cu", "slot", "pool")))
    assert need > 0
    before = g["pool"].clone()
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"), torch.empty(need + 16, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(ValueError):
            call_scan(gdn_lib, g, workspace=ws)
    with pytest.raises(ValueError):
        call_scan(gdn_lib, g, workspace=torch.empty(need, device="cuda"))
    assert torch.equal(g["pool"], before)


def test_scan_chunks_equal_the_whole(gdn_lib):
    """A prompt in chunks through its slot, then token by token, against the whole at once."""
    print("[case] chunks", flush=True)
    rng = np.random.default_rng(2)
    c, g = scan_case(rng, [700], 70, 16, 1, F32)
    parts = [(0, 300), (300, 301), (301, 690)] + [(k, k + 1) for k in range(690, 700)]
    out = torch.empty((700, 70), device="cuda")
    for a, b in parts:
        cut = {k: g[k][a:b] for k in ("x", "dt", "B", "C", "z")}
        if b - a > 1 or a == 300:
            call_scan(gdn_lib, {**g, **cut, "cu": i32([0, b - a])}, out=out[a:b])
        else:
            gdn_lib.selective_update(cut["x"], cut["dt"], g["A"], cut["B"], cut["C"], g["slot"], g["pool"], D=g["D"], z=cut["z"],
                                     dt_bias=g["dt_bias"], out=out[a:b])
    check_scan(c, out, g["pool"], F32, "chunks")


# ------------------------------------------------------------------ streams, graphs, sizes
def test_other_streams_and_two_at_once(gdn_lib):
    """Two streams at once, each with its own workspace, between work of the default stream."""
    print("[case] streams", flush=True)
    rng = np.random.default_rng(3)
    cases = [scan_case(rng, [1200, 40], 64, 16, 1, BF) for _ in range(2)]
    outs = []
    streams = [torch.cuda.Stream() for _ in cases]
    for s, (c, g) in zip(streams, cases):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            out = call_scan(gdn_lib, g, max_seqlen=1200)
            outs.append((out, gdn_lib.rms_norm(out, out_dtype=F8, group=64)))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for (c, g), (out, (codes, scale)) in zip(cases, outs):
        check_scan(c, out, g["pool"], BF, "stream")
        check_norm(dict(x=host(out), weight=None, residual=None, gate=None), (codes, scale), None, F8, 64, "stream norm")


def test_captured_steps(gdn_lib):
    """Two captured steps over static buffers (plan, norm with the residual, scan, update, norm,
    release), replayed in turn with eager work between: every replay equals the eager call."""
    print("[case] graph", flush=True)
    rng = np.random.default_rng(4)
    N, T, W, page = 5, 40, 64, 16
    graphs = []
    for k in range(2):
        c, g = scan_case(rng, [8, 0, 20, 1, 3], W, 16, 1, BF, pad=8)
        s = dict(g, held=i32([3, 16, -1, 40, 0]), new=i32([8, 1, 20, 1, 3]), table=torch.full((N, 6), -1, dtype=torch.int32, device="cuda"),
                 res=torch.randn(T, W, device="cuda").to(BF), pages=gdn_lib.page_pool(64), out=torch.zeros(T, W, dtype=BF, device="cuda"),
                 ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), y=torch.zeros(T, W, dtype=F8, device="cuda"),
                 sc=torch.zeros(T, 1, device="cuda"), u=torch.zeros(N, W, dtype=BF, device="cuda"))
        s["plan"] = gdn_lib.StepPlan(*(torch.zeros(n, dtype=d, device="cuda") for n, d in (
            (N + 1, torch.int32), (N, torch.int32), (N, torch.int32), (T, torch.int64), (T, torch.int32), (T, torch.int32))))

        def step(s=s):
            gdn_lib.plan_pages(s["pages"], s["table"], s["held"], s["new"], page, T, out=s["plan"])
            x = gdn_lib.rms_norm(s["x"], residual=s["res"], out=s["out"])
            y = gdn_lib.selective_scan(x, s["dt"], s["A"], s["B"], s["C"], s["plan"].cu_seqlens, s["slot"], s["pool"], D=s["D"],
                                       z=s["z"], dt_bias=s["dt_bias"], workspace=s["ws"])
            gdn_lib.selective_update(y[:N], s["dt"][:N], s["A"], s["B"][:N], s["C"][:N], s["slot"], s["pool"], D=s["D"], out=s["u"])
            gdn_lib.rms_norm(y, gate=s["z"].contiguous(), out=s["y"], scale=s["sc"])
            gdn_lib.release_pages(s["pages"], s["table"], s["plan"].cache_len, s["plan"].kv_len, page)

        names = ("table", "res", "out", "y", "sc", "u", "pool")
        flat = lambda s=s: [s[k].clone() for k in names] + [t.clone() for t in s["plan"]] + [s["pages"].state.clone()]  # noqa: E731

        def back(to, s=s):
            for dst, src in zip([s[k] for k in names] + list(s["plan"]) + [s["pages"].state], to):
                dst.copy_(src)
        start = flat()
        want = []
        for _ in range(3):
            step()
            want.append(flat())
        back(start)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        back(start)
        graphs.append((graph, flat, want))
    live = int(8 + 1 + 20 * 0 + 1 + 3)
    for turn in range(3):
        for graph, flat, want in graphs:
            graph.replay()
            torch.randn(1000, device="cuda").sum().item()
            for i, (a, b) in enumerate(zip(flat(), want[turn])):
                if i in (2, 3, 4):     # (rows of tokens that no sequence owns come from uninitialised scan rows)
                    a, b = a[:live], b[:live]
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (turn, i)


def test_large_pools_and_rows(gdn_lib):
    """Offsets past 2^31 elements: a pool's last slots, rows of a wide buffer, many long rows."""
    print("[case] large", flush=True)
    D, S, slots = 4096, 128, 4200
    pool = torch.empty((slots, D, S), device="cuda")          # 2.2e9 values
    pool[-2:] = 0.5
    pool[0] = 2.0
    rng = np.random.default_rng(5)
    c, g = scan_case(rng, [1, 1], D, S, 1, BF, slots=2)
    c["pool"], c["slot"] = np.full((2, D, S), 0.5), np.array([1, 0])
    g["slot"] = i32([slots - 1, slots - 2])
    out = gdn_lib.selective_update(g["x"], g["dt"], g["A"], g["B"], g["C"], g["slot"], pool, D=g["D"], z=g["z"], dt_bias=g["dt_bias"])
    check_scan(c, out, pool[-2:], BF, "last slots")
    pool[-2:] = 0.5
    out = call_scan(gdn_lib, {**g, "pool": pool})
    check_scan(c, out, pool[-2:], BF, "last slots, scan")
    assert (pool[0] == 2).all()
    del pool
    # rows 2^27 elements apart
    c, g = scan_case(rng, [20], 40, 16, 1, BF)
    far = torch.empty(19 * (1 << 27) + 40, dtype=BF, device="cuda").as_strided((20, 40), (1 << 27, 1))
    far.copy_(g["x"])
    to = torch.empty(19 * (1 << 27) + 40, dtype=BF, device="cuda").as_strided((20, 40), (1 << 27, 1))
    call_scan(gdn_lib, {**g, "x": far}, out=to)
    check_scan(c, to, g["pool"], BF, "far rows")
    x = torch.randn(3, 40, device="cuda").to(BF)
    far[17:] = x
    got = gdn_lib.rms_norm(far[17:], out=to[17:])
    assert torch.equal(got, gdn_lib.rms_norm(x))
    del far, to
    x = torch.empty((70000, 32768), dtype=BF, device="cuda")  # 2.3e9 values
    x[-1] = torch.randn(32768, device="cuda")
    x[:-1] = x[-1]
    codes, scale = gdn_lib.rms_norm(x, out_dtype=F8, group=128)
    first, s0 = gdn_lib.rms_norm(x[-1:].clone(), out_dtype=F8, group=128)
    assert torch.equal(codes[-1:].view(torch.uint8), first.view(torch.uint8)) and torch.equal(scale[-1:], s0)
    assert torch.equal(codes[65536:65537].view(torch.uint8), first.view(torch.uint8))


# ------------------------------------------------------------------ together
def test_a_step_of_a_hybrid_model(gdn_lib):
    """Prefill, then decode steps of a small model: pages planned on the GPU, a state space layer (norm
    with residual, conv, scan or update, gated norm to 8 bits), and softmax attention over the
    planned pages; every stage against its definition on the stage's own inputs.  The requests end
    and give their pages back."""
    print("[case] hybrid step", flush=True)
    rng = np.random.default_rng(6)
    W, S, page, H, Hkv, d, pages = 64, 16, 16, 4, 2, 64, 40
    N = 3
    w_in, w_x = (up(rounded(rng.normal(size=s) * 0.1, BF), BF) for s in ((W, 2 * W), (W, 8 + 2 * S)))
    w_dt, w_qkv, w_o = (up(rounded(rng.normal(size=s) * 0.1, BF), BF) for s in ((8, W), (W, (H + 2 * Hkv) * d), (W, W)))
    nw, gw = up(rounded(0.1 * rng.normal(size=W), BF), BF), up(rounded(1 + 0.1 * rng.normal(size=W), BF), BF)
    taps = up(rounded(rng.normal(size=(W, 4)) * 0.3, BF), BF)
    A, D = -torch.rand(W, S, device="cuda") * 2 - 0.1, torch.ones(W, device="cuda")
    dtb = torch.full((W,), -3.0, device="cuda")
    layer = SimpleNamespace(num_heads=H, num_kv_heads=Hkv, head_dim=d, layer_id=0)
    cache, pool = gdn_lib.kv_cache(pages, Hkv, d, page), gdn_lib.page_pool(pages)
    table = torch.full((N, 8), -1, dtype=torch.int32, device="cuda")
    slots_left = gdn_lib.page_pool(4)
    slot2 = torch.full((N, 1), -1, dtype=torch.int32, device="cuda")
    states, convs = torch.zeros(4, W, S, device="cuda"), torch.zeros(4, W, 3, dtype=BF, device="cuda")
    held = np.zeros(N, np.int64)
    stack, ref_table = list(range(pages - 1, -1, -1)), np.full((N, 8), -1)

    for turn, new in enumerate(([30, 1, 17], [1, 1, 1], [1, 1, 1])):
        T, decode = sum(new), turn > 0
        plan = gdn_lib.plan_pages(pool, table, i32(held), i32(new), page, T)
        want = os_.plan_pages(stack, pages, ref_table, held, new, page, T)
        stack, ref_table = want[0], want[1]
        assert plan.slots.tolist() == want[5] and plan.positions.tolist() == want[6] and np.array_equal(table.cpu().numpy(), ref_table)
        gdn_lib.plan_pages(slots_left, slot2, i32(held), i32(new), 1 << 30, T)      # a state slot for each request
        slot = slot2[:, 0].contiguous()
        assert sorted(slot.tolist()) == [0, 1, 2]
        x, res = (up(rounded(rng.normal(size=(T, W)), BF), BF) for _ in range(2))
        before = host(x), host(res)
        h = gdn_lib.rms_norm(x, nw, offset=1.0, residual=res)
        check_norm(dict(x=before[0], residual=before[1], weight=host(nw), gate=None), h, res, BF, 0, "norm in", residual=BF, offset=1.0)
        xz = h @ w_in
        has_init = i32([int(a > 0) for a in held])
        if decode:
            xc = gdn_lib.conv1d_update(xz[:, :W].contiguous(), taps, None, slot, convs)
        else:
            xc = gdn_lib.conv1d(xz[:, :W].contiguous(), taps, None, plan.cu_seqlens, slot, convs, has_init=has_init)
        proj = xc @ w_x
        dt = proj[:, :8].contiguous() @ w_dt
        kw = dict(D=D, z=xz[:, W:], dt_bias=dtb)
        was = host(states)
        Bm, Cm = proj[:, 8:8 + S], proj[:, 8 + S:]
        if decode:
            y = gdn_lib.selective_update(xc, dt, A, Bm, Cm, slot, states, **kw)
        else:
            y = gdn_lib.selective_scan(xc, dt, A, Bm, Cm, plan.cu_seqlens, slot, states, has_init=has_init, **kw)
        c = dict(x=host(xc), dt=host(dt), A=host(A), B=host(Bm)[:, None], C=host(Cm)[:, None], cu=plan.cu_seqlens.tolist(),
                 slot=slot.cpu().numpy(), pool=was, D=host(D), z=host(xz[:, W:]), dt_bias=host(dtb))
        check_scan(c, y, states, BF, "scan", has_init=has_init.tolist())
        codes, scale = gdn_lib.rms_norm(y, gw, gate=xz[:, W:], out_dtype=F8, group=64)
        check_norm(dict(x=host(y), weight=host(gw), gate=host(xz[:, W:]), residual=None), (codes, scale), None, F8, 64, "norm out")
        a_in = (codes.float() * scale).to(BF)
        q, k, v = (a_in @ w_qkv).split((H * d, Hkv * d, Hkv * d), 1)
        fb = SimpleNamespace(forward_mode="decode" if decode else "extend", kv_pool={0: cache}, block_table=table,
                             cache_len=plan.cache_len, cu_seqlens=plan.cu_seqlens)
        ref_cache = {n: host_codes(t) for n, t in (("k", cache.k), ("v", cache.v))}
        ref_cache.update(k_scale=host(cache.k_scale), v_scale=host(cache.v_scale), pos=None, weight=None)
        o = gdn_lib.forward_attn(layer, fb, q, k, v)
        heads = lambda t, n: host(t).reshape(T, n, d)  # noqa: E731
        if decode:
            ref_cache = oa.kv_store(ref_cache, heads(k, Hkv), heads(v, Hkv), np.arange(N + 1), held, ref_table, held)
            ref, mag = oa.attn_decode(heads(q, H), ref_cache, ref_table, held + 1, d ** -0.5)[:2]
        else:
            ref, mag = oa.attn_extend(heads(q, H), heads(k, Hkv), heads(v, Hkv), plan.cu_seqlens.tolist(), d ** -0.5, cache=ref_cache,
                                      table=ref_table, cache_len=held, start=held)
        ds = score_error(heads(q, H), max(row_norm(heads(k, Hkv)), cache_norm(ref_cache)), d ** -0.5)
        assert_out(host(o).reshape(T, H, d), ref, mag, ds, "attention")
        held = held + np.array(new)
        assert plan.kv_len.tolist() == held.tolist()
    zero = i32(np.zeros(N, np.int64))
    gdn_lib.release_pages(pool, table, zero, i32(held), page)
    gdn_lib.release_pages(slots_left, slot2, zero, i32(held), 1 << 30)
    assert int(pool.state[0]) == pages and sorted(pool.state[2:].tolist()) == list(range(pages))
    assert int(slots_left.state[0]) == 4


def host_codes(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("mode", ["extend", "decode"])
def test_forward_gdn_with_its_gated_norm(gdn_lib, mode):
    print("[case] forward_gdn z", mode, flush=True)
    rng = np.random.default_rng(7)
    T = 6
    layer = SimpleNamespace(num_k_heads=2, num_v_heads=4, head_k_dim=128, head_v_dim=128, layer_id=0,
                            A_log=up(rng.normal(size=4), F32), dt_bias=up(rng.normal(size=4), F32), norm_weight=up(rng.normal(size=128), BF))
    mixed = up(rng.normal(size=(T, 2 * 2 * 128 + 512)), BF)
    a, b, z = up(rng.normal(size=(T, 4)), BF), up(rng.normal(size=(T, 4)), BF), up(rng.normal(size=(T, 512)), BF)
    slots = list(range(T)) if mode == "decode" else [2, 0]
    fb = lambda: SimpleNamespace(forward_mode=mode, state_slots=i32(slots), cu_seqlens=i32([0, 4, T]),  # noqa: E731
                                 state_pool={0: torch.zeros(T, 4, 128, 128, device="cuda")})
    plain = gdn_lib.forward_gdn(layer, fb(), mixed, a, b)
    got = gdn_lib.forward_gdn(layer, fb(), mixed, a, b, z)
    assert got.shape == (T, 512)
    with pytest.raises(ValueError):
        gdn_lib.forward_gdn(SimpleNamespace(**{**vars(layer), "norm_weight": None}), fb(), mixed, a, b, z)
    with pytest.raises(ValueError):
        gdn_lib.forward_gdn(layer, fb(), mixed, a, b, z[:, :256])
    check_norm(dict(x=host(plain).reshape(T, 4, 128), weight=host(layer.norm_weight), gate=host(z).reshape(T, 4, 128), residual=None),
               got, None, BF, 0, "gated")


def test_run_to_run_bits(gdn_lib):
    """The same call twice gives the same bits (no order of arrival enters a sum)."""
    print("[case] bits", flush=True)
    rng = np.random.default_rng(8)
    c, g = scan_case(rng, [900, 700, 5], 130, 16, 1, BF)
    pools = [g["pool"].clone() for _ in range(3)]
    outs = [call_scan(gdn_lib, {**g, "pool": p}, max_seqlen=900) for p in pools]
    assert all(torch.equal(o, outs[0]) for o in outs) and all(torch.equal(p, pools[0]) for p in pools)
    x = torch.randn(300, 5000, device="cuda").to(BF)
    ys = [gdn_lib.rms_norm(x, out_dtype=F8) for _ in range(3)]
    assert all(torch.equal(y[0].view(torch.uint8), ys[0][0].view(torch.uint8)) and torch.equal(y[1], ys[0][1]) for y in ys)
