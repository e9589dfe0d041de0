"""GPU tests of the step operators at their edges: codes next to a border, factors that are
not finite, page tables with holes, requests that a plan does not serve, and every kernel that
the dispatch can choose."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import step as os_
from test_gpu_step import call_scan, check_norm, check_scan, i32, norm_case, scan_case, up

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ------------------------------------------------------------------ selective scan
@pytest.mark.parametrize("S,dtype", [(8, BF), (16, F32), (32, BF), (64, F32), (128, BF)])
@pytest.mark.parametrize("cut", [False, True])
def test_a_factor_that_is_minus_infinity_forgets(gdn_lib, S, dtype, cut):
    """exp(delta A) is 0 for A = -inf as for any large one: the same bits as with -1e30, in whole and
    partial tiles (whose missing tokens have no delta), cut and uncut, and token by token."""
    print("[case] A = -inf", S, dtype, cut, flush=True)
    rng = np.random.default_rng(S)
    lens = [1, 7, 16, 29, 700, 33, 0] if cut else [1, 7, 16, 29, 48, 33, 0]
    c, g = scan_case(rng, lens, 70, S, 1, dtype)
    some = torch.from_numpy(rng.random((70, S)) < 0.3).cuda()
    got = []
    for far in (float("-inf"), -1e30):
        h = {**g, "A": torch.where(some, far, g["A"]), "pool": g["pool"].clone()}
        out = call_scan(gdn_lib, h, max_seqlen=700 if cut else 48)
        last = gdn_lib.selective_update(g["x"][:7], g["dt"][:7], h["A"], g["B"][:7], g["C"][:7], g["slot"], h["pool"], D=g["D"])
        got.append((out, h["pool"], last))
    for name, a, b in zip(("out", "pool", "update"), *got):
        assert b.isfinite().all() and torch.equal(a, b), name


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("T,H,d", [(4096, 1, 4096), (3000, 1, 5003), (2000, 40, 100), (4000, 600, 5), (300, 1, 40000)])
@pytest.mark.parametrize("group", [0, 128])
def test_codes_are_rounded_quotients(gdn_lib, T, H, d, group):
    """Every code is the fp32 quotient of the value (which the call to fp32 gives) and its scale,
    rounded to nearest even: a product with the scale's reciprocal lands on the other side of a
    border about once in a million values."""
    print("[case] quotients", T, H, d, group, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    x = torch.randn((T, H, d) if H > 1 else (T, d), generator=gen, device="cuda")
    y = gdn_lib.rms_norm(x, out_dtype=F32).view(T, -1).cpu()
    codes, scale = gdn_lib.rms_norm(x, out_dtype=F8, group=group)
    W = y.shape[1]
    step = group or W
    want = torch.stack([p.abs().amax(1) for p in y.split(step, 1)], 1) / 448
    assert torch.equal(scale.cpu(), want)
    quotients = y / want.repeat_interleave(step, 1)[:, :W]
    off = int((codes.view(T, W).cpu().view(torch.uint8) != quotients.to(F8).view(torch.uint8)).sum())
    print(f"  {off} of {y.numel()} codes are another value", flush=True)
    assert off == 0


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("N,width,room", [(1, 3, 50), (5, 40, 1000), (3, 3000, 20000), (2, 9000, 4000), (256, 30, 9000),
                                          (300, 20, 100000), (700, 9, 2500), (4, 70, 0), (40, 600, 1)])
@pytest.mark.parametrize("holes", [0.0, 0.02, 0.6, 1.0])
def test_release_passes_over_entries_without_a_page(gdn_lib, N, width, room, holes):
    """A table may hold negative ids (rows whose page was given back before): they do not come to
    the stack, and what is behind them does, in order, as far as the capacity goes."""
    print("[case] release with holes", N, width, room, holes, flush=True)
    rng = np.random.default_rng(N + width)
    page, free = 16, 7
    table = rng.permutation(N * width).reshape(N, width) + 100
    table[rng.random((N, width)) < holes] = -1 - rng.integers(0, 2)
    held = rng.integers(-1, width * page + 1, N)
    held[-1] = width * page + 90                    # (more than the table has)
    keep = np.where(rng.random(N) < 0.3, rng.integers(-1, width * page, N), 0)
    state = torch.full((2 + free + room,), -7, dtype=torch.int32, device="cuda")
    state[:2 + free] = i32([free, 0] + list(range(free)))
    pool = gdn_lib.PagePool(state)
    for turn in range(2):                           # (the second as after any other call)
        before = state.clone()
        gdn_lib.release_pages(pool, i32(table), i32(keep), i32(held), page)
        want = os_.release_pages(before[2:2 + int(before[0])].tolist(), pool.capacity, table, keep, held, page)
        s = state.tolist()
        assert s[:2] == [len(want), 0] and s[2:2 + s[0]] == want, turn
        state[0] = free


def test_no_request_gets_a_page_that_is_none(gdn_lib):
    """The pages of a request with holes go back, and the next step's requests take them: every token has a slot."""
    print("[case] plan behind a release with holes", flush=True)
    pool, table = gdn_lib.page_pool(0), i32([[-1, 4, -1, 9], [-1] * 4])
    state = torch.zeros(2 + 10, dtype=torch.int32, device="cuda")
    pool = gdn_lib.PagePool(state)
    gdn_lib.release_pages(pool, table, i32([0, 0]), i32([64, 0]), 16)
    assert state.tolist()[:4] == [2, 0, 4, 9]
    plan = gdn_lib.plan_pages(pool, table, i32([0, 0]), i32([20, 5]), 16, 25)
    assert plan.cache_len.tolist() == [0, -1] and (plan.slots[:20] >= 0).all() and (plan.slots[20:] == -1).all()
    assert table[0].tolist() == [9, 4, -1, 9] and state[0] == 0


@pytest.mark.parametrize("tokens,free", [(47, 3), (30, 9)])
def test_layers_skip_requests_that_the_plan_does_not_serve(gdn_lib, tokens, free):
    """The stack or the room for tokens ends inside of the third request's need: with its slot masked by
    cache_len the layers leave its states and its rows (which the plan still counts, cut at the
    room) as they are, and serve the others as alone."""
    print("[case] unserved requests", tokens, free, flush=True)
    rng = np.random.default_rng(7)
    lens, page = [20, 1, 17, 9], 16
    c, g = scan_case(rng, lens, 40, 16, 1, BF)
    pool, table = gdn_lib.page_pool(free), torch.full((4, 4), -1, dtype=torch.int32, device="cuda")
    table[1, 0] = 100
    held = i32([0, 15, 0, 0])
    plan = gdn_lib.plan_pages(pool, table, held, i32(lens), page, tokens)
    assert plan.cache_len.tolist() == [0, 15, -1, -1] and plan.cu_seqlens.tolist() == [0, 20, 21, min(38, tokens), min(47, tokens)]
    slot = torch.where(plan.cache_len < 0, -1, g["slot"])
    before, out = g["pool"].clone(), torch.full((tokens, 40), 7.0, dtype=BF, device="cuda")
    g.update({k: g[k][:tokens] for k in ("x", "dt", "B", "C", "z")})
    call_scan(gdn_lib, {**g, "cu": plan.cu_seqlens, "slot": slot}, out=out)
    alone = before.clone()
    want = call_scan(gdn_lib, {**g, "cu": i32([0, 20, 21]), "slot": g["slot"][:2].contiguous(), "pool": alone})
    assert torch.equal(out[:21], want[:21]) and (out[21:] == 7).all() and torch.equal(g["pool"], alone)
    assert torch.equal(alone[g["slot"][2:].long()], before[g["slot"][2:].long()])
    # the linear-attention layer, by its batch's state_slots
    layer = SimpleNamespace(num_k_heads=1, num_v_heads=2, head_k_dim=64, head_v_dim=64, layer_id=0, A_log=torch.zeros(2, device="cuda"),
                            dt_bias=torch.zeros(2, device="cuda"), norm_weight=torch.ones(64, device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF)  # noqa: E731
    mixed, a, b, z, states = rand(tokens, 256), rand(tokens, 2), rand(tokens, 2), rand(tokens, 128), rand(6, 2, 64, 64).float()
    first = states.clone()
    fb = SimpleNamespace(forward_mode="extend", state_slots=slot, cu_seqlens=plan.cu_seqlens, state_pool={0: states})
    got = gdn_lib.forward_gdn(layer, fb, mixed, a, b, z)
    ref = SimpleNamespace(forward_mode="extend", state_slots=g["slot"][:2].contiguous(), cu_seqlens=i32([0, 20, 21]), state_pool={0: first.clone()})
    assert torch.equal(got[:21], gdn_lib.forward_gdn(layer, ref, mixed, a, b, z)[:21]) and torch.equal(states, ref.state_pool[0])
    rest = [k for k in range(6) if k not in g["slot"][:2].tolist()]
    assert torch.equal(states[rest], first[rest])


# ------------------------------------------------------------------ every kernel of the dispatch
@pytest.mark.parametrize("n,D,S,G,dtype", [(517, 512, 16, 1, BF), (1030, 512, 8, 4, F32), (411, 258, 32, 2, BF), (65, 1024, 64, 1, F32),
                                           (65, 512, 128, 1, BF), (129, 2048, 16, 1, F32)])
@pytest.mark.parametrize("aligned", [False, True])
def test_update_of_two_rows_a_workgroup(gdn_lib, n, D, S, G, dtype, aligned):
    """From 4096 workgroups of one row on, two share one: odd numbers of rows, padding rows as the first, the
    second and both of a pair and as the last, B and C in wide loads and at odd elements."""
    print("[case] update by pairs", n, D, S, G, dtype, aligned, flush=True)
    per = 1024 // S
    assert -(-(D // G) // per) * G * n >= 4096
    rng = np.random.default_rng(n + D)
    c, g = scan_case(rng, [1] * n, D, S, G, dtype, skip=(4, 11, 20, 21, n - 1))
    if aligned:
        g["B"], g["C"] = g["B"].contiguous(), g["C"].contiguous()
    out = torch.full((n, D), 7.0, dtype=dtype, device="cuda")
    gdn_lib.selective_update(g["x"], g["dt"], g["A"], g["B"], g["C"], g["slot"], g["pool"], D=g["D"], z=g["z"], dt_bias=g["dt_bias"], out=out)
    check_scan(c, out, g["pool"], dtype, "update by pairs", untouched=7.0)


@pytest.mark.parametrize("n,D,S", [(1, 300, 16), (5, 64, 64)])
def test_update_with_aligned_operands(gdn_lib, n, D, S):
    print("[case] update aligned", n, D, S, flush=True)
    c, g = scan_case(np.random.default_rng(n), [1] * n, D, S, 1, BF)
    out = gdn_lib.selective_update(g["x"], g["dt"], g["A"], g["B"].contiguous(), g["C"].contiguous(), g["slot"], g["pool"], D=g["D"],
                                   z=g["z"], dt_bias=g["dt_bias"])
    check_scan(c, out, g["pool"], BF, "update aligned")


# rows of a wave (1024 rows and more, also where the last workgroup is not full), of four and of sixteen,
# one to four pieces a thread; in aligned pieces, at any element, and in parts of any size
NORMS = [(1030, 4, 128), (1027, 1, 500), (1027, 1, 1000), (1030, 8, 128), (1030, 1, 1003), (1027, 5, 100), (1029, 9, 100),
         (3, 1, 1500), (3, 1, 2001), (3, 1, 3001), (3, 30, 100), (3, 1, 5600), (3, 1, 6001), (3, 50, 100), (2, 1, 7168), (3, 64, 128),
         (3, 1, 7001), (3, 70, 100), (3, 1, 12000), (2, 128, 128), (3, 1, 12001), (3, 120, 100), (2, 1, 20001), (2, 200, 100),
         (2, 1, 32768), (2, 1, 30001), (2, 300, 100), (5, 32, 80), (5, 40, 96), (3, 8, 192), (1026, 5, 96)]


@pytest.mark.parametrize("T,H,d", NORMS)
@pytest.mark.parametrize("out_dtype,group", [(BF, 0), (F8, 0), (F8, 128), (F8, 64), (F32, 0)])
def test_norm_in_every_kernel(gdn_lib, T, H, d, out_dtype, group):
    print("[case] norm", T, H, d, out_dtype, group, flush=True)
    rng = np.random.default_rng(T + d)
    for dtype, residual, gate, first, wdtype, offset in ((BF, BF, False, False, BF, 1.0), (BF, F32, False, False, F32, 0.0),
                                                         (F32, None, True, False, None, 0.0), (BF, None, True, True, BF, 1.0)):
        h = norm_case(rng, T, H, d, dtype, residual, gate, wdtype)
        r = up(h["residual"], residual)
        got = gdn_lib.rms_norm(up(h["x"], dtype), up(h["weight"], wdtype), eps=1e-5, offset=offset, residual=r,
                               gate=up(h["gate"], dtype), gate_first=first, out_dtype=out_dtype, group=group)
        check_norm(h, got, r, out_dtype, group, f"{dtype} {residual} {gate}", residual=residual, eps=1e-5, offset=offset,
                   gate_first=first)
