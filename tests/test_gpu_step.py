"""GPU tests of the step operators against oracle.step: the selective scan and its update, the
RMS norm, the pages of a step; sizes, types, strides, masks and values where they can go wrong."""
import numpy as np
import pytest
import torch

from oracle import step as os_

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}        # half a step, relative


def up(x, dtype=None):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def i32(x):
    return None if x is None else torch.from_numpy(np.asarray(x, np.int32)).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def rounded(x, dtype):
    """x as the values of dtype that the GPU gets."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(dtype).double().numpy()


# ------------------------------------------------------------------ selective scan
def scan_case(rng, lens, D, S, G, dtype, *, skip=(), pad=0, z=True, skipw=True, bias=True, softplus=True, slots=None):
    """A case on the host and on the GPU.  B and C are views of one projection, z one of a wider row."""
    T = sum(lens) + pad
    slots = slots or len(lens) + 2
    low = rng.uniform(np.log(1e-3), np.log(0.1), D)
    h = dict(x=rng.normal(size=(T, D)), dt=rng.normal(size=(T, D)) * 0.7, B=rng.normal(size=(T, G, S)), C=rng.normal(size=(T, G, S)))
    h = {k: rounded(v, dtype) for k, v in h.items()}
    f = {"A": -np.arange(1, S + 1) * np.exp(0.2 * rng.normal(size=(D, S))), "D": rng.normal(size=D),
         "dt_bias": np.exp(low) + np.log(-np.expm1(-np.exp(low))), "pool": rng.normal(size=(slots, D, S))}
    f = {k: rounded(v, F32) for k, v in f.items()}
    if not softplus:
        h["dt"] = rounded(np.abs(h["dt"]) * 0.1, dtype)
    h["z"] = rounded(rng.normal(size=(T, D)), dtype) if z else None
    slot = rng.permutation(slots)[:len(lens)]
    for n in skip:
        slot[n] = -1
    c = dict(h, **f, cu=np.concatenate([[0], np.cumsum(lens)]).astype(np.int64), slot=slot)
    if not skipw:
        c["D"] = None
    if not bias:
        c["dt_bias"] = None
    proj = up(np.concatenate([np.zeros((T, 3)), h["B"].reshape(T, G * S), h["C"].reshape(T, G * S)], 1), dtype)
    g = dict(x=up(h["x"], dtype), dt=up(h["dt"], dtype), A=up(f["A"], F32), B=proj[:, 3:3 + G * S].unflatten(1, (G, S)),
             C=proj[:, 3 + G * S:].unflatten(1, (G, S)), slot=i32(slot), pool=up(f["pool"], F32), cu=i32(c["cu"]),
             D=up(c["D"], F32), dt_bias=up(c["dt_bias"], F32), z=None)
    if z:
        g["z"] = up(np.concatenate([h["z"], h["z"]], 1), dtype)[:, D:]
    return c, g


def check_scan(c, got, pool, out_dtype, what, has_init=None, softplus=True, keep=False, untouched=None):
    ref, rpool, (err, perr) = os_.selective_scan(c["x"], c["dt"], c["A"], c["B"], c["C"], c["cu"], c["slot"], c["pool"], D=c["D"],
                                                 z=c["z"], dt_bias=c["dt_bias"], softplus=softplus, has_init=has_init)
    got, pool = host(got), host(pool)
    live = np.isfinite(ref)
    tol = err + HALF[out_dtype] * (np.abs(ref) + err) + 1e-37
    worst = float((np.abs(got - ref)[live] / tol[live]).max()) if live.any() else 0.0
    ptol = perr + HALF[F32] * np.abs(rpool) + 1e-37
    pworst = float((np.abs(pool - (c["pool"] if keep else rpool)) / ptol).max())
    print(f"  {what}: out {worst:.3f}, pool {pworst:.3f} of the bound", flush=True)
    assert worst <= 1 and pworst <= 1, what
    if untouched is not None:
        assert (got[~live] == untouched).all(), f"{what}: rows that no sequence writes"
    rest = [s for s in range(len(pool)) if s not in c["slot"]]
    assert np.array_equal(pool[rest], c["pool"][rest]), f"{what}: other slots"


def call_scan(gdn, g, **kw):
    return gdn.selective_scan(g["x"], g["dt"], g["A"], g["B"], g["C"], g["cu"], g["slot"], g["pool"], D=g["D"], z=g["z"],
                              dt_bias=g["dt_bias"], **kw)


SCANS = [
    ([1], 8, 8, 1, BF), ([29], 64, 16, 1, BF), ([7, 0, 1, 64, 65], 100, 16, 1, BF), ([130, 3], 65, 16, 1, F32),
    ([33], 258, 32, 2, BF), ([15, 16, 17, 31, 32, 33], 192, 32, 3, F32), ([40, 9], 130, 64, 1, BF), ([70], 36, 128, 4, F32),
    ([63, 1], 70, 128, 1, BF), ([700, 200, 1200], 64, 16, 1, F32), ([12] * 40, 24, 8, 2, BF), ([2500], 40, 16, 1, BF),
]


@pytest.mark.parametrize("lens,D,S,G,dtype", SCANS)
def test_scan(gdn_lib, lens, D, S, G, dtype):
    print("[case] scan", lens[:6], D, S, G, dtype, flush=True)
    rng = np.random.default_rng(sum(lens) + D)
    c, g = scan_case(rng, lens, D, S, G, dtype)
    out = call_scan(gdn_lib, g, max_seqlen=max(lens))
    check_scan(c, out, g["pool"], dtype, "scan")


@pytest.mark.parametrize("dtype,out_dtype", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("z,skipw,bias,softplus", [(False, True, True, True), (True, False, False, False), (False, False, True, True)])
def test_scan_options_and_masks(gdn_lib, dtype, out_dtype, z, skipw, bias, softplus):
    """Skipped and fresh sequences, padding tokens behind the last one, a given output, the pool kept."""
    print("[case] scan options", dtype, z, skipw, bias, softplus, flush=True)
    rng = np.random.default_rng(5)
    lens, init = [20, 33, 0, 0, 5, 48], [1, 0, 0, 1, 1, 1]
    for keep in (False, True):
        c, g = scan_case(rng, lens, 72, 16, 1, dtype, skip=(4,), pad=9, z=z, skipw=skipw, bias=bias, softplus=softplus)
        out = torch.full((sum(lens) + 9, 72), 7.0, dtype=out_dtype, device="cuda")
        got = call_scan(gdn_lib, g, has_init=i32(init), out=out, dt_softplus=softplus, keep_pool=keep)
        assert got is out
        check_scan(c, out, g["pool"], out_dtype, "options", has_init=init, softplus=softplus, keep=keep, untouched=7.0)


def test_scan_odd_addresses_and_strides(gdn_lib):
    """Every operand at an odd element, with its own row stride; the output in a wider buffer."""
    print("[case] scan strides", flush=True)
    rng = np.random.default_rng(6)
    c, g = scan_case(rng, [37, 90], 77, 16, 1, BF)
    T = 127

    def odd(t, lead, tail):
        w = torch.zeros((T, lead + t.shape[1] + tail), dtype=t.dtype, device="cuda")
        w[:, lead:lead + t.shape[1]] = t
        return w[:, lead:lead + t.shape[1]]
    for k, a, b in (("x", 1, 3), ("dt", 3, 0), ("z", 5, 2)):
        g[k] = odd(g[k], a, b)
    for k, a, b in (("B", 1, 2), ("C", 7, 1)):
        g[k] = odd(g[k].flatten(1), a, b)
    wide = torch.full((T, 90), 3.0, dtype=BF, device="cuda")
    call_scan(gdn_lib, g, out=wide[:, 5:82])
    check_scan(c, wide[:, 5:82], g["pool"], BF, "strides")
    assert (wide[:, :5] == 3).all() and (wide[:, 82:] == 3).all()


def test_scan_long_memory_and_sharp_decay(gdn_lib):
    """Decays near 1 over a long sequence, and decays that underflow at once."""
    print("[case] scan decays", flush=True)
    rng = np.random.default_rng(7)
    for size, dtype in ((1e-3, F32), (30.0, F32), (1e-3, BF)):
        c, g = scan_case(rng, [1800], 64, 16, 1, dtype)
        c["A"] = rounded(c["A"] * size, F32)
        g["A"] = up(c["A"], F32)
        out = call_scan(gdn_lib, g, max_seqlen=1800)
        check_scan(c, out, g["pool"], dtype, f"decay {size}")


def test_scan_values_that_are_not_finite_stay_in_their_channel_and_sequence(gdn_lib):
    print("[case] scan NaN", flush=True)
    rng = np.random.default_rng(8)
    c, g = scan_case(rng, [50, 60, 30], 80, 16, 1, BF, pad=6, skip=(2,))
    clean = call_scan(gdn_lib, {**g, "pool": g["pool"].clone()})
    g["x"][10, 3] = float("nan")
    g["dt"][70, 9] = float("inf")
    g["x"][110:] = float("nan")                  # a skipped sequence and the padding
    g["B"][110:] = float("nan")
    g["pool"][[s for s in range(5) if s not in c["slot"]]] = float("nan")
    out = torch.full_like(clean, 5.0)
    pool = g["pool"].clone()
    call_scan(gdn_lib, {**g, "pool": pool}, out=out)
    hit = torch.zeros(clean.shape, dtype=torch.bool, device="cuda")
    hit[10:50, 3] = True
    hit[70:110, 9] = True
    assert out[10:50, 3].isnan().all() and not out[70, 9].isfinite()
    assert torch.equal(out[:110][~hit[:110]], clean[:110][~hit[:110]]) and (out[110:] == 5).all()
    # limits that the formula has: delta = 0 for dt = -inf leaves the state; a delta of 100 and more forgets it
    c, g = scan_case(rng, [2], 16, 16, 1, F32, z=False, skipw=False, bias=False)
    g["dt"][:] = float("-inf")
    before = g["pool"].clone()
    call_scan(gdn_lib, g)
    assert torch.equal(g["pool"], before)
    g["dt"][:] = 3e4
    g["x"][:] = 1e-3
    call_scan(gdn_lib, g)
    want = 3e4 * g["x"][1, :, None] * g["B"][1]
    torch.testing.assert_close(g["pool"][int(c["slot"][0])], want, rtol=2.0 ** -21, atol=0)


@pytest.mark.parametrize("n,D,S,G,dtype", [(1, 2048, 16, 1, BF), (5, 100, 8, 1, F32), (37, 130, 32, 2, BF), (9, 66, 64, 1, F32),
                                           (64, 63, 16, 3, BF), (3, 40, 128, 1, BF), (130, 512, 16, 1, BF)])
def test_update(gdn_lib, n, D, S, G, dtype):
    print("[case] update", n, D, S, G, dtype, flush=True)
    rng = np.random.default_rng(n + D)
    skip = tuple(range(n - n // 8, n))
    c, g = scan_case(rng, [1] * n, D, S, G, dtype, skip=skip)
    out = torch.full((n, D), 7.0, dtype=dtype, device="cuda")
    got = gdn_lib.selective_update(g["x"], g["dt"], g["A"], g["B"], g["C"], g["slot"], g["pool"], D=g["D"], z=g["z"],
                                   dt_bias=g["dt_bias"], out=out)
    assert got is out
    check_scan(c, out, g["pool"], dtype, "update", untouched=7.0)


@pytest.mark.parametrize("dtype,out_dtype,z,skipw,bias,softplus", [(BF, F32, False, True, True, True), (F32, BF, True, False, False, False)])
def test_update_options(gdn_lib, dtype, out_dtype, z, skipw, bias, softplus):
    print("[case] update options", dtype, flush=True)
    rng = np.random.default_rng(11)
    c, g = scan_case(rng, [1] * 6, 90, 16, 1, dtype, z=z, skipw=skipw, bias=bias, softplus=softplus)
    out = gdn_lib.selective_update(g["x"], g["dt"], g["A"], g["B"][:, 0], g["C"][:, 0], g["slot"], g["pool"], D=g["D"], z=g["z"],
                                   dt_bias=g["dt_bias"], dt_softplus=softplus, out_dtype=out_dtype)
    assert out.dtype is out_dtype
    check_scan(c, out, g["pool"], out_dtype, "update options", softplus=softplus)


# ------------------------------------------------------------------ norm
def norm_case(rng, T, H, d, dtype, residual, gate, wdtype):
    shape = (T, H, d) if H > 1 else (T, d)
    size = np.exp2(rng.integers(-6, 6, (T,) + (1,) * (len(shape) - 1)))
    h = dict(x=rounded(rng.normal(size=shape) * size, dtype), residual=None, gate=None, weight=None)
    if residual is not None:
        h["residual"] = rounded(rng.normal(size=shape) * 3, residual)
    if gate:
        h["gate"] = rounded(rng.normal(size=shape) * 2, dtype)
    if wdtype is not None:
        h["weight"] = rounded(rng.normal(size=d), wdtype)
    return h


def check_norm(h, got, kept, out_dtype, group, what, *, residual=None, **kw):
    T, d = h["x"].shape[0], h["x"].shape[-1]
    full = lambda v: None if v is None else v.reshape(T, -1, d)  # noqa: E731
    y, u = os_.rms_norm(full(h["x"]), h["weight"], residual=full(h["residual"]), gate=full(h["gate"]), **kw)
    y = y.reshape(T, -1)
    # fp32: the sum of squares (a lane's d / 64 terms and six steps, at least 8 values a lane), u, root,
    # quotient, weight, gate
    rel = (max(d / 64, 8) + 48) * 2.0 ** -24
    if residual is not None:
        want = (torch.from_numpy(h["x"]).float() + torch.from_numpy(h["residual"]).float()).to(residual)
        assert torch.equal(kept.cpu(), want.view(kept.shape)), f"{what}: residual"
    if out_dtype is not F8:
        tol = (rel + HALF[out_dtype] * (1 + rel)) * np.abs(y) + 1e-38
        worst = float((np.abs(host(got).reshape(T, -1) - y) / tol).max())
    else:
        codes, scale = got
        s = os_.group_scales(y, group)
        assert scale.shape == s.shape
        assert (np.abs(host(scale) - s) <= (rel + 2.0 ** -23) * s).all(), f"{what}: scale"
        per = host(scale)[:, np.arange(y.shape[1]) // (group or y.shape[1])]
        v = os_.E4M3[codes.view(torch.uint8).cpu().numpy().reshape(T, -1)] * per
        # half a step of e4m3 (of its subnormals below 2^-6), and the value's own error
        tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * per) * (1 + 4 * rel) + 4 * rel * np.abs(y)
        worst = float((np.abs(v - y) / tol).max())
    print(f"  {what}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1, what


@pytest.mark.parametrize("T,H,d", [(1, 1, 2048), (3, 1, 1), (5, 1, 77), (4, 1, 512), (130, 1, 4096), (7, 1, 5003), (2, 1, 20000),
                                   (9, 32, 128), (6, 3, 100), (33, 4, 64), (5, 2, 256), (3, 64, 24), (2, 1, 40004), (1, 1, 1 << 20),
                                   (1500, 5, 9), (1100, 37, 27), (4, 37, 100), (3, 11, 8), (2, 700, 17), (2, 3, 5000), (2, 31, 1000),
                                   (5, 13, 3), (3, 400, 110), (2, 2, 12)])
@pytest.mark.parametrize("out_dtype,group", [(BF, 0), (F8, 0), (F8, 128), (F8, 64), (F32, 0)])
def test_norm(gdn_lib, T, H, d, out_dtype, group):
    print("[case] norm", T, H, d, out_dtype, group, flush=True)
    rng = np.random.default_rng(T + d)
    for dtype, residual, gate, first, wdtype, offset in ((BF, BF, False, False, BF, 1.0), (BF, None, True, False, F32, 0.0),
                                                         (F32, F32, False, False, None, 0.0), (F32, None, True, True, BF, 1.0)):
        h = norm_case(rng, T, H, d, dtype, residual, gate, wdtype)
        r = up(h["residual"], residual)
        got = gdn_lib.rms_norm(up(h["x"], dtype), up(h["weight"], wdtype), eps=1e-5, offset=offset, residual=r,
                               gate=up(h["gate"], dtype), gate_first=first, out_dtype=out_dtype, group=group)
        check_norm(h, got, r, out_dtype, group, f"{dtype} {residual} {gate}", residual=residual, eps=1e-5, offset=offset,
                   gate_first=first)


def test_norm_strides_and_given_outputs(gdn_lib):
    """Rows inside of wider ones, aligned and at odd elements; outputs given; what is beside them stays."""
    print("[case] norm strides", flush=True)
    rng = np.random.default_rng(3)
    for lead, extra in ((8, 16), (3, 2)):
        for d in (256, 130):
            h = norm_case(rng, 11, 4, d, BF, BF, False, BF)
            width = 4 * d

            def inside(v, dtype, fill=9.0):
                w = torch.full((11, lead + width + extra), fill, dtype=F32, device="cuda").to(dtype)
                if v is not None:
                    w[:, lead:lead + width] = up(v, dtype).view(11, width)
                return w, w[:, lead:lead + width].unflatten(1, (4, d))
            xw, x = inside(h["x"], BF)
            rw, r = inside(h["residual"], BF)
            ow, o = inside(None, F8)
            scale = torch.empty(11, -(-width // 64), device="cuda")
            before = rw.clone(), ow.clone()
            got = gdn_lib.rms_norm(x, up(h["weight"], BF), residual=r, out=o, scale=scale, group=64)
            assert got[0] is o and got[1] is scale
            check_norm(h, (o, scale), r.reshape(11, 4, d), F8, 64, f"strides {lead} {d}", residual=BF)
            for w, b in ((rw, before[0]), (ow.view(torch.uint8), before[1].view(torch.uint8))):
                assert torch.equal(w[:, :lead], b[:, :lead]) and torch.equal(w[:, lead + width:], b[:, lead + width:])


def test_norm_zero_rows_and_values_that_are_not_finite(gdn_lib):
    print("[case] norm values", flush=True)
    for d in (128, 333):
        x = torch.randn(4, 2, d, device="cuda")
        x[1] = 0
        x[2, 0, 5] = float("nan")
        x[3, 1, 7] = float("inf")
        codes, scale = gdn_lib.rms_norm(x, out_dtype=F8, group=0)
        v = codes.float()
        assert (v[1] == 0).all() and scale[1, 0] == 2.0 ** -64
        assert v[2, 0].isnan().all() and v[2, 1].isfinite().all() and scale[2].isfinite().all()
        assert v[3, 1, 7].isnan() and (v[3, 1, :7] == 0).all() and v[3, 0].isfinite().all()
        ref, s0 = gdn_lib.rms_norm(x[:1].contiguous(), out_dtype=F8, group=0)
        assert torch.equal(ref.view(torch.uint8), codes[:1].view(torch.uint8)) and torch.equal(s0, scale[:1])


# ------------------------------------------------------------------ pages
def pages_case(rng, N, page, hi, held, pad, short, width=None):
    h = rng.integers(0, held + 1, N)
    new = np.minimum(rng.integers(0, hi + 1, N), hi) if hi > 1 else np.ones(N, np.int64)
    h[rng.permutation(N)[:pad]] = -1
    owned = [-(-max(int(a), 0) // page) for a in h]
    need = [max(0, -(-(int(a) + int(b)) // page) - o) if a >= 0 else 0 for a, b, o in zip(h, new, owned)]
    free = sum(need) * 2 // 3 if short else sum(need) + 7
    perm = rng.permutation(sum(owned) + free)
    width = width or max(a + b for a, b in zip(owned, need)) + 2
    table = np.full((N, width), -5, np.int64)
    at = 0
    for n, o in enumerate(owned):
        table[n, :min(o, width)] = perm[at:at + o][:width]
        at += o
    return h, new, table, list(perm[at:])


def run_plan(gdn, h, new, table, stack, page, T, start=None, capacity=None):
    capacity = capacity or len(stack) + 20
    state = torch.zeros(2 + capacity, dtype=torch.int32, device="cuda")
    state[0] = len(stack)
    state[2:2 + len(stack)] = i32(stack)
    pool, t = gdn.PagePool(state), i32(table)
    return pool, t, gdn.plan_pages(pool, t, i32(h), i32(new), page, T, start=i32(start))


def check_plan(want, pool, t, plan, what):
    stack, table, cu, cl, kv, slots, pos, seq = want
    s = pool.state.cpu().numpy()
    assert s[0] == len(stack) and s[1] == 0 and s[2:2 + len(stack)].tolist() == [int(x) for x in stack], f"{what}: pool"
    assert np.array_equal(t.cpu().numpy(), table), f"{what}: table"
    for got, ref, name in zip(plan, (cu, cl, kv, slots, pos, seq), plan._fields):
        assert got.cpu().numpy().tolist() == [int(x) for x in ref], f"{what}: {name}"


@pytest.mark.parametrize("N,page,hi,held,pad,short", [
    (1, 16, 1, 0, 0, False), (1, 64, 300, 5, 0, False), (5, 16, 40, 100, 1, False), (256, 64, 1, 4096, 4, False),
    (257, 32, 1, 200, 30, True), (64, 64, 3000, 600, 0, False), (64, 128, 3000, 600, 3, True), (700, 16, 20, 60, 50, True),
    (3000, 16, 3, 50, 100, False), (3, 1, 50, 20, 0, False), (2, 64, 20000, 1, 0, False)])
def test_plan_and_release(gdn_lib, N, page, hi, held, pad, short):
    print("[case] pages", N, page, hi, held, pad, short, flush=True)
    rng = np.random.default_rng(N + page + hi)
    h, new, table, stack = pages_case(rng, N, page, hi, held, pad, short)
    total = int(new[h >= 0].sum())
    for T, start in ((total, None), (total + 13, h + 1000), (max(1, total * 2 // 3), None)):
        pool, t, plan = run_plan(gdn_lib, h, new, table, stack, page, T, start)
        want = os_.plan_pages(stack, len(stack) + 20, table, h, new, page, T, start)
        check_plan(want, pool, t, plan, f"T {T}")
        # half of the new rows go back (a rejected draft), then all that is held
        keep = [-1 if a < 0 else a + (b - a) // 2 for a, b in zip(want[3], want[4])]
        gdn_lib.release_pages(pool, t, i32(keep), plan.kv_len, page)
        stack2 = os_.release_pages(want[0], len(stack) + 20, want[1], keep, want[4], page)
        s = pool.state.cpu().numpy()
        assert s[0] == len(stack2) and s[1] == 0 and s[2:2 + len(stack2)].tolist() == [int(x) for x in stack2]
        zero = [0 if k >= 0 else -1 for k in keep]
        gdn_lib.release_pages(pool, t, i32(zero), i32(keep), page)
        stack3 = os_.release_pages(stack2, len(stack) + 20, want[1], zero, keep, page)
        s = pool.state.cpu().numpy()
        assert s[0] == len(stack3) and s[2:2 + len(stack3)].tolist() == [int(x) for x in stack3]


def test_plan_edges(gdn_lib):
    """No request; a table too narrow; negative ids; counts out of range; given outputs; state slots."""
    print("[case] pages edges", flush=True)
    pool = gdn_lib.page_pool(6)
    assert pool.capacity == 6 and pool.state.tolist() == [6, 0, 5, 4, 3, 2, 1, 0]
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    plan = gdn_lib.plan_pages(pool, torch.empty((0, 3), dtype=torch.int32, device="cuda"), e, e, 16, 5)
    assert plan.cu_seqlens.tolist() == [0] and plan.slots.tolist() == [-1] * 5 and pool.state[0] == 6
    rng = np.random.default_rng(0)
    h, new = np.array([0, 40, 3, 2 ** 31 - 3]), np.array([33, 5, 9, 10])
    table = np.full((4, 2), -1)
    table[2, 0] = 77
    pool, t, plan = run_plan(gdn_lib, h, new, table, list(range(9)), 16, 60)
    check_plan(os_.plan_pages(list(range(9)), 29, table, h, new, 16, 60), pool, t, plan, "narrow")
    assert plan.cache_len.tolist() == [-1, -1, 3, -1]
    for count, seen in ((-3, 0), (500, 8)):
        state = torch.arange(10, dtype=torch.int32, device="cuda")
        state[0], state[1] = count, 0
        pool = gdn_lib.PagePool(state)
        t = i32(np.full((1, 4), -1))
        plan = gdn_lib.plan_pages(pool, t, i32([0]), i32([20]), 16, 20)
        assert plan.kv_len.tolist() == [20 if seen else -1] and int(state[0]) == (seen - 2 if seen else 0)
        assert t.tolist() == [[9, 8, -1, -1] if seen else [-1] * 4]
    # one state slot for each request that has none: a page that no sequence fills
    pool, t = gdn_lib.page_pool(4), i32(np.full((3, 1), -1))
    gdn_lib.plan_pages(pool, t, i32([0, -1, 0]), i32([700, 3, 1]), 1 << 30, 701)
    assert t.tolist() == [[0], [-1], [1]] and pool.state.tolist()[:4] == [2, 0, 3, 2]
    # static buffers
    pool, t = gdn_lib.page_pool(40), i32(np.full((3, 8), -1))
    out = gdn_lib.StepPlan(*(torch.full((k,), 9, dtype=d, device="cuda") for k, d in
                             ((4, torch.int32), (3, torch.int32), (3, torch.int32), (30, torch.int64), (30, torch.int32), (30, torch.int32))))
    assert gdn_lib.plan_pages(pool, t, i32([0, 5, -1]), i32([10, 4, 6]), 16, 30, out=out) is out
    assert out.cu_seqlens.tolist() == [0, 10, 14, 14] and out.seq.tolist() == [0] * 10 + [1] * 4 + [-1] * 16
    assert out.slots[10:14].tolist() == [-1] * 4, "request 1 holds rows on a page that the table lacks"
