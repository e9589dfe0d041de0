"""Small cases of the softmax-attention operators: numpy inputs, their upload, and bounds on
how far a kernel may be from oracle.attention."""
import numpy as np
import torch

from oracle import attention as oa

BF = 2.0 ** -8          # half a step of bf16, relative


def bf16(x):
    """x rounded to bf16 values, as float32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def make_cache(rng, pages, H, page, d, track=False):
    """A cache with every row filled; scales differ from page to page."""
    x = rng.normal(0, 1, (2, pages, H, page, d)) * 2.0 ** rng.integers(-2, 2, (2, pages, H, 1, 1))
    c = dict(pos=None, weight=None)
    for name, y in zip("kv", x):
        s = np.array([[oa.page_scale(y[p, h]) for h in range(H)] for p in range(pages)])
        c[name], c[name + "_scale"] = oa.e4m3_encode(y / s[:, :, None, None]), s
    if track:
        c["pos"] = np.zeros((pages, H, page), np.int64)
        c["weight"] = rng.random((pages, H, page)).astype(np.float32).astype(np.float64)
    return c


def make_table(rng, counts, page, pages, width=None):
    """Block table over distinct random pages; unused entries are -1."""
    need = [-(-max(c, 0) // page) for c in counts]
    width = max(max(need), 1) if width is None else width
    perm = list(rng.permutation(pages)[:sum(need)])
    t = np.full((len(counts), width), -1, np.int64)
    for n, m in enumerate(need):
        t[n, :m] = [perm.pop() for _ in range(m)]
    return t


def spread_positions(rng, cache, table, counts):
    """Ascending positions with gaps on every sequence's rows (per kv head)."""
    page, H = cache["k"].shape[2], cache["k"].shape[1]
    last = []
    for n, count in enumerate(counts):
        top = 0
        for h in range(H):
            pos = np.cumsum(rng.integers(1, 4, max(count, 0)))
            for r, x in enumerate(pos):
                cache["pos"][table[n, r // page], h, r % page] = x
            top = max(top, int(pos[-1]) if len(pos) else 0)
        last.append(top)
    return last


def up(x, dtype=None):
    if x is None:
        return None
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def i32(x):
    return None if x is None else torch.from_numpy(np.asarray(x, np.int32)).cuda()


def upload_cache(gdn, c):
    f8 = lambda x: up(x).view(torch.float8_e4m3fn)  # noqa: E731
    return gdn.KVCache(f8(c["k"]), f8(c["v"]), up(c["k_scale"], torch.float32), up(c["v_scale"], torch.float32),
                       None if c["pos"] is None else up(c["pos"], torch.int32),
                       None if c["weight"] is None else up(c["weight"], torch.float32))


def host_cache(c):
    return dict(k=c.k.view(torch.uint8).cpu().numpy(), v=c.v.view(torch.uint8).cpu().numpy(),
                k_scale=c.k_scale.double().cpu().numpy(), v_scale=c.v_scale.double().cpu().numpy(),
                pos=None if c.pos is None else c.pos.cpu().numpy().astype(np.int64),
                weight=None if c.weight is None else c.weight.double().cpu().numpy())


def assert_same_cache(got, want, what):
    for a in ("k", "v", "k_scale", "v_scale", "pos", "weight"):
        if want[a] is not None:
            assert np.array_equal(got[a], want[a], equal_nan=True), f"{what}: cache.{a} differs"


def row_norm(x):
    """Largest norm of a row (last axis) of finite values."""
    return float(np.sqrt(np.nan_to_num(np.square(np.asarray(x, np.float64)), nan=0.0, posinf=0.0).sum(-1).max()))


def cache_norm(c):
    """Largest norm of a cached key."""
    x = np.nan_to_num(oa.E4M3[c["k"]]) * c["k_scale"][:, :, None, None]
    return row_norm(x)


def score_error(q, knorm, scale, softcap=0.0, slope=0.0, dist=0):
    """How far a score's fp32 value can be from the exact one: d products summed in any
    order ((d + 4) roundings of at most sum |q k| <= |q| |k|), the scaling, the log2 e and the
    exponent's argument (relative to the score), the cap's tanh (a few units of 2^-24 times
    cap) and the bias."""
    d = q.shape[-1]
    top = scale * row_norm(q) * knorm
    size = top if softcap == 0 else min(top, softcap)
    return (d + 4) * 2.0 ** -24 * top + 2.0 ** -21 * (size + softcap + slope * dist)


def assert_out(got, ref, mag, ds, what):
    """|got - ref| <= bf16 rounding of the output and of every weight, and weights that are
    off by 2 ds relative (numerator and normaliser)."""
    got = np.asarray(got, np.float64)
    live = np.isfinite(ref)
    assert np.isfinite(got[live]).all(), f"{what}: non-finite output"
    tol = (BF * (np.abs(ref) + mag) + 2 * ds * mag) * (1 + 2 * BF) + 1e-30
    worst = float((np.abs(got - ref)[live] / tol[live]).max()) if live.any() else 0.0
    print(f"  {what}: worst error {worst:.3f} of the bound (score error {ds:.1e})", flush=True)
    assert worst <= 1, f"{what}: {worst:.3f} of the bound"
