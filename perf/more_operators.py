"""What a hybrid model's serving step runs beside its linear and softmax attention, as cases
that can be timed and checked: the selective state space scan of packed prompts
(selective_scan) and its step of one token per sequence (selective_update), the
root-mean-square norm with the residual's addition, a gate and an output in 8 bits
(rms_norm), and the block tables and slot maps of a step, built on the GPU from the
requests' lengths (plan_pages, release_pages).

`run` computes a case with elementary torch operations in 32 bits, or, with `own` set,
with the calls of the package.  `exact` gives the same outputs in 64 bits from the
definitions.

Definitions.
Scan: channel c of group g = c // (d / groups) with its state h [states], token by token
  delta = softplus(dt[t, c] + dt_bias[c])
  h_i   = exp(delta A[c, i]) h_i + delta x[t, c] B[t, g, i]
  y     = (sum_i C[t, g, i] h_i + D[c] x[t, c]) * z sigmoid(z),  z = z[t, c]
A sequence starts from its slot of the pool, or from zeros, and leaves its last state there.
Norm: u = x + residual (the sum is also the new residual), or u = x, or u = x g sigmoid(g)
  y = u / sqrt(mean(u^2) + eps) * (weight + offset) [* g sigmoid(g)]
over the last dimension; in 8 bits y = code * scale, the scale of a group of values being
their largest magnitude / 448, at least 2^-64, the code y / scale to the nearest e4m3 value.
Pages: request n holds held[n] rows and brings new[n] tokens.  It needs the pages
ceil(held / page) .. ceil((held + new) / page) - 1 of its row of the table, and gets them in
order of the requests from the top of the stack of free pages, as long as the stack and the
room for tokens last; those after that get none, and their lengths become -1.  A token's slot
is (its page) * page + (its row there).  The release pushes a request's pages back in order.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
DEVICE = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt: latency
        dict(name="scan one prompt of 29", op="scan", n=1, lo=29, hi=29, d=1024, states=16, groups=1, f32=False,
             z=True, init=False),
        # a ragged batch that continues cached states, in 32 bits, odd channels, two groups
        dict(name="scan ragged 24 in fp32", op="scan", n=24, lo=1, hi=3000, d=1000, states=32, groups=2, f32=True,
             z=False, init=True),
        # one long document
        dict(name="scan one of 30000", op="scan", n=1, lo=30000, hi=30000, d=2048, states=16, groups=1, f32=False,
             z=True, init=False),
        # the batched prefill
        dict(name="scan 8 x 4096", op="scan", n=8, lo=4096, hi=4096, d=4096, states=16, groups=1, f32=False, z=True,
             init=False),
        # one chat's next token: latency
        dict(name="update 1", op="update", n=1, pad=0, d=2048, states=16, groups=1, f32=False, z=True),
        # the batched decode, some rows of the static batch being padding
        dict(name="update 256", op="update", n=256, pad=6, d=4096, states=16, groups=1, f32=False, z=True),
        # one token between two layers: latency
        dict(name="norm 1 x 2048 in e4m3", op="norm", t=1, heads=1, d=2048, residual="bf16", gate="", out="e4m3", group=0),
        # the same for a batched prefill
        dict(name="norm 32768 x 4096 in e4m3", op="norm", t=32768, heads=1, d=4096, residual="bf16", gate="", out="e4m3",
             group=0),
        # the gated norm behind a linear-attention layer, a scale for each head's 128 values
        dict(name="norm gated 32768 x 32 x 128", op="norm", t=32768, heads=32, d=128, residual="", gate="after", out="e4m3",
             group=128),
        # odd rows, the residual kept in 32 bits
        dict(name="norm 777 x 5003", op="norm", t=777, heads=1, d=5003, residual="f32", gate="", out="bf16", group=0),
        # a decode step of 256 requests (every 64th needs a page), and its pages given back
        dict(name="pages of 256 decoding", op="pages", n=256, pad=4, lo=1, hi=1, held=4096, page=64, short=False),
        # a step of 64 ragged prompts, 131072 tokens at most, and their pages given back
        dict(name="pages of 64 ragged prompts", op="pages", n=64, pad=0, lo=1, hi=8192, held=600, page=64, short=False),
    ]


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["scan", "scan", "update", "norm", "norm", "pages"])
    if op in ("scan", "update"):
        groups = rng.choice([1, 1, 1, 2, 4])
        c = dict(op=op, d=groups * log(8, 5000 // groups), states=rng.choice([8, 16, 16, 32, 64, 128]), groups=groups,
                 f32=rng.random() < 0.3, z=rng.random() < 0.7)
        area = c["d"] * c["states"]
        if op == "scan":
            hi = min(log(1, 20000), max(1, int(4.0e8 / area)))
            n = max(1, min(log(1, 200), int(4.0e8 / (area * hi))))
            c.update(n=n, lo=max(1, hi // rng.choice([1, 5, 100])), hi=hi, init=rng.random() < 0.5)
        else:
            n = max(1, min(log(1, 600), int(1.6e7 / area)))
            c.update(n=n, pad=rng.choice([0, n // 8]))
        return c
    if op == "norm":
        heads = rng.choice([1, 1, log(2, 64)])
        d = log(1, 20000) if heads == 1 else rng.choice([64, 128, 256, log(8, 300)])
        t = max(1, min(log(1, 60000), int(1.2e8 / (heads * d))))
        gate = rng.choice(["", "after", "first"])
        return dict(op=op, t=t, heads=heads, d=d, residual="" if gate else rng.choice(["", "bf16", "f32"]), gate=gate,
                    out=rng.choice(["bf16", "f32", "e4m3", "e4m3"]), group=rng.choice([0, 64, 128]))
    hi = rng.choice([1, log(2, 8192)])
    n = max(1, min(log(1, 4000), int(131072 / hi)))
    return dict(op=op, n=n, pad=n // 16, lo=max(1, hi // rng.choice([1, 5, 1000])), hi=hi, held=rng.choice([0, log(1, 8000)]),
                page=rng.choice([16, 32, 64, 128]), short=rng.random() < 0.3)


def _lengths(case):
    """The case's ragged lengths: log-uniform in [lo, hi], the longest among them."""
    r = random.Random(1000 * case["n"] + case["hi"])
    a, b = case["lo"], case["hi"]
    got = [min(b, max(a, int(round(math.exp(r.uniform(math.log(a), math.log(b))))))) for _ in range(case["n"])]
    got[-1] = b
    return got


def work(case):
    if case["op"] in ("scan", "update"):
        d, ds, g, size = case["d"], case["states"], case["groups"], 4 if case["f32"] else 2
        rows = sum(_lengths(case)) if case["op"] == "scan" else case["n"] - case["pad"]
        seqs = case["n"] if case["op"] == "scan" else rows
        kept = seqs * d * ds * 4 * (2 if case["op"] == "update" or case["init"] else 1)
        return {"bytes": rows * size * (d * (4 if case["z"] else 3) + 2 * g * ds) + kept + d * (ds + 2) * 4,
                "flops": rows * d * (7 * ds + 12)}
    if case["op"] == "norm":
        w = case["heads"] * case["d"]
        out = {"bf16": 2, "f32": 4, "e4m3": 1}[case["out"]]
        kept = {"": 0, "bf16": 4, "f32": 8}[case["residual"]]
        scales = (-(-w // case["group"]) if case["group"] else 1) * 4 if case["out"] == "e4m3" else 0
        return {"bytes": case["t"] * (w * (2 + out + kept + (2 if case["gate"] else 0)) + scales) + 2 * case["d"],
                "flops": case["t"] * w * (12 if case["gate"] else 6)}
    lens = _lengths(case)
    pages = sum(lens) / case["page"]
    return {"bytes": 20 * case["n"] + 16 * sum(lens) + 24 * pages, "flops": 10 * case["n"] + 4 * sum(lens)}


# ------------------------------------------------------------------ inputs
def _scan_inputs(case, rows, gen, dev):
    """x (behind the short conv and its SiLU), dt, B, C and z as the projections leave them:
    B and C next to dt's low-rank part, z next to x's half; A, D, dt_bias as such a layer starts."""
    d, ds, g = case["d"], case["states"], case["groups"]
    kind = torch.float32 if case["f32"] else torch.bfloat16
    rand = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    rank = max(8, d // 16 // 8 * 8)
    x = rand(rows, d)
    proj = rand(rows, rank + 2 * g * ds).to(kind)
    start = torch.exp(torch.empty(d, device=dev).uniform_(math.log(1e-3), math.log(0.1), generator=gen))
    s = dict(x=(x / (1 + torch.exp(-x))).to(kind), dt=(0.7 * rand(rows, d)).to(kind),
             B=proj[:, rank:rank + g * ds].unflatten(1, (g, ds)), C=proj[:, rank + g * ds:].unflatten(1, (g, ds)),
             A=-(torch.arange(1, ds + 1, device=dev) * torch.exp(0.2 * rand(d, ds))), D=1 + 0.1 * rand(d),
             dt_bias=start + torch.log(-torch.expm1(-start)), z=None)
    if case["z"]:
        s["z"] = rand(rows, 2 * d).to(kind)[:, d:]
    return s


def prepare(case, seed):
    dev = DEVICE
    gen = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    op = case["op"]
    if op == "scan":
        lens = _lengths(case)
        n, slots = case["n"], case["n"] + 3
        s = _scan_inputs(case, sum(lens), gen, dev)
        s.update(op=op, cu=i32([0] + torch.tensor(lens).cumsum(0).tolist()), longest=max(lens),
                 slot=torch.randperm(slots, generator=gen, device=dev)[:n].to(torch.int32),
                 pool=0.3 * rand(slots, case["d"], case["states"]),
                 has_init=i32([1 - k % 4 // 3 if case["init"] else 0 for k in range(n)]))
        return s
    if op == "update":
        n, slots = case["n"], 2 * case["n"]
        s = _scan_inputs(case, n, gen, dev)
        slot = torch.randperm(slots, generator=gen, device=dev)[:n].to(torch.int32)
        slot[n - case["pad"]:] = -1                      # the static batch's last rows are padding
        s.update(op=op, slot=slot, live=n - case["pad"], pool=0.3 * rand(slots, case["d"], case["states"]),
                 out=torch.zeros_like(s["x"]))
        return s
    if op == "norm":
        t, h, d = case["t"], case["heads"], case["d"]
        shape = (t, h, d) if h > 1 else (t, d)
        s = dict(op=op, x=rand(*shape).to(torch.bfloat16), weight=(0.1 * rand(d)).to(torch.bfloat16), residual=None, gate=None,
                 first=case["gate"] == "first", group=case["group"],
                 out={"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": F8}[case["out"]])
        if case["gate"]:
            s["gate"] = rand(*shape).to(torch.bfloat16)
        if case["residual"]:
            s["residual"] = (3 * rand(*shape)).to(torch.bfloat16 if case["residual"] == "bf16" else torch.float32)
        return s
    n, page, lens = case["n"], case["page"], _lengths(case)
    r = random.Random(seed)
    held = [r.randint(case["held"] // 2, case["held"]) for _ in range(n)]
    for k in range(case["pad"]):                         # the static batch's padding rows
        held[n - 1 - k] = -1
    owned = [-(-max(a, 0) // page) for a in held]
    need = [-(-(a + b) // page) - -(-a // page) if a >= 0 else 0 for a, b in zip(held, lens)]
    free = sum(need) * 3 // 4 if case["short"] else sum(need) + 1000
    most = [(case["held"] + a) // page + 2 for a in lens]
    total = sum(most) + 1050                             # (some pages belong to requests that do not run now)
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    width = max(most) + 8
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    table[torch.arange(width, device=dev)[None] < torch.tensor(owned, device=dev)[:, None]] = perm[:sum(owned)]
    pool = torch.zeros(total + 2, dtype=torch.int32, device=dev)      # [free pages, 0, the stack of free pages]
    pool[0] = free
    pool[2:2 + free] = perm[sum(owned):sum(owned) + free]
    return dict(op=op, pool=pool, table=table, held=i32(held), new=i32(lens), page=page, tokens=sum(lens) + 5)


# ------------------------------------------------------------------ plain forms
def _silu(x):
    return x / (1 + torch.exp(-x))


def _terms(s):
    """exp(delta A) and delta x B as [rows, groups, channels of a group, states]; x; delta."""
    rows, d = s["x"].shape
    g, ds = s["B"].shape[1:]
    x, v = s["x"].float(), s["dt"].float() + s["dt_bias"]
    delta = v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))
    a = torch.exp_(delta[..., None] * s["A"]).view(rows, g, d // g, ds)
    b = (delta * x).view(rows, g, d // g, 1) * s["B"].float()[:, :, None]
    return a, b, x


def _outputs(s, h, x):
    y = (h * s["C"].float()[:, :, None]).sum(-1).view(x.shape) + s["D"] * x
    return (y if s["z"] is None else y * _silu(s["z"].float())).to(s["x"].dtype)


def _scan(s):
    a, b, x = _terms(s)
    cu, slot = s["cu"].long(), s["slot"].long()
    first, last = cu[:-1], cu[1:] - 1                    # (no sequence of a case is empty)
    start = torch.where(s["has_init"].bool()[:, None, None], s["pool"][slot], 0.0).view(len(slot), *b.shape[1:])
    b[first] += a[first] * start
    a[first] = 0
    k = 1
    while k < s["longest"]:      # b: the sum over 2k tokens up to each, a: the product of their factors
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    s["pool"][slot] = b[last].view(len(slot), *s["pool"].shape[1:])
    return {"out": _outputs(s, b, x), "pool": s["pool"]}


def _update(s):
    a, b, x = _terms(s)
    m, slot = s["live"], s["slot"][:s["live"]].long()
    b[:m] += a[:m] * s["pool"][slot].view(m, *b.shape[1:])
    s["pool"][slot] = b[:m].view(m, *s["pool"].shape[1:])
    s["out"][:m] = _outputs(s, b, x)[:m]
    return {"out": s["out"], "pool": s["pool"]}


def _norm(s):
    u = s["x"].float()
    if s["residual"] is not None:
        u = u + s["residual"].float()
        s["residual"].copy_(u)
    gate = _silu(s["gate"].float()) if s["gate"] is not None else 1.0
    if s["first"]:
        u = u * gate
    y = u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS) * (s["weight"].float() + 1.0)
    if not s["first"]:
        y = y * gate
    if s["out"] != F8:
        return {"out": y.to(s["out"]), "residual": s["residual"]}
    rows = y.flatten(1)
    width, group = rows.shape[1], s["group"] or rows.shape[1]
    count = -(-width // group)
    parts = torch.cat([rows, rows.new_zeros((len(rows), count * group - width))], 1).view(-1, count, group)
    scale = (parts.abs().amax(-1) / 448).clamp(min=2.0 ** -64)
    codes = (parts / scale[..., None]).flatten(1)[:, :width].view(y.shape).to(F8)
    return {"out": codes, "scale": scale, "residual": s["residual"]}


def _plan(s):
    pool, table, page, room = s["pool"], s["table"], s["page"], s["tokens"]
    n, width = table.shape
    held, new = s["held"].long(), s["new"].long()
    live = (held >= 0) & (new >= 0)
    tokens = torch.where(live, new, 0)
    lo, hi = (held + page - 1) // page, (held + tokens + page - 1) // page
    live = live & (hi <= width)
    need = torch.where(live, hi - lo, 0)
    ends, taken = tokens.cumsum(0), need.cumsum(0)
    live = live & (taken <= pool[0]) & (ends <= room)
    at = taken - need                                    # pages that those before a request take
    p = torch.arange(width, device=table.device)[None]
    fresh = live[:, None] & (p >= lo[:, None]) & (p < hi[:, None])
    place = (pool[0] - 1 - (at[:, None] + p - lo[:, None])).clamp(0, len(pool) - 3)
    table.copy_(torch.where(fresh, pool[2 + place], table))
    pool[0] -= torch.where(live, need, 0).sum()
    t = torch.arange(room, device=table.device)
    seq = torch.searchsorted(ends, t, right=True)
    q = seq.clamp(max=n - 1)
    used = (seq < n) & live[q]
    pos = held[q] + t - (ends - tokens)[q]
    ids = table[q, (pos // page).clamp(0, width - 1)].long()
    pick = lambda m, x: torch.where(m, x, -1)  # noqa: E731
    cu = torch.cat([ends.new_zeros(1), ends]).clamp(max=room).to(torch.int32)
    return dict(cu_seqlens=cu, cache_len=pick(live, held).to(torch.int32), kv_len=pick(live, held + new).to(torch.int32),
                slots=pick(used & (ids >= 0), ids * page + pos % page), positions=pick(used, pos).to(torch.int32),
                seq=pick(used, seq).to(torch.int32))


def _release(s, keep, held):
    pool, table, page = s["pool"], s["table"], s["page"]
    n, width = table.shape
    lo, hi = (keep.long() + page - 1) // page, (held.long() + page - 1) // page
    give = torch.where((keep >= 0) & (held >= keep), hi - lo, 0)
    at = give.cumsum(0) - give
    p = torch.arange(width, device=table.device)[None]
    back = (p >= lo[:, None]) & (p < (lo + give)[:, None])
    place = torch.where(back, pool[0] + at[:, None] + p - lo[:, None], 0)
    pool[2 + place[back]] = table[back]
    pool[0] += give.sum()


def _pages(s):
    plan = _plan(s)
    _release(s, plan["cache_len"], plan["kv_len"])
    return {**plan, "table": s["table"], "pool": s["pool"]}


# ------------------------------------------------------------------ the package's calls
def _own_calls(s):
    import hybrid_model_linear_amd as gdn
    op = s["op"]
    if op == "scan":
        out = gdn.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], s["slot"], s["pool"], D=s["D"], z=s["z"],
                                 dt_bias=s["dt_bias"], has_init=s["has_init"], max_seqlen=s["longest"])
        return {"out": out, "pool": s["pool"]}
    if op == "update":
        gdn.selective_update(s["x"], s["dt"], s["A"], s["B"], s["C"], s["slot"], s["pool"], D=s["D"], z=s["z"],
                             dt_bias=s["dt_bias"], out=s["out"])
        return {"out": s["out"], "pool": s["pool"]}
    if op == "norm":
        got = gdn.rms_norm(s["x"], s["weight"], eps=EPS, offset=1.0, residual=s["residual"], gate=s["gate"],
                           gate_first=s["first"], out_dtype=s["out"], group=s["group"])
        if s["out"] != F8:
            return {"out": got, "residual": s["residual"]}
        return {"out": got[0], "scale": got[1], "residual": s["residual"]}
    pool = gdn.PagePool(s["pool"])
    plan = gdn.plan_pages(pool, s["table"], s["held"], s["new"], s["page"], s["tokens"])
    gdn.release_pages(pool, s["table"], plan.cache_len, plan.kv_len, s["page"])
    return {**plan._asdict(), "table": s["table"], "pool": s["pool"]}


def run(state):
    if own:
        return _own_calls(state)
    return {"scan": _scan, "update": _update, "norm": _norm, "pages": _pages}[state["op"]](state)


# ------------------------------------------------------------------ exact values
def _exact_step(s, k, h):
    """One token of every sequence in 64 bits: rows k of the inputs, states h [n, d, states] -> (y, h)."""
    d, g = s["x"].shape[1], s["B"].shape[1]
    x = s["x"][k].double()
    v = s["dt"][k].double() + s["dt_bias"].double()
    delta = torch.logaddexp(v, torch.zeros_like(v))
    own_group = torch.arange(d, device=x.device) // (d // g)
    h = h * torch.exp(delta[..., None] * s["A"].double()) + (delta * x)[..., None] * s["B"][k].double()[:, own_group]
    y = (h * s["C"][k].double()[:, own_group]).sum(2) + s["D"].double() * x
    if s["z"] is not None:
        z = s["z"][k].double()
        y = y * z * torch.sigmoid(z)
    return y, h


def _exact_norm(case, s):
    u = s["x"].double()
    if s["residual"] is not None:
        u = u + s["residual"].double()
    kept = u if s["residual"] is not None else None
    g = s["gate"].double() if s["gate"] is not None else None
    if s["first"]:
        u = u * g * torch.sigmoid(g)
    y = u * torch.rsqrt(u.square().sum(-1, keepdim=True) / case["d"] + EPS) * (1.0 + s["weight"].double())
    if g is not None and not s["first"]:
        y = y * g * torch.sigmoid(g)
    if s["out"] != F8:
        return {"out": y, "residual": kept}
    rows = y.reshape(case["t"], -1)
    step = case["group"] or rows.shape[1]
    scale = torch.stack([rows[:, a:a + step].abs().max(1).values for a in range(0, rows.shape[1], step)], 1) / 448.0
    scale = torch.clamp(scale, min=2.0 ** -64)
    v = rows / scale[:, torch.arange(rows.shape[1], device=rows.device) // step]
    size = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -300))).clamp(min=-6) - 3)   # e4m3's steps
    return {"out": (torch.round(v / size) * size).view(y.shape), "scale": scale, "residual": kept}


def exact(case, seed):
    if case["op"] == "pages":                            # (whole numbers)
        return None
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "update":
        m, pool, out = s["live"], s["pool"].double(), s["out"].double()
        slot = s["slot"][:m].long()
        out[:m], pool[slot] = _exact_step(s, slice(0, m), pool[slot])
        return {"out": out, "pool": pool}
    if case["hi"] * case["d"] * case["states"] * case["n"] > 3.0e9:
        return None
    pool, out = s["pool"].double(), torch.empty(s["x"].shape, dtype=torch.float64, device=s["x"].device)
    lens, cu, slot = _lengths(case), s["cu"].tolist(), s["slot"].long()
    order = sorted(range(case["n"]), key=lambda k: -lens[k])          # longest first: those that still run stand in front
    h = (pool[slot] * s["has_init"][:, None, None])[order]
    begin = torch.tensor([cu[k] for k in order], device=out.device)
    running = case["n"]
    for t in range(max(lens)):
        while lens[order[running - 1]] <= t:
            running -= 1
        k = begin[:running] + t
        out[k], h[:running] = _exact_step(s, k, h[:running])
    pool[slot[order]] = h
    return {"out": out, "pool": pool}
