"""The softmax-attention operators of a hybrid model, as cases that can be timed and
checked: attention of new tokens (attn_extend), attention of one token per sequence over
the 8-bit paged cache (attn_decode), the writing of that cache (kv_store) and its
eviction by accumulated attention weight (kv_evict).

`run` computes a case with elementary torch operations in 32 bits, or, with `own` set,
with the calls of the package.  `exact` gives the same outputs in 64 bits from the
definitions.

Definitions.  Query head h reads kv head h // (H / Hkv).  With p_i, p_j the positions of
a query and a key:
  s_ij = scale q_i.k_j;  capped: cap tanh(s / cap);  biased: s - slope_h |p_i - p_j|
  visible(i, j) = (j <= i, or j among the sequence's first `visible` tokens)
                  and (no window, or |p_i - p_j| < window) and (doc_i == doc_j >= 0)
  o_i = softmax over the visible j of s_ij, applied to v_j (a row that sees nothing: 0)
A cached value is code * scale, the code in e4m3, the scale a power of two per (page, kv
head): the smallest one with max |x| <= 448 scale over the page's rows, at least 2^-64.
Rows appended to a page that holds older ones raise its scale if they need it; the older
codes are then rounded to the new scale.  An eviction keeps `budget` rows per kv head:
those with pos > max pos - recent first, then by weight, ties to the lowest row; the
kept rows at or past `budget` move, in order, into the dropped rows before it, in order.
The scale of a page that receives rows grows to the largest of its own and theirs, and
its rows before `budget` are rounded to it.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
DEVICE = "cuda"
PAGE_SPARE = 3          # pages of the cache that no sequence owns


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt whose first tokens see each other (prefix mask): latency
        dict(name="extend one prompt of 19", op="extend", n=1, lo=19, hi=19, heads=8, kv=2, d=64, cap=0.0,
             bias=False, window=0, docs=0, visible=5, cached=0, page=16),
        # ragged batch of packed documents, capped scores
        dict(name="extend ragged documents", op="extend", n=6, lo=1, hi=4095, heads=16, kv=4, d=128, cap=50.0,
             bias=False, window=0, docs=5, visible=0, cached=0, page=64),
        # the batched prefill, 8 prompts of 4096 tokens
        dict(name="extend 8 x 4096", op="extend", n=8, lo=4096, hi=4096, heads=32, kv=8, d=128, cap=0.0,
             bias=False, window=0, docs=0, visible=0, cached=0, page=64),
        # a chunk of each prompt over its cached part, distance bias, wide heads
        dict(name="extend chunk over cache", op="extend", n=4, lo=512, hi=512, heads=16, kv=2, d=256, cap=0.0,
             bias=True, window=0, docs=0, visible=0, cached=7000, page=64),
        # one chat, short context: latency
        dict(name="decode 1 x 300", op="decode", n=1, lo=300, hi=300, heads=8, kv=2, d=64, cap=0.0, bias=False,
             window=0, track=False, page=16),
        # the batched decode of 256 sequences, ragged contexts
        dict(name="decode 256 ragged", op="decode", n=256, lo=512, hi=4096, heads=32, kv=8, d=128, cap=0.0,
             bias=False, window=0, track=False, page=64),
        # few sequences with long contexts, capped scores, wide heads
        dict(name="decode 2 x 131000", op="decode", n=2, lo=131000, hi=131000, heads=16, kv=2, d=256, cap=30.0,
             bias=False, window=0, track=False, page=128),
        # decode that accumulates the weights an eviction goes by, with distance bias
        dict(name="decode accumulating 32", op="decode", n=32, lo=2000, hi=8192, heads=32, kv=8, d=128, cap=0.0,
             bias=True, window=0, track=True, page=64),
        # the new token of every sequence of a decode batch
        dict(name="store 256 tokens", op="store", n=256, lo=1, hi=1, kv=8, d=128, cached=2000, track=True, page=64),
        # the keys and values of a batched prefill
        dict(name="store 8 x 4096", op="store", n=8, lo=4096, hi=4096, kv=8, d=128, cached=0, track=False, page=64),
        # a few short caches cut to half
        dict(name="evict 4 x 1000 to 500", op="evict", n=4, lo=1000, hi=1000, kv=2, d=64, budget=500, recent=64,
             page=16),
        # a batch of long caches cut to half
        dict(name="evict 32 x 8192 to 4096", op="evict", n=32, lo=8192, hi=8192, kv=8, d=128, budget=4096,
             recent=256, page=64),
    ]


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["extend", "extend", "decode", "decode", "store", "evict"])
    d = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, kv=kv, d=d, page=rng.choice([16, 32, 64, 128]))
    if op == "extend":
        hi = log(3, 4096)
        heads = kv * rng.choice([1, 3, 4, 8])
        heads = heads if heads <= 32 else 32
        cached = rng.choice([0, 0, log(5, 6000)])
        area = heads * hi * (hi + cached)
        n = max(1, min(log(1, 40), int(2.0e9 / area)))
        docs = rng.choice([0, 0, 3]) if not cached else 0
        c.update(n=n, lo=max(1, hi // rng.choice([1, 4, 50])), hi=hi, heads=heads, cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                 bias=rng.random() < 0.3, window=rng.choice([0, 0, 0, log(8, 2000)]), docs=docs,
                 visible=rng.choice([0, 0, log(1, 200)]), cached=cached)
    elif op == "decode":
        hi = log(1, 60000)
        n = max(1, min(log(1, 300), int(4.0e8 / (hi * kv * d))))
        c.update(n=n, lo=max(1, hi // rng.choice([1, 3, 30])), hi=hi, heads=kv * rng.choice([1, 4, 7, 8]),
                 cap=rng.choice([0.0, 0.0, 30.0]), bias=rng.random() < 0.3, window=rng.choice([0, 0, log(16, 4000)]),
                 track=rng.random() < 0.4)
    elif op == "store":
        hi = rng.choice([1, log(2, 4096)])
        n = max(1, min(log(1, 300), int(3.0e7 / (hi * kv * d))))
        c.update(n=n, lo=max(1, hi // rng.choice([1, 20])), hi=hi, cached=rng.choice([0, log(1, 1500)]),
                 track=rng.random() < 0.5)
    else:
        hi = log(40, 16000)
        n = max(1, min(log(1, 60), int(2.5e8 / (hi * kv * d))))
        budget = max(8, int(hi * rng.uniform(0.2, 0.95)))
        c.update(n=n, lo=max(1, hi // rng.choice([1, 2])), hi=hi, budget=budget, recent=rng.choice([0, budget // 8, budget // 2]))
    return c


def _lengths(case):
    """The case's ragged lengths: log-uniform in [lo, hi], the longest among them."""
    r = random.Random(1000 * case["n"] + case["hi"])
    a, b = case["lo"], case["hi"]
    got = [min(b, max(a, int(round(math.exp(r.uniform(math.log(a), math.log(b))))))) for _ in range(case["n"])]
    got[-1] = b
    return got


def _cached(case):
    """Cached tokens of each sequence: from half of `cached` up to all of it."""
    r = random.Random(case["n"] + case["cached"])
    return [r.randint((case["cached"] + 1) // 2, case["cached"]) for _ in range(case["n"])]


def _documents(case, lens):
    """Document ids of every packed token: each sequence cut into about `docs` runs; the
    last tokens of a document-cut sequence are padding (-1), which sees nothing."""
    r = random.Random(7 + case["n"])
    ids = []
    for length in lens:
        cuts = sorted(r.randint(0, length) for _ in range(case["docs"] - 1))
        run, at = [], 0
        for i, c in enumerate(cuts + [length]):
            run += [i] * (c - at)
            at = c
        pad = min(length // 16, 20)
        ids += run[:length - pad] + [-1] * pad
    return ids


def _pairs(case, lens):
    """Visible (query, key) pairs of one head."""
    cached = _cached(case)
    docs = torch.tensor(_documents(case, lens)) if case["docs"] else None
    total, at = 0, 0
    for n, length in enumerate(lens):
        i = torch.arange(length, dtype=torch.int64)
        w = case["window"] or (1 << 40)
        if docs is None:
            lo, hi = (i - w + 1).clamp(min=0), i + 1
            if case["visible"]:
                seen = torch.minimum(torch.full_like(i, min(case["visible"], length)), i + w)
                hi = torch.maximum(hi, seen)
            total += int((hi - lo).clamp(min=0).sum())
        else:
            own_docs = docs[at:at + length]
            for doc in own_docs[own_docs >= 0].unique().tolist():
                j = i[own_docs == doc]
                m = len(j)
                r = torch.arange(m, dtype=torch.int64)
                seen = int((j < case["visible"]).sum())
                lo, hi = (r - w + 1).clamp(min=0), torch.maximum(r + 1, torch.minimum(torch.full_like(r, seen), r + w))
                total += int((hi - lo).clamp(min=0).sum())
        p = cached[n]
        total += int(torch.minimum(torch.full_like(i, p), (w - 1 - i).clamp(min=0)).sum())
        at += length
    return total


def work(case):
    kv, d = case["kv"], case["d"]
    lens = _lengths(case)
    if case["op"] == "extend":
        tokens, old = sum(lens), sum(_cached(case)) if case["cached"] else 0
        return {"bytes": tokens * d * (4 * case["heads"] + 4 * kv) + old * kv * 2 * d,
                "flops": 4 * d * case["heads"] * _pairs(case, lens)}
    if case["op"] == "decode":
        w = case["window"] or (1 << 40)
        rows = sum(min(n, w // 2 if case["track"] else w) for n in lens)   # (thinned out caches: every second token)
        return {"bytes": rows * kv * (2 * d + 8 / case["page"] + (12 if case["track"] else 0))
                + case["n"] * case["heads"] * d * 4,
                "flops": 4 * d * case["heads"] * rows}
    if case["op"] == "store":
        return {"bytes": sum(lens) * kv * (6 * d + (8 if case["track"] else 0)), "flops": 2 * sum(lens) * kv * d}
    rows = sum(lens)
    moved = sum(min(max(0, n - case["budget"]), case["budget"]) / 2 for n in lens)   # about half are survivors
    return {"bytes": kv * (8 * rows + moved * 2 * (2 * d + 8)), "flops": 4 * kv * rows}


# ------------------------------------------------------------------ inputs
def _page_scales(x):
    """Scales of pages whose rows are x [pages, kv, rows, d]: the smallest power of two
    with max |x| <= 448 scale, at least 2^-64."""
    top = x.abs().amax((2, 3))
    m, e = torch.frexp(top)
    e = torch.where(top > 0, e - 9 + (m > 0.875), -64).clamp(min=-64)
    return torch.ldexp(torch.ones_like(top), e)


def _codes(x, scale):
    return (x / scale[..., None, None]).to(F8)


def _table(counts, page, gen, dev, spare=PAGE_SPARE):
    """Block table [n, width] for sequences of these many rows, over shuffled pages."""
    need = [-(-c // page) for c in counts]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen, device=dev)
    width = max(max(need), 1)
    owned = torch.arange(width, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=dev)
    table[owned] = perm[:sum(need)].to(torch.int32)
    return table, total


def _filled(total, kv, page, d, gen, dev):
    """A cache with every row filled: keys and values whose size differs from page to page."""
    size = torch.exp2(torch.randint(-2, 2, (total, kv, 1, 1), generator=gen, device=dev).float())
    k, v = (torch.randn((total, kv, page, d), generator=gen, device=dev) * size for _ in range(2))
    ks, vs = _page_scales(k), _page_scales(v)
    return dict(k=_codes(k, ks), v=_codes(v, vs), k_scale=ks, v_scale=vs, pos=None, weight=None)


def prepare(case, seed):
    dev = DEVICE
    gen = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device=dev).to(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    kv, d, page, n = case["kv"], case["d"], case["page"], case["n"]
    lens = _lengths(case)
    s = dict(op=case["op"], scale=d ** -0.5, lens=i32(lens))
    if case["op"] in ("extend", "store"):
        total = sum(lens)
        s["cu"] = i32([0] + list(torch.tensor(lens).cumsum(0).tolist()))
        s["longest"] = max(lens)
        s["k"], s["v"] = rand(total, kv, d), rand(total, kv, d)
    if case["op"] in ("extend", "decode"):
        heads = case["heads"]
        s["cap"], s["window"] = case["cap"], case["window"]
        s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, heads + 1, device=dev) / heads) if case["bias"] else None)
    if case["op"] == "extend":
        s["q"] = rand(total, heads, d)
        s["doc"] = i32(_documents(case, lens)) if case["docs"] else None
        s["visible"] = i32([min(case["visible"], length) for length in lens]) if case["visible"] else None
        s["cache"] = s["table"] = s["old"] = None
        if case["cached"]:
            old = _cached(case)
            s["table"], pages = _table(old, page, gen, dev)
            s["cache"], s["old"] = _filled(pages, kv, page, d, gen, dev), i32(old)
    elif case["op"] == "decode":
        s["q"] = rand(n, heads, d)
        s["table"], pages = _table(lens, page, gen, dev)
        s["cache"] = _filled(pages, kv, page, d, gen, dev)
        s["q_pos"] = None
        if case["track"]:                       # a cache that evictions have thinned out: about every second token left
            gaps = torch.randint(1, 4, (n, kv, s["table"].shape[1] * page), generator=gen, device=dev)
            pos = (gaps.cumsum(2) - 1).to(torch.int32)
            s["cache"]["pos"] = torch.zeros((pages, kv, page), dtype=torch.int32, device=dev)
            s["cache"]["weight"] = torch.rand((pages, kv, page), generator=gen, device=dev)
            own_pages = s["table"] >= 0
            s["cache"]["pos"][s["table"][own_pages].long()] = pos.unflatten(2, (-1, page)).transpose(1, 2)[own_pages]
            s["q_pos"] = i32([2 * length for length in lens])
    elif case["op"] == "store":
        old = _cached(case) if case["cached"] else [0] * n
        s["table"], pages = _table([a + b for a, b in zip(old, lens)], page, gen, dev)
        s["cache"], s["old"] = _filled(pages, kv, page, d, gen, dev), i32(old)
        if case["track"]:
            s["cache"]["pos"] = torch.zeros((pages, kv, page), dtype=torch.int32, device=dev)
            s["cache"]["weight"] = torch.rand((pages, kv, page), generator=gen, device=dev)
    else:
        s["table"], pages = _table(lens, page, gen, dev)
        s["cache"] = _filled(pages, kv, page, d, gen, dev)
        s["cache"]["pos"] = torch.zeros((pages, kv, page), dtype=torch.int32, device=dev)
        rows = torch.arange(s["table"].shape[1] * page, device=dev).to(torch.int32)
        own_pages = s["table"] >= 0
        s["cache"]["pos"][s["table"][own_pages].long()] = (
            rows.view(1, -1, 1, page).expand(n, -1, kv, page)[own_pages])
        # accumulated weights fall off like 1 / rank, in eighths so that some are equal
        w = torch.rand((pages, kv, page), generator=gen, device=dev)
        s["weight0"] = ((1.0 / (w + 1e-3)) * 8).round() / 8
        s["pos0"] = s["cache"]["pos"].clone()
        s["cache"]["weight"] = s["weight0"].clone()
        s["budget"], s["recent"] = case["budget"], case["recent"]
    return s


# ------------------------------------------------------------------ plain forms
def _rows(table, kv_len, page):
    """For [n, rows] of a block table: page, row in it, and whether the row is held."""
    r = torch.arange(table.shape[1] * page, device=table.device)
    held = r[None] < kv_len[:, None]
    pages = table.long().repeat_interleave(page, 1).clamp(min=0)
    return pages, (r % page)[None].expand_as(pages), held


def _dequantised(codes, scale, table, page):
    """The cached rows of each sequence, [n, kv, rows, d] in 32 bits."""
    t = table.long().clamp(min=0)
    x = codes[t].float() * scale[t][..., None, None]            # [n, pages, kv, page, d]
    return x.transpose(1, 2).flatten(2, 3)


def _paged(x, table):
    return x[table.long().clamp(min=0)].transpose(1, 2).flatten(2, 3)   # [n, kv, rows]


def _softmax_rows(scores, hidden):
    """In place: exp(scores - max) with 0 where hidden, and the rows' sums."""
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    return scores.sum(-1, keepdim=True)


def _scores(q, k, s, dist):
    """q [n, kv, g, rows, d], k [n, kv, keys, d] -> capped and biased scores; dist
    broadcasts to [n, kv, 1, rows, keys]."""
    n, kv, g, rows, d = q.shape
    x = torch.matmul(q.reshape(n, kv, g * rows, d), k.transpose(2, 3).contiguous()).mul_(s["scale"])
    x = x.view(n, kv, g, rows, -1)
    if s["cap"]:
        x.div_(s["cap"]).tanh_().mul_(s["cap"])
    if s["slopes"] is not None:
        x.addcmul_(s["slopes"].view(1, kv, g, 1, 1), dist.abs().float(), value=-1.0)
    return x


def _extend(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"].long()
    (total, heads, d), kv, dev = q.shape, k.shape[1], q.device
    n, longest = cu.numel() - 1, s["longest"]
    i = torch.arange(longest, device=dev)
    live = i[None] < s["lens"][:, None]                          # [n, longest]
    at = (cu[:-1, None] + i[None]).clamp(max=total - 1)
    group = lambda x, h: x[at].float().transpose(1, 2)  # noqa: E731   [n, h, longest, d]
    qs = group(q, heads).unflatten(1, (kv, heads // kv))
    start = s["old"].long() if s["old"] is not None else torch.zeros(n, dtype=torch.long, device=dev)
    seen = i[None, :] <= i[:, None]
    if s["visible"] is not None:
        seen = seen[None] | (i[None, None] < s["visible"][:, None, None])
    seen = seen & live[:, None]                                  # [n, rows, keys]
    if s["doc"] is not None:
        doc = s["doc"][at]
        seen = seen & (doc[:, :, None] == doc[:, None]) & (doc >= 0)[:, :, None]
    dist = (i[:, None] - i[None]).expand(n, -1, -1)
    ks, vs = group(k, kv), group(v, kv)
    if s["cache"] is not None:                                   # the cached rows stand in front
        c, page = s["cache"], s["cache"]["k"].shape[2]
        _, _, held = _rows(s["table"], s["old"], page)
        ks = torch.cat([_dequantised(c["k"], c["k_scale"], s["table"], page), ks], 2)
        vs = torch.cat([_dequantised(c["v"], c["v_scale"], s["table"], page), vs], 2)
        p = torch.arange(held.shape[1], device=dev)
        dist = torch.cat([(start[:, None, None] + i[None, :, None]) - p[None, None], dist], 2)
        seen = torch.cat([held[:, None].expand(-1, longest, -1), seen], 2)
    if s["window"]:
        seen = seen & (dist.abs() < s["window"])
    x = _scores(qs, ks, s, dist[:, None, None])
    total_w = _softmax_rows(x, ~seen[:, None, None])
    o = torch.matmul(x.flatten(2, 3), vs).view(*x.shape[:4], d)
    o.div_(torch.where(total_w > 0, total_w, torch.ones_like(total_w)))
    return o.flatten(1, 2).transpose(1, 2)[live].to(torch.bfloat16)


def _decode(s):
    q, c, table = s["q"].float(), s["cache"], s["table"]
    n, heads, d = q.shape
    kv, page = c["k"].shape[1], c["k"].shape[2]
    pages, rows, held = _rows(table, s["lens"], page)
    ks, vs = (_dequantised(c[a], c[a + "_scale"], table, page) for a in ("k", "v"))
    r = torch.arange(pages.shape[1], device=q.device).expand(n, kv, -1)
    pos = _paged(c["pos"], table).long() if c["pos"] is not None else r
    q_pos = s["q_pos"].long() if s["q_pos"] is not None else s["lens"].long() - 1
    dist = q_pos[:, None, None] - pos                            # [n, kv, rows]
    seen = held[:, None].expand(n, kv, -1)
    if s["window"]:
        seen = seen & (dist.abs() < s["window"])
    x = _scores(q.view(n, kv, heads // kv, 1, d), ks, s, dist[:, :, None, None])
    total = _softmax_rows(x, ~seen[:, :, None, None])
    x.div_(torch.where(total > 0, total, torch.ones_like(total)))
    o = torch.matmul(x.flatten(2, 3), vs).reshape(n, heads, d).to(torch.bfloat16)
    if c["weight"] is None:
        return {"out": o}
    w = x.sum((2, 3)).transpose(1, 2)                            # [n, rows, kv]
    c["weight"].transpose(1, 2).index_put_((pages[held], rows[held]), w[held], accumulate=True)
    return {"out": o, "weight": c["weight"]}


def _store(s):
    c, table, cu, old = s["cache"], s["table"].long(), s["cu"].long(), s["old"].long()
    page, width, dev = c["k"].shape[2], table.shape[1], table.device
    n, kv, d = table.shape[0], c["k"].shape[1], c["k"].shape[3]
    r = torch.arange(width * page, device=dev)[None]
    new = (r >= old[:, None]) & (r < (old + s["lens"])[:, None])               # [n, rows]
    kept = (r < old[:, None]).unflatten(1, (width, page))
    touched = new.unflatten(1, (width, page)).any(2)                           # [n, width]
    src = (cu[:-1, None] + r - old[:, None]).clamp(0, s["k"].shape[0] - 1)
    src, fresh, kept = (x.unflatten(1, (width, page))[touched] for x in (src, new, kept.flatten(1)))
    ids = table[touched]
    for name in ("k", "v"):
        x = s[name][src].float().transpose(1, 2) * fresh[:, None, :, None]     # [pages, kv, page, d]
        need, was = _page_scales(x), c[name + "_scale"][ids]
        scale = torch.where(kept.any(1)[:, None], torch.maximum(was, need), need)
        held = c[name].view(torch.uint8)[ids]
        again = _codes(held.view(F8).float() * was[..., None, None], scale).view(torch.uint8)
        codes = torch.where(kept[:, None, :, None], again, held)
        codes = torch.where(fresh[:, None, :, None], _codes(x, scale).view(torch.uint8), codes)
        c[name].view(torch.uint8)[ids] = codes
        c[name + "_scale"][ids] = scale
    if c["pos"] is not None:
        at = r.unflatten(1, (width, page)).expand(n, -1, -1)[touched][:, None].expand(-1, kv, -1)
        c["pos"][ids] = torch.where(fresh[:, None], at.to(torch.int32), c["pos"][ids])
        c["weight"][ids] = c["weight"][ids] * ~fresh[:, None]
    return {k: x for k, x in c.items() if x is not None}


def _evict(s):
    c, table, page = s["cache"], s["table"], s["cache"]["k"].shape[2]
    n, kv, budget, dev = table.shape[0], c["k"].shape[1], s["budget"], table.device
    _, _, held = _rows(table, s["lens"], page)
    rows = held.shape[1]
    w, pos = _paged(c["weight"], table), _paged(c["pos"], table).long()       # [n, kv, rows]
    held = held[:, None].expand_as(w)
    last = pos.masked_fill(~held, -1).amax(2, keepdim=True)
    key = torch.where(pos > last - s["recent"], math.inf, w.double()).masked_fill(~held, -math.inf)
    order = key.sort(dim=2, descending=True, stable=True).indices[:, :, :budget]
    keep = torch.zeros_like(held).scatter_(2, order, True) & held
    r = torch.arange(rows, device=dev).expand_as(w)
    hole = ~keep & (r < budget) & held
    mover = keep & (r >= budget)
    first = lambda m: torch.where(m, r, r + rows).sort(2).values  # noqa: E731   the marked rows first, in order
    count = mover.sum(2, keepdim=True)
    live = r < count
    dst, src = first(hole).clamp(max=rows - 1)[live], first(mover).clamp(max=rows - 1)[live]
    seq, head = (torch.arange(m, device=dev).view(*v).expand_as(r)[live] for m, v in ((n, (n, 1, 1)), (kv, (1, kv, 1))))
    t = table.long().clamp(min=0)
    to, of = t[seq, dst // page], t[seq, src // page]
    dst, src = dst % page, src % page
    alive = torch.zeros((c["k"].shape[0], page), dtype=torch.bool, device=dev)   # rows before `budget`
    alive[table[table >= 0].long()] = (r[0, 0] < budget).expand(n, rows).unflatten(1, (-1, page))[table >= 0]
    again = torch.unique(to * kv + head)                                       # (page, kv head)s that receive rows
    for name in ("k", "v"):
        scale, codes = c[name + "_scale"], c[name].view(torch.uint8)
        grown = scale.view(-1).scatter_reduce(0, to * kv + head, scale[of, head], "amax").view_as(scale)
        moved = codes[of, head, src].view(F8).float() * (scale[of, head] / grown[to, head])[:, None]
        flat = codes.view(-1, page, codes.shape[3])
        rounded = (flat[again].view(F8).float() * (scale.view(-1)[again] / grown.view(-1)[again])[:, None, None]).to(F8)
        flat[again] = torch.where(alive[again // kv][..., None], rounded.view(torch.uint8), flat[again])
        codes[to, head, dst] = moved.to(F8).view(torch.uint8)
        scale.copy_(grown)
    for name in ("pos", "weight"):
        c[name][to, head, dst] = c[name][of, head, src]
    return {**c, "new_len": s["lens"].clamp(max=budget)}


# ------------------------------------------------------------------ the package's calls
def _own_calls(s):
    import hybrid_model_linear_amd as gdn
    c = gdn.KVCache(**s["cache"]) if s.get("cache") is not None else None
    if s["op"] == "extend":
        return gdn.attn_extend(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"], softcap=s["cap"], slopes=s["slopes"],
                               window=s["window"], doc=s["doc"], visible=s["visible"], cache=c, block_table=s["table"],
                               cache_len=s["old"])
    if s["op"] == "decode":
        o = gdn.attn_decode(s["q"], c, s["table"], s["lens"], scale=s["scale"], softcap=s["cap"], slopes=s["slopes"],
                            window=s["window"], q_pos=s["q_pos"], accumulate=c.weight is not None)
        return {"out": o} if c.weight is None else {"out": o, "weight": c.weight}
    if s["op"] == "store":
        gdn.kv_store(s["k"], s["v"], s["cu"], c, s["table"], s["old"])
        return {k: x for k, x in s["cache"].items() if x is not None}
    new_len = gdn.kv_evict(c, s["table"], s["lens"], s["budget"], recent=s["recent"])
    return {**s["cache"], "new_len": new_len}


def run(state):
    if state["op"] == "evict":      # the weights that the decode steps since the last eviction have left
        state["cache"]["weight"].copy_(state["weight0"])
        state["cache"]["pos"].copy_(state["pos0"])
    if own:
        return _own_calls(state)
    return {"extend": _extend, "decode": _decode, "store": _store, "evict": _evict}[state["op"]](state)


# ------------------------------------------------------------------ exact values
def _round_e4m3(x):
    """x (64 bits, |x| <= 448) to the nearest e4m3 value, ties to even, from the format:
    three fraction bits, smallest normal exponent -6."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -300))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _need(top):
    """The smallest power of two s, at least 2^-64, with top <= 448 s."""
    e = math.ceil(math.log2(top / 448.0)) if top > 0 else -64
    while top > 448.0 * 2.0 ** e:
        e += 1
    while top <= 448.0 * 2.0 ** (e - 1) and e > -64:
        e -= 1
    return 2.0 ** max(e, -64)


def _exact_rows(c, table, length, head):
    """A sequence's cached rows of one head in 64 bits: k, v [rows, d]."""
    page = c["k"].shape[2]
    ids = table[: -(-length // page)].long()
    return [(c[a][ids, head].double() * c[a + "_scale"][ids, head].double()[:, None, None]).flatten(0, 1)[:length]
            for a in ("k", "v")]


def _exact_attention(q, k, v, seen, dist, s, slopes):
    """q [rows, d], k, v [keys, d] in 64 bits; seen, dist [rows, keys]."""
    x = s["scale"] * (q @ k.T)
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    if slopes is not None:
        x = x - float(slopes) * dist.abs()
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    top = x.max(1, keepdim=True).values
    p = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    z = p.sum(1, keepdim=True)
    p = p / torch.where(z > 0, z, torch.ones_like(z))
    return p @ v, p


def exact(case, seed):
    s = prepare(case, seed)
    kv, dev = case["kv"], s["lens"].device
    lens = s["lens"].tolist()
    if case["op"] == "extend":
        g, out = case["heads"] // kv, torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        cu = s["cu"].tolist()
        for n, length in enumerate(lens):
            a, b = cu[n], cu[n + 1]
            p = int(s["old"][n]) if s["old"] is not None else 0
            i, j = torch.arange(length, device=dev)[:, None] + p, torch.arange(p + length, device=dev)[None]
            seen = j <= i
            if s["visible"] is not None:
                seen = seen | (j < int(s["visible"][n]) + p)
            if s["doc"] is not None:
                doc = s["doc"][a:b]
                seen = seen & (doc[:, None] == doc[None]) & (doc[:, None] >= 0)
            if s["window"]:
                seen = seen & ((i - j).abs() < s["window"])
            for h in range(kv):
                k, v = s["k"][a:b, h].double(), s["v"][a:b, h].double()
                if p:
                    ko, vo = _exact_rows(s["cache"], s["table"][n], p, h)
                    k, v = torch.cat([ko, k]), torch.cat([vo, v])
                for x in range(h * g, h * g + g):
                    out[a:b, x] = _exact_attention(s["q"][a:b, x].double(), k, v, seen, i - j, s,
                                                   s["slopes"][x] if s["slopes"] is not None else None)[0]
        return out
    c = s["cache"]
    page = c["k"].shape[2]
    if case["op"] == "decode":
        g, out = case["heads"] // kv, torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        weight = c["weight"].double() if c["weight"] is not None else None
        for n, length in enumerate(lens):
            r = torch.arange(length, device=dev)
            ids = s["table"][n].long()[r // page]
            for h in range(kv):
                k, v = _exact_rows(c, s["table"][n], length, h)
                pos = c["pos"][ids, h, r % page].long() if c["pos"] is not None else r
                dist = ((int(s["q_pos"][n]) if s["q_pos"] is not None else length - 1) - pos).expand(g, -1)
                seen = dist.abs() < s["window"] if s["window"] else torch.ones_like(dist, dtype=torch.bool)
                x = slice(h * g, h * g + g)
                q = s["q"][n, x].double()
                t = dict(s, slopes=None)
                if s["slopes"] is None:
                    o, p = _exact_attention(q, k, v, seen, dist, t, None)
                else:
                    both = [_exact_attention(q[i:i + 1], k, v, seen[:1], dist[:1], t, s["slopes"][h * g + i]) for i in range(g)]
                    o, p = torch.cat([b[0] for b in both]), torch.cat([b[1] for b in both])
                out[n, x] = o
                if weight is not None:
                    weight[ids, h, r % page] += p.sum(0)
        return {"out": out} if weight is None else {"out": out, "weight": weight}
    if case["op"] == "store":
        if sum(-(-(n + page) // page) for n in lens) * kv > 6000:
            return None
        got = {k: x.double() for k, x in c.items() if x is not None}
        cu, old, table = s["cu"].tolist(), s["old"].tolist(), s["table"].tolist()
        for n, length in enumerate(lens):
            for p in range(old[n] // page, (old[n] + length - 1) // page + 1):
                lo, hi = max(old[n], p * page), min(old[n] + length, (p + 1) * page)
                a, b, at = lo - p * page, hi - p * page, table[n][p]
                rows = slice(cu[n] + lo - old[n], cu[n] + hi - old[n])
                for name in ("k", "v"):
                    x = s[name][rows].double().transpose(0, 1)                  # [kv, rows, d]
                    tops = x.abs().amax((1, 2)).tolist()
                    for h in range(kv):
                        need, was = _need(tops[h]), float(c[name + "_scale"][at, h])
                        scale = max(need, was) if a else need
                        if a and scale > was:
                            got[name][at, h, :a] = _round_e4m3(got[name][at, h, :a] * (was / scale))
                        got[name][at, h, a:b] = _round_e4m3(x[h] / scale)
                        got[name + "_scale"][at, h] = scale
                if "weight" in got:
                    got["weight"][at, :, a:b] = 0.0
                    got["pos"][at, :, a:b] = torch.arange(lo, hi, device=dev).double()
        return {**got, **({"pos": None} if "pos" in got else {})}
    return _exact_evict(case, s, lens)


def _exact_evict(case, s, lens):
    c, kv, page, budget = s["cache"], case["kv"], s["cache"]["k"].shape[2], case["budget"]
    dev = s["lens"].device
    got = {k: x.double() for k, x in c.items()}
    old_scale = {k: got[k].clone() for k in ("k_scale", "v_scale")}
    for n, length in enumerate(lens):
        if length <= budget:
            continue
        r = torch.arange(length, device=dev)
        table = s["table"][n].long()
        ids = table[r // page]
        for h in range(kv):
            w, pos = c["weight"][ids, h, r % page].double(), c["pos"][ids, h, r % page].long()
            newest = pos > pos.max() - case["recent"]
            rank = torch.argsort(-w, stable=True)                   # by weight, ties to the lowest row,
            rank = rank[torch.argsort((~newest[rank]).to(torch.int8), stable=True)]   # behind the newest
            keep = torch.zeros(length, dtype=torch.bool, device=dev)
            keep[rank[:budget]] = True
            dst, src = torch.nonzero(~keep[:budget])[:, 0], torch.nonzero(keep[budget:])[:, 0] + budget
            if not len(dst):
                continue
            to, of = ids[dst], ids[src]
            for name in ("k", "v"):
                sc = got[name + "_scale"]
                new = sc[:, h].scatter_reduce(0, to, old_scale[name + "_scale"][of, h], "amax")
                moved = _round_e4m3(c[name][of, h, src % page].double() * (sc[of, h] / new[to])[:, None])
                for p in range(-(-budget // page)):
                    at, rows = int(table[p]), min(page, budget - p * page)
                    if new[at] != sc[at, h]:
                        got[name][at, h, :rows] = _round_e4m3(got[name][at, h, :rows] * (sc[at, h] / new[at]))
                got[name][to, h, dst % page] = moved
                sc[:, h] = new
            got["weight"][to, h, dst % page] = w[src]
    got["pos"] = None
    return {**got, "new_len": None}
