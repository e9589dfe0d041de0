"""fp64 reference of the softmax-attention operators over a paged 8-bit cache: plain
definitions, one row at a time where that matters, no tiling, splitting or blocking.

A cache is a dict of numpy arrays: k, v uint8 codes [pages, H_kv, page, d] (OCP e4m3),
k_scale, v_scale float64 [pages, H_kv], pos int64 and weight float64 [pages, H_kv, page]
or None.  A block table is an int array [N, width]; a page id outside [0, pages) holds
nothing."""
import math

import numpy as np


# ------------------------------------------------------------------ e4m3
def _e4m3_table():
    """Value of every code: sign, 4 exponent bits (bias 7), 3 fraction bits; exponent 0
    is subnormal, 0x7f / 0xff are NaN, and there are no infinities."""
    out = np.empty(256)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        out[c] = math.nan if c & 0x7f == 0x7f else (-x if c & 0x80 else x)
    return out


E4M3 = _e4m3_table()
_POS = E4M3[:0x7f]                   # the non-negative values, ascending


def e4m3_encode(x):
    """Codes of the nearest e4m3 values (ties to the even code); NaN for NaN, infinities
    and anything that rounds past 448."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_POS, a), 1, 0x7e)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        up = a - _POS[lo], _POS[hi] - a
        code = np.where(up[0] < up[1], lo, np.where(up[0] > up[1], hi, np.where(lo % 2 == 0, lo, hi)))
        code = np.where(~np.isfinite(a) | (a > 464), 0x7f, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def page_scale(x):
    """Smallest power of two s >= 2^-64 with max |x| <= 448 s over the finite x."""
    a = np.abs(np.asarray(x, np.float64))
    a = a[np.isfinite(a)]
    top = a.max() if a.size else 0.0
    s = 2.0 ** -64
    while top > 448 * s:
        s *= 2
    return s


# ------------------------------------------------------------------ cache
def _held(cache, table_row, rows):
    """(page, row in it) of the rows, page -1 where nothing is held."""
    page, width = cache["k"].shape[2], len(table_row)
    out = []
    for r in rows:
        j = int(r) // page
        p = int(table_row[j]) if j < width else -1
        out.append((p if 0 <= p < cache["k"].shape[0] else -1, int(r) % page))
    return out


def kv_store(cache, k, v, cu, cache_len, table, start=None):
    """Returns the cache after the store; k, v [T, H_kv, d], cu None: one token each."""
    c = {a: None if b is None else b.copy() for a, b in cache.items()}
    page, H = c["k"].shape[2], c["k"].shape[1]
    for n, old in enumerate(int(o) for o in cache_len):
        t0, t1 = (n, n + 1) if cu is None else (int(cu[n]), int(cu[n + 1]))
        if old < 0 or t1 <= t0:
            continue
        rows = np.arange(old, old + t1 - t0)
        where = _held(c, table[n], rows)
        for j in sorted({r // page for r in rows}):
            mine = [i for i, r in enumerate(rows) if r // page == j]
            p = where[mine[0]][0]
            if p < 0:
                continue
            kept = max(0, min(page, old - j * page))              # earlier rows of the page
            for name, x in (("k", k), ("v", v)):
                for h in range(H):
                    new = np.stack([x[t0 + i, h] for i in mine]).astype(np.float64)
                    s, was = page_scale(new), c[name + "_scale"][p, h]
                    if kept:
                        s = max(s, was)
                        if s > was:
                            c[name][p, h, :kept] = e4m3_encode(E4M3[c[name][p, h, :kept]] * (was / s))
                    c[name + "_scale"][p, h] = s
                    for i, row in zip(mine, new):
                        c[name][p, h, where[i][1]] = e4m3_encode(row / s)
            for i in mine:
                if c["pos"] is not None:
                    c["pos"][p, :, where[i][1]] = (old if start is None else int(start[n])) + i
                if c["weight"] is not None:
                    c["weight"][p, :, where[i][1]] = 0.0
    return c


def cached_rows(cache, table_row, length, h):
    """k, v [rows, d], positions and validity of a sequence's first `length` rows."""
    length = min(int(length), len(table_row) * cache["k"].shape[2])
    where = _held(cache, table_row, range(length))
    d = cache["k"].shape[3]
    k, v, pos = np.zeros((length, d)), np.zeros((length, d)), np.arange(length)
    ok = np.array([p >= 0 for p, _ in where], bool)
    for i, (p, r) in enumerate(where):
        if p >= 0:
            k[i] = E4M3[cache["k"][p, h, r]] * cache["k_scale"][p, h]
            v[i] = E4M3[cache["v"][p, h, r]] * cache["v_scale"][p, h]
            if cache["pos"] is not None:
                pos[i] = cache["pos"][p, h, r]
    return k, v, pos, ok, where


# ------------------------------------------------------------------ attention
def attend(q, k, v, seen, dist, scale, softcap=0.0, slope=0.0):
    """One query over its keys: (output, weights, sum of weights * |v|).  Keys that are not
    seen take no part, whatever they hold."""
    idx = np.flatnonzero(seen)
    w = np.zeros(len(seen))
    if not len(idx):
        return np.zeros(v.shape[1]), w, np.zeros(v.shape[1])
    s = scale * (k[idx] @ q)
    if softcap > 0:
        s = softcap * np.tanh(s / softcap)
    s = s - slope * np.abs(dist[idx])
    p = np.exp(s - s.max())
    p = p / p.sum()
    w[idx] = p
    return p @ v[idx], w, p @ np.abs(v[idx])


def attn_extend(q, k, v, cu, scale, *, causal=True, softcap=0.0, slopes=None, window=0, doc=None, visible=None,
                cache=None, table=None, cache_len=None, start=None):
    """(out [T, H, d], sum p |v|): NaN rows where nothing is written."""
    T, H, d = q.shape
    G = H // k.shape[1]
    out, mag = np.full((T, H, d), math.nan), np.full((T, H, d), math.nan)
    for n in range(len(cu) - 1):
        t0, t1 = int(cu[n]), int(cu[n + 1])
        old = 0 if cache is None else int(cache_len[n])
        if old < 0:
            continue
        first = old if start is None else int(start[n])
        L = t1 - t0
        for h in range(H):
            kk, vv = k[t0:t1, h // G].astype(np.float64), v[t0:t1, h // G].astype(np.float64)
            if cache is not None:
                ck, cv, cpos, cok, _ = cached_rows(cache, table[n], old, h // G)
                kk, vv = np.concatenate([ck, kk]), np.concatenate([cv, vv])
            else:
                cpos, cok = np.zeros(0, int), np.zeros(0, bool)
            for i in range(L):
                dist = np.concatenate([first + i - cpos, i - np.arange(L)])
                j = np.arange(L)
                seen = (j <= i) | (not causal)
                if visible is not None:
                    seen |= j < int(visible[n])
                if doc is not None:
                    seen &= (doc[t0:t1] == doc[t0 + i]) & (doc[t0 + i] >= 0)
                seen = np.concatenate([cok, seen])
                if window:
                    seen = seen & (np.abs(dist) < window)
                out[t0 + i, h], _, mag[t0 + i, h] = attend(q[t0 + i, h].astype(np.float64), kk, vv, seen, dist, scale,
                                                           softcap, 0.0 if slopes is None else float(slopes[h]))
    return out, mag


def attn_decode(q, cache, table, kv_len, scale, *, softcap=0.0, slopes=None, window=0, q_pos=None):
    """(out [N, H, d], sum p |v|, the cache's weight after accumulation); NaN rows for padding."""
    N, H, d = q.shape
    G = H // cache["k"].shape[1]
    out, mag = np.full((N, H, d), math.nan), np.full((N, H, d), math.nan)
    weight = None if cache["weight"] is None else cache["weight"].copy()
    for n in range(N):
        if kv_len[n] < 0:
            continue
        at = int(kv_len[n]) - 1 if q_pos is None else int(q_pos[n])
        for h in range(H):
            k, v, pos, ok, where = cached_rows(cache, table[n], kv_len[n], h // G)
            seen = ok & (np.abs(at - pos) < window) if window else ok
            out[n, h], w, mag[n, h] = attend(q[n, h].astype(np.float64), k, v, seen, at - pos, scale, softcap,
                                             0.0 if slopes is None else float(slopes[h]))
            if weight is not None:
                for (p, r), x in zip(where, w):
                    if p >= 0:
                        weight[p, h // G, r] += x
    return out, mag, weight


# ------------------------------------------------------------------ eviction
def kv_evict(cache, table, kv_len, budget, recent=0):
    """(cache, new lengths) after the eviction."""
    c = {a: b.copy() for a, b in cache.items()}
    page = c["k"].shape[2]
    new_len = np.array([min(int(x), budget) for x in kv_len])
    for n, L in enumerate(int(x) for x in kv_len):
        L = min(L, len(table[n]) * page)
        if L <= budget:
            continue
        where = _held(cache, table[n], range(L))
        if any(p < 0 for p, _ in where):
            new_len[n] = int(kv_len[n])
            continue
        for h in range(c["k"].shape[1]):
            w = np.array([cache["weight"][p, h, r] for p, r in where])
            pos = np.array([cache["pos"][p, h, r] for p, r in where])
            newest = pos > pos.max() - recent
            # newest, then by weight, NaN last; ties to the lowest row
            rank = sorted(range(L), key=lambda i: (0, 0.0, i) if newest[i] else
                          (2, 0.0, i) if math.isnan(w[i]) else (1, -w[i], i))
            keep = set(rank[:budget])
            moves = list(zip([i for i in range(budget) if i not in keep], sorted(i for i in keep if i >= budget)))
            for name in ("k", "v"):
                s0 = cache[name + "_scale"][:, h]
                for dst, src in moves:
                    s1 = c[name + "_scale"][:, h]
                    s1[where[dst][0]] = max(s1[where[dst][0]], s0[where[src][0]])
                for i in range(budget):
                    p, r = where[i]
                    f = s0[p] / c[name + "_scale"][p, h]
                    if f != 1:
                        c[name][p, h, r] = e4m3_encode(E4M3[cache[name][p, h, r]] * f)
                for dst, src in moves:
                    (p, r), (a, b) = where[dst], where[src]
                    f = s0[a] / c[name + "_scale"][p, h]
                    x = cache[name][a, h, b]
                    c[name][p, h, r] = x if f == 1 else e4m3_encode(E4M3[x] * f)
            for dst, src in moves:
                (p, r), (a, b) = where[dst], where[src]
                c["pos"][p, h, r], c["weight"][p, h, r] = cache["pos"][a, h, b], cache["weight"][a, h, b]
    return c, new_len
