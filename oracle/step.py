"""fp64 reference of a serving step's operators beside the attention layers: the selective
scan token by token, the RMS norm, and the pages of a step request by request.  Plain
definitions, no splitting or blocking."""
import math

import numpy as np

from .attention import E4M3, e4m3_encode

U = 2.0 ** -24            # half a step of fp32, relative


def _silu(z):
    with np.errstate(over="ignore", invalid="ignore"):
        return z / (1 + np.exp(-z))


# ------------------------------------------------------------------ selective scan
def selective_scan(x, dt, A, B, C, cu, slot, pool, *, D=None, z=None, dt_bias=None, softplus=True, has_init=None):
    """x, dt, z [T, D], A [D, S], B, C [T, G, S], pool [slots, D, S].  Returns (out [T, D] with NaN
    in rows that no sequence writes, pool, bound): `bound` has the same two parts and says how
    far fp32 arithmetic may be from them, followed through the recurrence:
      delta        off by (|dt + bias| + 16) U relative: the rounded sum moves log softplus by at most
                   its own error, the functions are good to a few units;
      exp(delta A) relative: |delta A| (that + 2 U for the two products + L U for a fold over L
                   summed deltas) + 4 U (the exponential and the product with h);
      delta x B    relative: that of delta + 3 U;  the sum with it: U;
      y            (S + 3) U of the sum of its terms' magnitudes, and 32 U for the gate."""
    x, dt, A, B, C = (np.asarray(v, np.float64) for v in (x, dt, A, B, C))
    T, width = x.shape
    of = np.arange(width) // (width // B.shape[1])
    out, err = np.full((T, width), np.nan), np.zeros((T, width))
    pool = np.array(pool, np.float64)
    pool_err = np.zeros_like(pool)
    for n in range(len(slot)):
        if slot[n] < 0:
            continue
        L = cu[n + 1] - cu[n]
        h = pool[slot[n]].copy() if has_init is None or has_init[n] else np.zeros_like(pool[slot[n]])
        size, e = np.abs(h), np.zeros_like(h)
        for t in range(cu[n], cu[n + 1]):
            v = dt[t] + (0 if dt_bias is None else dt_bias)
            delta = np.logaddexp(v, 0) if softplus else v
            rd = (np.abs(v) + 16) * U
            a = np.exp(delta[:, None] * A)
            new = (delta * x[t])[:, None] * B[t][of]
            r = np.abs(delta[:, None] * A) * (rd[:, None] + (2 + L) * U) + 4 * U
            h = a * h + new
            e = a * (e + size * r) + np.abs(new) * (rd[:, None] + 3 * U)
            size = a * size + np.abs(new)
            e += size * U
            y, mag = (C[t][of] * h).sum(1), (np.abs(C[t][of]) * size).sum(1)
            ye = (np.abs(C[t][of]) * e).sum(1)
            if D is not None:
                y, mag = y + D * x[t], mag + np.abs(D * x[t])
            g = 1.0 if z is None else _silu(np.asarray(z[t], np.float64))
            out[t], err[t] = y * g, (ye + mag * (A.shape[1] + 3) * U) * np.abs(g) + 32 * U * np.abs(y * g)
        pool[slot[n]], pool_err[slot[n]] = h, e
    return out, pool, (err, pool_err)


def selective_update(x, dt, A, B, C, slot, pool, **kw):
    n = len(slot)
    return selective_scan(x, dt, A, B, C, np.arange(n + 1), slot, pool, **kw)


# ------------------------------------------------------------------ norm
def rms_norm(x, weight=None, *, eps=1e-6, offset=0.0, residual=None, gate=None, gate_first=False):
    """x [T, H, d]; returns (y, u): the normalised rows, and x + residual."""
    u = np.asarray(x, np.float64)
    if residual is not None:
        u = u + np.asarray(residual, np.float64)
    kept = u
    if gate is not None and gate_first:
        u = u * _silu(np.asarray(gate, np.float64))
    y = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * (np.asarray(weight, np.float64) + offset)
    if gate is not None and not gate_first:
        y = y * _silu(np.asarray(gate, np.float64))
    return y, kept


def group_scales(y, group):
    """y [T, W] -> scales [T, groups]: max of the finite |y| / 448, at least 2^-64."""
    W = y.shape[1]
    a = np.where(np.isfinite(y), np.abs(y), 0)
    step = group or W
    return np.stack([np.maximum(a[:, k:k + step].max(1) / 448, 2.0 ** -64) for k in range(0, W, step)], 1)


def e4m3_codes(y, scale, group):
    step = group or y.shape[1]
    with np.errstate(invalid="ignore"):
        return e4m3_encode(y / scale[:, np.arange(y.shape[1]) // step])


# ------------------------------------------------------------------ pages
def plan_pages(stack, capacity, table, held, new, page, T, start=None):
    """stack: list of free page ids, the top last.  Returns (stack, table, cu_seqlens, cache_len,
    kv_len, slots, positions, seq)."""
    stack, table = list(stack), np.array(table)
    N, width = table.shape
    cu, cache_len, kv_len = [0], [-1] * N, [-1] * N
    slots, positions, seq = [-1] * T, [-1] * T, [-1] * T
    tokens, full = 0, False
    for n in range(N):
        h, m = int(held[n]), int(new[n])
        if h < 0 or m < 0:
            cu.append(min(tokens, T))
            continue
        lo, hi = math.ceil(h / page), math.ceil((h + m) / page)
        fits = hi <= width and h + m < 2 ** 31
        full = full or tokens + m > T or (fits and hi - lo > len(stack))
        if fits and not full:
            for p in range(lo, hi):
                table[n, p] = stack.pop()
            cache_len[n], kv_len[n] = h, h + m
            for i in range(m):
                p = int(table[n, (h + i) // page])
                slots[tokens + i] = p * page + (h + i) % page if p >= 0 else -1
                positions[tokens + i] = (h if start is None else int(start[n])) + i
                seq[tokens + i] = n
        tokens += m
        cu.append(min(tokens, T))
    return stack, table, cu, cache_len, kv_len, slots, positions, seq


def release_pages(stack, capacity, table, keep, held, page):
    stack = list(stack)
    for n in range(len(held)):
        if keep[n] >= 0 and held[n] > keep[n]:
            for p in range(math.ceil(keep[n] / page), min(math.ceil(held[n] / page), table.shape[1])):
                if table[n, p] >= 0 and len(stack) < capacity:
                    stack.append(int(table[n, p]))
    return stack


__all__ = ["E4M3", "selective_scan", "selective_update", "rms_norm", "group_scales", "e4m3_codes", "plan_pages",
           "release_pages"]
