"""What a hybrid model's serving step runs beside its linear and softmax attention.

  selective_scan     state space scan with a decay matrix, packed prompts -> gdn_selective_scan
  selective_update   the same, one token per row                          -> gdn_selective_update
  rms_norm           norm with residual, gate and an output in 8 bits     -> gdn_rms_norm
  page_pool          allocate a stack of free pages                       -> PagePool
  plan_pages         a step's lengths, block tables and slot maps         -> gdn_plan_pages
  release_pages      pages back on the stack                              -> gdn_release_pages

As in the rest of the binding the operators run in the library's HIP kernels; this module
checks tensors, allocates what the caller did not supply and passes pointers.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib
from ._lib import GDN_BF16, GDN_E4M3, GDN_F32, GDN_SELECTIVE_UNCUT
from .attention import _at, _attach, _need, _place, _run, _table, _vec

_BF16, _F32, _I32, _I64, _F8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn
_CODES = {_BF16: GDN_BF16, _F32: GDN_F32}
_MOST = 2 ** 31 - 1          # (ctypes cuts larger numbers silently)
_MOST_F32 = torch.finfo(_F32).max
_OUT_CODES = {_BF16: GDN_BF16, _F32: GDN_F32, _F8: GDN_E4M3}


# ------------------------------------------------------------------ helpers
def _code(t, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    return code


def _matrix(t, name: str, shape, dtype) -> int:
    """Row stride of a matrix of this shape and type with unit column stride."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {tuple(t.shape)}")
    row, col = t.stride()
    if col != 1 and shape[1] > 1 and shape[0] > 0:
        raise ValueError(f"{name} must have unit column stride (strides {t.stride()})")
    return row if shape[0] > 1 else shape[1]


def _grouped(t, name: str, n: int, states: int, dtype) -> tuple[int, int]:
    """(token stride, groups) of B or C: [n, G, states] with contiguous groups, or [n, states]."""
    if t.dim() == 2:
        return _matrix(t, name, (n, states), dtype), 1
    if t.dtype is not dtype or t.dim() != 3 or t.shape[0] != n or t.shape[2] != states:
        raise ValueError(f"{name} must be {dtype} [{n}, G, {states}] or [{n}, {states}], got {t.dtype} {tuple(t.shape)}")
    g = t.shape[1]
    row, group, col = t.stride()
    if n > 0 and ((states > 1 and col != 1) or (g > 1 and group != states)):
        raise ValueError(f"{name} must have contiguous groups (strides {t.stride()})")
    return row if n > 1 else g * states, g


# ------------------------------------------------------------------ selective scan
def _selective_args(x, dt, A, B, C, cu_seqlens, slot, pool, D, z, dt_bias, dt_softplus, has_init, out, out_dtype,
                    max_seqlen, keep_pool):
    if x.dim() != 2 or A.dim() != 2:
        raise ValueError(f"x must be [T, D] and A [D, states], got {tuple(x.shape)} and {tuple(A.shape)}")
    shape = x.shape
    T, width = shape
    states, N = A.shape[1], slot.shape[0]
    i = _place(x, dt, A, B, C, cu_seqlens, slot, pool, D, z, dt_bias, has_init, out)
    kind = x.dtype
    code = _code(x, "x")
    if A.dtype is not _F32 or A.shape != (width, states) or not A.is_contiguous():
        raise ValueError(f"A must be contiguous fp32 [{width}, states], got {A.dtype} {tuple(A.shape)}")
    if pool.dtype is not _F32 or pool.dim() != 3 or pool.shape[1:] != (width, states) or not pool.is_contiguous():
        raise ValueError(f"pool must be contiguous fp32 [num_slots, {width}, {states}], got {pool.dtype} {tuple(pool.shape)}")
    bs, G = _grouped(B, "B", T, states, kind)
    cs, G2 = _grouped(C, "C", T, states, kind)
    if G != G2:
        raise ValueError(f"B and C must have the same groups, got {G} and {G2}")
    if out is None:   # (a query of the workspace reads no buffer: an aligned stand-in for the output)
        o, os, oc = 256, width, _CODES.get(out_dtype, -1)
    else:
        o, os, oc = out.data_ptr(), _matrix(out, "out", shape, out.dtype), _code(out, "out")
    return _lib.SelectiveArgs(
        code, oc, N, G, T, width, states, 1 if dt_softplus else 0, x.data_ptr(), _matrix(x, "x", shape, kind),
        dt.data_ptr(), _matrix(dt, "dt", shape, kind), B.data_ptr(), bs, C.data_ptr(), cs, _at(z),
        0 if z is None else _matrix(z, "z", shape, kind), A.data_ptr(), _vec(D, "D", width, _F32),
        _vec(dt_bias, "dt_bias", width, _F32), _vec(cu_seqlens, "cu_seqlens", N + 1), _vec(slot, "slot", N),
        _vec(has_init, "has_init", N), pool.data_ptr(), pool.shape[0], o, os, min(max_seqlen, _MOST), 1 if keep_pool else 0, None, 0), i


def _new_out(x, out_dtype):
    if x.is_contiguous():
        return torch.empty_like(x) if out_dtype is None else torch.empty_like(x, dtype=out_dtype)
    return x.new_empty(x.shape, dtype=x.dtype if out_dtype is None else out_dtype)


def selective_scan(x, dt, A, B, C, cu_seqlens, slot, pool, *, D=None, z=None, dt_bias=None, dt_softplus: bool = True,
                   has_init=None, out=None, out_dtype=None, max_seqlen: int = 0, keep_pool: bool = False,
                   workspace: torch.Tensor | None = None):
    """Selective state space scan of packed sequences over a pool of states.  Per channel c
    with states h, delta = softplus(dt + dt_bias) (dt + dt_bias without dt_softplus):
        h = exp(delta A[c]) h + delta x B,  y = C.h + D[c] x,  out = y z sigmoid(z) (y without z)
    x, dt, z [T, D] and B, C [T, G, states] (or [T, states]) bf16 or fp32, one type, rows may
    be strided; channel c reads group c // (D / G).  A fp32 [D, states] (states 8, 16, 32, 64
    or 128), D, dt_bias fp32 [D].  cu_seqlens int32 [N+1], slot int32 [N] (negative skips),
    has_init int32 [N] or None (= all 1), pool fp32 [num_slots, D, states] as in extend
    (updated in place unless keep_pool).
    max_seqlen: host hint of the longest sequence (speed only).  workspace: uint8 device
    tensor of selective_scan_workspace_size bytes (else one is allocated where long sequences
    are cut into segments).
    Returns out [T, D] in x's dtype or out_dtype (bf16, fp32)."""
    lib = _lib.load()
    if out is None:
        out = _new_out(x, out_dtype)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
    args, i = _selective_args(x, dt, A, B, C, cu_seqlens, slot, pool, D, z, dt_bias, dt_softplus, has_init, out, None,
                              max_seqlen, keep_pool)
    # (calls that are too short to be cut feel the query)
    ws = None
    if workspace is not None or args.T > GDN_SELECTIVE_UNCUT:
        ws = _attach("gdn_selective_scan", lib.gdn_selective_scan_workspace_size, args, i, workspace)
    _run("gdn_selective_scan", lib.gdn_selective_scan, args, i)
    del ws
    return out


def selective_scan_workspace_size(x, dt, A, B, C, cu_seqlens, slot, pool, *, D=None, z=None, dt_bias=None,
                                  dt_softplus: bool = True, has_init=None, out_dtype=None, max_seqlen: int = 0,
                                  keep_pool: bool = False) -> int:
    """Bytes of workspace with which selective_scan cuts sequences of these arguments (0: it
    does not)."""
    lib = _lib.load()
    args, i = _selective_args(x, dt, A, B, C, cu_seqlens, slot, pool, D, z, dt_bias, dt_softplus, has_init, None,
                              x.dtype if out_dtype is None else out_dtype, max_seqlen, keep_pool)
    # (apart from the inputs, and aligned whatever they are)
    args.out = (max(args.x or 0, args.dt or 0, args.B or 0, args.C or 0, args.z or 0, args.pool or 0) + (1 << 50)) & -256
    return _need("gdn_selective_scan_workspace_size", lib.gdn_selective_scan_workspace_size, args, i)


def selective_update(x, dt, A, B, C, slot, pool, *, D=None, z=None, dt_bias=None, dt_softplus: bool = True, out=None,
                     out_dtype=None):
    """One token per row of selective_scan's recurrence: row b continues pool[slot[b]] in
    place (slot[b] < 0 marks a padding row: its output row and every slot stay untouched).
    x, dt, z [N, D], B, C [N, G, states] (or [N, states]); the rest as in selective_scan."""
    lib = _lib.load()
    if out is None:
        out = _new_out(x, out_dtype)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
    if x.shape[0] != slot.shape[0]:
        raise ValueError(f"one token per row: {x.shape[0]} tokens, {slot.shape[0]} slots")
    args, i = _selective_args(x, dt, A, B, C, None, slot, pool, D, z, dt_bias, dt_softplus, None, out, None, 0, False)
    _run("gdn_selective_update", lib.gdn_selective_update, args, i)
    return out


# ------------------------------------------------------------------ norm
def _token_rows(t, name: str, shape, dtype=None) -> int:
    """Token stride of a tensor of this shape whose rows are contiguous."""
    if t.shape != shape or (dtype is not None and t.dtype is not dtype):
        raise ValueError(f"{name} must be {dtype or 'a tensor'} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    st = t.stride()
    if shape[0] > 0 and ((shape[-1] > 1 and st[-1] != 1) or (len(shape) == 3 and shape[1] > 1 and st[1] != shape[2])):
        raise ValueError(f"{name} must have contiguous rows (strides {st})")
    if shape[0] > 1:
        return st[0]
    return shape[1] * shape[2] if len(shape) == 3 else shape[1]


def rms_norm(x, weight=None, *, eps: float = 1e-6, offset: float = 0.0, residual=None, gate=None, gate_first: bool = False,
             out=None, out_dtype=None, scale=None, group: int = 0):
    """Root-mean-square norm over the last dimension of x [T, d] or [T, H, d] (bf16 or fp32):
        y = u / sqrt(mean(u^2) + eps) * (weight + offset),  u = x
    weight [d] bf16 or fp32, or None (y without it and offset).  residual (x's shape, bf16 or
    fp32): u = x + residual, and residual becomes u, in place.  gate (like x): y times g
    sigmoid(g), or with gate_first u = x g sigmoid(g); not together with a residual.
    out_dtype bf16 or fp32 (default x's), or float8_e4m3fn: then y = code * scale, and the
    result is (codes, scale fp32 [T, groups]) with one scale for each `group` (64 or 128)
    values of a token's row, or for the whole row (0).  Rows may be strided."""
    lib = _lib.load()
    if x.dim() not in (2, 3):
        raise ValueError(f"x must be [T, d] or [T, H, d], got {tuple(x.shape)}")
    T, d = x.shape[0], x.shape[-1]
    H = x.shape[1] if x.dim() == 3 else 1
    code = _code(x, "x")
    if out is None:
        out = _new_out(x, out_dtype)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
    out_code = _OUT_CODES.get(out.dtype)
    if out_code is None:
        raise ValueError(f"out must be bf16, fp32 or float8_e4m3fn, got {out.dtype}")
    f8 = out_code == GDN_E4M3
    if group not in (0, 64, 128):
        raise ValueError(f"group must be 0, 64 or 128, got {group}")
    if f8:
        groups = -(-H * d // group) if group else 1
        if scale is None:
            scale = x.new_empty((T, groups), dtype=_F32)
        elif scale.dtype is not _F32 or scale.shape != (T, groups) or not scale.is_contiguous():
            raise ValueError(f"scale must be contiguous fp32 [{T}, {groups}], got {scale.dtype} {tuple(scale.shape)}")
    elif scale is not None:
        raise ValueError("scale goes with a float8_e4m3fn output")
    i = _place(x, weight, residual, gate, out, scale)
    if weight is not None and (weight.shape != (d,) or not weight.is_contiguous()):
        raise ValueError(f"weight must be a contiguous [{d}] vector, got {tuple(weight.shape)}")
    args = _lib.RmsNormArgs(
        code, out_code, GDN_F32 if weight is None else _code(weight, "weight"),
        GDN_F32 if residual is None else _code(residual, "residual"), T, H, d, x.data_ptr(), _token_rows(x, "x", x.shape),
        _at(gate), 0 if gate is None else _token_rows(gate, "gate", x.shape, x.dtype), _at(residual),
        0 if residual is None else _token_rows(residual, "residual", x.shape), _at(weight), out.data_ptr(),
        _token_rows(out, "out", x.shape), _at(scale), eps, offset, 1 if gate_first else 0, group)
    _run("gdn_rms_norm", lib.gdn_rms_norm, args, i)
    return (out, scale) if f8 else out


def check_gated_norm(like, H: int, d: int, gate, weight, eps: float) -> None:
    """Refuses what rms_norm would refuse of a gate [T, H d] and a weight [d] for an output [T, H, d]
    of the type and on the device of `like`."""
    width = H * d
    if _token_rows(gate, "z", (like.shape[0], width), like.dtype) < width:
        raise ValueError(f"z must have rows of {width} values apart from each other (strides {gate.stride()})")
    _code(weight, "norm_weight")
    if weight.shape != (d,) or not weight.is_contiguous():
        raise ValueError(f"norm_weight must be a contiguous [{d}] vector, got {tuple(weight.shape)}")
    if not 0.0 <= eps <= _MOST_F32:
        raise ValueError(f"norm_eps must be finite and at least 0, got {eps}")
    _place(like, gate, weight)


# ------------------------------------------------------------------ pages
class PagePool:
    """A stack of free pages in device memory, checked once: state int32 [2 + capacity] holds
    the number of free pages, a 0 that is the library's own, and their ids, the next one to be
    taken last."""
    __slots__ = ("_state", "_capacity")

    def __init__(self, state):
        if state.dtype is not _I32 or state.dim() != 1 or state.shape[0] < 2 or not state.is_contiguous():
            raise ValueError(f"state must be a contiguous int32 vector [2 + capacity], got {state.dtype} {tuple(state.shape)}")
        _place(state)
        self._state, self._capacity = state, state.shape[0] - 2

    # (fixed, since the calls use what was checked above)
    state = property(lambda self: self._state)
    capacity = property(lambda self: self._capacity)


def page_pool(num_pages: int, *, device="cuda") -> PagePool:
    """All of the pages 0 .. num_pages - 1 free, the lowest to be taken first."""
    state = torch.arange(num_pages + 1, -1, -1, dtype=_I32, device=device)   # (the ids end in num_pages - 1 .. 0)
    state[0], state[1] = num_pages, 0
    return PagePool(state)


class StepPlan(NamedTuple):
    """plan_pages' outputs: what a forward batch carries (cu_seqlens, cache_len; kv_len behind
    the step), and per token its row of the cache (page id * page + row), its position, its request."""
    cu_seqlens: torch.Tensor
    cache_len: torch.Tensor
    kv_len: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    seq: torch.Tensor


def _page(page: int) -> None:
    if not 1 <= page <= 1 << 30:
        raise ValueError(f"page must be in [1, 2^30], got {page}")


def plan_pages(pool: PagePool, block_table, held, new, page: int, tokens: int, *, start=None,
               out: StepPlan | None = None) -> StepPlan:
    """The lengths, block-table entries and slot maps of a step, formed on the GPU.  Request n
    holds held[n] rows and brings new[n] tokens (int32 [N]; negative: a padding row); it takes
    the pages it lacks from `pool`, requests in order, into its row of block_table (int32 [N,
    width], updated in place).  From the first request on for which the pages or the room for
    `tokens` tokens do not last, and where the table is too narrow, nothing is served: cache_len
    and kv_len are -1, as for padding rows.  cu_seqlens still counts the tokens of such requests
    (up to `tokens`): layers that go by slots skip them with slot = torch.where(plan.cache_len < 0, -1, slot).
    Returns StepPlan: cu_seqlens int32 [N+1]; cache_len = held, kv_len = held + new int32 [N];
    slots int64 [tokens], positions, seq int32 [tokens] (-1 for tokens of no served request).
    start int32 [N]: the first tokens' positions (default held).  out: a StepPlan to be
    written (static buffers of a graph)."""
    lib = _lib.load()
    N = held.shape[0]
    i = _place(pool._state, block_table, held, new, start)
    ts, tw = _table(block_table, N)
    _page(page)
    if not 0 <= tokens <= _MOST:
        raise ValueError(f"tokens must be in [0, 2^31), got {tokens}")
    if out is None:      # (two allocations; the tensors are parts of them)
        small = held.new_empty(3 * N + 1 + 2 * tokens).split_with_sizes((N + 1, N, N, tokens, tokens))
        out = StepPlan(small[0], small[1], small[2], held.new_empty(tokens, dtype=_I64), small[3], small[4])
        at = [t.data_ptr() for t in out]
    else:
        _place(pool._state, *out)
        at = [_vec(t, name, n, dtype) for t, name, n, dtype in zip(
            out, StepPlan._fields, (N + 1, N, N, tokens, tokens, tokens), (_I32, _I32, _I32, _I64, _I32, _I32))]
    args = _lib.PlanPagesArgs(
        pool._state.data_ptr(), pool._capacity, N, page, tokens, _vec(held, "held", N), _vec(new, "new", N),
        _vec(start, "start", N), block_table.data_ptr(), ts, tw, 0, *at)
    _run("gdn_plan_pages", lib.gdn_plan_pages, args, i)
    return out


def release_pages(pool: PagePool, block_table, keep, held, page: int) -> None:
    """Request n keeps its first keep[n] rows of held[n] (int32 [N]): the pages behind them go
    back to `pool`, requests and pages in order (keep[n] = 0: all of them; keep[n] < 0 or
    held[n] <= keep[n]: none; negative entries of the table are passed over).  block_table is
    left as it is."""
    lib = _lib.load()
    _page(page)
    N = held.shape[0]
    i = _place(pool._state, block_table, keep, held)
    ts, tw = _table(block_table, N)
    args = _lib.ReleasePagesArgs(pool._state.data_ptr(), pool._capacity, N, page, _vec(keep, "keep", N),
                                 _vec(held, "held", N), block_table.data_ptr(), ts, tw, 0)
    _run("gdn_release_pages", lib.gdn_release_pages, args, i)
