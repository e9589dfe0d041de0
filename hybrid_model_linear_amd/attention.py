"""Softmax attention of the hybrid model's full-attention layers, over a paged 8-bit cache.

  kv_cache       allocate a cache                                  -> KVCache
  kv_store       quantise new keys and values into its pages       -> gdn_kv_store
  attn_extend    packed varlen new tokens (+ a cached prefix)      -> gdn_attn_extend
  attn_decode    one token per sequence over the cache             -> gdn_attn_decode
  kv_evict       keep a budget of rows by accumulated weight       -> gdn_kv_evict
and the layer call of the pages:
  forward_attn(layer, forward_batch, q, k, v)   (pymllm RadixAttention.forward)

As in the rest of the binding the operators run in the library's HIP kernels; this module
checks tensors, allocates what the caller did not supply and passes pointers.  (forward_attn
forms a decode step's lengths, cache_len + 1, with torch.)
"""
from __future__ import annotations

import ctypes as ct

import torch

from . import _lib, _is_target_verify, _mode_kind
from ._lib import GDN_BF16

_PAGES = (16, 32, 64, 128)
_NO_CACHE = _lib.KVCacheArgs()
_BF16, _F32, _I32, _U8, _F8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn
_current_device, _raw_stream = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream


# ------------------------------------------------------------------ helpers
# (A decode step is a few microseconds of GPU work: the checks below look at each tensor
# once, and arguments go into their struct in one positional call.)
def _place(first, *ts) -> int:
    """Device index that all given tensors share."""
    i = first.get_device()
    if i < 0:
        raise ValueError("all tensors must live on the GPU")
    for t in ts:
        if t is not None and t.get_device() != i:
            raise ValueError("all tensors must live on the GPU" if t.get_device() < 0
                             else "all tensors must be on the same device")
    return i


def _at(t):
    return None if t is None else t.data_ptr()


def _vec(t, name: str, n: int, dtype=_I32):
    """Address of a contiguous vector of n elements, None for None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == (n,) and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} vector of length {n}, got {t.dtype} {tuple(t.shape)}")


def _heads(t, name: str, n: int, heads: int, d: int) -> int:
    """Token stride of a bf16 [n, heads, d] view whose heads are contiguous."""
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be bf16, got {t.dtype}")
    if t.shape != (n, heads, d):
        raise ValueError(f"{name} must be [{n}, {heads}, {d}], got {tuple(t.shape)}")
    if t.is_contiguous():
        return heads * d
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != d):
        raise ValueError(f"{name} must have contiguous heads (strides {st})")
    return st[0] if n > 1 else heads * d


def _table(t, n: int) -> tuple[int, int]:
    """(row stride, width) of a block table."""
    if t.dtype is _I32 and t.dim() == 2:
        rows, w = t.shape
        if rows == n:
            if t.is_contiguous():
                return w, w
            if w == 1 or t.stride(1) == 1:
                return (t.stride(0) if n > 1 else w), w
    raise ValueError(f"block_table must be int32 [{n}, width] with unit column stride, got "
                     f"{t.dtype} {tuple(t.shape)} / {t.stride()}")


def _like(q):
    """A contiguous output of q's shape and type."""
    return torch.empty_like(q) if q.is_contiguous() else torch.empty_like(q, memory_format=torch.contiguous_format)


def _run(name: str, fn, args, i: int) -> None:
    """The call on device i's current stream."""
    if _current_device() == i:
        st = fn(ct.byref(args), _raw_stream(i))
    else:
        with torch.cuda.device(i):
            st = fn(ct.byref(args), _raw_stream(i))
    if st:
        _lib.check(name, st)


def _need(name: str, fn, args, i: int) -> int:
    """A workspace query on device i."""
    if _current_device() == i:
        need = fn(ct.byref(args))
    else:
        with torch.cuda.device(i):
            need = fn(ct.byref(args))
    if need < 0:
        _lib.check(name, int(-need))
    return need


def _attach(name: str, fn, args, i: int, workspace):
    """Attach a call's workspace: the caller's uint8 tensor, or a fresh allocation."""
    if workspace is None:
        need = _need(name, fn, args, i)
        if need == 0:
            return None
        workspace = torch.empty(need, dtype=_U8, device=torch.device("cuda", i))
    elif workspace.dtype is not _U8 or workspace.dim() != 1 or not workspace.is_contiguous() \
            or workspace.get_device() != i:
        raise ValueError("workspace must be a contiguous uint8 vector on the call's device")
    args.workspace, args.workspace_bytes = workspace.data_ptr(), workspace.numel()
    return workspace


# ------------------------------------------------------------------ the cache
class KVCache:
    """The tensors of a paged 8-bit key/value cache (gdn_kv_cache), checked once: k, v
    float8_e4m3fn [num_pages, H_kv, page, d]; k_scale, v_scale fp32 [num_pages, H_kv], powers
    of two (a cached value is code * scale); optional pos int32 and weight fp32 [num_pages,
    H_kv, page]: the rows' positions and the softmax weights accumulated on them (an eviction
    needs both)."""
    __slots__ = ("_k", "_v", "_k_scale", "_v_scale", "_pos", "_weight", "_args", "_device")

    def __init__(self, k, v, k_scale, v_scale, pos=None, weight=None):
        shape = k.shape
        if len(shape) != 4 or k.dtype is not _F8 or not k.is_contiguous():
            raise ValueError("cache.k must be contiguous float8_e4m3fn [num_pages, H_kv, page, d]")
        pages, H_kv, page, d = shape
        if v.shape != shape or v.dtype is not _F8 or not v.is_contiguous():
            raise ValueError("cache.v must be like cache.k")
        for t, nm in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype is not _F32 or t.shape != (pages, H_kv) or not t.is_contiguous():
                raise ValueError(f"cache.{nm} must be contiguous fp32 [{pages}, {H_kv}]")
        for t, nm, dt in ((pos, "pos", _I32), (weight, "weight", _F32)):
            if t is not None and (t.dtype is not dt or t.shape != (pages, H_kv, page) or not t.is_contiguous()):
                raise ValueError(f"cache.{nm} must be contiguous {dt} [{pages}, {H_kv}, {page}]")
        self._device = _place(k, v, k_scale, v_scale, pos, weight)
        self._k, self._v, self._k_scale, self._v_scale, self._pos, self._weight = k, v, k_scale, v_scale, pos, weight
        self._args = _lib.KVCacheArgs(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _at(pos),
                                      _at(weight), pages, page, H_kv, d, 0)

    # (fixed, since the calls use the addresses taken above)
    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)
    pos = property(lambda self: self._pos)
    weight = property(lambda self: self._weight)
    page = property(lambda self: self._args.page)


def kv_cache(num_pages: int, H_kv: int, d: int, page: int = 64, *, track: bool = False,
             device="cuda") -> KVCache:
    """An empty cache of num_pages pages of `page` rows (16, 32, 64 or 128); `track` adds
    the positions and accumulated weights that kv_evict goes by."""
    if page not in _PAGES:
        raise ValueError(f"page must be one of {_PAGES}, got {page}")
    rows = (num_pages, H_kv, page)
    codes = [torch.zeros(rows + (d,), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full(rows[:2], 2.0 ** -64, dtype=torch.float32, device=device) for _ in range(2)]
    return KVCache(*codes, *scales, torch.zeros(rows, dtype=torch.int32, device=device) if track else None,
                   torch.zeros(rows, dtype=torch.float32, device=device) if track else None)


def kv_store(k, v, cu_seqlens, cache: KVCache, block_table, cache_len, *, start=None) -> None:
    """Quantise the new tokens' keys and values (k, v bf16 [T, H_kv, d]) into the cache: the
    tokens of sequence n (cu_seqlens int32 [N+1]; None: one token per sequence) become its
    rows cache_len[n], cache_len[n] + 1, ... over the pages block_table[n] (int32 [N,
    width]).  start int32 [N]: the first token's position (default cache_len), for a cache
    that keeps positions.  cache_len[n] < 0 skips the sequence."""
    lib = _lib.load()
    ca = cache._args
    T, N, H_kv, d = k.shape[0], cache_len.shape[0], ca.H_kv, ca.d
    i = _place(cache._k, k, v, cu_seqlens, block_table, cache_len, start)
    if cu_seqlens is None and T != N:
        raise ValueError(f"without cu_seqlens there is one token per sequence: {T} tokens, {N} sequences")
    ts, tw = _table(block_table, N)
    args = _lib.KVStoreArgs(ca, GDN_BF16, N, T, k.data_ptr(), _heads(k, "k", T, H_kv, d), v.data_ptr(),
                            _heads(v, "v", T, H_kv, d), _vec(cu_seqlens, "cu_seqlens", N + 1),
                            _vec(cache_len, "cache_len", N), _vec(start, "start", N), block_table.data_ptr(), ts, tw)
    _run("gdn_kv_store", lib.gdn_kv_store, args, i)


# ------------------------------------------------------------------ attention
def _extend_args(q, k, v, cu_seqlens, scale, causal, softcap, slopes, window, doc, visible, cache, block_table,
                 cache_len, start, out, max_cached=0):
    T, H, d = q.shape
    H_kv, N = k.shape[1], cu_seqlens.shape[0] - 1
    if cache is not None:
        if block_table is None or cache_len is None:
            raise ValueError("a cache needs block_table and cache_len")
        ca = cache._args
        i = _place(cache._k, q, k, v, cu_seqlens, slopes, doc, visible, block_table, cache_len, start, out)
        ts, tw = _table(block_table, N)
    else:
        if block_table is not None or cache_len is not None:
            raise ValueError("block_table and cache_len need a cache")
        ca, ts, tw = _NO_CACHE, 0, 0
        i = _place(q, k, v, cu_seqlens, slopes, doc, visible, start, out)
    # (a query of the workspace reads no buffer: an aligned stand-in for the output)
    o, os = (256, H * d) if out is None else (out.data_ptr(), _heads(out, "out", T, H, d))
    return _lib.AttnExtendArgs(
        ca, GDN_BF16, GDN_BF16, N, H, H_kv, d, T, q.data_ptr(), _heads(q, "q", T, H, d), k.data_ptr(),
        _heads(k, "k", T, H_kv, d), v.data_ptr(), _heads(v, "v", T, H_kv, d), o, os,
        _vec(cu_seqlens, "cu_seqlens", N + 1), _vec(cache_len, "cache_len", N),
        _vec(start, "start", N), _at(block_table), ts, tw, 1 if causal else 0, _vec(visible, "visible", N),
        _vec(doc, "doc", T), _vec(slopes, "slopes", H, _F32), window, d ** -0.5 if scale is None else scale,
        softcap, max_cached), i


def attn_extend(q, k, v, cu_seqlens, *, scale=None, causal: bool = True, softcap: float = 0.0, slopes=None,
                window: int = 0, doc=None, visible=None, cache: KVCache | None = None, block_table=None,
                cache_len=None, start=None, max_cached: int = 0, out=None, workspace: torch.Tensor | None = None):
    """Attention of packed new tokens over their own keys and values and, with `cache`, the
    cache_len[n] rows that each sequence holds already.  q [T, H, d], k, v [T, H_kv, d]
    bf16; cu_seqlens int32 [N+1].
    softcap: scores become softcap * tanh(score / softcap) (0: none).  slopes fp32 [H]: a
    bias of -slope * |distance|.  window: only keys closer than this (0: all).  visible
    int32 [N]: the first visible[n] tokens are seen by every token of the sequence (prefix
    mask); causal=False lets every token see every other.  doc int32 [T]: a token sees only
    tokens with its own id; a negative id sees nothing and is not seen (output 0).
    start int32 [N]: position of each first token (default: behind the cached rows).
    max_cached: host hint of the longest cache_len, else the table's width counts (speed
    only: how the keys of few rows are split).
    workspace: uint8 device tensor of attn_extend_workspace_size bytes (else one is
    allocated where the keys of few rows are split).
    Returns out [T, H, d] bf16 (rows behind the last sequence, and those of sequences with
    cache_len[n] < 0, are not written)."""
    lib = _lib.load()
    if out is None:
        out = _like(q)
    args, i = _extend_args(q, k, v, cu_seqlens, scale, causal, softcap, slopes, window, doc, visible, cache,
                           block_table, cache_len, start, out, max_cached)
    # (fewer than 512 keys are not split: no query, which short calls would feel)
    ws = None
    if workspace is not None or cache is not None or q.shape[0] >= 512:
        ws = _attach("gdn_attn_extend", lib.gdn_attn_extend_workspace_size, args, i, workspace)
    _run("gdn_attn_extend", lib.gdn_attn_extend, args, i)
    del ws
    return out


def attn_extend_workspace_size(q, k, v, cu_seqlens, *, scale=None, causal: bool = True, softcap: float = 0.0,
                               slopes=None, window: int = 0, doc=None, visible=None, cache: KVCache | None = None,
                               block_table=None, cache_len=None, start=None, max_cached: int = 0) -> int:
    """Bytes of workspace with which attn_extend splits the keys of these arguments (0: no
    split)."""
    lib = _lib.load()
    args, i = _extend_args(q, k, v, cu_seqlens, scale, causal, softcap, slopes, window, doc, visible, cache,
                           block_table, cache_len, start, None, max_cached)
    return _need("gdn_attn_extend_workspace_size", lib.gdn_attn_extend_workspace_size, args, i)


def _decode_args(q, cache, block_table, kv_len, scale, softcap, slopes, window, q_pos, accumulate, max_kvlen, out):
    N, H, d = q.shape
    ca = cache._args
    i = _place(cache._k, q, block_table, kv_len, slopes, q_pos, out)
    if accumulate and cache._weight is None:
        raise ValueError("accumulate needs cache.weight (kv_cache(track=True))")
    if ca.d != d:
        raise ValueError(f"q must be [N, H, {ca.d}], got {tuple(q.shape)}")
    ts, tw = _table(block_table, N)
    # (a query of the workspace reads no buffer: an aligned stand-in for the output)
    o, os = (256, H * d) if out is None else (out.data_ptr(), _heads(out, "out", N, H, d))
    return _lib.AttnDecodeArgs(
        ca, GDN_BF16, GDN_BF16, N, H, q.data_ptr(), _heads(q, "q", N, H, d), o, os, _vec(kv_len, "kv_len", N),
        _vec(q_pos, "q_pos", N), block_table.data_ptr(), ts, tw, max_kvlen, _vec(slopes, "slopes", H, _F32),
        window, d ** -0.5 if scale is None else scale, softcap, 1 if accumulate else 0, None, 0), i


def attn_decode(q, cache: KVCache, block_table, kv_len, *, scale=None, softcap: float = 0.0, slopes=None,
                window: int = 0, q_pos=None, accumulate: bool = False, max_kvlen: int = 0, out=None,
                workspace: torch.Tensor | None = None):
    """One token per sequence (q bf16 [N, H, d]) over the rows 0 .. kv_len[n] - 1 of the
    cache, the token's own among them.  softcap, slopes, window as in attn_extend; q_pos
    int32 [N]: the queries' positions (default kv_len - 1).  accumulate adds each row's
    softmax weight, summed over the query heads of its kv head, to cache.weight.
    kv_len[n] = 0 gives zeros, kv_len[n] < 0 is a padding row whose output is not written.
    max_kvlen: host hint of the longest kv_len (speed only).  workspace: uint8 device
    tensor of attn_decode_workspace_size bytes (else one is allocated)."""
    lib = _lib.load()
    if out is None:
        out = _like(q)
    args, i = _decode_args(q, cache, block_table, kv_len, scale, softcap, slopes, window, q_pos, accumulate,
                           max_kvlen, out)
    ws = _attach("gdn_attn_decode", lib.gdn_attn_decode_workspace_size, args, i, workspace)
    _run("gdn_attn_decode", lib.gdn_attn_decode, args, i)
    del ws
    return out


def attn_decode_workspace_size(q, cache: KVCache, block_table, kv_len, *, scale=None, softcap: float = 0.0,
                               slopes=None, window: int = 0, q_pos=None, accumulate: bool = False,
                               max_kvlen: int = 0) -> int:
    """Bytes of workspace attn_decode wants for these arguments (0: none)."""
    lib = _lib.load()
    args, i = _decode_args(q, cache, block_table, kv_len, scale, softcap, slopes, window, q_pos, accumulate,
                           max_kvlen, None)
    return _need("gdn_attn_decode_workspace_size", lib.gdn_attn_decode_workspace_size, args, i)


# ------------------------------------------------------------------ eviction
def _evict_args(cache, block_table, kv_len, budget, recent, new_len):
    i = _place(cache._k, block_table, kv_len, new_len)
    if cache._pos is None or cache._weight is None:
        raise ValueError("an eviction needs cache.pos and cache.weight (kv_cache(track=True))")
    N = kv_len.shape[0]
    ts, tw = _table(block_table, N)
    # (a query of the workspace reads no buffer: an aligned stand-in for the new lengths)
    return _lib.KVEvictArgs(cache._args, N, budget, recent, tw, _vec(kv_len, "kv_len", N),
                            256 if new_len is None else _vec(new_len, "new_len", N), block_table.data_ptr(), ts, None, 0), i


def kv_evict(cache: KVCache, block_table, kv_len, budget: int, *, recent: int = 0, new_len=None,
             workspace: torch.Tensor | None = None):
    """Cut every sequence to at most `budget` rows per kv head, in place: the `recent`
    newest positions and the rows of largest accumulated weight stay, rows that stay past
    `budget` move into the places of dropped ones.  Returns new_len int32 [N] = min(kv_len,
    budget) (may be given, kv_len itself included).  workspace: uint8 device tensor of
    kv_evict_workspace_size bytes (else one is allocated)."""
    lib = _lib.load()
    if new_len is None:
        new_len = torch.empty_like(kv_len)
    args, i = _evict_args(cache, block_table, kv_len, budget, recent, new_len)
    ws = _attach("gdn_kv_evict", lib.gdn_kv_evict_workspace_size, args, i, workspace)
    _run("gdn_kv_evict", lib.gdn_kv_evict, args, i)
    del ws
    return new_len


def kv_evict_workspace_size(cache: KVCache, block_table, kv_len, budget: int, *, recent: int = 0) -> int:
    """Bytes of workspace kv_evict wants for these arguments."""
    lib = _lib.load()
    args, i = _evict_args(cache, block_table, kv_len, budget, recent, None)
    return _need("gdn_kv_evict_workspace_size", lib.gdn_kv_evict_workspace_size, args, i)


# ------------------------------------------------------------------ layer call
def _check_layer(layer) -> None:
    """Refuses layers that ask for another attention than forward_attn's."""
    if getattr(layer, "is_cross_attention", False):
        raise ValueError("forward_attn is self-attention: is_cross_attention is not supported")
    kind = getattr(layer, "attn_type", None)
    if kind is not None and str(getattr(kind, "value", kind)).lower() != "decoder":
        raise ValueError(f"forward_attn is a decoder's causal attention, got attn_type {kind!r} (attn_extend has causal=False)")
    d_v = getattr(layer, "v_head_dim", None)
    if d_v not in (None, -1, layer.head_dim):
        raise ValueError(f"keys and values have one head size: head_dim {layer.head_dim}, v_head_dim {d_v}")


def forward_attn(layer, forward_batch, q, k, v, save_kv_cache: bool = True):
    """Full-attention layer call of a hybrid model (pymllm RadixAttention.forward), the
    counterpart of forward_gdn: stores the new tokens in the layer's cache and attends.

    layer: num_heads, num_kv_heads, head_dim, layer_id; optional scaling (default head_dim
           ** -0.5), logit_cap (tanh cap, 0 = none), sliding_window_size (-1 or 0 = none; w:
           a token sees itself and the w - 1 before it), alibi_slopes fp32 [num_heads].  A
           layer with is_cross_attention, an attn_type other than "decoder" or a v_head_dim
           other than head_dim raises ValueError.
    forward_batch: forward_mode; kv_pool indexable by layer_id -> KVCache; block_table int32
           [N, width]; cache_len int32 [N], the rows each sequence holds before this call
           (negative: a padding row); optional positions int32 [N] of each sequence's first
           new token (default cache_len; needed once rows have been evicted); for extend
           modes cu_seqlens int32 [N+1]; optional accumulate_weights (decode: add the
           softmax weights to the cache's); optional max_kvlen, a host hint of the longest
           sequence.
    q [T, num_heads * head_dim], k, v [T, num_kv_heads * head_dim] (or [T, heads, head_dim]).
    save_kv_cache=False leaves the cache as it is (draft models; extend modes only, since a
    decode step attends to its own stored row).  Target verify leaves it as it is too: the
    accepted tokens are the caller's to store; token trees (spec_parents) raise ValueError.
    Returns out [T, num_heads * head_dim] bf16."""
    _check_layer(layer)
    kind = _mode_kind(forward_batch.forward_mode)
    H, H_kv, d = layer.num_heads, layer.num_kv_heads, layer.head_dim
    T = q.shape[0]
    if T == 0:
        return q.new_empty((0, H * d))
    q, k, v = q.unflatten(1, (H, d)) if q.dim() == 2 else q, *(
        x.unflatten(1, (H_kv, d)) if x.dim() == 2 else x for x in (k, v))
    fb = forward_batch
    cache, table, held = fb.kv_pool[layer.layer_id], fb.block_table, fb.cache_len
    start = getattr(fb, "positions", None)
    window = int(getattr(layer, "sliding_window_size", 0) or 0)
    kw = dict(scale=getattr(layer, "scaling", None), softcap=float(getattr(layer, "logit_cap", 0.0) or 0.0),
              window=max(window, 0), slopes=getattr(layer, "alibi_slopes", None))
    if kind == "decode":
        if not save_kv_cache:
            raise ValueError("a decode step attends to its own stored row: save_kv_cache must be True")
        kv_store(k, v, None, cache, table, held, start=start)
        # a padding row (negative) must not become a row of length 0
        kv_len = torch.where(held >= 0, held + 1, held)
        o = attn_decode(q, cache, table, kv_len, q_pos=start, accumulate=bool(getattr(fb, "accumulate_weights", False)),
                        max_kvlen=int(getattr(fb, "max_kvlen", 0) or 0), **kw)
    else:
        verify = _is_target_verify(fb.forward_mode)
        if verify and getattr(fb, "spec_parents", None) is not None:
            raise ValueError("forward_attn has no token trees: verify a chain")
        o = attn_extend(q, k, v, fb.cu_seqlens, cache=cache, block_table=table, cache_len=held, start=start,
                        max_cached=int(getattr(fb, "max_kvlen", 0) or 0), **kw)
        if save_kv_cache and not verify:
            kv_store(k, v, fb.cu_seqlens, cache, table, held, start=start)
    return o.view(T, H * d)
