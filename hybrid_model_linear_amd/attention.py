"""Softmax attention of the hybrid model's full-attention layers, over a paged 8-bit cache.

  kv_cache       allocate a cache                                  -> KVCache
  kv_store       quantise new keys and values into its pages       -> gdn_kv_store
  attn_extend    packed varlen new tokens (+ a cached prefix)      -> gdn_attn_extend
  attn_decode    one token per sequence over the cache             -> gdn_attn_decode
  kv_evict       keep a budget of rows by accumulated weight       -> gdn_kv_evict
and the layer call of the pages:
  forward_attn(layer, forward_batch, q, k, v)   (pymllm RadixAttention.forward)

As in the rest of the binding every step runs in the library's HIP kernels; this module
checks tensors, allocates what the caller did not supply and passes pointers.
"""
from __future__ import annotations

import ctypes as ct
from dataclasses import dataclass

import torch

from . import _i32, _lib, _mode_kind, _on_gpu, _ptr, _rows, _same_rows, _stream, _is_target_verify
from ._lib import GDN_BF16

_PAGES = (16, 32, 64, 128)


@dataclass
class KVCache:
    """The tensors of a paged 8-bit key/value cache (gdn_kv_cache): k, v float8_e4m3fn
    [num_pages, H_kv, page, d]; k_scale, v_scale fp32 [num_pages, H_kv], powers of two (a
    cached value is code * scale); optional pos int32 and weight fp32 [num_pages, H_kv,
    page]: the rows' positions and the softmax weights accumulated on them (an eviction
    needs both)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    pos: torch.Tensor | None = None
    weight: torch.Tensor | None = None

    @property
    def page(self) -> int:
        return self.k.shape[2]


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


def _cache_args(c: KVCache, track: bool = False) -> _lib.KVCacheArgs:
    k = c.k
    if k.dim() != 4 or k.dtype != torch.float8_e4m3fn or not k.is_contiguous():
        raise ValueError("cache.k must be contiguous float8_e4m3fn [num_pages, H_kv, page, d]")
    pages, H_kv, page, d = k.shape
    if c.v.shape != k.shape or c.v.dtype != k.dtype or not c.v.is_contiguous():
        raise ValueError("cache.v must be like cache.k")
    for t, nm in ((c.k_scale, "k_scale"), (c.v_scale, "v_scale")):
        if t.shape != (pages, H_kv) or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"cache.{nm} must be contiguous fp32 [{pages}, {H_kv}]")
    for t, nm, dt in ((c.pos, "pos", torch.int32), (c.weight, "weight", torch.float32)):
        if t is None:
            if track:
                raise ValueError(f"this call needs cache.{nm} (kv_cache(track=True))")
        elif t.shape != (pages, H_kv, page) or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"cache.{nm} must be contiguous {dt} [{pages}, {H_kv}, {page}]")
    return _lib.KVCacheArgs(_ptr(k), _ptr(c.v), _ptr(c.k_scale), _ptr(c.v_scale), _ptr(c.pos), _ptr(c.weight),
                            pages, page, H_kv, d)


def _cache_device(c: KVCache, *ts):
    return _on_gpu(c.k, c.v, c.k_scale, c.v_scale, c.pos, c.weight, *ts)


def _table(t: torch.Tensor, n: int) -> tuple[int, int]:
    """(row stride, width) of a block table."""
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != n or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"block_table must be int32 [{n}, width] with unit column stride, got "
                         f"{t.dtype} {tuple(t.shape)}")
    return (t.stride(0) if n > 1 else t.shape[1]), t.shape[1]


def _bf16(**ts):
    for nm, t in ts.items():
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{nm} must be bf16")


def _slopes(t, H):
    if t is not None and (t.dtype != torch.float32 or t.shape != (H,) or not t.is_contiguous()):
        raise ValueError(f"slopes must be contiguous fp32 [{H}]")


def _stride(t, name, heads, d):
    s = _rows(t, name, heads, d)
    return s if t.shape[0] > 1 else heads * d


def kv_store(k, v, cu_seqlens, cache: KVCache, block_table, cache_len, *, start=None) -> None:
    """Quantise the new tokens' keys and values (k, v bf16 [T, H_kv, d]) into the cache: the
    tokens of sequence n (cu_seqlens int32 [N+1]; None: one token per sequence) become its
    rows cache_len[n], cache_len[n] + 1, ... over the pages block_table[n] (int32 [N,
    width]).  start int32 [N]: the first token's position (default cache_len), for a cache
    that keeps positions.  cache_len[n] < 0 skips the sequence."""
    lib = _lib.load()
    dev = _cache_device(cache, k, v, cu_seqlens, block_table, cache_len, start)
    ca = _cache_args(cache)
    T, N = k.shape[0], cache_len.shape[0]
    _same_rows(T, "the tokens of k", v=v)
    _bf16(k=k, v=v)
    _i32(cache_len, "cache_len", N)
    if cu_seqlens is not None:
        _i32(cu_seqlens, "cu_seqlens", N + 1)
    elif T != N:
        raise ValueError(f"without cu_seqlens there is one token per sequence: {T} tokens, {N} sequences")
    if start is not None:
        _i32(start, "start", N)
    ts, tw = _table(block_table, N)
    args = _lib.KVStoreArgs(cache=ca, in_dtype=GDN_BF16, N=N, T=T, k=_ptr(k), k_stride=_stride(k, "k", ca.H_kv, ca.d),
                            v=_ptr(v), v_stride=_stride(v, "v", ca.H_kv, ca.d), cu_seqlens=_ptr(cu_seqlens),
                            cache_len=_ptr(cache_len), start=_ptr(start), block_table=_ptr(block_table),
                            table_stride=ts, table_width=tw)
    with torch.cuda.device(dev):
        _lib.check("gdn_kv_store", lib.gdn_kv_store(ct.byref(args), _stream(dev)))


def attn_extend(q, k, v, cu_seqlens, *, scale=None, causal: bool = True, softcap: float = 0.0, slopes=None,
                window: int = 0, doc=None, visible=None, cache: KVCache | None = None, block_table=None,
                cache_len=None, start=None, out=None):
    """Attention of packed new tokens over their own keys and values and, with `cache`, the
    cache_len[n] rows that each sequence holds already.  q [T, H, d], k, v [T, H_kv, d]
    bf16; cu_seqlens int32 [N+1].
    softcap: scores become softcap * tanh(score / softcap) (0: none).  slopes fp32 [H]: a
    bias of -slope * |distance|.  window: only keys closer than this (0: all).  visible
    int32 [N]: the first visible[n] tokens are seen by every token of the sequence (prefix
    mask); causal=False lets every token see every other.  doc int32 [T]: a token sees only
    tokens with its own id; a negative id sees nothing and is not seen (output 0).
    start int32 [N]: position of each first token (default: behind the cached rows).
    Returns out [T, H, d] bf16 (rows behind the last sequence, and those of sequences with
    cache_len[n] < 0, are not written)."""
    lib = _lib.load()
    T, H, d = q.shape
    H_kv, N = k.shape[1], cu_seqlens.shape[0] - 1
    ts_all = (q, k, v, cu_seqlens, slopes, doc, visible, block_table, cache_len, start, out)
    args = _lib.AttnExtendArgs()
    if cache is not None:
        if block_table is None or cache_len is None:
            raise ValueError("a cache needs block_table and cache_len")
        dev = _cache_device(cache, *ts_all)
        args.cache = _cache_args(cache)
        args.table_stride, args.table_width = _table(block_table, N)
        _i32(cache_len, "cache_len", N)
    else:
        if block_table is not None or cache_len is not None:
            raise ValueError("block_table and cache_len need a cache")
        dev = _on_gpu(*ts_all)
    _same_rows(T, "the tokens of q", k=k, v=v, out=out, doc=doc)
    _bf16(q=q, k=k, v=v)
    _i32(cu_seqlens, "cu_seqlens", N + 1)
    for t, nm, n in ((visible, "visible", N), (start, "start", N), (doc, "doc", T)):
        if t is not None:
            _i32(t, nm, n)
    _slopes(slopes, H)
    if out is None:
        out = torch.empty((T, H, d), dtype=torch.bfloat16, device=dev)
    _bf16(out=out)
    args.in_dtype = args.out_dtype = GDN_BF16
    args.N, args.H, args.H_kv, args.d, args.T = N, H, H_kv, d, T
    args.q, args.q_stride = _ptr(q), _stride(q, "q", H, d)
    args.k, args.k_stride = _ptr(k), _stride(k, "k", H_kv, d)
    args.v, args.v_stride = _ptr(v), _stride(v, "v", H_kv, d)
    args.out, args.out_stride = _ptr(out), _stride(out, "out", H, d)
    args.cu_seqlens, args.cache_len, args.start = _ptr(cu_seqlens), _ptr(cache_len), _ptr(start)
    args.block_table, args.causal = _ptr(block_table), int(bool(causal))
    args.visible, args.doc, args.slopes = _ptr(visible), _ptr(doc), _ptr(slopes)
    args.window, args.softcap = int(window), float(softcap)
    args.scale = float(d ** -0.5 if scale is None else scale)
    with torch.cuda.device(dev):
        _lib.check("gdn_attn_extend", lib.gdn_attn_extend(ct.byref(args), _stream(dev)))
    return out


def _workspace_for(lib_size, fn, args, dev, workspace):
    """Attach a call's workspace: the caller's uint8 tensor, or a fresh allocation."""
    if workspace is None:
        need = lib_size(ct.byref(args))
        if need < 0:
            _lib.check(fn, int(-need))
        if need == 0:
            return None
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous() \
            or workspace.device != dev:
        raise ValueError("workspace must be a contiguous uint8 vector on the call's device")
    args.workspace, args.workspace_bytes = _ptr(workspace), workspace.numel()
    return workspace


def _decode_args(q, cache, block_table, kv_len, scale, softcap, slopes, window, q_pos, accumulate, max_kvlen, out):
    N, H, d = q.shape
    dev = _cache_device(cache, q, block_table, kv_len, slopes, q_pos, out)
    args = _lib.AttnDecodeArgs()
    args.cache = ca = _cache_args(cache)
    if accumulate and cache.weight is None:
        raise ValueError("accumulate needs cache.weight (kv_cache(track=True))")
    if ca.d != d:
        raise ValueError(f"q must be [N, H, {ca.d}], got {tuple(q.shape)}")
    _bf16(q=q)
    _i32(kv_len, "kv_len", N)
    if q_pos is not None:
        _i32(q_pos, "q_pos", N)
    _slopes(slopes, H)
    args.in_dtype = args.out_dtype = GDN_BF16
    args.N, args.H = N, H
    args.q, args.q_stride = _ptr(q), _stride(q, "q", H, d)
    if out is not None:
        _same_rows(N, "one token per sequence of q", out=out)
        _bf16(out=out)
        args.out, args.out_stride = _ptr(out), _stride(out, "out", H, d)
    args.kv_len, args.q_pos, args.block_table = _ptr(kv_len), _ptr(q_pos), _ptr(block_table)
    args.table_stride, args.table_width = _table(block_table, N)
    args.max_kvlen, args.slopes, args.window = int(max_kvlen), _ptr(slopes), int(window)
    args.scale = float(d ** -0.5 if scale is None else scale)
    args.softcap, args.accumulate = float(softcap), int(bool(accumulate))
    return args, dev


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
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    args, dev = _decode_args(q, cache, block_table, kv_len, scale, softcap, slopes, window, q_pos, accumulate,
                             max_kvlen, out)
    with torch.cuda.device(dev):
        ws = _workspace_for(lib.gdn_attn_decode_workspace_size, "gdn_attn_decode", args, dev, workspace)
        _lib.check("gdn_attn_decode", lib.gdn_attn_decode(ct.byref(args), _stream(dev)))
        del ws
    return out


def attn_decode_workspace_size(q, cache: KVCache, block_table, kv_len, *, scale=None, softcap: float = 0.0,
                               slopes=None, window: int = 0, q_pos=None, accumulate: bool = False,
                               max_kvlen: int = 0) -> int:
    """Bytes of workspace attn_decode wants for these arguments (0: none)."""
    lib = _lib.load()
    args, dev = _decode_args(q, cache, block_table, kv_len, scale, softcap, slopes, window, q_pos, accumulate,
                             max_kvlen, None)
    # the host-side query reads no buffer: an aligned stand-in for the output
    args.out, args.out_stride = ct.c_void_p(256), q.shape[1] * q.shape[2]
    with torch.cuda.device(dev):
        need = lib.gdn_attn_decode_workspace_size(ct.byref(args))
    if need < 0:
        _lib.check("gdn_attn_decode_workspace_size", int(-need))
    return int(need)


def _evict_args(cache, block_table, kv_len, budget, recent, new_len):
    dev = _cache_device(cache, block_table, kv_len, new_len)
    N = kv_len.shape[0]
    _i32(kv_len, "kv_len", N)
    args = _lib.KVEvictArgs()
    args.cache = _cache_args(cache, track=True)
    args.N, args.budget, args.recent, args.kv_len = N, int(budget), int(recent), _ptr(kv_len)
    args.block_table = _ptr(block_table)
    args.table_stride, args.table_width = _table(block_table, N)
    if new_len is not None:
        args.new_len = _ptr(_i32(new_len, "new_len", N))
    return args, dev


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
    args, dev = _evict_args(cache, block_table, kv_len, budget, recent, new_len)
    with torch.cuda.device(dev):
        ws = _workspace_for(lib.gdn_kv_evict_workspace_size, "gdn_kv_evict", args, dev, workspace)
        _lib.check("gdn_kv_evict", lib.gdn_kv_evict(ct.byref(args), _stream(dev)))
        del ws
    return new_len


def kv_evict_workspace_size(cache: KVCache, block_table, kv_len, budget: int, *, recent: int = 0) -> int:
    """Bytes of workspace kv_evict wants for these arguments."""
    lib = _lib.load()
    args, _ = _evict_args(cache, block_table, kv_len, budget, recent, None)
    args.new_len = ct.c_void_p(256)          # (not read by the query)
    need = lib.gdn_kv_evict_workspace_size(ct.byref(args))
    if need < 0:
        _lib.check("gdn_kv_evict_workspace_size", int(-need))
    return int(need)


def forward_attn(layer, forward_batch, q, k, v, save_kv_cache: bool = True):
    """Full-attention layer call of a hybrid model (pymllm RadixAttention.forward), the
    counterpart of forward_gdn: stores the new tokens in the layer's cache and attends.

    layer: num_heads, num_kv_heads, head_dim, layer_id; optional scaling (default head_dim
           ** -0.5), logit_cap (tanh cap, 0 = none), sliding_window_size (-1 or 0 = none),
           alibi_slopes fp32 [num_heads].
    forward_batch: forward_mode; kv_pool indexable by layer_id -> KVCache; block_table int32
           [N, width]; cache_len int32 [N], the rows each sequence holds before this call
           (negative: a padding row); optional positions int32 [N] of each sequence's first
           new token (default cache_len; needed once rows have been evicted); for extend
           modes cu_seqlens int32 [N+1]; optional accumulate_weights (decode: add the
           softmax weights to the cache's); optional max_kvlen, a host hint.
    q [T, num_heads * head_dim], k, v [T, num_kv_heads * head_dim] (or [T, heads, head_dim]).
    save_kv_cache=False leaves the cache as it is (draft models; extend modes only, since a
    decode step attends to its own stored row).  Target verify leaves it as it is too: the
    accepted tokens are the caller's to store; token trees (spec_parents) raise ValueError.
    Returns out [T, num_heads * head_dim] bf16."""
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
        o = attn_extend(q, k, v, fb.cu_seqlens, cache=cache, block_table=table, cache_len=held, start=start, **kw)
        if save_kv_cache and not verify:
            kv_store(k, v, fb.cu_seqlens, cache, table, held, start=start)
    return o.view(T, H * d)
