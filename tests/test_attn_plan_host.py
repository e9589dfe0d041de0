"""Host-side tests of how attn_extend and attn_decode cut a call and of what they refuse for its
size (no GPU: workspace queries and calls that fail validation launch nothing)."""
import ctypes as ct
from unittest import mock

import pytest
import torch

import hybrid_model_linear_amd as gdn
from hybrid_model_linear_amd import _lib, attention
from test_attn_host import P, _batch, _cache, _decode, _evict, _extend, _layer, _store

CUS = 256            # what the library assumes without a device
KEYS = 7000


def _parts(n, tokens, H, H_kv, d, keys=KEYS, page=64, **kw):
    """Parts into which the keys of n sequences of so many tokens over `keys` cached rows are cut."""
    width, T = -(-keys // page), n * tokens
    a = _extend(_cache(H_kv=H_kv, d=d, page=page, pos=None, num_pages=1 << 20), N=n, T=T, H=H, H_kv=H_kv, d=d, q=P, q_stride=H * d,
                k=P, k_stride=H_kv * d, v=P, v_stride=H_kv * d, out=1 << 50, out_stride=H * d, table_width=width,
                table_stride=width, **kw)
    need = gdn.load().gdn_attn_extend_workspace_size(ct.byref(a))
    assert need >= 0
    return max(need // (T * H * (d + 2) * 4), 1)


@pytest.mark.parametrize("n,tokens,H,H_kv,d", [(1, 16, 32, 8, 128), (8, 4, 32, 8, 128), (16, 4, 32, 8, 128), (16, 1, 32, 8, 128),
                                               (32, 4, 32, 8, 128), (8, 4, 16, 2, 256), (32, 4, 16, 2, 256), (64, 4, 16, 2, 128),
                                               (5, 30, 16, 4, 128), (6, 256, 32, 8, 64)])
def test_parts_have_a_place_at_once(n, tokens, H, H_kv, d):
    """Row tiles do not cross sequences: there is one per sequence and kv head at least."""
    tiles = n * -(-tokens * (H // H_kv) // 128) * H_kv
    places = CUS * (2 if d <= 128 else 1)
    parts = _parts(n, tokens, H, H_kv, d)
    assert parts * tiles <= places * 9 // 8 or parts <= 4
    assert parts > 1 or 2 * tiles > places // 2


@pytest.mark.parametrize("n,tokens,H,H_kv,d,keys", [(64, 4, 32, 8, 128, 7000), (128, 4, 32, 8, 128, 4000), (48, 4, 32, 8, 128, 7000),
                                                    (64, 4, 16, 2, 256, 7000), (24, 4, 32, 8, 256, 7000)])
def test_batches_that_fill_the_chip_are_cut_in_four_at_most(n, tokens, H, H_kv, d, keys):
    assert _parts(n, tokens, H, H_kv, d, keys) <= 4


def test_chunks_that_fill_the_chip_are_not_cut():
    assert _parts(4, 512, 16, 2, 256) == _parts(4, 512, 32, 8, 128) == 1


def test_a_hint_of_the_cached_rows_counts_instead_of_the_table():
    wide = dict(n=8, tokens=16, H=32, H_kv=8, d=128, keys=32768)
    assert _parts(**wide) > 1
    assert _parts(**wide, max_cached=200) == 1
    assert _parts(**wide, max_cached=32768) == _parts(**wide, max_cached=1 << 30) == _parts(**wide)
    assert 1 < _parts(**dict(wide, n=1), max_cached=1500) < _parts(**dict(wide, n=1))
    a = _extend(_cache(), max_cached=-1)
    assert gdn.load().gdn_attn_extend(ct.byref(a), None) == _lib.GDN_E_SHAPE


def test_forward_attn_passes_its_hint_on():
    x = torch.zeros(2, 4 * 64), torch.zeros(2, 2 * 64), torch.zeros(2, 2 * 64)
    with mock.patch.object(attention, "kv_store"), mock.patch.object(attention, "attn_extend") as ex:
        ex.return_value = torch.zeros(2, 4, 64)
        for kw, hint in ((dict(max_kvlen=77), 77), (dict(max_kvlen=None), 0), ({}, 0)):
            gdn.forward_attn(_layer(), _batch("extend", **kw), *x)
            assert ex.call_args.kwargs["max_cached"] == hint


# A launch has fewer than 2^32 threads in a dimension, 2^24 - 1 workgroups of 256.
def test_decode_calls_past_the_largest_launch_are_refused():
    lib = gdn.load()
    for H_kv, fits in ((255, True), (256, True), (257, False), (1000, False)):
        a = _decode(_cache(H_kv=H_kv, d=64), N=65535, H=H_kv, q_stride=H_kv * 64, out_stride=H_kv * 64, out=1 << 50)
        need = lib.gdn_attn_decode_workspace_size(ct.byref(a))
        assert (need >= 0) == fits and (fits or need == -_lib.GDN_E_UNSUPPORTED)
        if not fits:
            assert lib.gdn_attn_decode(ct.byref(a), None) == _lib.GDN_E_UNSUPPORTED
    a = _decode(_cache(H_kv=9000, d=64), N=1, H=9000, q_stride=9000 * 64, out_stride=9000 * 64, out=1 << 50, accumulate=1,
                table_width=1 << 24, table_stride=1 << 24)
    assert lib.gdn_attn_decode_workspace_size(ct.byref(a)) == -_lib.GDN_E_UNSUPPORTED


def test_extend_calls_past_the_largest_launch_are_refused():
    for N, fits in ((1 << 23, True), (1 << 24, False)):
        a = _extend(N=N, T=1, H=1, H_kv=1, d=64, q_stride=64, k_stride=64, v_stride=64, out_stride=64)
        need = gdn.load().gdn_attn_extend_workspace_size(ct.byref(a))
        assert need == (0 if fits else -_lib.GDN_E_UNSUPPORTED)


def test_store_and_evict_calls_past_the_largest_launch_are_refused():
    lib = gdn.load()
    many = 1 << 23
    assert lib.gdn_kv_store(ct.byref(_store(N=many, T=many)), None) == _lib.GDN_E_UNSUPPORTED
    assert lib.gdn_kv_store(ct.byref(_store(_cache(H_kv=64, d=64), N=1 << 20, T=1 << 20, k_stride=4096, v_stride=4096)), None) == \
        _lib.GDN_E_UNSUPPORTED
    wide = dict(table_width=1 << 26, table_stride=1 << 26, budget=1 << 30, N=1)
    assert lib.gdn_kv_evict_workspace_size(ct.byref(_evict(_cache(page=16), **wide))) == -_lib.GDN_E_UNSUPPORTED
    assert lib.gdn_kv_evict_workspace_size(ct.byref(_evict(_cache(page=16), **dict(wide, budget=1 << 27)))) > 0
