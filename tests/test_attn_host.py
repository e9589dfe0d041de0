"""Host-side tests of the softmax-attention entry points (no GPU): struct layouts, the
refusals of the C ABI (nothing is launched: every call fails validation first) and of the
binding, the workspace queries, and forward_attn's dispatch with the calls mocked."""
import ctypes as ct
import os
import subprocess
import tempfile
from types import SimpleNamespace
from unittest import mock

import pytest
import torch

import hybrid_model_linear_amd as gdn
from hybrid_model_linear_amd import _lib, attention

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdn.h")
OK, NULL, SHAPE, DTYPE, UNSUP = (_lib.GDN_OK, _lib.GDN_E_NULL, _lib.GDN_E_SHAPE, _lib.GDN_E_DTYPE,
                                 _lib.GDN_E_UNSUPPORTED)
P = 0x10000          # aligned stand-ins, never dereferenced
Q = 0x20000000
NAN, INF = float("nan"), float("inf")


def test_struct_layouts_match_header():
    structs = {"gdn_kv_cache": _lib.KVCacheArgs, "gdn_kv_store_args": _lib.KVStoreArgs,
               "gdn_attn_extend_args": _lib.AttnExtendArgs, "gdn_attn_decode_args": _lib.AttnDecodeArgs,
               "gdn_kv_evict_args": _lib.KVEvictArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void){"]
    for c, cls in structs.items():
        lines.append(f'printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in cls._fields_]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(src, "w").write("\n".join(lines + ["return 0;}"]))
        subprocess.run(["gcc", "-std=c99", "-o", exe, src], check=True)
        got = {tuple(x.split()[:2]): int(x.split()[2]) for x in
               subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()}
    for c, cls in structs.items():
        assert got[(c, "size")] == ct.sizeof(cls), c
        for f, _ in cls._fields_:
            assert got[(c, f)] == getattr(cls, f).offset, (c, f)


def _cache(**kw):
    base = dict(k=P, v=P, k_scale=P, v_scale=P, pos=P, weight=P, num_pages=10, page=64, H_kv=2, d=128)
    base.update(kw)
    return _lib.KVCacheArgs(**base)


CACHE = [(dict(d=96), UNSUP), (dict(d=512), UNSUP), (dict(page=8), UNSUP), (dict(page=48), UNSUP), (dict(page=256), UNSUP),
         (dict(H_kv=0), SHAPE), (dict(H_kv=70000), SHAPE), (dict(num_pages=0), SHAPE), (dict(v=None), NULL),
         (dict(k_scale=None), NULL), (dict(v_scale=None), NULL), (dict(k=P + 8), SHAPE), (dict(v=P + 4), SHAPE),
         (dict(pos=P + 4), SHAPE), (dict(weight=P + 8), SHAPE), (dict(k_scale=P + 2), SHAPE)]
TABLE = [(dict(block_table=None), NULL), (dict(table_width=0), SHAPE), (dict(table_stride=3), SHAPE),
         (dict(table_width=1 << 26, table_stride=1 << 26), SHAPE), (dict(block_table=P + 2), SHAPE)]


def _store(cache=None, **kw):
    base = dict(cache=cache or _cache(), in_dtype=1, N=3, T=7, k=P, k_stride=256, v=P, v_stride=256, cu_seqlens=P,
                cache_len=P, start=None, block_table=P, table_stride=4, table_width=4)
    base.update(kw)
    return _lib.KVStoreArgs(**base)


def _extend(cache=None, **kw):
    base = dict(cache=cache or _lib.KVCacheArgs(), in_dtype=1, out_dtype=1, N=2, H=4, H_kv=2, d=128, T=9, q=P, q_stride=512,
                k=P, k_stride=256, v=P, v_stride=256, out=Q, out_stride=512, cu_seqlens=P, causal=1, scale=0.1)
    if cache is not None:
        base.update(cache_len=P, block_table=P, table_stride=4, table_width=4)
    base.update(kw)
    return _lib.AttnExtendArgs(**base)


def _decode(cache=None, **kw):
    base = dict(cache=cache or _cache(), in_dtype=1, out_dtype=1, N=3, H=4, q=P, q_stride=512, out=Q, out_stride=512,
                kv_len=P, block_table=P, table_stride=4, table_width=4, scale=0.1)
    base.update(kw)
    return _lib.AttnDecodeArgs(**base)


def _evict(cache=None, **kw):
    base = dict(cache=cache or _cache(), N=3, budget=20, recent=4, table_width=4, kv_len=P, new_len=P, block_table=P,
                table_stride=4)
    base.update(kw)
    return _lib.KVEvictArgs(**base)


@pytest.mark.parametrize("kw,status", [(dict(in_dtype=0), DTYPE), (dict(N=-1), SHAPE), (dict(T=-1), SHAPE),
                                       (dict(T=1 << 31), SHAPE), (dict(cu_seqlens=None), SHAPE), (dict(k=None), NULL),
                                       (dict(v=None), NULL), (dict(cache_len=None), NULL), (dict(k=P + 8), SHAPE),
                                       (dict(k_stride=248), SHAPE), (dict(v_stride=260), SHAPE),
                                       (dict(v_stride=1 << 23), SHAPE), (dict(N=0, T=0), OK), (dict(T=0), OK)] + TABLE)
def test_store_refusals(kw, status):
    assert gdn.load().gdn_kv_store(ct.byref(_store(**kw)), None) == status


@pytest.mark.parametrize("kw,status", CACHE)
def test_cache_refusals(kw, status):
    lib, c = gdn.load(), _cache(**kw)
    assert lib.gdn_kv_store(ct.byref(_store(c)), None) == status
    assert lib.gdn_attn_decode(ct.byref(_decode(c, H=c.H_kv * 2 or 2)), None) == status
    assert lib.gdn_kv_evict(ct.byref(_evict(c)), None) == status
    if "k" in kw or "v" in kw or "H_kv" not in kw:
        assert lib.gdn_attn_extend(ct.byref(_extend(c)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(in_dtype=0), DTYPE), (dict(out_dtype=0), DTYPE), (dict(d=96), UNSUP), (dict(N=-1), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=1 << 31), SHAPE), (dict(H=5), SHAPE), (dict(H=0), SHAPE), (dict(H_kv=0), SHAPE), (dict(scale=NAN), SHAPE),
    (dict(softcap=-1.0), SHAPE), (dict(softcap=INF), SHAPE), (dict(window=-1), SHAPE), (dict(q=None), NULL), (dict(k=None), NULL),
    (dict(out=None), NULL), (dict(cu_seqlens=None), NULL), (dict(q=P + 8), SHAPE), (dict(out=Q + 4), SHAPE),
    (dict(q_stride=504), SHAPE), (dict(k_stride=258), SHAPE), (dict(out_stride=1 << 23), SHAPE), (dict(out=P), SHAPE),
    (dict(out=P + 1024), SHAPE), (dict(cache_len=P), NULL), (dict(block_table=P), NULL), (dict(T=1 << 30), UNSUP),
    (dict(T=0), OK), (dict(N=0, T=0), OK)])
def test_extend_refusals(kw, status):
    if kw.get("T") == 1 << 30:           # (out out of the inputs' way)
        kw = dict(kw, out=1 << 50)
    assert gdn.load().gdn_attn_extend(ct.byref(_extend(**kw)), None) == status


@pytest.mark.parametrize("kw,status", TABLE + [(dict(doc=P), UNSUP), (dict(cache_len=None), NULL)])
def test_extend_over_cache_refusals(kw, status):
    lib = gdn.load()
    assert lib.gdn_attn_extend(ct.byref(_extend(_cache(), **kw)), None) == status
    assert lib.gdn_attn_extend(ct.byref(_extend(_cache(d=64))), None) == SHAPE
    assert lib.gdn_attn_extend(ct.byref(_extend(_cache(H_kv=4))), None) == SHAPE


@pytest.mark.parametrize("kw,status", TABLE + [
    (dict(in_dtype=0), DTYPE), (dict(out_dtype=0), DTYPE), (dict(N=-1), SHAPE), (dict(N=70000), SHAPE), (dict(H=3), SHAPE),
    (dict(H=0), SHAPE), (dict(max_kvlen=-1), SHAPE), (dict(scale=INF), SHAPE), (dict(softcap=NAN), SHAPE),
    (dict(window=-2), SHAPE), (dict(q=None), NULL), (dict(out=None), NULL), (dict(kv_len=None), NULL), (dict(q=P + 2), SHAPE),
    (dict(q_stride=500), SHAPE), (dict(out=P), SHAPE), (dict(N=0), OK)])
def test_decode_refusals(kw, status):
    lib = gdn.load()
    assert lib.gdn_attn_decode(ct.byref(_decode(**kw)), None) == status
    assert lib.gdn_attn_decode_workspace_size(ct.byref(_decode(**kw))) == -status
    if status != OK:
        assert lib.gdn_attn_decode(ct.byref(_decode(_cache(weight=None), accumulate=1)), None) == NULL


@pytest.mark.parametrize("kw,status", TABLE + [
    (dict(N=-1), SHAPE), (dict(N=70000), SHAPE), (dict(budget=0), SHAPE), (dict(recent=-1), SHAPE), (dict(recent=21), SHAPE),
    (dict(kv_len=None), NULL), (dict(new_len=None), NULL), (dict(N=0), OK)])
def test_evict_refusals(kw, status):
    lib = gdn.load()
    assert lib.gdn_kv_evict(ct.byref(_evict(**kw)), None) == status
    assert lib.gdn_kv_evict_workspace_size(ct.byref(_evict(**kw))) == -status
    for c in (_cache(pos=None), _cache(weight=None)):
        assert lib.gdn_kv_evict(ct.byref(_evict(c)), None) == NULL
    assert lib.gdn_kv_evict(ct.byref(_evict(_cache(num_pages=1 << 27))), None) == UNSUP


def test_workspaces():
    lib = gdn.load()
    assert lib.gdn_attn_decode_workspace_size(ct.byref(_decode())) == 0       # 256 rows: no split
    wide = dict(table_width=4096, table_stride=4096)
    need = lib.gdn_attn_decode_workspace_size(ct.byref(_decode(**wide)))
    assert need > 0 and need % 256 == 0
    assert lib.gdn_attn_decode_workspace_size(ct.byref(_decode(max_kvlen=100, **wide))) == 0
    assert lib.gdn_attn_decode_workspace_size(ct.byref(_decode(_cache(pos=None), window=100, **wide))) == 0
    acc = lib.gdn_attn_decode_workspace_size(ct.byref(_decode(accumulate=1, **wide)))
    assert acc >= need + 3 * 4 * 4096 * 64 * 4
    for ws, nbytes, status in ((None, 0, NULL), (P, need - 1, SHAPE), (P + 64, need, SHAPE)):
        assert lib.gdn_attn_decode(ct.byref(_decode(workspace=ws, workspace_bytes=nbytes, **wide)), None) == status
    need = lib.gdn_kv_evict_workspace_size(ct.byref(_evict()))
    assert need > 0
    for ws, nbytes, status in ((None, 0, NULL), (P, need - 1, SHAPE), (P + 64, need, SHAPE)):
        assert lib.gdn_kv_evict(ct.byref(_evict(workspace=ws, workspace_bytes=nbytes)), None) == status
    # a budget past the table's rows needs no longer lists
    assert lib.gdn_kv_evict_workspace_size(ct.byref(_evict(budget=1 << 30))) == \
        lib.gdn_kv_evict_workspace_size(ct.byref(_evict(budget=256)))


@pytest.mark.parametrize("softcap,scale,status", [(8192.0, 0.1, OK), (8193.0, 0.1, UNSUP), (1e30, 0.1, UNSUP),
                                                  (1e-38, 10.0, UNSUP), (1e-30, 1.0, OK)])
def test_caps_that_fp32_cannot_hold(softcap, scale, status):
    lib, kw = gdn.load(), dict(softcap=softcap, scale=scale)
    assert lib.gdn_attn_extend(ct.byref(_extend(T=0, **kw)), None) == status
    assert lib.gdn_attn_decode(ct.byref(_decode(N=0, **kw)), None) == status


def test_extend_workspace():
    lib = gdn.load()
    size = lambda *a, **kw: lib.gdn_attn_extend_workspace_size(ct.byref(_extend(*a, **kw)))  # noqa: E731
    wide = dict(table_width=4096, table_stride=4096)
    assert size() == 0 and size(_cache()) == 0                                # too few keys
    need = size(_cache(), **wide)
    assert need > 0 and need % 256 == 0
    assert size(_cache(pos=None), window=100, **wide) == 0                    # a window leaves too few
    assert size(_cache(), window=100, **wide) == need                         # (not where rows hold positions of their own)
    assert size(T=40000, N=1) == 0                                            # rows enough
    assert size(T=2000, N=1) > 0 and size(T=2000, N=40) == 0
    assert size(H=0) == -SHAPE and size(d=96) == -UNSUP
    for ws, nbytes in ((P, need - 1), (P + 64, need)):
        assert lib.gdn_attn_extend(ct.byref(_extend(_cache(), workspace=ws, workspace_bytes=nbytes, **wide)), None) == SHAPE


# ------------------------------------------------------------------ binding
def _tensors(**kw):
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)  # noqa: E731
    f8 = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    t = dict(k=f8(6, 2, 16, 64), v=f8(6, 2, 16, 64), k_scale=z(6, 2), v_scale=z(6, 2), pos=z(6, 2, 16, dt=torch.int32),
             weight=z(6, 2, 16))
    t.update(kw)
    return t


@pytest.fixture
def on_gpu():
    """CPU tensors that count as device 0's, calls that launch nothing."""
    calls = []
    with mock.patch.object(attention, "_place", lambda *ts: 0), \
            mock.patch.object(attention, "_run", lambda name, fn, args, i: calls.append((name, args))), \
            mock.patch.object(attention, "_attach", lambda *a: None):
        yield calls


def test_cpu_tensors_are_refused():
    with pytest.raises(ValueError, match="GPU"):
        gdn.KVCache(**_tensors())
    with pytest.raises(ValueError, match="GPU"):
        gdn.attn_extend(torch.zeros(2, 2, 64).bfloat16(), torch.zeros(2, 2, 64).bfloat16(), torch.zeros(2, 2, 64).bfloat16(),
                        torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("name,bad", [
    ("k", torch.zeros(6, 2, 16, 64, dtype=torch.uint8)), ("k", torch.zeros(6, 16, 64).to(torch.float8_e4m3fn)),
    ("v", torch.zeros(6, 2, 16, 128).to(torch.float8_e4m3fn)), ("k_scale", torch.zeros(6, 1)),
    ("v_scale", torch.zeros(6, 2).half()), ("pos", torch.zeros(6, 2, 16)), ("weight", torch.zeros(6, 2, 8)),
    ("weight", torch.zeros(6, 16, 2).transpose(1, 2))])
def test_kv_cache_checks(on_gpu, name, bad):
    with pytest.raises(ValueError):
        gdn.KVCache(**_tensors(**{name: bad}))
    c = gdn.KVCache(**_tensors())
    assert c.page == 16
    with pytest.raises(AttributeError):
        c.k = bad


def test_binding_checks(on_gpu):
    c = gdn.KVCache(**_tensors())
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, k, tab = bf(3, 4, 64), bf(3, 2, 64), i(3, 5)
    gdn.attn_decode(q, c, tab, i(3))
    gdn.attn_decode(bf(3, 512).view(3, 8, 64)[:, :4], c, i(3, 9)[:, :5], i(3), q_pos=i(3), slopes=torch.ones(4), accumulate=True)
    gdn.kv_store(k, k, None, c, tab, i(3))
    gdn.attn_extend(q, k, k, i(2), doc=i(3), visible=i(1))
    gdn.attn_extend(q, k, k, i(4), cache=c, block_table=tab, cache_len=i(3), start=i(3))
    gdn.kv_evict(c, tab, i(3), 7)
    assert [n for n, _ in on_gpu] == ["gdn_attn_decode"] * 2 + ["gdn_kv_store"] + ["gdn_attn_extend"] * 2 + ["gdn_kv_evict"]
    a = on_gpu[1][1]
    assert (a.q_stride, a.table_stride, a.table_width, a.accumulate, a.H) == (512, 9, 5, 1, 4)
    e = on_gpu[4][1]
    assert (e.N, e.T, e.H, e.H_kv, e.d, e.causal, e.cache.num_pages) == (3, 3, 4, 2, 64, 1, 6)
    assert on_gpu[3][1].cache.k is None and abs(e.scale - 0.125) < 1e-7
    for bad in (lambda: gdn.attn_decode(q.float(), c, tab, i(3)), lambda: gdn.attn_decode(bf(3, 4, 128), c, tab, i(3)),
                lambda: gdn.attn_decode(q, c, i(2, 5), i(3)), lambda: gdn.attn_decode(q, c, tab, i(4)),
                lambda: gdn.attn_decode(q, c, tab.long(), i(3)), lambda: gdn.attn_decode(q, c, tab, i(3).long()),
                lambda: gdn.attn_decode(q, c, tab, i(3), slopes=torch.ones(2)),
                lambda: gdn.attn_decode(q, c, tab, i(3), out=bf(3, 4, 32)),
                lambda: gdn.attn_decode(q.transpose(0, 1), c, i(4, 5), i(4)),
                lambda: gdn.kv_store(k, k, None, c, tab, i(2)), lambda: gdn.kv_store(k, bf(2, 2, 64), i(4), c, tab, i(3)),
                lambda: gdn.kv_store(k, bf(3, 1, 64), i(4), c, tab, i(3)), lambda: gdn.kv_store(k, k, i(3), c, tab, i(3)),
                lambda: gdn.attn_extend(q, k, k, i(2), doc=i(2)), lambda: gdn.attn_extend(q, k, k, i(2), cache=c),
                lambda: gdn.attn_extend(q, k, k, i(2), block_table=tab), lambda: gdn.attn_extend(q, bf(3, 2, 32), k, i(2)),
                lambda: gdn.kv_evict(c, tab, i(3), 7, new_len=i(2))):
        with pytest.raises(ValueError):
            bad()
    slim = gdn.KVCache(**_tensors(pos=None, weight=None))
    with pytest.raises(ValueError, match="track"):
        gdn.attn_decode(q, slim, tab, i(3), accumulate=True)
    with pytest.raises(ValueError, match="track"):
        gdn.kv_evict(slim, tab, i(3), 7)
    with pytest.raises(ValueError, match="page"):
        gdn.kv_cache(4, 2, 64, page=20, device="cpu")


def _layer(**kw):
    return SimpleNamespace(num_heads=4, num_kv_heads=2, head_dim=64, layer_id=7, **kw)


def _batch(mode, **kw):
    return SimpleNamespace(forward_mode=mode, kv_pool={7: "cache"}, block_table="table",
                           cache_len=torch.tensor([3, -1], dtype=torch.int32), cu_seqlens="cu", **kw)


def test_forward_attn_dispatch():
    x = torch.zeros(2, 4 * 64), torch.zeros(2, 2 * 64), torch.zeros(2, 2 * 64)
    with mock.patch.object(attention, "kv_store") as st, mock.patch.object(attention, "attn_decode") as de, \
            mock.patch.object(attention, "attn_extend") as ex:
        de.return_value = ex.return_value = torch.zeros(2, 4, 64)
        out = gdn.forward_attn(_layer(logit_cap=30.0, sliding_window_size=-1), _batch("decode", accumulate_weights=True), *x)
        assert out.shape == (2, 256) and st.call_args.args[2:4] == (None, "cache") and not ex.called
        kw = de.call_args
        assert kw.args[3].tolist() == [4, -1] and kw.kwargs["softcap"] == 30.0 and kw.kwargs["window"] == 0
        assert kw.kwargs["accumulate"] is True and kw.args[0].shape == (2, 4, 64)
        st.reset_mock()
        gdn.forward_attn(_layer(sliding_window_size=128, scaling=0.5), _batch("extend"), *x)
        assert ex.call_args.kwargs["window"] == 128 and ex.call_args.kwargs["scale"] == 0.5 and st.called
        for mode, keep in (("target_verify", True), ("extend", False)):
            st.reset_mock()
            gdn.forward_attn(_layer(), _batch(mode), *x, save_kv_cache=keep)
            assert not st.called
        with pytest.raises(ValueError, match="tree"):
            gdn.forward_attn(_layer(), _batch("target_verify", spec_parents=1), *x)
        with pytest.raises(ValueError, match="save_kv_cache"):
            gdn.forward_attn(_layer(), _batch("decode"), *x, save_kv_cache=False)
        with pytest.raises(ValueError, match="forward mode"):
            gdn.forward_attn(_layer(), _batch("train"), *x)
    assert gdn.forward_attn(_layer(), _batch("decode"), *(t[:0] for t in x)).shape == (0, 256)
