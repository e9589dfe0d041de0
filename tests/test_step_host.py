"""Host-side tests of the step operators (no GPU): struct layouts, the refusals of the C ABI
(nothing is launched: every call fails validation first) and of the binding."""
import ctypes as ct
import os
import subprocess
import tempfile

import pytest
import torch

import hybrid_model_linear_amd as gdn
from hybrid_model_linear_amd import _lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdn.h")
OK, NULL, SHAPE, DTYPE, UNSUP = (_lib.GDN_OK, _lib.GDN_E_NULL, _lib.GDN_E_SHAPE, _lib.GDN_E_DTYPE,
                                 _lib.GDN_E_UNSUPPORTED)
P = [0x10000000 * k for k in range(1, 24)]          # aligned stand-ins far apart, never dereferenced
NAN, INF = float("nan"), float("inf")


def test_struct_layouts_match_header():
    structs = {"gdn_selective_args": _lib.SelectiveArgs, "gdn_rms_norm_args": _lib.RmsNormArgs,
               "gdn_plan_pages_args": _lib.PlanPagesArgs, "gdn_release_pages_args": _lib.ReleasePagesArgs}
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


# ------------------------------------------------------------------ C ABI
def _selective(**kw):
    base = dict(in_dtype=1, out_dtype=1, N=3, G=2, T=7, D=64, states=16, dt_softplus=1, x=P[0], x_stride=64, dt=P[1],
                dt_stride=64, B=P[2], B_stride=32, C=P[3], C_stride=32, z=P[4], z_stride=128, A=P[5], D_skip=P[6],
                dt_bias=P[7], cu_seqlens=P[8], slot=P[9], has_init=P[10], pool=P[11], num_slots=4, out=P[12], out_stride=64)
    base.update(kw)
    return _lib.SelectiveArgs(**base)


SELECTIVE = [
    (dict(in_dtype=2), DTYPE), (dict(out_dtype=2), DTYPE), (dict(in_dtype=-1), DTYPE), (dict(N=-1), SHAPE), (dict(G=0), SHAPE),
    (dict(G=3), SHAPE), (dict(D=0), SHAPE), (dict(D=1 << 25), SHAPE), (dict(states=4), UNSUP), (dict(states=24), UNSUP),
    (dict(states=256), UNSUP), (dict(A=None), NULL), (dict(pool=None), NULL), (dict(slot=None), NULL), (dict(x=None), NULL),
    (dict(dt=None), NULL), (dict(B=None), NULL), (dict(C=None), NULL), (dict(out=None), NULL), (dict(x_stride=63), SHAPE),
    (dict(dt_stride=63), SHAPE), (dict(B_stride=31), SHAPE), (dict(C_stride=31), SHAPE), (dict(z_stride=63), SHAPE),
    (dict(out_stride=63), SHAPE), (dict(x=P[0] + 1), SHAPE), (dict(in_dtype=0, dt=P[1] + 2), SHAPE), (dict(A=P[5] + 4), SHAPE),
    (dict(pool=P[11] + 8), SHAPE), (dict(slot=P[9] + 2), SHAPE), (dict(out=P[0]), SHAPE), (dict(out=P[4] + 64), SHAPE),
    (dict(out=P[11] + 1024), SHAPE), (dict(out=P[2]), SHAPE), (dict(num_slots=-1), SHAPE), (dict(max_seqlen=-1), SHAPE),
]


@pytest.mark.parametrize("kw,want", SELECTIVE + [
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(cu_seqlens=None), NULL), (dict(cu_seqlens=P[8] + 1), SHAPE),
    (dict(has_init=P[10] + 2), SHAPE), (dict(N=1 << 24), UNSUP)])
def test_selective_scan_refusals(kw, want):
    lib = gdn.load()
    assert lib.gdn_selective_scan(ct.byref(_selective(**kw)), None) == want
    assert lib.gdn_selective_scan_workspace_size(ct.byref(_selective(**kw))) == -want


@pytest.mark.parametrize("kw,want", SELECTIVE[:-1] + [(dict(T=8), SHAPE), (dict(T=3, N=4), SHAPE)])
def test_selective_update_refusals(kw, want):
    kw = {**dict(T=3, cu_seqlens=None, has_init=None), **kw}
    if kw.get("N") == -1:
        kw["T"] = -1
    assert gdn.load().gdn_selective_update(ct.byref(_selective(**kw)), None) == want


def test_empty_calls_launch_nothing():
    lib = gdn.load()
    assert lib.gdn_selective_scan(ct.byref(_selective(N=0, T=0, slot=None, cu_seqlens=None)), None) == OK
    assert lib.gdn_selective_update(ct.byref(_selective(N=0, T=0, x=None, out=None)), None) == OK
    assert lib.gdn_rms_norm(ct.byref(_norm(T=0, x=None, out=None)), None) == OK
    assert lib.gdn_release_pages(ct.byref(_release(N=0, keep=None)), None) == OK
    for fn in (lib.gdn_selective_scan, lib.gdn_selective_update, lib.gdn_rms_norm, lib.gdn_plan_pages, lib.gdn_release_pages):
        assert fn(None, None) == NULL
    assert lib.gdn_selective_scan_workspace_size(None) == -NULL


def _norm(**kw):
    base = dict(in_dtype=1, out_dtype=2, weight_dtype=1, residual_dtype=1, T=5, H=2, d=100, x=P[0], x_stride=200, gate=None,
                gate_stride=0, residual=P[2], residual_stride=200, weight=P[3], out=P[4], out_stride=200, scale=P[5],
                eps=1e-6, offset=0.0, gate_first=0, group=64)
    base.update(kw)
    return _lib.RmsNormArgs(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(in_dtype=2), DTYPE), (dict(out_dtype=3), DTYPE), (dict(weight_dtype=2), DTYPE), (dict(residual_dtype=2), DTYPE),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(H=0), SHAPE), (dict(H=8193), SHAPE), (dict(d=0), SHAPE),
    (dict(d=1 << 20), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE), (dict(eps=INF), SHAPE), (dict(offset=NAN), SHAPE),
    (dict(group=32), UNSUP), (dict(group=-64), UNSUP), (dict(gate=P[1], gate_stride=200), UNSUP), (dict(x=None), NULL),
    (dict(out=None), NULL), (dict(scale=None), NULL), (dict(x_stride=199), SHAPE), (dict(residual_stride=100), SHAPE),
    (dict(out_stride=199), SHAPE), (dict(residual=None, gate=P[1], gate_stride=199), SHAPE), (dict(x=P[0] + 1), SHAPE),
    (dict(residual=P[2] + 1), SHAPE), (dict(weight=P[3] + 1), SHAPE), (dict(out_dtype=1, out=P[4] + 1), SHAPE),
    (dict(scale=P[5] + 2), SHAPE), (dict(out=P[0] + 1000), SHAPE), (dict(residual=P[0]), SHAPE), (dict(out=P[2]), SHAPE),
    (dict(scale=P[4] + 900), SHAPE), (dict(weight=P[5] + 64), SHAPE), (dict(T=1 << 24), UNSUP)])
def test_rms_norm_refusals(kw, want):
    if kw.get("T") == 1 << 24:      # (rows apart at this size)
        kw = {**kw, "H": 1, "d": 1, "x_stride": 1, "residual": None, "out_stride": 1}
    assert gdn.load().gdn_rms_norm(ct.byref(_norm(**kw)), None) == want


def _plan(**kw):
    base = dict(pool=P[0], capacity=100, N=3, page=16, T=20, held=P[1], new_len=P[2], start=None, block_table=P[3],
                table_stride=8, table_width=8, cu_seqlens=P[4], cache_len=P[5], kv_len=P[6], slots=P[7], positions=P[8], seq=P[9])
    base.update(kw)
    return _lib.PlanPagesArgs(**base)


def _release(**kw):
    base = dict(pool=P[0], capacity=100, N=3, page=16, keep=P[1], held=P[2], block_table=P[3], table_stride=8, table_width=8)
    base.update(kw)
    return _lib.ReleasePagesArgs(**base)


POOL = [(dict(capacity=-1), SHAPE), (dict(capacity=1 << 31), SHAPE), (dict(N=-1), SHAPE), (dict(N=65536), SHAPE),
        (dict(page=0), SHAPE), (dict(page=(1 << 30) + 1), SHAPE), (dict(table_width=0), SHAPE), (dict(table_stride=7), SHAPE),
        (dict(pool=None), NULL), (dict(block_table=None), NULL), (dict(held=None), NULL), (dict(pool=P[0] + 2), SHAPE),
        (dict(block_table=P[3] + 1), SHAPE), (dict(held=P[1] + 1), SHAPE), (dict(block_table=P[0] + 400), SHAPE)]


@pytest.mark.parametrize("kw,want", POOL + [
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(new_len=None), NULL), (dict(cu_seqlens=None), NULL),
    (dict(cache_len=None), NULL), (dict(kv_len=None), NULL), (dict(slots=P[7] + 4), SHAPE), (dict(positions=P[8] + 2), SHAPE),
    (dict(seq=P[9] + 2), SHAPE), (dict(start=P[9] + 2), SHAPE), (dict(cache_len=P[1]), SHAPE), (dict(kv_len=P[2] + 8), SHAPE),
    (dict(cu_seqlens=P[4], cache_len=P[4] + 12), SHAPE), (dict(slots=P[8] - 152), SHAPE), (dict(start=P[6]), SHAPE)])
def test_plan_pages_refusals(kw, want):
    assert gdn.load().gdn_plan_pages(ct.byref(_plan(**kw)), None) == want


@pytest.mark.parametrize("kw,want", POOL + [(dict(keep=None), NULL), (dict(keep=P[1] + 2), SHAPE), (dict(keep=P[0] + 8), SHAPE)])
def test_release_pages_refusals(kw, want):
    assert gdn.load().gdn_release_pages(ct.byref(_release(**kw)), None) == want


# ------------------------------------------------------------------ binding
def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    A, B = torch.zeros(16, 8), torch.zeros(4, 8, dtype=torch.bfloat16)
    cu, slot, pool = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 16, 8)
    with pytest.raises(ValueError, match="GPU"):
        gdn.selective_scan(x, x, A, B, B, cu, slot, pool)
    with pytest.raises(ValueError, match="one token per row"):
        gdn.selective_update(x, x, A, B, B, slot, pool)
    with pytest.raises(ValueError, match=r"\[T, D\]"):
        gdn.selective_scan(x[0], x, A, B, B, cu, slot, pool, out=x)
    with pytest.raises(ValueError, match="out_dtype"):
        gdn.selective_scan(x, x, A, B, B, cu, slot, pool, out=x, out_dtype=torch.float32)
    with pytest.raises(ValueError, match="GPU"):
        gdn.rms_norm(x)
    with pytest.raises(ValueError, match=r"\[T, d\]"):
        gdn.rms_norm(x[0])
    with pytest.raises(ValueError, match="bf16 or fp32"):
        gdn.rms_norm(x.half())
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        gdn.rms_norm(x, out_dtype=torch.float16)
    for group in (32, 1 << 32):
        with pytest.raises(ValueError, match="group must be"):
            gdn.rms_norm(x, out_dtype=torch.float8_e4m3fn, group=group)
    with pytest.raises(ValueError, match="scale goes with"):
        gdn.rms_norm(x, scale=torch.zeros(4, 1))
    with pytest.raises(ValueError, match="scale must be"):
        gdn.rms_norm(x, out_dtype=torch.float8_e4m3fn, scale=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="GPU"):
        gdn.page_pool(5, device="cpu")
    with pytest.raises(ValueError, match="int32 vector"):
        gdn.PagePool(torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="int32 vector"):
        gdn.PagePool(torch.zeros(9))


def test_pages_refuse_numbers_that_do_not_fit():
    pool = object.__new__(gdn.PagePool)
    t, e = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pool._state, pool._capacity = torch.zeros(9, dtype=torch.int32), 7
    from unittest import mock
    from hybrid_model_linear_amd import step
    with mock.patch.object(step, "_place", return_value=0):
        for page, tokens in ((0, 4), ((1 << 32) + 16, 4), (16, -1), (16, 1 << 31)):
            with pytest.raises(ValueError):
                gdn.plan_pages(pool, t, e, e, page, tokens)
        for page in (0, (1 << 32) + 16):
            with pytest.raises(ValueError):
                gdn.release_pages(pool, t, e, e, page)


def test_shape_helpers():
    from hybrid_model_linear_amd import step
    bf = torch.bfloat16
    p = torch.zeros(5, 40, dtype=bf)
    assert step._grouped(p[:, 8:40].unflatten(1, (2, 16)), "B", 5, 16, bf) == (40, 2)
    assert step._grouped(p[:, 8:24], "B", 5, 16, bf) == (40, 1)
    assert step._matrix(p[:1, 3:9], "x", (1, 6), bf) == 6
    assert step._token_rows(p[:, 8:].unflatten(1, (4, 8)), "x", torch.Size((5, 4, 8))) == 40
    for bad in (lambda: step._grouped(p.unflatten(1, (2, 20))[:, :, :16], "B", 5, 16, bf),
                lambda: step._grouped(p.unflatten(1, (2, 20)), "B", 5, 16, bf),
                lambda: step._matrix(p.T, "x", (40, 5), bf), lambda: step._matrix(p, "x", (5, 40), torch.float32),
                lambda: step._matrix(p[:, ::2], "x", (5, 20), bf),
                lambda: step._token_rows(p.unflatten(1, (4, 10))[:, :, :8], "x", torch.Size((5, 4, 8)))):
        with pytest.raises(ValueError):
            bad()
