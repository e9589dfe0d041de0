"""Host-side tests of the step operators at the limits of their arguments (no GPU: no call here
passes validation)."""
import ctypes as ct
from unittest import mock

import pytest
import torch

import hybrid_model_linear_amd as gdn
from hybrid_model_linear_amd import _lib

SHAPE, UNSUP = _lib.GDN_E_SHAPE, _lib.GDN_E_UNSUPPORTED
P = [(k << 44) + 0x10000000 for k in range(1, 14)]      # aligned stand-ins 16 TiB apart, never dereferenced


# ------------------------------------------------------------------ launches
@pytest.mark.parametrize("H,d,most", [(1, 8192, (1 << 24) - 1), (1, 8193, (1 << 22) - 1), (1, 8200, (1 << 22) - 1),
                                      (90, 100, (1 << 22) - 1), (1, 32768, (1 << 22) - 1), (1, 32769, (1 << 24) - 1),
                                      (3000, 3, (1 << 24) - 1), (1, 1, (1 << 24) - 1)])
def test_rms_norm_launches_have_fewer_than_2_32_threads(H, d, most):
    """Rows of 8193 to 32768 values in parts of 8 or more take workgroups of 1024 threads, all others of 256."""
    W = H * d
    args = dict(in_dtype=1, out_dtype=1, H=H, d=d, x=P[0], x_stride=W, out=P[1], out_stride=W, eps=1e-6)
    lib = gdn.load()
    assert lib.gdn_rms_norm(ct.byref(_lib.RmsNormArgs(T=most + 1, **args)), None) == UNSUP
    # one row less: as far as the output that meets the input
    assert lib.gdn_rms_norm(ct.byref(_lib.RmsNormArgs(T=most, **{**args, "out": P[0]})), None) == SHAPE


# ------------------------------------------------------------------ forward_gdn's gated norm
def _gdn_call(z, mode, **layer):
    from types import SimpleNamespace
    layer = dict(dict(num_k_heads=2, num_v_heads=4, head_k_dim=128, head_v_dim=128, A_log=object(), dt_bias=object(), layer_id=3,
                      conv_weight=torch.zeros(1024, 4), norm_weight=torch.zeros(128)), **layer)
    fb = SimpleNamespace(forward_mode=mode, state_pool={3: object()}, conv_pool={3: object()}, state_slots=object(),
                         cu_seqlens=object())
    mixed, ab = torch.zeros(5, 1024, dtype=torch.bfloat16), torch.zeros(5, 4)
    with mock.patch.object(gdn, "conv1d", return_value=mixed) as mc, mock.patch.object(gdn, "conv1d_update", return_value=mixed) as mu, \
            mock.patch.object(gdn, "gdn_gate_inputs", return_value=SimpleNamespace(dtype=mixed.dtype)), \
            mock.patch.object(gdn, "extend", return_value=torch.zeros(5, 4, 128)) as me, \
            mock.patch.object(gdn, "decode", return_value=torch.zeros(5, 4, 128)) as md:
        with pytest.raises(ValueError) as e:
            gdn.forward_gdn(SimpleNamespace(**layer), fb, mixed, ab, ab, z)
    for m in (mc, mu, me, md):
        m.assert_not_called()
    return str(e.value)


@pytest.mark.parametrize("mode", ["extend", "decode"])
def test_forward_gdn_refuses_its_gated_norm_before_any_state_moves(mode):
    """The conv and the layer change their pools in place: whatever the norm behind them would
    refuse is refused in front of them."""
    z = torch.zeros(5, 512, dtype=torch.bfloat16)
    for bad, kw in ((z.float(), {}), (z[:, :256], {}), (z[:4], {}), (z[0], {}), (z.view(5, 4, 128), {}),
                    (torch.zeros(512, 5, dtype=torch.bfloat16).T, {}), (torch.zeros(5, 1024, dtype=torch.bfloat16)[:, ::2], {}),
                    (z[:1].expand(5, 512), {}), (z, dict(norm_weight=None)), (z, dict(norm_weight=torch.zeros(64))),
                    (z, dict(norm_weight=torch.zeros(4, 128))), (z, dict(norm_weight=torch.zeros(256)[::2])),
                    (z, dict(norm_weight=torch.zeros(128, dtype=torch.float16))), (z, dict(norm_eps=-1e-6)),
                    (z, dict(norm_eps=float("nan"))), (z, dict(norm_eps=float("inf"))), (z, dict(norm_eps=1e39))):
        assert "GPU" not in _gdn_call(bad, mode, **kw)
    assert "GPU" in _gdn_call(z, mode)          # (all else in order: a gate in host memory)


# ------------------------------------------------------------------ selective_scan's workspace
@pytest.mark.parametrize("lead", [0, 1, 3])
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_the_workspace_query_takes_what_the_call_takes(lead, out_dtype):
    """Operands at any element: the query's stand-in for the output is aligned whatever they are."""
    from hybrid_model_linear_amd import step
    T, D, S = 3000, 37, 16
    bf = torch.bfloat16
    A, pool = torch.zeros(D, S), torch.zeros(2, D, S)
    cu, slot = torch.tensor([0, T], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    flat = torch.zeros(T * 200, dtype=bf)          # x, dt, B, C and z in one buffer, z highest
    at = lambda k, w: flat[40 * T * k + lead:].as_strided((T, w), (w, 1))  # noqa: E731
    with mock.patch.object(step, "_place", return_value=0), mock.patch.object(step, "_need", lambda name, fn, args, i: fn(ct.byref(args))):
        need = gdn.selective_scan_workspace_size(at(0, D), at(1, D), A, at(2, S), at(3, S), cu, slot, pool, z=at(4, D),
                                                 out_dtype=out_dtype)
    assert need > 0


def test_the_workspace_query_without_tokens():
    from hybrid_model_linear_amd import step
    e = torch.zeros((0, 8), dtype=torch.bfloat16)
    cu, slot = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with mock.patch.object(step, "_place", return_value=0), mock.patch.object(step, "_need", lambda name, fn, args, i: fn(ct.byref(args))):
        assert gdn.selective_scan_workspace_size(e, e, torch.zeros(8, 8), e, e, cu, slot, torch.zeros(1, 8, 8)) == 0


def test_calls_that_skip_the_query_are_not_cut():
    """The binding asks for no workspace where the header says that no sequence is cut; one token
    more, and a sequence can be."""
    import re
    from test_step_host import HEADER
    uncut = int(re.search(r"#define GDN_SELECTIVE_UNCUT (\d+)", open(HEADER).read()).group(1))
    assert _lib.GDN_SELECTIVE_UNCUT == uncut
    query = gdn.load().gdn_selective_scan_workspace_size

    def need(T, N, D, S, hint):
        return query(ct.byref(_lib.SelectiveArgs(
            in_dtype=1, out_dtype=1, N=N, G=1, T=T, D=D, states=S, x=P[0], x_stride=D, dt=P[1], dt_stride=D, B=P[2], B_stride=S, C=P[3],
            C_stride=S, A=P[4], cu_seqlens=P[5], slot=P[6], pool=P[7], num_slots=4, out=P[8], out_stride=D, max_seqlen=hint)))
    for S in (8, 16, 32, 64, 128):
        for D in (8, 100, 4096, 1 << 20):
            assert all(need(T, N, D, S, h) == 0 for T in (1, 33, uncut) for N in (1, 3) for h in (0, T, 1 << 30)), (S, D)
    assert need(uncut + 1, 1, 64, 16, 0) > 0


# ------------------------------------------------------------------ extents
def test_extents_past_62_bits_are_refused():
    """A row operand whose last element lies past 2^62 bytes would wrap around the overlap checks."""
    lib = gdn.load()
    base = dict(in_dtype=1, out_dtype=1, N=0, G=1, T=1 << 30, D=64, states=16, x=P[0], x_stride=64, dt=P[1], dt_stride=64, B=P[2],
                B_stride=16, C=P[3], C_stride=16, A=P[4], pool=P[5], num_slots=4, out=P[6], out_stride=64)
    call = lambda **kw: lib.gdn_selective_scan(ct.byref(_lib.SelectiveArgs(**{**base, **kw})), None)  # noqa: E731
    assert call() == _lib.GDN_OK
    for kw in (dict(x_stride=1 << 40), dict(out_stride=1 << 40), dict(out_stride=1 << 40, out=P[0]), dict(B_stride=1 << 33),
               dict(num_slots=1 << 52), dict(num_slots=1 << 62)):
        assert call(**kw) == SHAPE, kw
    norm = dict(in_dtype=1, out_dtype=1, T=(1 << 24) - 1, H=1, d=8, x=P[0], x_stride=8, out=P[1], out_stride=8, eps=1e-6)
    for kw in (dict(x_stride=1 << 39), dict(out_stride=1 << 39), dict(residual=P[2], residual_stride=1 << 40)):
        assert lib.gdn_rms_norm(ct.byref(_lib.RmsNormArgs(**{**norm, **kw})), None) == SHAPE, kw
