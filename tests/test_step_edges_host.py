"""Host-side tests of the step operators at the limits of their arguments (no GPU: no call here
passes validation)."""
import ctypes as ct

import pytest

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
