"""GPU tests of the step operators at their edges: codes next to a border, factors that are
not finite, page tables with holes, requests that a plan does not serve, and every kernel that
the dispatch can choose."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("T,H,d", [(4096, 1, 4096), (3000, 1, 5003), (2000, 40, 100), (4000, 600, 5), (300, 1, 40000)])
@pytest.mark.parametrize("group", [0, 128])
def test_codes_are_rounded_quotients(gdn_lib, T, H, d, group):
    """Every code is the fp32 quotient of the value (which the call to fp32 gives) and its scale,
    rounded to nearest even: a product with the scale's reciprocal lands on the other side of a
    border about once in a million values."""
    print("[case] quotients", T, H, d, group, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    x = torch.randn((T, H, d) if H > 1 else (T, d), generator=gen, device="cuda")
    y = gdn_lib.rms_norm(x, out_dtype=F32).view(T, -1).cpu()
    codes, scale = gdn_lib.rms_norm(x, out_dtype=F8, group=group)
    W = y.shape[1]
    step = group or W
    want = torch.stack([p.abs().amax(1) for p in y.split(step, 1)], 1) / 448
    assert torch.equal(scale.cpu(), want)
    quotients = y / want.repeat_interleave(step, 1)[:, :W]
    off = int((codes.view(T, W).cpu().view(torch.uint8) != quotients.to(F8).view(torch.uint8)).sum())
    print(f"  {off} of {y.numel()} codes are another value", flush=True)
    assert off == 0
