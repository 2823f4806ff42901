"""Activations in 8 bits at the small end: what bf16 holds of blocks whose maximum is
near 2^-116.  E4M3's smallest step under a block's scale 2^se is 2^(se - 9) and bf16's
is 2^-133, so se >= -124, which is a maximum of 2^-116 or more, is exact; MXINT8's
step is 2^(se - 6) with se >= -120, exact always."""
import numpy as np
import pytest
import torch

from oracle import act8 as ref
from spectral_domain_quantization_b200 import api

pytestmark = pytest.mark.gpu


def to_bf16(v):
    """float64 values rounded to bf16's nearest, ties to even, down to its subnormals (step 2^-133)."""
    e = np.maximum(np.frexp(v)[1] - 1, -126)
    step = np.exp2(e - 7.0)
    return np.rint(v / step) * step


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("pad", [0, 1])
def test_restore_near_the_smallest_steps(fmt, pad):
    # a row a block maximum 2^-130 .. 2^-110; E4M3's smallest steps, their multiples and
    # values between them
    tops = np.arange(-130, -109)
    X = np.zeros((len(tops), 32 + pad), np.float64)
    X[:, 0] = np.exp2(tops)
    k = np.arange(1, 32)
    X[:, 1:32] = np.exp2(np.maximum(tops - 8, -126))[:, None] * 2.0 ** -9 * np.where(k % 2, k, -k / 2)
    Xd = torch.from_numpy(X.astype(np.float32)).cuda()[:, :32]
    a = api.save_act8(Xd, fmt)
    codes, scales = ref.save(Xd.double().cpu().numpy(), fmt)
    assert np.array_equal(a.codes.cpu().numpy(), codes) and np.array_equal(a.scales.cpu().numpy(), scales)
    held = ref.load(codes, scales, 32, fmt)
    assert np.array_equal(api.restore_act8(a, torch.float32).double().cpu().numpy(), held)
    out = torch.empty((len(tops), 32 + pad), dtype=torch.bfloat16, device="cuda")[:, :32]
    got = api.restore_act8(a, out=out).double().cpu().numpy()
    assert np.array_equal(got, to_bf16(held))
    exact = (got == held).all(1)
    assert exact[tops >= -116].all()
    assert exact.all() if fmt == "mxint8" else not exact[tops < -116].any()
