"""The layer norm at the ends of float32's range.

Tolerances: those of tests/test_gpu_layer_norm.py."""
import pytest
import torch

from spectral_domain_quantization_b200 import api

from test_gpu_layer_norm import check_bwd, check_fwd, data, mat, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [40, 1000, 1001, 4096, 9001, 14336, 33000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_row_and_smallest_eps(cols, dtype):
    # rstd is 10^20: its square is past float32, the gradient is not
    x, dy, w, b = data(6, cols, seed=70)
    x[1] = 0
    x[4] = 0
    X, dY, w, b = mat(x, dtype), mat(dy, dtype), w.cuda(), b.cuda()
    r = api.layer_norm_fwd(X, w, b, eps=1e-40)
    eps = float(torch.tensor(1e-40, dtype=torch.float32))
    check_fwd(r, X, w, b, eps)
    assert torch.equal(r.Y[1], b.to(r.Y.dtype)) and np64(r.rstd)[1] > 0.99e20
    got = api.layer_norm_bwd(dY, X, r.mean, r.rstd, w)
    assert torch.isfinite(got[0]).all()
    check_bwd(got, dY, np64(X), r.mean, r.rstd, w)
