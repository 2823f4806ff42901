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


@pytest.mark.parametrize("cols", [40, 1000, 1001, 4096, 9001, 14336, 33000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sums_past_float32(cols, dtype):
    # what the header says of such rows, and nothing of it in the others
    x, dy, w, b = data(8, cols, seed=71)
    X, dY, w, b = mat(x, dtype), mat(dy, dtype), w.cuda(), b.cuda()
    rest = torch.tensor([0, 1, 3, 5, 7], device="cuda")
    clean = api.layer_norm_fwd(X, w, b)
    dclean = api.layer_norm_bwd(dY, X, clean.mean, clean.rstd, w)
    X[2] *= 1e25                          # squared deviations
    X[4] = 3e38                           # the sum of the values
    X[6] = -1e35
    X[6, ::2] = 1e35                      # squares again, of a row whose sum stays
    r = api.layer_norm_fwd(X, w, b)
    assert torch.equal(r.Y[rest], clean.Y[rest]) and torch.equal(r.rstd[rest], clean.rstd[rest])
    assert torch.isnan(r.Y[4]).all() and not torch.isfinite(r.mean[4])
    for k in (2, 6):
        assert float(r.rstd[k]) == 0 and torch.equal(r.Y[k], b.to(r.Y.dtype))
    dX = api.layer_norm_bwd(dY, X, r.mean, r.rstd, w)[0]
    assert torch.equal(dX[rest], dclean[0][rest])
    assert not dX[2].any() and not dX[6].any() and torch.isnan(dX[4]).all()
