"""A forward norm in place at the widths whose rows start anywhere and are too wide to
be shifted (32762 to 32768 columns): each element is read through the row's image and
written by itself, next to rows that other CTAs have on their way."""
import pytest
import torch

from spectral_domain_quantization_b200 import api

from test_gpu_layer_norm import check_fwd, data, mat

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols,offset,pad", [(32762, 0, 0), (32763, 5, 0), (32765, 1, 2), (32767, 0, 0), (32768, 1, 1),
                                             (32768, 3, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_in_place(cols, offset, pad, dtype):
    x, _, w, b = data(150, cols, seed=90)
    w, b = w.cuda(), b.cuda()
    apart = mat(x, dtype, pad, offset)
    want = api.layer_norm_fwd(mat(x, dtype, pad, offset), w, b, save="mxint8", out=apart)
    check_fwd(want, mat(x, dtype, pad, offset), w, b)
    Y = mat(x, dtype, pad, offset)
    got = api.layer_norm_fwd(Y, w, b, save="mxint8", out=Y)
    assert torch.equal(Y, want.Y) and torch.equal(got.mean, want.mean) and torch.equal(got.rstd, want.rstd)
    assert torch.equal(got.saved.codes, want.saved.codes) and torch.equal(got.saved.scales, want.saved.scales)
