"""The layer norm's backward pass where a thread has columns that are not the row's:
widths that fill the layout of the threads in part only.  What such columns read
stands for nothing, so no value of a row, its statistics or the weight may turn it
into a part of the row's sums.

Tolerances: those of tests/test_gpu_layer_norm.py."""
import numpy as np
import pytest
import torch

from oracle import norm
from spectral_domain_quantization_b200 import api

from test_gpu_layer_norm import check_bwd, data, mat, np64

pytestmark = pytest.mark.gpu

# every spread of rows over threads, whole and ragged
WIDTHS = [40, 64, 100, 200, 264, 500, 1000, 1001, 1027, 1100, 2000, 4001, 4096, 4104, 9000, 9001, 12000, 14335, 17000,
          20001]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind,gdtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("mxint8", "bf16"),
                                         ("mxfp8", "f32")])
@pytest.mark.parametrize("lie", ["alike", "differently"])
def test_large_constant_row(cols, kind, gdtype, lie):
    # 2^109 in every column and eps 1e-12: rstd is 10^6, and mean * rstd is past
    # float32's range while every xh is 0
    x, dy, w, _ = data(7, cols, seed=60)
    x[2] = 2.0 ** 109
    x[5] = -2.0 ** 109
    a8 = kind.startswith("mx")
    X, dY, w = mat(x, "bf16" if a8 else kind), mat(dy, gdtype, 0 if lie == "alike" else 1), w.cuda()
    r = api.layer_norm_fwd(X, w, eps=1e-12, save=kind if a8 else None)
    m = np64(r.mean)
    assert m[2] == 2.0 ** 109 and m[5] == -2.0 ** 109 and abs(m[2] * np64(r.rstd)[2]) > 3.5e38
    x64 = np64(X if not a8 else api.restore_act8(r.saved, torch.float32))
    got = api.layer_norm_bwd(dY, X if not a8 else r.saved, r.mean, r.rstd, w)
    assert all(torch.isfinite(t).all() for t in got)
    check_bwd(got, dY, x64, r.mean, r.rstd, w)


@pytest.mark.parametrize("cols", [8200, 8449, 9001, 10239, 12281, 12288, 12320, 13000, 14335, 14336, 16377, 16384])
@pytest.mark.parametrize("kind,gdtype", [("bf16", "bf16"), ("mxint8", "bf16"), ("mxint8", "f32"), ("mxfp8", "f32")])
def test_long_rows(cols, kind, gdtype):
    # rows of one CTA and of a cluster, fewer of them than an SM holds and more
    for rows in (1, 5, 400):
        x, dy, w, _ = data(rows, cols, seed=62)
        a8 = kind.startswith("mx")
        X, dY, w = mat(x, "bf16" if a8 else kind), mat(dy, gdtype), w.cuda()
        r = api.layer_norm_fwd(X, w, save=kind if a8 else None)
        given = r.saved if a8 else X
        x64 = np64(X if not a8 else api.restore_act8(r.saved, torch.float32))
        got = api.layer_norm_bwd(dY, given, r.mean, r.rstd, w)
        check_bwd(got, dY, x64, r.mean, r.rstd, w)
        # over dY, and one output alone: the same values
        over = dY.clone()
        part = api.layer_norm_bwd(over, given, r.mean, r.rstd, w, want_db=False, out=over)
        assert torch.equal(over, got[0]) and torch.equal(part[1], got[1]) and part[2] is None
