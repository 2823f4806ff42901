"""The layer norm on the GPU against float64.

Tolerances.  u = 2^-24 is float32's half step, uo the output type's
(finfo.eps / 2).  A sum of n terms spread over threads passes through at most D
additions, so it is off by at most D u times the sum of the magnitudes.

Forward: d = (x - m0) - m1 is rounded twice, and the mean m0 + m1 is off by at
most D u mean|x - m0| <= D u / rstd, so xh is off by (2 |xh| + D) u plus rstd's
relative error ((D + 2) / 2 + 4) u, and y = xh w + b adds one rounding:
  |y - y*| <= uo |y*| + u (|w| ((D / 2 + 8) |xh| + D) + |y*|).
Backward (mean and rstd given): xh has two roundings, c1 = mean(g xh) and c2 =
mean(g) a sum each:
  |dx - dx*| <= uo |dx*| + u rstd (4 |g| + (D + 6) mean|g| + |xh| (D + 12) mean|g xh|)
  |dw - dw*| <= u (D2 + 4) sum|dy xh|,  |db - db*| <= u D2 sum|dy|
with D2 the additions a column's sum passes through.  D <= cols / 1024 + 64 and
D2 <= rows / 16 + 64 for every kernel here."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import act8 as act8_ref
from oracle import norm
from spectral_domain_quantization_b200 import api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def half_step(t):
    return torch.finfo(t.dtype).eps / 2


def mat(x, dtype, pad=0, offset=0):
    rows, cols = x.shape
    buf = torch.zeros(offset + rows * (cols + pad), dtype=DT[dtype], device="cuda")
    v = buf[offset:].view(rows, cols + pad)[:, :cols]
    v.copy_(x)
    return v


def data(rows, cols, seed=0, shift=0.0):
    g = torch.Generator().manual_seed(7 * rows + cols + seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(torch.randn((rows, 1), generator=g)) + shift
    dy = torch.randn((rows, cols), generator=g) * 0.1
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    b = 0.2 * torch.randn(cols, generator=g)
    return x, dy, w, b


def np64(t):
    return t.double().cpu().numpy()


def check_fwd(r, X, w, b, eps=1e-5):
    n = X.shape[1]
    D = n / 1024 + 64
    w64 = np.ones(n) if w is None else np64(w)
    b64 = None if b is None else np64(b)
    y, mean, rstd = norm.forward(np64(X), w64, b64, eps)
    xh = (np64(X) - mean[:, None]) * rstd[:, None]
    tol = half_step(r.Y) * np.abs(y) + U * (np.abs(w64) * ((D / 2 + 8) * np.abs(xh) + D) + np.abs(y))
    assert np.all(np.abs(np64(r.Y) - y) <= tol)
    if r.mean is not None:
        assert np.all(np.abs(np64(r.mean) - mean) <= U * (np.abs(mean) + (D + 2) / rstd))
        assert np.all(np.abs(np64(r.rstd) - rstd) <= U * (D / 2 + 8) * rstd)


def check_bwd(got, dY, x64, mean, rstd, w):
    rows, n = dY.shape
    D, D2 = n / 1024 + 64, rows / 16 + 64
    dX, dw, db = got
    w64 = np.ones(n) if w is None else np64(w)
    m64, r64 = np64(mean), np64(rstd)
    want = norm.backward(np64(dY), x64, m64, r64, w64)
    xh = (x64 - m64[:, None]) * r64[:, None]
    g = np64(dY) * w64
    if dX is not None:
        tol = half_step(dX) * np.abs(want[0]) + U * r64[:, None] * (
            4 * np.abs(g) + (D + 6) * np.abs(g).mean(1, keepdims=True)
            + np.abs(xh) * (D + 12) * np.abs(g * xh).mean(1, keepdims=True))
        assert np.all(np.abs(np64(dX) - want[0]) <= tol)
    if dw is not None:
        assert np.all(np.abs(np64(dw) - want[1]) <= U * (D2 + 4) * np.abs(np64(dY) * xh).sum(0))
    if db is not None:
        assert np.all(np.abs(np64(db) - want[2]) <= U * D2 * np.abs(np64(dY)).sum(0))


# rows, cols, row padding, offset of the first element
SHAPES = [(1, 1, 0, 0), (3, 1, 0, 0), (1, 4096, 0, 0), (2, 7, 0, 0), (37, 32, 0, 0), (5, 64, 0, 0), (9, 65, 0, 0),
          (300, 200, 0, 0), (11, 256, 0, 0), (70, 257, 0, 0), (33, 1000, 24, 0), (6, 1003, 0, 0), (5, 1024, 1, 1),
          (4, 1027, 0, 0), (3, 2048, 0, 0), (3, 2056, 8, 8), (5, 4095, 0, 0), (700, 4096, 0, 0), (3, 4097, 0, 0),
          (40, 5000, 0, 0), (9, 8200, 0, 0), (3, 14336, 0, 0), (2, 16391, 0, 0), (2, 32768, 0, 0), (2, 32765, 0, 0), (9, 16383, 0, 0), (20, 8190, 0, 3), (2, 32771, 0, 0),
          (1, 40000, 0, 0), (2000, 72, 0, 0), (5000, 33, 0, 0), (700, 57, 0, 0), (90, 121, 0, 5), (301, 255, 0, 1), (40, 510, 2, 0),
          (77, 2046, 0, 0), (19, 128, 4, 4)]


@pytest.mark.parametrize("dtype,wdtype,out", [("bf16", "f32", "bf16"), ("f32", "f32", "f32"), ("bf16", "bf16", "f32"),
                                              ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_forward(rows, cols, pad, offset, dtype, wdtype, out):
    x, _, w, b = data(rows, cols)
    X, w, b = mat(x, dtype, pad, offset), w.to(DT[wdtype]).cuda(), b.to(DT[wdtype]).cuda()
    fmt = "mxint8" if wdtype == "f32" else "mxfp8"
    r = api.layer_norm_fwd(X, w, b, out_dtype=DT[out], save=fmt)
    check_fwd(r, X, w, b)
    # the 8-bit copy is the one save_act8 makes
    a = api.save_act8(X, fmt)
    assert torch.equal(a.codes, r.saved.codes) and torch.equal(a.scales, r.saved.scales)
    assert torch.equal(a.amax.max(), r.saved.amax.max())
    # without the copy and the statistics: the same Y, here into a strided tensor
    buf = torch.full((rows, cols + 9), 7.0, dtype=DT[out], device="cuda")
    plain = api.layer_norm_fwd(X, w, b, stats=False, out=buf[:, 8:cols + 8])
    assert plain.mean is None and plain.rstd is None and plain.saved is None
    check_fwd(plain, X, w, b)
    assert (buf[:, :8] == 7).all() and (buf[:, cols + 8:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "f32", "mxint8", "mxfp8"])
@pytest.mark.parametrize("gdtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_backward(rows, cols, pad, offset, gdtype, out, kind):
    x, dy, w, b = data(rows, cols, seed=1)
    X = mat(x, "bf16" if kind == "bf16" else "f32", pad, offset)
    dY, w = mat(dy, gdtype, pad, offset), w.cuda()
    r = api.layer_norm_fwd(X, w, save=kind if kind in act8_ref.FORMATS else None)
    given = X if r.saved is None else r.saved
    x64 = np64(X) if r.saved is None else act8_ref.load(*act8_ref.save(np64(X), kind), cols, kind)
    got = api.layer_norm_bwd(dY, given, r.mean, r.rstd, w, out_dtype=DT[out])
    check_bwd(got, dY, x64, r.mean, r.rstd, w)
    # the same sums on every call
    again = api.layer_norm_bwd(dY, given, r.mean, r.rstd, w, out_dtype=DT[out])
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("cols", [40, 515, 4096, 6000, 33000])
def test_parts_of_the_backward(cols):
    x, dy, w, _ = data(50, cols, seed=2)
    X, dY, w = mat(x, "bf16"), mat(dy, "bf16"), w.cuda()
    r = api.layer_norm_fwd(X)
    full = api.layer_norm_bwd(dY, X, r.mean, r.rstd, w)
    for want in [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)]:
        got = api.layer_norm_bwd(dY, X, r.mean, r.rstd, w, want_dx=want[0], want_dw=want[1], want_db=want[2])
        for f, g, on in zip(full, got, want):
            assert (g is None) == (not on) and (g is None or torch.equal(f, g))
    check_bwd(api.layer_norm_bwd(dY, X, r.mean, r.rstd), dY, np64(X), r.mean, r.rstd, None)


def test_many_rows():
    x, dy, w, b = data(20000, 96, seed=3)
    X, dY, w, b = mat(x, "bf16"), mat(dy, "f32"), w.cuda(), b.cuda()
    r = api.layer_norm_fwd(X, w, b)
    check_fwd(r, X, w, b)
    check_bwd(api.layer_norm_bwd(dY, X, r.mean, r.rstd, w), dY, np64(X), r.mean, r.rstd, w)


@pytest.mark.parametrize("cols", [64, 1000, 4096, 6001, 33000])
@pytest.mark.parametrize("shift", [1000.0, -30000.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_offset(cols, shift, dtype):
    # a row far from zero: no cancellation in the variance, no bits lost in the mean
    x, _, w, b = data(4, cols, seed=4, shift=shift)
    X = mat(x, dtype)
    check_fwd(api.layer_norm_fwd(X, w.cuda(), b.cuda(), out_dtype=torch.float32), X, w, b)


@pytest.mark.parametrize("cols", [64, 255, 1000, 4096, 6000, 33000])
def test_special_rows(cols):
    x, dy, w, b = data(6, cols, seed=5)
    X, dY, w, b = mat(x, "f32"), mat(dy, "f32"), w.cuda(), b.cuda()
    clean = api.layer_norm_fwd(X, w, b)
    cg = api.layer_norm_bwd(dY, X, clean.mean, clean.rstd, w)[0]
    X[1, cols // 2] = float("nan")
    X[3, 0] = float("inf")
    X[4] = 2.5                        # constant: y = b
    r = api.layer_norm_fwd(X, w, b, save="mxint8")
    for k in (0, 2, 5):
        assert torch.equal(r.Y[k], clean.Y[k])
    assert torch.isnan(r.Y[1]).all() and torch.isnan(r.Y[3]).all()
    assert torch.equal(r.Y[4], b)
    d = api.layer_norm_bwd(dY, X, r.mean, r.rstd, w)[0]
    for k in (0, 2, 5):
        assert torch.equal(d[k], cg[k])
    assert torch.isnan(d[1]).all() and torch.isfinite(d[4]).all()
    z = api.layer_norm_bwd(dY, r.saved, r.mean, r.rstd, w)[0]
    assert torch.isnan(z[1]).all() and torch.isfinite(z[0]).all() and torch.isfinite(z[5]).all()
    # eps = 0 on a constant row is a division by zero, in that row alone
    r = api.layer_norm_fwd(X, w, b, eps=0.0)
    assert torch.isnan(r.Y[4]).all() and torch.isfinite(r.Y[0]).all()


@pytest.mark.parametrize("cols", [48, 1000, 3001, 4096, 9000, 33000])
def test_in_place(cols):
    x, dy, w, b = data(300, cols, seed=6)
    X, dY, w, b = mat(x, "bf16"), mat(dy, "bf16"), w.cuda(), b.cuda()
    r = api.layer_norm_fwd(X, w, b, save="mxfp8")
    want = api.layer_norm_bwd(dY, X, r.mean, r.rstd, w)
    X2, dY2 = X.clone(), dY.clone()
    r2 = api.layer_norm_fwd(X2, w, b, save="mxfp8", out=X2)
    assert torch.equal(X2, r.Y) and torch.equal(r2.saved.codes, r.saved.codes) and torch.equal(r2.rstd, r.rstd)
    got = api.layer_norm_bwd(dY2, X, r.mean, r.rstd, w, out=dY2)
    assert torch.equal(dY2, want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_no_rows():
    X = torch.zeros((0, 40), device="cuda")
    w = torch.ones(40, device="cuda")
    r = api.layer_norm_fwd(X, w, w, save="mxint8")
    assert r.Y.shape == (0, 40) and r.mean.shape == (0,) and not r.saved.amax.any()
    dX, dw, db = api.layer_norm_bwd(X, X, r.mean, r.rstd, w)
    assert dX.shape == (0, 40) and not dw.any() and not db.any()
    assert not api.layer_norm_bwd(X, r.saved, r.mean, r.rstd, w)[1].any()


def test_gradient_against_differences():
    # float32 all through: the directional derivative of sum(dY Y) by central differences
    x, dy, w, b = data(4, 96, seed=8)
    X, dY, w, b = mat(x, "f32"), mat(dy, "f32"), w.cuda(), b.cuda()
    r = api.layer_norm_fwd(X, w, b)
    dX, dw, db = api.layer_norm_bwd(dY, X, r.mean, r.rstd, w)
    g = torch.Generator().manual_seed(9)
    for arr, grad, at in ((X, dX, 0), (w, dw, 1), (b, db, 2)):
        v = torch.randn(arr.shape, generator=g).cuda()
        v = v / v.norm()
        h = 0.02
        args = [[X, w, b], [X, w, b]]
        args[0][at], args[1][at] = arr + h * v, arr - h * v
        y = [api.layer_norm_fwd(*a).Y.double() for a in args]
        num = float((dY.double() * (y[0] - y[1])).sum()) / (2 * h)
        want = float((grad.double() * v.double()).sum())
        # truncation h^2 / 6 of the third derivative (|x| / sigma < 4 here), and
        # float32's 400 outputs of size up to 8 with 70 u each, over 2 h
        tol = 1e-3 * float(grad.norm()) + 70 * U * 8 * float(dY.abs().sum()) / (2 * h)
        assert abs(num - want) <= tol


def test_other_stream_and_two_graphs():
    x, dy, w, b = data(500, 1000, seed=10)
    X, dY, w, b = mat(x, "bf16"), mat(dy, "bf16"), w.cuda(), b.cuda()

    def step(scale=1.0):
        r = api.layer_norm_fwd(X, w, b, save="mxint8")
        return [r.Y, r.mean, r.rstd] + list(api.layer_norm_bwd(dY, r.saved, r.mean, r.rstd, w))

    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    # two captured graphs replayed at once, between eager calls
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    step()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(want, o))


def test_first_call_in_a_capture():
    # a fresh process whose first call of each kernel is captured
    code = (
        "import torch\n"
        "from spectral_domain_quantization_b200 import api\n"
        "X = torch.randn(64, 1000, device='cuda').bfloat16()\n"
        "w = torch.ones(1000, device='cuda')\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    r = api.layer_norm_fwd(X, w, save='mxint8')\n"
        "    d = api.layer_norm_bwd(X, r.saved, r.mean, r.rstd, w)\n"
        "    q = api.quantize_fp4_act8(r.saved, 'mx', axis=0)\n"
        "g.replay()\n"
        "torch.cuda.synchronize()\n"
        "r2 = api.layer_norm_fwd(X, w, save='mxint8')\n"
        "d2 = api.layer_norm_bwd(X, r2.saved, r2.mean, r2.rstd, w)\n"
        "q2 = api.quantize_fp4_act8(r2.saved, 'mx', axis=0)\n"
        "assert torch.equal(r.Y, r2.Y) and all(torch.equal(a, b) for a, b in zip(d, d2))\n"
        "assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales) and float(q.tensor_scale) == 1\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


def test_two_threads_on_one_stream():
    cases = []
    for k in range(2):
        x, dy, w, _ = data(3000, 520, seed=20 + k)
        X, dY, w = mat(x, "bf16"), mat(dy, "bf16"), w.cuda()
        r = api.layer_norm_fwd(X, w)
        cases.append((dY, X, r.mean, r.rstd, w))
    want = [api.layer_norm_bwd(*c) for c in cases]
    torch.cuda.synchronize()
    got = [[], []]

    def work(k):
        for _ in range(200):
            got[k].append(api.layer_norm_bwd(*cases[k])[1:])

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in range(2):
        assert len(got[k]) == 200
        for dw, db in got[k]:
            assert torch.equal(dw, want[k][1]) and torch.equal(db, want[k][2])


@pytest.mark.parametrize("cols", [515, 769, 1021, 1026, 1275, 1277, 1531, 2041, 2049, 10243, 16373, 16381])
@pytest.mark.parametrize("dtype,gdtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_every_begin(cols, dtype, gdtype):
    # rows that begin and end at every place of a 16-byte word, and of two
    for offset in (range(8) if cols < 2000 else (1, 6)):
        x, dy, w, b = data(9, cols, seed=offset)
        X, dY, w, b = mat(x, dtype, 0, offset), mat(dy, gdtype, 0, offset), w.cuda(), b.cuda()
        r = api.layer_norm_fwd(X, w, b)
        check_fwd(r, X, w, b)
        check_bwd(api.layer_norm_bwd(dY, X, r.mean, r.rstd, w), dY, np64(X), r.mean, r.rstd, w)


@pytest.mark.parametrize("cols", [1100, 1272, 1280, 10240, 10248, 11000, 12288, 16384])
@pytest.mark.parametrize("kind", ["bf16", "mxint8", "mxfp8"])
def test_backward_of_few_long_rows(cols, kind):
    for rows in (1, 3, 200):
        x, dy, w, _ = data(rows, cols, seed=30)
        X, dY, w = mat(x, "bf16"), mat(dy, "bf16"), w.cuda()
        r = api.layer_norm_fwd(X, w, save=None if kind == "bf16" else kind)
        given = X if r.saved is None else r.saved
        x64 = np64(X) if r.saved is None else act8_ref.load(*act8_ref.save(np64(X), kind), cols, kind)
        for weight in (w, None):
            check_bwd(api.layer_norm_bwd(dY, given, r.mean, r.rstd, weight), dY, x64, r.mean, r.rstd, weight)


def test_between_other_work():
    # the launches overlap the end of what runs before them: copies, fills and
    # library kernels that write their inputs, on one stream, over a fork and a
    # join, eagerly and captured
    x, dy, w, _ = data(2016, 1000, seed=40)
    X0, dY0, w = mat(x, "bf16"), mat(dy, "bf16"), w.cuda()
    X, dY = torch.zeros_like(X0), torch.zeros_like(dY0)
    side = torch.cuda.Stream()

    def step():
        X.copy_(X0)
        r = api.layer_norm_fwd(X, w, save="mxint8")
        X.fill_(7)                                 # behind the forward's reads
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            back = api.restore_act8(r.saved)
            kept = api.save_act8(back, "mxfp8")
        dY.zero_()
        dY.copy_(dY0)
        d = api.layer_norm_bwd(dY, r.saved, r.mean, r.rstd, w)
        dY.fill_(3)
        torch.cuda.current_stream().wait_stream(side)
        q = api.quantize_fp4_act8(kept, "nv", axis=0)
        return [r.Y, r.mean, r.rstd, back, kept.codes, q.codes, q.scales] + list(d)

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    check_bwd(want[-3:], dY0, act8_ref.load(*act8_ref.save(np64(X0), "mxint8"), 1000, "mxint8"), want[1], want[2], w)
    for _ in range(20):
        got = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(20):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got))


@pytest.mark.parametrize("cols", [130, 1001, 4001, 11003, 17001])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("kind", ["bf16", "f32", "mxint8"])
def test_special_rows_stay_alone(cols, pad, kind):
    # rows next to one another in words, and matrices that lie differently
    x, dy, w, b = data(12, cols, seed=50)
    dt = "f32" if kind == "f32" else "bf16"
    w, b = w.cuda(), b.cuda()
    plain, dY = mat(x, dt, pad), mat(dy, dt)
    bad = x.clone()
    bad[2, 0], bad[5, cols - 1], bad[9, cols // 2] = float("inf"), float("nan"), float("-inf")
    special = mat(bad, dt, pad)
    rows = torch.tensor([2, 5, 9], device="cuda")
    rest = torch.tensor([r for r in range(12) if r not in (2, 5, 9)], device="cuda")
    fmt = kind if kind in act8_ref.FORMATS else None
    got, want = api.layer_norm_fwd(special, w, b, save=fmt), api.layer_norm_fwd(plain, w, b, save=fmt)
    assert torch.isnan(got.Y[rows]).all() and torch.equal(got.Y[rest], want.Y[rest])
    dgot = api.layer_norm_bwd(dY, got.saved or special, got.mean, got.rstd, w)
    dwant = api.layer_norm_bwd(dY, want.saved or plain, want.mean, want.rstd, w)
    assert torch.isnan(dgot[0][rows]).all() and torch.equal(dgot[0][rest], dwant[0][rest])
    assert torch.isnan(dgot[1]).all() and torch.equal(dgot[2], dwant[2])


@pytest.mark.parametrize("cols", [130, 1001, 4001, 4096, 11003, 17001])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_in_place_of_another_lie(cols, dtype):
    # dX over dY, X elsewhere against the words; and Y over X at every begin
    x, dy, w, b = data(60, cols, seed=51)
    X, dY, w, b = mat(x, dtype, 3, 1), mat(dy, dtype), w.cuda(), b.cuda()
    r = api.layer_norm_fwd(X, w, b)
    want = api.layer_norm_bwd(dY, X, r.mean, r.rstd, w)
    over = dY.clone()
    got = api.layer_norm_bwd(over, X, r.mean, r.rstd, w, out=over)
    assert got[0] is over and all(torch.equal(p, q) for p, q in zip(got, want))
    # (sums run in an order that depends on how the matrices lie: the same here)
    Y = mat(x, dtype, 0, 5)
    ref = api.layer_norm_fwd(mat(x, dtype, 0, 5), w, b, save="mxfp8", out=mat(x, dtype, 0, 5))
    res = api.layer_norm_fwd(Y, w, b, save="mxfp8", out=Y)
    check_fwd(res, mat(x, dtype, 0, 5), w, b)
    assert torch.equal(Y, ref.Y) and torch.equal(res.saved.codes, ref.saved.codes)


def test_offsets_past_32_bits():
    # 2.3e9 elements: the rows at the end against the same rows alone
    rows, cols, tail = 70000, 32768, 40
    X = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    X.normal_(generator=torch.Generator(device="cuda").manual_seed(11))
    w = 1 + 0.1 * torch.randn(cols, device="cuda")
    r = api.layer_norm_fwd(X, w, w, save="mxint8")
    t = api.layer_norm_fwd(X[-tail:].clone(), w, w, save="mxint8")
    assert torch.equal(r.Y[-tail:], t.Y) and torch.equal(r.mean[-tail:], t.mean)
    assert torch.equal(r.saved.codes[-tail:], t.saved.codes) and torch.equal(r.saved.scales[-tail:], t.saved.scales)
    a = api.save_act8(X)
    assert torch.equal(a.codes, r.saved.codes) and torch.equal(a.scales, r.saved.scales)
    del r.Y
    out = api.restore_act8(a)
    assert torch.equal(out[-tail:], api.restore_act8(t.saved))
    dX = api.layer_norm_bwd(X, a, r.mean, r.rstd, w, want_dw=False, want_db=False, out=out)[0]
    assert torch.equal(dX[-tail:], api.layer_norm_bwd(X[-tail:].clone(), t.saved, t.mean, t.rstd, w)[0])
    rows = rows // 32 * 32
    b = api.Act8("mxint8", rows, cols, codes=a.codes[:rows], scales=a.scales[:rows], amax=a.amax)
    q = api.quantize_fp4_act8(b, "nv", axis=1)
    c = api.Act8("mxint8", 32, cols, codes=a.codes[rows - 32:rows], scales=a.scales[rows - 32:rows], amax=a.amax)
    assert torch.equal(q.codes[-16 * cols:], api.quantize_fp4_act8(c, "nv", axis=1).codes)
    q = api.quantize_fp4_act8(b, "nv", axis=0).codes.view(cols, rows // 2)
    assert torch.equal(q[:, -16:], api.quantize_fp4_act8(c, "nv", axis=0).codes.view(cols, 16))


def test_refusals():
    X = torch.zeros((4, 32), device="cuda")
    w, m = torch.ones(32, device="cuda"), torch.zeros(4, device="cuda")
    a = api.Act8("mxint8", 4, 64)
    for call in (lambda: api.layer_norm_fwd(X, w[:31]), lambda: api.layer_norm_fwd(X, w.cpu()),
                 lambda: api.layer_norm_fwd(X, eps=-1e-5), lambda: api.layer_norm_fwd(X.t()),
                 lambda: api.layer_norm_fwd(X, save="int8"), lambda: api.layer_norm_fwd(X, out=X[:3]),
                 lambda: api.layer_norm_fwd(X, torch.ones(64, device="cuda")[::2]),
                 lambda: api.layer_norm_fwd(X[None]),
                 lambda: api.layer_norm_fwd(X.view(2, 64)[:, :32], out=X.view(-1)[:64].view(2, 32)),
                 lambda: api.layer_norm_bwd(X, X[:3], m, m), lambda: api.layer_norm_bwd(X, a, m, m),
                 lambda: api.layer_norm_bwd(X, X, m[:3], m),
                 lambda: api.layer_norm_bwd(X, X, m, m, want_dx=False, want_dw=False, want_db=False)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: api.layer_norm_fwd(X.half()), lambda: api.layer_norm_fwd(X, w, w.bfloat16()),
                 lambda: api.layer_norm_fwd(X, out_dtype=torch.float16),
                 lambda: api.layer_norm_bwd(X, X, m.double(), m)):
        with pytest.raises(TypeError):
            call()
