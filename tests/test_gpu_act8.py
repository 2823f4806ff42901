"""Activations kept in 8 bits on the GPU: bytes against the oracle's, the way
back, and the FP4 operand made from them against metis_quantize_fp4."""
import numpy as np
import pytest
import torch

from oracle import act8 as ref
from spectral_domain_quantization_b200 import api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(rows, cols, dtype="bf16", pad=0, offset=0, seed=0, spread=20):
    """A rows x cols view with row stride cols + pad, starting `offset` elements into its buffer."""
    g = torch.Generator().manual_seed(1000 * rows + cols + seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (rows, 1), generator=g))
    buf = torch.zeros(offset + rows * (cols + pad), dtype=DT[dtype], device="cuda")
    v = buf[offset:].view(rows, cols + pad)[:, :cols] if rows else buf[offset:].view(0, cols + pad)[:, :cols]
    v.copy_(x)
    return v


def check(a, X):
    codes, scales = ref.save(X.float().cpu().numpy(), a.fmt)
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    assert np.array_equal(a.codes.cpu().numpy(), codes)
    assert float(a.amax.max()) == ref.amax(codes, scales, a.fmt)
    assert float(a.amax.min()) >= 0


SHAPES = [(1, 1, 0, 0), (1, 32, 0, 0), (3, 31, 0, 0), (2, 33, 0, 0), (7, 8, 0, 0), (5, 100, 4, 0), (64, 96, 0, 0),
          (33, 257, 0, 0), (17, 1027, 5, 3), (40, 512, 1, 0), (9, 64, 0, 1), (300, 776, 8, 8), (2, 14336, 0, 0),
          (1, 70001, 0, 0), (4099, 40, 0, 0)]


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_save_and_restore(fmt, dtype, rows, cols, pad, offset):
    X = make(rows, cols, dtype, pad, offset)
    a = api.save_act8(X, fmt)
    check(a, X)
    want = ref.load(a.codes.cpu().numpy(), a.scales.cpu().numpy(), cols, fmt)
    y32, y16 = api.restore_act8(a, torch.float32), api.restore_act8(a)
    assert np.array_equal(y32.double().cpu().numpy(), want)
    assert np.array_equal(y16.double().cpu().numpy(), want)   # 8 bits fit in bf16's significand
    # into a strided and unaligned tensor; what lies between its rows stays
    buf = torch.full((rows, cols + 3), 7.0, dtype=DT[dtype], device="cuda")
    api.restore_act8(a, out=buf[:, 1:cols + 1])
    assert np.array_equal(buf[:, 1:cols + 1].double().cpu().numpy(), want)
    assert (buf[:, 0] == 7).all() and (buf[:, cols + 1:] == 7).all()


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("pad", [0, 1])
def test_special_values(fmt, pad):
    X = make(8, 96, "f32", pad, spread=3)
    X[0, 3] = float("nan")
    X[1, 40] = float("inf")
    X[2, 70] = -float("inf")
    X[3] = 0
    X[4, :32] = 1e-45
    X[5, :32] = -3.4028234663852886e38
    X[6, :32] = 2.0 ** -125
    X[7, :32] = -0.0
    a = api.save_act8(X, fmt)
    check(a, X)
    y = api.restore_act8(a, torch.float32)
    want = ref.load(a.codes.cpu().numpy(), a.scales.cpu().numpy(), 96, fmt)
    assert np.array_equal(y.double().cpu().numpy(), want, equal_nan=True)
    assert torch.isnan(y[0, :32]).all() and not torch.isnan(y[0, 32:]).any()


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_every_element_code(fmt):
    # scaled values at and next to every rounding border, under one block scale
    levels = np.arange(0, 127.25, 0.25) / 64 if fmt == "mxint8" else None
    if levels is None:
        lv = ref.e4m3_value(np.arange(0x7F))
        levels = np.concatenate([lv, (lv[1:] + lv[:-1]) / 2]) / 256
    v = np.float32(levels)
    v = np.concatenate([v, np.nextafter(v, np.float32(9)), np.nextafter(v, np.float32(-9)), -v])
    v = np.clip(v, -1.9999999, 1.9999999).astype(np.float32)
    n = (len(v) + 30) // 31
    X = np.full((n, 32), 1.0, np.float32)            # column 0 holds the block's exponent
    X[:, 1:].reshape(-1)
    flat = np.zeros(n * 31, np.float32)
    flat[:len(v)] = v
    X[:, 1:] = flat.reshape(n, 31)
    Xd = torch.from_numpy(X).cuda()
    check(api.save_act8(Xd, fmt), Xd)


@pytest.mark.parametrize("rows", [0])
def test_no_rows(rows):
    X = torch.zeros((0, 40), dtype=torch.bfloat16, device="cuda")
    a = api.save_act8(X, "mxfp8")
    assert not a.amax.any() and api.restore_act8(a).shape == (0, 40)


def same_fp4(a, b):
    assert (a.outer, a.inner) == (b.outer, b.inner)
    assert torch.equal(a.codes, b.codes)
    assert torch.equal(a.scales, b.scales)
    assert torch.equal(a.tensor_scale, b.tensor_scale)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("fp4", ["nv", "mx"])
@pytest.mark.parametrize("axis,rows,cols", [(1, 1, 32), (1, 5, 96), (1, 129, 160), (1, 300, 1056), (1, 64, 4096),
                                            (0, 32, 1), (0, 32, 33), (0, 96, 100), (0, 544, 257), (0, 288, 1003),
                                            (0, 2048, 520), (0, 4128, 130)])
def test_fp4_from_8_bits(fmt, fp4, axis, rows, cols):
    a = api.save_act8(make(rows, cols, "bf16", spread=4), fmt)
    got = api.quantize_fp4_act8(a, fp4, axis, linear=True)
    # the quantizer on the restored float32 matrix (rows padded to 16 bytes for it)
    full = torch.zeros((rows, (cols + 3) // 4 * 4), dtype=torch.float32, device="cuda")
    api.restore_act8(a, out=full[:, :cols])
    want = api.quantize_fp4(full[:, :cols], fp4, axis, linear=True)
    same_fp4(got, want)
    assert torch.equal(got.scales_linear, want.scales_linear)


@pytest.mark.parametrize("fp4", ["nv", "mx"])
@pytest.mark.parametrize("axis", [0, 1])
def test_fp4_of_zeros_nan_and_small(fp4, axis):
    X = make(64, 64, "f32", spread=2)
    X[:, :32] = 0
    X[3, 40] = float("nan")
    X[40:, 32:] *= 1e-30
    a = api.save_act8(X)
    same_fp4(api.quantize_fp4_act8(a, fp4, axis), api.quantize_fp4(api.restore_act8(a, torch.float32), fp4, axis))
    a = api.save_act8(torch.zeros((32, 32), device="cuda"))
    same_fp4(api.quantize_fp4_act8(a, fp4, axis), api.quantize_fp4(torch.zeros((32, 32), device="cuda"), fp4, axis))


def test_other_stream_and_graph():
    X = make(96, 200, "bf16", spread=2)
    a0 = api.save_act8(X)
    q0 = api.quantize_fp4_act8(a0, "nv", 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a1 = api.save_act8(X)
        q1 = api.quantize_fp4_act8(a1, "nv", 0)
    s.synchronize()
    assert torch.equal(a0.codes, a1.codes) and torch.equal(a0.amax.max(), a1.amax.max())
    same_fp4(q0, q1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a2 = api.save_act8(X)
        q2 = api.quantize_fp4_act8(a2, "nv", 0)
        y2 = api.restore_act8(a2)
    for k in range(2):
        X.mul_(1.5)
        g.replay()
        torch.cuda.synchronize()
        a = api.save_act8(X)
        assert torch.equal(a.codes, a2.codes) and torch.equal(a.scales, a2.scales)
        same_fp4(api.quantize_fp4_act8(a, "nv", 0), q2)
        assert torch.equal(api.restore_act8(a), y2)


def test_refusals():
    X = make(32, 40)
    a = api.save_act8(X)
    for call in (lambda: api.quantize_fp4_act8(a, "nv", 1),              # 40 columns
                 lambda: api.quantize_fp4_act8(a, "nv", 2),
                 lambda: api.restore_act8(a, out=torch.zeros((32, 41), device="cuda")),
                 lambda: api.restore_act8(a, out=torch.zeros((32, 40))),
                 lambda: api.save_act8(X.t()),
                 lambda: api.save_act8(X, "mxint8", out=api.Act8("mxfp8", 32, 40)),
                 lambda: api.save_act8(X[:1].expand(32, 40)),
                 lambda: api.save_act8(torch.zeros((4, 0), device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        api.restore_act8(a, torch.float16)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_tensor_scale_is_the_results_own(fmt):
    # writing one result's scale reaches no other
    X = torch.randn(64, 96, device="cuda")
    a = api.save_act8(X)
    first = [api.quantize_fp4_act8(a, fmt, 0), api.quantize_fp4(X, fmt, 0)]
    want = [float(q.tensor_scale) for q in first]
    assert fmt == "nv" or want == [1.0, 1.0]
    for q in first:
        q.tensor_scale.fill_(7)
    second = [api.quantize_fp4_act8(a, fmt, 0), api.quantize_fp4(X, fmt, 0)]
    assert [float(q.tensor_scale) for q in second] == want
