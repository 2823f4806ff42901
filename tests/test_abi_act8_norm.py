"""Host-side checks of the 8-bit activation and layer norm entry points: every
call below is refused, or only sizes a workspace, before any device work, so
its pointers are never followed."""
import ctypes

import pytest
import torch

from spectral_domain_quantization_b200 import api

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_ARG = 0, 1, 2, 3, 4, 5, 7
X, Y, W, B, ST = 0x40000, 0x80000, 0xC0000, 0xC8000, 0xD0000


def act8(rows=64, cols=128, fmt=api.MXINT8, codes=0x10000, scales=0x20001, amax=0x30000):
    return api.Act8Struct(fmt, rows, cols, codes, scales, amax)


def ref(s):
    return None if s is None else ctypes.byref(s)


def fp4(fmt, outer, inner, **kw):
    s = api.FP4Struct()
    s.fmt, s.outer, s.inner = fmt, outer, inner
    s.codes, s.scales, s.tensor_scale = 0x10000, 0x20000, 0x30000
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_struct_layout_and_sizes():
    S = api.Act8Struct
    assert ctypes.sizeof(S) == 48
    assert [S.fmt.offset, S.rows.offset, S.cols.offset, S.codes.offset, S.scales.offset, S.amax.offset] == \
        [0, 8, 16, 24, 32, 40]
    hdr = open(api.HEADER).read()
    assert f"#define METIS_ACT8_AMAX {api.ACT8_AMAX}" in hdr
    L = api.lib()
    assert [L.metis_act8_codes_bytes(3, c) for c in (1, 32, 33)] == [96, 96, 192]
    assert [L.metis_act8_scales_bytes(3, c) for c in (1, 32, 33)] == [3, 3, 6]
    assert L.metis_act8_codes_bytes(0, 5) == 0 and L.metis_act8_codes_bytes(-1, 5) == 0
    assert L.metis_act8_codes_bytes(5, 0) == 0


def save(rows=64, cols=128, ld=None, dtype=api.BF16, x=X, out=False):
    out = act8(rows, cols) if out is False else out
    return api.lib().metis_act8_save(x, dtype, rows, cols, cols if ld is None else ld, ref(out), None)


def test_save_refusals():
    assert save(x=None) == ERR_NULL
    assert save(out=None) == ERR_NULL
    assert save(dtype=7) == ERR_ARG
    assert save(cols=0) == ERR_SHAPE
    assert save(rows=-1) == ERR_SHAPE
    assert save(ld=100) == ERR_SHAPE
    assert save(cols=1 << 31) == ERR_SHAPE
    assert save(rows=1 << 41, cols=1) == ERR_SHAPE
    assert save(rows=1 << 30, ld=1 << 40) == ERR_SHAPE
    assert save(x=X + 1) == ERR_ALIGN and save(x=X + 2, dtype=api.F32) == ERR_ALIGN
    assert save(out=act8(63, 128)) == ERR_SHAPE and save(out=act8(64, 127)) == ERR_SHAPE
    assert save(out=act8(fmt=2)) == ERR_ARG
    assert save(out=act8(codes=None)) == ERR_NULL and save(out=act8(scales=None)) == ERR_NULL
    assert save(out=act8(amax=None)) == ERR_NULL
    assert save(out=act8(codes=0x10008)) == ERR_ALIGN and save(out=act8(amax=0x30004)) == ERR_ALIGN
    if not torch.cuda.is_available():
        assert save() == ERR_UNSUPPORTED


def test_restore_and_quantize_refusals():
    L = api.lib()

    def restore(a, y=Y, dtype=api.BF16, ld=128):
        return L.metis_act8_restore(ref(a), y, dtype, ld, None)

    assert restore(None) == ERR_NULL and restore(act8(), y=None) == ERR_NULL
    assert restore(act8(), dtype=9) == ERR_ARG
    assert restore(act8(), ld=127) == ERR_SHAPE
    assert restore(act8(), y=Y + 1) == ERR_ALIGN

    def quant(a, axis, out):
        return L.metis_act8_quantize_fp4(ref(a), axis, ref(out), None)

    nv = api.NVFP4
    assert quant(None, 1, fp4(nv, 64, 128)) == ERR_NULL and quant(act8(), 1, None) == ERR_NULL
    assert quant(act8(), 2, fp4(nv, 64, 128)) == ERR_ARG
    assert quant(act8(), 0, fp4(nv, 64, 128)) == ERR_SHAPE           # axis 0: 128 x 64
    assert quant(act8(fmt=5), 1, fp4(nv, 64, 128)) == ERR_ARG
    assert quant(act8(64, 100), 1, fp4(nv, 64, 100)) == ERR_SHAPE    # blocked dimension not a multiple of 32
    assert quant(act8(0, 128), 1, fp4(nv, 0, 128)) == ERR_SHAPE
    assert quant(act8(), 1, fp4(3, 64, 128)) == ERR_ARG
    assert quant(act8(), 1, fp4(nv, 64, 128, tensor_scale=None)) == ERR_NULL
    assert quant(act8(), 1, fp4(nv, 64, 128, inner_sum=0x50000)) == ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        assert restore(act8()) == ERR_UNSUPPORTED
        assert quant(act8(), 1, fp4(nv, 64, 128)) == ERR_UNSUPPORTED
        assert quant(act8(64, 100), 0, fp4(api.MXFP4, 100, 64)) == ERR_UNSUPPORTED


def fwd(rows=64, cols=128, ldx=None, x=X, dtype=api.BF16, w=W, b=B, wdt=api.F32, eps=1e-5, y=Y, ydt=api.BF16, ldy=None,
        mean=0xE0000, rstd=0xE8000, saved=None):
    return api.lib().metis_layer_norm_fwd(x, dtype, rows, cols, cols if ldx is None else ldx, w, b, wdt, eps, y, ydt,
                                          cols if ldy is None else ldy, mean, rstd, ref(saved), None)


def test_layer_norm_fwd_refusals():
    assert fwd(x=None) == ERR_NULL and fwd(y=None) == ERR_NULL
    assert fwd(dtype=4) == ERR_ARG and fwd(ydt=4) == ERR_ARG and fwd(wdt=4) == ERR_ARG
    assert fwd(w=None, b=None, wdt=4) in (ERR_UNSUPPORTED, OK) if not torch.cuda.is_available() else True
    assert fwd(eps=-1.0) == ERR_ARG and fwd(eps=float("nan")) == ERR_ARG
    assert fwd(cols=0) == ERR_SHAPE and fwd(ldx=100) == ERR_SHAPE and fwd(ldy=100) == ERR_SHAPE
    assert fwd(x=X + 1) == ERR_ALIGN and fwd(y=Y + 1) == ERR_ALIGN and fwd(w=W + 2) == ERR_ALIGN
    assert fwd(b=B + 1, wdt=api.BF16) == ERR_ALIGN and fwd(mean=0xE0002) == ERR_ALIGN and fwd(rstd=0xE8001) == ERR_ALIGN
    assert fwd(saved=act8(64, 127)) == ERR_SHAPE and fwd(saved=act8(fmt=-1)) == ERR_ARG
    if not torch.cuda.is_available():
        assert fwd() == ERR_UNSUPPORTED and fwd(saved=act8(), w=None, b=None, mean=None, rstd=None) == ERR_UNSUPPORTED


def bwd(rows=64, cols=128, dy=X, gdt=api.BF16, ldg=None, x=Y, xdt=api.BF16, ldx=None, saved=None, mean=0xE0000,
        rstd=0xE8000, w=W, wdt=api.F32, dx=0x100000, ddt=api.BF16, ldd=None, dw=0xF0000, db=0xF8000, ws=None, wsb=0):
    size = ctypes.c_size_t(wsb)
    st = api.lib().metis_layer_norm_bwd(dy, gdt, rows, cols, cols if ldg is None else ldg, x, xdt,
                                        cols if ldx is None else ldx, ref(saved), mean, rstd, w, wdt, dx, ddt,
                                        cols if ldd is None else ldd, dw, db, ws, ctypes.byref(size), None)
    return st, size.value


def test_layer_norm_bwd_refusals_and_workspace_query():
    st, need = bwd()
    assert st == OK and need >= 256
    assert bwd(dx=None)[0] == OK and bwd(dw=None, db=None)[0] == OK
    assert bwd(dx=None, dw=None, db=None)[0] == ERR_NULL
    assert bwd(dy=None)[0] == ERR_NULL and bwd(x=None)[0] == ERR_NULL
    assert bwd(mean=None)[0] == ERR_NULL and bwd(rstd=None)[0] == ERR_NULL
    assert bwd(x=None, saved=act8())[0] == OK
    assert bwd(saved=act8())[0] == ERR_ARG                            # both forms of X
    assert bwd(x=None, saved=act8(64, 96))[0] == ERR_SHAPE
    assert bwd(gdt=5)[0] == ERR_ARG and bwd(xdt=5)[0] == ERR_ARG and bwd(ddt=5)[0] == ERR_ARG and bwd(wdt=5)[0] == ERR_ARG
    assert bwd(cols=0)[0] == ERR_SHAPE and bwd(rows=-2)[0] == ERR_SHAPE
    assert bwd(ldg=64)[0] == ERR_SHAPE and bwd(ldx=64)[0] == ERR_SHAPE and bwd(ldd=64)[0] == ERR_SHAPE
    assert bwd(dy=X + 1)[0] == ERR_ALIGN and bwd(dw=0xF0002)[0] == ERR_ALIGN and bwd(mean=0xE0001)[0] == ERR_ALIGN
    ws = ctypes.c_void_p(0x200000)
    assert bwd(ws=ws, wsb=need - 1)[0] == ERR_WORKSPACE
    assert bwd(ws=ctypes.c_void_p(0x200010), wsb=need)[0] == ERR_WORKSPACE
    # no rows: nothing but the zeros of the sums
    assert bwd(rows=0, dy=None, x=None, mean=None, rstd=None, dx=None)[0] == OK
    if not torch.cuda.is_available():
        assert bwd(ws=ws, wsb=need)[0] == ERR_UNSUPPORTED
    L = api.lib()
    assert L.metis_layer_norm_bwd(X, 0, 4, 4, 4, Y, 0, 4, None, X, X, None, 0, None, 0, 4, W, None, None, None,
                                  None) == ERR_NULL


def test_python_refusals_before_the_device():
    t = torch.zeros((4, 32))
    for call in (lambda: api.save_act8(t), lambda: api.layer_norm_fwd(t), lambda: api.save_act8(torch.zeros(4)),
                 lambda: api.layer_norm_bwd(t, t, t[:, 0], t[:, 0]),
                 lambda: api.Act8("int8", 4, 32, "cpu"), lambda: api.Act8("mxint8", 4, 0, "cpu"),
                 lambda: api.Act8("mxint8", 4, 32, codes=torch.zeros((4, 32), dtype=torch.uint8),
                                  scales=torch.zeros((4, 1), dtype=torch.uint8), amax=torch.zeros(4))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        api.save_act8(torch.zeros((4, 32), dtype=torch.float16))
    with pytest.raises(TypeError):
        api.restore_act8(t)
    with pytest.raises(TypeError):
        api.quantize_fp4_act8(t, "nv")
