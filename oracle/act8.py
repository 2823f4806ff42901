"""Activations kept in 8 bits: MXINT8 and MXFP8 (E4M3) blocks (oracle side).

Test infrastructure only (see ``oracle/__init__.py``).

The pages quantize the layer's input again in the backward pass (along the
batch, for dW = X^T dY) without saying in what form it is kept until then; the
library offers the 8-bit element types of the OCP Microscaling v1.0
specification under its E8M0 scale, 32 consecutive columns a block, the last
block of a row possibly shorter.

Per block, a = max |x|:
    a not finite : scale code 255, codes 0, every value reads NaN
    a == 0       : scale code 0, codes 0
    MXINT8       : se = clamp(floor(log2 a), -120, 127)
                   code = rint(x * 2**(6 - se)) clamped to +-127
                   value = code * 2**(se - 6)
    MXFP8        : se = clamp(floor(log2 a) - 8, -126, 127)
                   code = E4M3(x * 2**-se), nearest even, saturating at 448
                   value = e4m3 * 2**se
    scale code = se + 127
Everything here runs in float64, which holds every scaled float32 exactly, so
the one rounding is the element's.
"""
import numpy as np

BLOCK = 32
FORMATS = ("mxint8", "mxfp8")


def e4m3_value(code):
    """Value of E4M3 codes (uint8 array): s|e3..e0|m2..m0, bias 7; 0x7F and 0xFF are NaN."""
    code = np.asarray(code, np.uint8)
    e = ((code >> 3) & 15).astype(np.int64)
    m = (code & 7).astype(np.float64)
    mag = np.where(e == 0, m * 2.0 ** -9, (8.0 + m) * np.exp2(e - 10.0))
    mag = np.where((code & 0x7F) == 0x7F, np.nan, mag)
    return np.where(code & 0x80, -mag, mag)


_LEVELS = e4m3_value(np.arange(0x7F))         # the finite magnitudes, ascending


def e4m3_code(q):
    """E4M3 codes of float64 values: the nearest level, ties to the even code, at most 448."""
    mag = np.minimum(np.abs(q), 448.0)
    hi = np.searchsorted(_LEVELS, mag)           # the first level >= mag
    lo = np.maximum(hi - 1, 0)
    dl, dh = mag - _LEVELS[lo], _LEVELS[hi] - mag
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(q), 0x80, 0)).astype(np.uint8)


def save(X, fmt):
    """codes (rows x 32 blocks, uint8), scales (rows x blocks, uint8) of a float32 matrix."""
    X = np.asarray(X, np.float64)
    m, n = X.shape
    nb = (n + BLOCK - 1) // BLOCK
    xb = np.zeros((m, nb * BLOCK))
    xb[:, :n] = X
    xb = xb.reshape(m, nb, BLOCK)
    a = np.max(np.abs(xb), axis=2)               # NaN where the block has one
    bad = ~np.isfinite(a)
    safe = np.where(bad | (a == 0), 1.0, a)
    top = np.frexp(safe)[1] - 1                  # floor(log2 a), exact
    xb = np.where(bad[:, :, None], 0.0, xb)
    if fmt == "mxint8":
        se = np.clip(top, -120, 127)
        code = np.clip(np.rint(xb * np.exp2(6.0 - se)[:, :, None]), -127, 127)
        codes = code.astype(np.int8).view(np.uint8)
    else:
        se = np.clip(top - 8, -126, 127)
        codes = e4m3_code(xb * np.exp2(-se.astype(np.float64))[:, :, None])
    scales = np.where(bad, 255, np.where(a == 0, 0, se + 127)).astype(np.uint8)
    codes = np.where(bad[:, :, None], np.uint8(0), codes)
    return codes.reshape(m, nb * BLOCK), scales


def load(codes, scales, cols, fmt):
    """The float64 values (rows x cols) of codes and scales."""
    m, nb = scales.shape
    c = codes.reshape(m, nb, BLOCK)
    elem = c.view(np.int8).astype(np.float64) if fmt == "mxint8" else e4m3_value(c)
    factor = np.exp2(scales.astype(np.float64) - (133.0 if fmt == "mxint8" else 127.0))
    factor = np.where(scales == 255, np.nan, factor)
    return (elem * factor[:, :, None]).reshape(m, nb * BLOCK)[:, :cols]


def amax(codes, scales, fmt):
    """The largest magnitude held; blocks that read NaN are left out."""
    v = np.abs(load(codes, scales, codes.shape[1], fmt))
    v = v[np.isfinite(v)]
    return float(v.max()) if v.size else 0.0
