"""Python binding of the C ABI in include/metis.h (ctypes).

Argument marshalling only: torch tensors provide device memory and the current
CUDA stream; every arithmetic step runs in the CUDA kernels of
``libmetis_b200.so``.  There is no fallback: if the library is missing or the
device is not sm_100, calls raise.
"""
import ctypes
import functools
import os
import re
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmetis_b200.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "metis.h")

OK = 0
ERR_WORKSPACE = 5
BF16, F32 = 0, 1
MXFP4, NVFP4 = 0, 1
SKETCH_GAUSSIAN, SKETCH_SPARSE_SIGN = 0, 1
MXINT8, MXFP8 = 0, 1
ACT8_AMAX = 1024
DEV_NUMERIC, DEV_TIMEOUT, DEV_SAMPLING = 1, 2, 4

FMT = {"mx": MXFP4, "nv": NVFP4, MXFP4: MXFP4, NVFP4: NVFP4}
FMT_NAME = {MXFP4: "mx", NVFP4: "nv"}
ACT8_FMT = {"mxint8": MXINT8, "mxfp8": MXFP8}


class MetisError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        detail = ""
        if status == 6:
            try:
                detail = " [" + lib().metis_last_error().decode() + "]"
            except Exception:  # pragma: no cover
                pass
        super().__init__(f"{what}: {status_string(status)} (status {status}){detail}")


class FP4Struct(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("outer", ctypes.c_int64), ("inner", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("scales_linear", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("inner_sum", ctypes.c_void_p)]


class Act8Struct(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("amax", ctypes.c_void_p)]


class SplitParams(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("p", ctypes.c_int32), ("power_iters", ctypes.c_int32),
                ("seed", ctypes.c_uint64), ("sketch", ctypes.c_int32),
                ("sparse_nnz", ctypes.c_int32), ("sample_rows", ctypes.c_int64),
                ("fmt", ctypes.c_int32), ("max_core_iters", ctypes.c_int32),
                ("compensate", ctypes.c_int32)]


class OperandStruct(ctypes.Structure):
    _fields_ = [("R", ctypes.POINTER(FP4Struct)), ("k", ctypes.c_int32),
                ("P", ctypes.POINTER(FP4Struct)), ("F", ctypes.POINTER(FP4Struct)),
                ("S", ctypes.c_void_p), ("flags", ctypes.c_int32)]


REQUANT_LOWRANK = 1


_lib = None

_VP, _I32, _I64, _SZP = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)
_FP = ctypes.POINTER(FP4Struct)
_OP = ctypes.POINTER(OperandStruct)
_AP = ctypes.POINTER(Act8Struct)

_SIGS = {
    "metis_fp4_codes_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "metis_fp4_scales_bytes": (ctypes.c_size_t, [_I32, _I64, _I64]),
    "metis_status_string": (ctypes.c_char_p, [_I32]),
    "metis_device_supported": (_I32, []),
    "metis_last_error": (ctypes.c_char_p, []),
    "metis_quantize_fp4": (_I32, [_VP, _I32, _I64, _I64, _I64, _I32, _VP, _FP, _VP, _SZP, _VP]),
    "metis_quantize_fp4_noalloc": (_I32, [_VP, _I32, _I64, _I64, _I64, _I32, _VP, _FP, _VP]),
    "metis_noalloc_scratch_bytes": (ctypes.c_size_t, []),
    "metis_selftest_wait_timeout": (_I32, [ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p]),
    "metis_split": (_I32, [_VP, _I32, _I64, _I64, _I64, ctypes.POINTER(SplitParams), _VP, _VP, _VP,
                           _FP, _FP, _FP, _FP, _VP, _VP, _VP, _SZP, _VP, _VP]),
    "metis_linear_fwd": (_I32, [_OP, _OP, _I64, _I64, _I64, _VP, _I32, _I64, _VP, _SZP, _VP, _VP]),
    "metis_linear_bwd": (_I32, [_OP, _OP, _OP, _OP, _I64, _I64, _I64, _VP, _I64, _VP, _I64, _I32,
                                _VP, _SZP, _VP, _VP]),
    "averis_split": (_I32, [_VP, _I32, _I64, _I64, _I64, _I32, _VP, _FP, _FP, _FP, _VP, _VP, _SZP,
                            _VP, _VP]),
    "metis_spectral_scale": (_I32, [_VP, _I64, _I64, _I64, _VP, _VP, _VP, _I32, ctypes.c_float, _VP, _VP, _SZP,
                                    _VP, _VP]),
    "metis_act8_codes_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "metis_act8_scales_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "metis_act8_save": (_I32, [_VP, _I32, _I64, _I64, _I64, _AP, _VP]),
    "metis_act8_restore": (_I32, [_AP, _VP, _I32, _I64, _VP]),
    "metis_act8_quantize_fp4": (_I32, [_AP, _I32, _FP, _VP]),
    "metis_layer_norm_fwd": (_I32, [_VP, _I32, _I64, _I64, _I64, _VP, _VP, _I32, ctypes.c_float, _VP, _I32, _I64,
                                    _VP, _VP, _AP, _VP]),
    "metis_layer_norm_bwd": (_I32, [_VP, _I32, _I64, _I64, _I64, _VP, _I32, _I64, _AP, _VP, _VP, _VP, _I32, _VP,
                                    _I32, _I64, _VP, _VP, _VP, _SZP, _VP]),
}


def lib():
    """Load libmetis_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmetis_b200.so is not built: run __graft_entry__.build() "
                               "or python spectral_domain_quantization_b200/build.py")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def header_functions():
    """Names of the functions declared in include/metis.h."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:METIS_API\s+)?(?:const\s+)?[a-z_0-9]+\s*\**\s+\**(\w+)\s*\(", src,
                                 flags=re.M)))


def status_string(status):
    try:
        return lib().metis_status_string(int(status)).decode()
    except Exception:  # pragma: no cover - only when the library is absent
        return "status"


def _check(status, what):
    if status != OK:
        raise MetisError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(index):
    """The current stream of device `index` (a cudaStream_t as an integer)."""
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


def _stream():
    return _stream_of(torch.cuda.current_device())


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError("only bfloat16 and float32 inputs are supported")


class _Workspace(threading.local):
    """Grow-only workspace per thread, device and stream (allocated by torch, the
    caller side), so that calls enqueued on different streams never share
    scratch memory, nor do two threads' calls on one stream, whose kernels may
    be enqueued in turn (ctypes releases the interpreter during a call).  A call that is captured into a graph gets memory of its
    own, from the graph's pool: graphs captured on one stream may be replayed
    at the same time, and live longer than a buffer that grows."""

    def __init__(self):
        self.buf = {}

    def held(self, device):
        """The stream's buffer as it is; None if there is none, or in a capture."""
        if torch.cuda.is_current_stream_capturing():
            return None
        index = device.index if device.index is not None else torch.cuda.current_device()
        return self.buf.get((index, _stream_of(index)))

    def get(self, nbytes, device):
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        index = device.index if device.index is not None else torch.cuda.current_device()
        key = (index, _stream_of(index))
        cur = self.buf.get(key)
        if cur is None or cur.numel() < nbytes:
            cur = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
            self.buf[key] = cur
        return cur


_ws = _Workspace()


def _call_with_workspace(fn, args_before_ws, args_after_ws, device, what, workspace=None):
    """Provide a workspace (the caller's uint8 tensor when given, else the
    thread's own for the stream, grown to the size the call asks for), then run
    the call."""
    if workspace is None:
        ws = _ws.held(device)
        if ws is not None:
            # large enough in most calls: the library refuses it otherwise,
            # before anything is launched
            size = ctypes.c_size_t(ws.numel())
            status = fn(*args_before_ws, ws.data_ptr(), ctypes.byref(size), *args_after_ws)
            if status != ERR_WORKSPACE:
                _check(status, what)
                return
    size = ctypes.c_size_t(0)
    _check(fn(*args_before_ws, None, ctypes.byref(size), *args_after_ws), what + " (workspace query)")
    if workspace is not None:
        if workspace.dtype != torch.uint8 or workspace.numel() < size.value:
            raise ValueError(f"{what}: the workspace needs {size.value} bytes (uint8)")
        ws = workspace
    else:
        ws = _ws.get(size.value, device)
    size2 = ctypes.c_size_t(ws.numel())
    _check(fn(*args_before_ws, _ptr(ws), ctypes.byref(size2), *args_after_ws), what)


# --------------------------------------------------------------------------
# FP4 tensors
# --------------------------------------------------------------------------

@functools.lru_cache(maxsize=4096)
def _fp4_bytes(fmt, outer, inner):
    """Bytes of an FP4 matrix's codes and scales."""
    L = lib()
    return L.metis_fp4_codes_bytes(outer, inner), L.metis_fp4_scales_bytes(fmt, outer, inner)


class _Ones(threading.local):
    """Floats on the device that hold 1, each handed out once: the tensor scales of
    MXFP4 results, which no kernel writes.  Filled many at a time on the stream they
    are for, so that a result costs no launch of its own."""

    def __init__(self):
        self.ready = {}          # by device and stream: a tensor of ones, and how many are taken

    def take(self, device):
        """A tensor and the index of the 1 in it."""
        if torch.cuda.is_current_stream_capturing():
            return torch.ones(1, dtype=torch.float32, device=device), 0      # the graph's, as the codes are
        key = (device.index, _stream_of(device.index))
        have = self.ready.get(key)
        if have is None or have[1] == have[0].numel():
            have = self.ready[key] = [torch.ones(256, dtype=torch.float32, device=device), 0]
        have[1] += 1
        return have[0], have[1] - 1


_ones = _Ones()


class QTensor:
    """An FP4 matrix (outer x inner, blocks along inner) held in torch buffers:
    codes, scales and tensor_scale (1 for MXFP4), and scales_linear and inner_sum
    or None.  Those that a quantizer's call allocates are parts of one storage:
    each keeps all of it alive, and is to be cloned before it is saved alone."""

    def __init__(self, fmt, outer, inner, device="cuda", linear=False, inner_sum=False, written=False):
        # written: for a call that writes all of it now.  codes, scales and
        # tensor_scale are then parts of one buffer, and tensors when asked for
        self.fmt = FMT[fmt]
        self.outer, self.inner = int(outer), int(inner)
        self.block = 32 if self.fmt == MXFP4 else 16
        nc, ns = _fp4_bytes(self.fmt, self.outer, self.inner)
        if written:
            at = (nc + 255) // 256 * 256
            end = (at + ns + 255) // 256 * 256
            self._parts = (nc, at, ns, end)
            self._buf = torch.empty(end + 4, dtype=torch.uint8, device=device)
            self.device = self._buf.device
            if self.fmt == MXFP4:
                self._one = _ones.take(self.device)
        else:
            self.codes = torch.empty(nc, dtype=torch.uint8, device=device)
            self.scales = torch.empty(ns, dtype=torch.uint8, device=device)
            self.tensor_scale = torch.ones(1, dtype=torch.float32, device=device)
            self.device = self.codes.device
        self.scales_linear = (torch.empty(self.outer * (self.inner // self.block), dtype=torch.uint8,
                                          device=device) if linear else None)
        self.inner_sum = torch.empty(self.outer, dtype=torch.float32, device=device) if inner_sum else None

    def __getattr__(self, name):
        # reached for what is not set yet
        if name in ("codes", "scales", "tensor_scale") and "_buf" in self.__dict__:
            nc, at, ns, end = self._parts
            if name == "codes":
                self.codes = self._buf[:nc]
            elif name == "scales":
                self.scales = self._buf[at:at + ns]
            elif self.fmt == NVFP4:
                self.tensor_scale = self._buf[end:].view(torch.float32)
            else:
                ones, k = self._one
                self.tensor_scale = ones[k:k + 1]
            return self.__dict__[name]
        raise AttributeError(name)

    def struct(self):
        s = FP4Struct()
        s.fmt, s.outer, s.inner = self.fmt, self.outer, self.inner
        has = self.__dict__
        if "_buf" in has:
            base, (_, at, _, end) = self._buf.data_ptr(), self._parts
            s.codes, s.scales = base, base + at
            s.tensor_scale = base + end if self.fmt == NVFP4 else None
        if "codes" in has:
            s.codes = self.codes.data_ptr()
        if "scales" in has:
            s.scales = self.scales.data_ptr()
        if "tensor_scale" in has:
            s.tensor_scale = self.tensor_scale.data_ptr()
        s.scales_linear = self.scales_linear.data_ptr() if self.scales_linear is not None else None
        s.inner_sum = self.inner_sum.data_ptr() if self.inner_sum is not None else None
        self._s = s          # keep alive while pointers are in use
        return s


def quantize_fp4(X, fmt, axis=1, sub_col=None, linear=False, inner_sum=False, out=None):
    """FP4 block quantization of a 2-D bf16/f32 CUDA tensor (metis_quantize_fp4)."""
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a row-major 2-D tensor")
    rows, cols = X.shape
    outer, inner = (rows, cols) if axis == 1 else (cols, rows)
    if out is None:
        out = QTensor(fmt, outer, inner, X.device, linear=linear, inner_sum=inner_sum,
                      written=True)
    s = out.struct()
    L = lib()
    _call_with_workspace(
        L.metis_quantize_fp4,
        (_ptr(X), _dtype_code(X), rows, cols, X.stride(0), axis, _ptr(sub_col), ctypes.byref(s)),
        (_stream(),), X.device, "metis_quantize_fp4")
    return out


def quantize_fp4_noalloc(X, fmt, axis=1, sub_col=None, linear=False, inner_sum=False, out=None):
    """metis_quantize_fp4_noalloc: the same quantization with the library's
    fixed scratch instead of a workspace (for callers that cannot allocate)."""
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a row-major 2-D tensor")
    rows, cols = X.shape
    outer, inner = (rows, cols) if axis == 1 else (cols, rows)
    if out is None:
        out = QTensor(fmt, outer, inner, X.device, linear=linear, inner_sum=inner_sum)
    s = out.struct()
    _check(lib().metis_quantize_fp4_noalloc(_ptr(X), _dtype_code(X), rows, cols, X.stride(0), axis,
                                            _ptr(sub_col), ctypes.byref(s), _stream()),
           "metis_quantize_fp4_noalloc")
    return out


# --------------------------------------------------------------------------
# split-linear products
# --------------------------------------------------------------------------

class Operand:
    """One operand of an FP4 product (see metis_operand in metis.h).

    left operand  A (M x K) = R + F diag(S) P^T
    right operand B (K x N) = R + P diag(S) F^T
    R: QTensor quantized along K; P: QTensor (outer k, inner K) or None for
    the all-ones vector; F: QTensor (outer k, inner M or N) or None for ones;
    S: CUDA float tensor of k values or None (ones).
    requant: re-quantize the low-rank intermediate formed from this
    operand's factors to FP4 along its k (METIS_REQUANT_LOWRANK)."""

    def __init__(self, R, k=0, P=None, F=None, S=None, requant=False):
        self.R, self.k, self.P, self.F, self.S = R, int(k), P, F, S
        self.requant = bool(requant)

    def struct(self):
        o = OperandStruct()
        self._r = self.R.struct()
        o.R = ctypes.pointer(self._r)
        o.k = self.k
        self._p = self.P.struct() if self.P is not None else None
        self._f = self.F.struct() if self.F is not None else None
        o.P = ctypes.pointer(self._p) if self._p is not None else None
        o.F = ctypes.pointer(self._f) if self._f is not None else None
        o.S = self.S.data_ptr() if self.S is not None else None
        o.flags = REQUANT_LOWRANK if self.requant else 0
        self._o = o
        return o


def _out_dtype(dt):
    return F32 if dt == torch.float32 else BF16


def linear_fwd(X, W, M, N, K, out_dtype=torch.float32, Y=None, dev_status=None):
    """Y = X W on FP4 operands (metis_linear_fwd).  X, W: Operand."""
    dev = X.R.device
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=dev)
    if dev_status is None:
        dev_status = torch.empty(1, dtype=torch.int32, device=dev)      # nobody reads it
    xs, ws_ = X.struct(), W.struct()
    _call_with_workspace(
        lib().metis_linear_fwd,
        (ctypes.byref(xs), ctypes.byref(ws_), M, N, K, _ptr(Y), _out_dtype(Y.dtype), Y.stride(0)),
        (_ptr(dev_status), _stream()), dev, "metis_linear_fwd")
    return Y


def linear_bwd(dY_n, Wt, Xt, dY_m, M, N, K, out_dtype=torch.float32, dX=None, dW=None,
               want_dx=True, want_dw=True, dev_status=None):
    """dX = dY W^T and dW = X^T dY on FP4 operands (metis_linear_bwd)."""
    dev = (dY_n or Xt).R.device
    if want_dx and dX is None:
        dX = torch.empty((M, K), dtype=out_dtype, device=dev)
    if want_dw and dW is None:
        dW = torch.empty((K, N), dtype=out_dtype, device=dev)
    if dev_status is None:
        dev_status = torch.empty(1, dtype=torch.int32, device=dev)      # nobody reads it
    a = ctypes.byref(dY_n.struct()) if want_dx else None
    b = ctypes.byref(Wt.struct()) if want_dx else None
    c = ctypes.byref(Xt.struct()) if want_dw else None
    d = ctypes.byref(dY_m.struct()) if want_dw else None
    dt = _out_dtype(out_dtype)
    _call_with_workspace(
        lib().metis_linear_bwd,
        (a, b, c, d, M, N, K, _ptr(dX) if want_dx else None, dX.stride(0) if want_dx else 0,
         _ptr(dW) if want_dw else None, dW.stride(0) if want_dw else 0, dt),
        (_ptr(dev_status), _stream()), dev, "metis_linear_bwd")
    return dX, dW


# --------------------------------------------------------------------------
# spectral split
# --------------------------------------------------------------------------

SKETCH = {"gaussian": SKETCH_GAUSSIAN, "sparse_sign": SKETCH_SPARSE_SIGN}


class Split:
    """Outputs of metis_split: U (m x k), S (k), V (n x k) float32; FP4 U_q
    (k x m), V_q (k x n), R_rows (m x n, blocks along n), R_cols (n x m,
    blocks along m); optional float32 residual tap and sample indices."""

    def __init__(self, **kw):
        self.__dict__.update(kw)

    def operand(self, side, axis_rows=True):
        """Operand of a product: side "right" for W in X W (residual quantized
        along K = rows of W), "left" for X in X W (residual along its columns)."""
        if side == "right":
            return Operand(self.R_cols if axis_rows else self.R_rows, self.k, self.U_q, self.V_q, self.S)
        return Operand(self.R_rows, self.k, self.V_q, self.U_q, self.S)


def split(A, k, p, q=1, seed=0, fmt="nv", sketch="gaussian", nnz=4, sample_rows=0, max_iters=64,
          rows=True, cols=True, factors=True, tap=False, compensate=False, dev_status=None, workspace=None):
    """Spectral split A = U diag(S) V^T + R with FP4 outputs (metis_split).
    compensate: R = A - deq(U_q) diag(S) deq(V_q)^T (needs factors=True).
    workspace: optional caller-owned uint8 CUDA tensor (see sketch_tap)."""
    if A.dim() != 2 or A.stride(1) != 1:
        raise ValueError("A must be a row-major 2-D tensor")
    m, n = A.shape
    dev = A.device
    f = FMT[fmt]
    U = torch.empty((m, k), dtype=torch.float32, device=dev)
    S = torch.empty(k, dtype=torch.float32, device=dev)
    V = torch.empty((n, k), dtype=torch.float32, device=dev)
    U_q = QTensor(f, k, m, dev) if factors else None
    V_q = QTensor(f, k, n, dev) if factors else None
    R_rows = QTensor(f, m, n, dev) if rows else None
    R_cols = QTensor(f, n, m, dev) if cols else None
    R_f32 = torch.empty((m, n), dtype=torch.float32, device=dev) if tap else None
    idx = torch.empty(sample_rows, dtype=torch.int32, device=dev) if sample_rows else None
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
    prm = SplitParams(k=k, p=p, power_iters=q, seed=seed, sketch=SKETCH[sketch], sparse_nnz=nnz,
                      sample_rows=sample_rows, fmt=f, max_core_iters=max_iters, compensate=int(bool(compensate)))
    st = [t.struct() if t is not None else None for t in (U_q, V_q, R_rows, R_cols)]
    refs = [ctypes.byref(s) if s is not None else None for s in st]
    _call_with_workspace(
        lib().metis_split,
        (_ptr(A), _dtype_code(A), m, n, A.stride(0), ctypes.byref(prm), _ptr(U), _ptr(S), _ptr(V), *refs,
         _ptr(R_f32), _ptr(idx)),
        (_ptr(dev_status), _stream()), dev, "metis_split", workspace=workspace)
    return Split(U=U, S=S, V=V, U_q=U_q, V_q=V_q, R_rows=R_rows, R_cols=R_cols, R_f32=R_f32, idx=idx,
                 dev_status=dev_status, k=k, fmt=f)


def sketch_tap(workspace, n, k, p):
    """The sketch Omega (n x l, float32 from bf16) that the last metis_split
    on `workspace` used: the first round_up(l, 16) x round_up(n, 8) bf16
    values of the workspace hold Omega^T (the tap metis.h documents)."""
    l = k + p
    lp = (l + 15) // 16 * 16
    ldn = (n + 7) // 8 * 8
    omt = workspace[: lp * ldn * 2].view(torch.bfloat16).view(lp, ldn)
    return omt, omt[:l, :n].float().t()


# --------------------------------------------------------------------------
# Averis
# --------------------------------------------------------------------------

class AverisSplit:
    """Outputs of averis_split: mean (n), mean_q (1 x n), R_rows (m x n,
    blocks along n), R_cols (n x m, blocks along m, with inner sums), tap."""

    def __init__(self, **kw):
        self.__dict__.update(kw)

    def left(self):
        """X as the left operand of X W (contraction over n): 1 mu^T + R."""
        return Operand(self.R_rows, 1, self.mean_q, None, None)

    def left_t(self):
        """X^T as the left operand of X^T dY (contraction over m): mu 1^T + R^T."""
        return Operand(self.R_cols, 1, None, self.mean_q, None)

    def right_m(self):
        """dY as the right operand of X^T dY (contraction over m): 1 nu^T + R."""
        return Operand(self.R_cols, 1, None, self.mean_q, None)


def averis_split(X, fmt="nv", rows=True, cols=True, tap=False, dev_status=None):
    """Mean / residual split with FP4 outputs (averis_split)."""
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a row-major 2-D tensor")
    m, n = X.shape
    dev = X.device
    f = FMT[fmt]
    mean = torch.empty(n, dtype=torch.float32, device=dev)
    mean_q = QTensor(f, 1, n, dev)
    R_rows = QTensor(f, m, n, dev, inner_sum=True) if rows else None
    R_cols = QTensor(f, n, m, dev, inner_sum=True) if cols else None
    R_f32 = torch.empty((m, n), dtype=torch.float32, device=dev) if tap else None
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
    st = [t.struct() if t is not None else None for t in (mean_q, R_rows, R_cols)]
    refs = [ctypes.byref(s) if s is not None else None for s in st]
    _call_with_workspace(
        lib().averis_split,
        (_ptr(X), _dtype_code(X), m, n, X.stride(0), f, _ptr(mean), *refs, _ptr(R_f32)),
        (_ptr(dev_status), _stream()), dev, "averis_split")
    return AverisSplit(mean=mean, mean_q=mean_q, R_rows=R_rows, R_cols=R_cols, R_f32=R_f32,
                       dev_status=dev_status, fmt=f)


# --------------------------------------------------------------------------
# mean + spectral composite
# --------------------------------------------------------------------------

class CompositeSplit:
    """A = 1 mu^T + U diag(S) V^T + R2 from averis_split then metis_split of
    the float32 mean-free residual.  The mean and the spectral part form one
    rank-(k + 1) low-rank part F diag(S1) P^T with F = [1 | U], P = [mu | V],
    S1 = [1, S]; F_q (outer k + 1, inner m) and P_q (outer k + 1, inner n) are
    their FP4 quantizations along the long axis.  F32 and P32 are float32
    column views of the factors as quantized (leading dimension padded)."""

    def __init__(self, **kw):
        self.__dict__.update(kw)

    def operand(self, side, axis_rows=True):
        """As Split.operand: "right" for W in X W, "left" for X in X W."""
        if side == "right":
            return Operand(self.R_cols if axis_rows else self.R_rows, self.k1, self.F_q, self.P_q, self.S1)
        return Operand(self.R_rows, self.k1, self.P_q, self.F_q, self.S1)


def composite_split(A, k, p, q=1, seed=0, fmt="nv", sketch="gaussian", nnz=4, max_iters=64,
                    rows=True, cols=True, tap=False, dev_status=None):
    """Mean removal (averis_split, float32 residual tap) followed by the
    spectral split of the residual (metis_split), then the FP4 factors of the
    rank-(k + 1) low-rank part (metis_quantize_fp4).  Every step runs in the
    library's kernels; this function only arranges buffers."""
    if A.dim() != 2 or A.stride(1) != 1:
        raise ValueError("A must be a row-major 2-D tensor")
    m, n = A.shape
    dev = A.device
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
    av = averis_split(A, fmt, rows=False, cols=False, tap=True, dev_status=dev_status)
    sp = split(av.R_f32, k, p, q, seed, fmt, sketch=sketch, nnz=nnz, max_iters=max_iters, rows=rows,
               cols=cols, factors=False, tap=tap, dev_status=dev_status)
    k1 = k + 1
    ldk = (k1 + 3) // 4 * 4                     # rows start on 16-byte boundaries
    Fbuf = torch.zeros((m, ldk), dtype=torch.float32, device=dev)
    Pbuf = torch.zeros((n, ldk), dtype=torch.float32, device=dev)
    Fbuf[:, 0] = 1.0
    Fbuf[:, 1:k1] = sp.U
    Pbuf[:, 0] = av.mean
    Pbuf[:, 1:k1] = sp.V
    F32, P32 = Fbuf[:, :k1], Pbuf[:, :k1]
    F_q = quantize_fp4(F32, fmt, 0)
    P_q = quantize_fp4(P32, fmt, 0)
    S1 = torch.cat([torch.ones(1, dtype=torch.float32, device=dev), sp.S])
    return CompositeSplit(mean=av.mean, R1=av.R_f32, U=sp.U, S=sp.S, V=sp.V, F32=F32, P32=P32, F_q=F_q,
                          P_q=P_q, S1=S1, R_rows=sp.R_rows, R_cols=sp.R_cols, R2_f32=sp.R_f32, k=k, k1=k1,
                          fmt=sp.fmt, dev_status=dev_status)


def spectral_scale(G, U, S, V, cap, out=None, dev_status=None):
    """Adaptive spectral learning (metis_spectral_scale): G' = P_L G P_R with
    the gains min(S_1 / S_i, cap) along the split's singular directions.
    G: K x N float32 CUDA tensor; U (K x k), S (k), V (N x k) from split()."""
    if G.dim() != 2 or G.stride(1) != 1 or G.dtype != torch.float32:
        raise ValueError("G must be a row-major float32 2-D tensor")
    if not (U.is_contiguous() and S.is_contiguous() and V.is_contiguous()):
        raise ValueError("U, S and V must be contiguous")
    K, N = G.shape
    k = U.shape[1]
    if out is None:
        out = torch.empty((K, N), dtype=torch.float32, device=G.device)
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=G.device)
    _call_with_workspace(
        lib().metis_spectral_scale,
        (_ptr(G), K, N, G.stride(0), _ptr(U), _ptr(S), _ptr(V), k,
         ctypes.c_float(cap), _ptr(out)),
        (_ptr(dev_status), _stream()), G.device, "metis_spectral_scale")
    return out


# --------------------------------------------------------------------------
# activations kept in 8 bits, and the layer norm
# --------------------------------------------------------------------------

_DTYPE_CODE = {torch.bfloat16: BF16, torch.float32: F32}


def _matrix(t, name, device=None):
    """Check a row-major 2-D bf16/f32 CUDA tensor (any row stride of at least
    its width); returns its leading dimension."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a row-major 2-D tensor")
    if t.dtype not in _DTYPE_CODE:
        raise TypeError("only bfloat16 and float32 inputs are supported")
    rows, cols = t.shape
    ld, inner = t.stride()
    if cols == 0:
        raise ValueError(f"{name} must have at least one column")
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must be a row-major 2-D tensor")
    if rows < 2 and ld < cols:
        ld = cols                            # the stride of at most one row is never used
    if ld < cols:
        raise ValueError(f"{name}: rows overlap (stride {ld}, {cols} columns)")
    _on_device(t, name, device)
    return ld


def _on_device(t, name, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _vector(t, name, n, device, dtypes):
    """Check a contiguous vector of n elements on `device`."""
    if not isinstance(t, torch.Tensor) or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} elements")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _out_matrix(t, name, shape, device):
    ld = _matrix(t, name, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
    return ld


def _status_on(device, fn, *args):
    """fn(*args, stream)'s status with `device` current (the library launches on
    the current device) and that device's current stream."""
    index = device.index
    if torch.cuda.current_device() == index:
        return fn(*args, _stream_of(index))
    with torch.cuda.device(device):
        return fn(*args, _stream_of(index))


def _run_on(device, fn, what, *args):
    _check(_status_on(device, fn, *args), what)


class Act8:
    """A matrix kept in 8 bits (metis_act8_tensor): rows x cols, blocks of 32
    columns under one E8M0 scale, "mxint8" or "mxfp8" (E4M3) elements.

    codes: uint8 (rows, 32 * blocks); scales: uint8 (rows, blocks) with blocks
    = ceil(cols / 32); amax: float32 (ACT8_AMAX), whose largest is the largest
    magnitude held.  Without buffers an empty one is allocated; a program that
    stores an activation elsewhere (host memory, a file) keeps the three
    tensors and passes them back in.  (The tensors may be written to, not
    replaced.)"""

    def __init__(self, fmt, rows, cols, device="cuda", codes=None, scales=None, amax=None):
        if fmt not in ACT8_FMT:
            raise ValueError("the 8-bit formats are mxint8 and mxfp8")
        self.fmt, self.rows, self.cols = fmt, int(rows), int(cols)
        if self.rows < 0 or self.cols < 1:
            raise ValueError("an 8-bit matrix has at least 0 rows and 1 column")
        self.blocks = nb = (self.cols + 31) // 32
        if codes is None and scales is None and amax is None:
            # one buffer; the tensors of its parts are made when they are asked for
            n = self.rows * nb
            self._buf = torch.empty(4 * ACT8_AMAX + 33 * n, dtype=torch.uint8, device=device)
            self.device = self._buf.device
            at = self._buf.data_ptr()
            at = (at, at + 4 * ACT8_AMAX, at + 4 * ACT8_AMAX + 32 * n)
        else:
            for name, t, shape, dt in (("codes", codes, (self.rows, 32 * nb), torch.uint8),
                                       ("scales", scales, (self.rows, nb), torch.uint8),
                                       ("amax", amax, (ACT8_AMAX,), torch.float32)):
                if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dt or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {shape}")
                _on_device(t, name, codes.device)
            self.codes, self.scales, self.amax = codes, scales, amax
            self.device = codes.device
            at = (amax.data_ptr(), codes.data_ptr(), scales.data_ptr())
        self._s = Act8Struct(ACT8_FMT[fmt], self.rows, self.cols, at[1], at[2], at[0])

    def __getattr__(self, name):
        # reached for what is not set yet
        if name in ("codes", "scales", "amax") and "_buf" in self.__dict__:
            n, a = self.rows * self.blocks, 4 * ACT8_AMAX
            self.amax = self._buf[:a].view(torch.float32)
            self.codes = self._buf[a:a + 32 * n].view(self.rows, 32 * self.blocks)
            self.scales = self._buf[a + 32 * n:].view(self.rows, self.blocks)
            return self.__dict__[name]
        raise AttributeError(name)

    @property
    def nbytes(self):
        return 33 * self.rows * self.blocks + 4 * ACT8_AMAX


def _act8_out(out, fmt, rows, cols, device):
    if out is None:
        return Act8(fmt, rows, cols, device)
    if not isinstance(out, Act8) or (out.fmt, out.rows, out.cols) != (fmt, rows, cols):
        raise ValueError(f"out must be an Act8 of {rows} x {cols} in {fmt}")
    if out.device != device:
        raise ValueError(f"out is on {out.device}, not on {device}")
    return out


def save_act8(X, fmt="mxint8", out=None):
    """Put an activation (2-D bf16/f32 CUDA tensor, any row stride) into 8 bits
    (metis_act8_save); returns an Act8."""
    ld = _matrix(X, "X")
    rows, cols = X.shape
    out = _act8_out(out, fmt, rows, cols, X.device)
    _run_on(X.device, lib().metis_act8_save, "metis_act8_save",
            X.data_ptr(), _DTYPE_CODE[X.dtype], rows, cols, ld, ctypes.byref(out._s))
    return out


def restore_act8(a, dtype=torch.bfloat16, out=None):
    """The matrix an Act8 holds, in bf16 or f32 (metis_act8_restore)."""
    if not isinstance(a, Act8):
        raise TypeError("a must be an Act8")
    if out is None:
        if dtype not in _DTYPE_CODE:
            raise TypeError("only bfloat16 and float32 outputs are supported")
        out = torch.empty(a.rows, a.cols, dtype=dtype, device=a.device)
        ld = a.cols
    else:
        ld = _out_matrix(out, "out", (a.rows, a.cols), a.device)
    _run_on(a.device, lib().metis_act8_restore, "metis_act8_restore",
            ctypes.byref(a._s), out.data_ptr(), _DTYPE_CODE[out.dtype], ld)
    return out


def quantize_fp4_act8(a, fmt, axis=1, linear=False, out=None):
    """quantize_fp4 of the float32 matrix an Act8 holds, in one pass over the 8
    bits (metis_act8_quantize_fp4): axis 0 gives the X^T operand of
    dW = X^T dY."""
    if not isinstance(a, Act8):
        raise TypeError("a must be an Act8")
    if axis not in (0, 1):
        raise ValueError("axis is 0 or 1")
    outer, inner = (a.rows, a.cols) if axis == 1 else (a.cols, a.rows)
    if inner % 32 or outer == 0 or inner == 0:
        raise ValueError(f"the blocked dimension must be a multiple of 32 (it is {inner}) and no dimension 0")
    if out is None:
        out = QTensor(fmt, outer, inner, a.device, linear=linear, written=True)
    elif (out.fmt, out.outer, out.inner) != (FMT[fmt], outer, inner) or out.device != a.device:
        raise ValueError(f"out must be a QTensor of {outer} x {inner} on {a.device}")
    _run_on(a.device, lib().metis_act8_quantize_fp4, "metis_act8_quantize_fp4",
            ctypes.byref(a._s), axis, ctypes.byref(out.struct()))
    return out


class LayerNorm:
    """Outputs of layer_norm_fwd: Y, mean and rstd (None without stats) and
    saved, the input in 8 bits (None unless asked for)."""

    __slots__ = ("Y", "mean", "rstd", "saved")

    def __init__(self, Y, mean, rstd, saved):
        self.Y, self.mean, self.rstd, self.saved = Y, mean, rstd, saved


def _affine(weight, bias, cols, device):
    """Pointers of weight and bias (either may be None) and their dtype code."""
    w = b = None
    code = BF16
    if weight is not None:
        _vector(weight, "weight", cols, device, _DTYPE_CODE)
        code, w = _DTYPE_CODE[weight.dtype], weight.data_ptr()
    if bias is not None:
        _vector(bias, "bias", cols, device, _DTYPE_CODE)
        if weight is not None and weight.dtype != bias.dtype:
            raise TypeError("weight and bias must have one dtype")
        code, b = _DTYPE_CODE[bias.dtype], bias.data_ptr()
    return w, b, code


def layer_norm_fwd(X, weight=None, bias=None, eps=1e-5, out_dtype=None, save=None, stats=True, out=None):
    """Layer norm over the columns of X (metis_layer_norm_fwd).

    X: 2-D bf16/f32 CUDA tensor, any row stride; weight, bias: vectors (bf16 or
    f32) or None.  out_dtype: dtype of Y (X's).  save: "mxint8" or "mxfp8" also
    keeps X in 8 bits; pass the result's ``saved`` to layer_norm_bwd in place of
    X.  (One pass over X where the rows of X and Y begin on 16-byte boundaries
    and are a multiple of 8 columns, at most 32768; save_act8's kernel first
    otherwise.)  stats=False: Y alone (inference).  out: Y's tensor (X itself is
    allowed if it has Y's dtype, no other overlap)."""
    ldx = _matrix(X, "X")
    dev = X.device
    rows, cols = X.shape
    w, b, wdt = _affine(weight, bias, cols, dev)
    if not eps >= 0:
        raise ValueError("eps must be 0 or more")
    if out is None:
        out = torch.empty(rows, cols, dtype=out_dtype or X.dtype, device=dev)
        if out.dtype not in _DTYPE_CODE:
            raise TypeError("only bfloat16 and float32 outputs are supported")
        ldy = cols
    else:
        ldy = _out_matrix(out, "out", (rows, cols), dev)
        if out.data_ptr() == X.data_ptr() and rows and (out.dtype != X.dtype or ldy != ldx):
            raise ValueError("out may be X itself, not another view of its memory")
    saved = None if save is None else Act8(save, rows, cols, dev)
    mean = rstd = mp = rp = None
    if stats:
        mean = torch.empty(rows, dtype=torch.float32, device=dev)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    _run_on(dev, lib().metis_layer_norm_fwd, "metis_layer_norm_fwd",
            X.data_ptr(), _DTYPE_CODE[X.dtype], rows, cols, ldx, w, b, wdt, eps, out.data_ptr(),
            _DTYPE_CODE[out.dtype], ldy, mp, rp, None if saved is None else ctypes.byref(saved._s))
    return LayerNorm(out, mean, rstd, saved)


_norm_ws = {}     # workspace bytes of layer_norm_bwd by device and sizes


def layer_norm_bwd(dY, X, mean, rstd, weight=None, out_dtype=None, want_dx=True, want_dw=True, want_db=True,
                   out=None):
    """(dX, dweight, dbias) of layer_norm_fwd (metis_layer_norm_bwd).

    X: the forward's input, or the Act8 it kept; mean, rstd: the forward's.
    out_dtype: dtype of dX (dY's); dweight and dbias are float32.  An output
    that is not wanted is None.  out: dX's tensor (dY itself is allowed if it has
    dX's dtype, no other overlap with an input)."""
    ldg = _matrix(dY, "dY")
    dev = dY.device
    rows, cols = dY.shape
    if not (want_dx or want_dw or want_db):
        raise ValueError("at least one gradient must be wanted")
    xp, xdt, ldx, sp = None, BF16, cols, None
    if isinstance(X, Act8):
        if (X.rows, X.cols) != (rows, cols):
            raise ValueError(f"X is {X.rows} x {X.cols}, dY {rows} x {cols}")
        if X.device != dev:
            raise ValueError(f"X is on {X.device}, not on {dev}")
        sp = ctypes.byref(X._s)
    else:
        ldx = _matrix(X, "X", dev)
        if X.shape != dY.shape:
            raise ValueError(f"X is {tuple(X.shape)}, dY {tuple(dY.shape)}")
        xp, xdt = X.data_ptr(), _DTYPE_CODE[X.dtype]
    _vector(mean, "mean", rows, dev, (torch.float32,))
    _vector(rstd, "rstd", rows, dev, (torch.float32,))
    w, _, wdt = _affine(weight, None, cols, dev)
    ldd, dp, ddt = cols, None, BF16
    if want_dx:
        if out is None:
            out = torch.empty(rows, cols, dtype=out_dtype or dY.dtype, device=dev)
            if out.dtype not in _DTYPE_CODE:
                raise TypeError("only bfloat16 and float32 outputs are supported")
        else:
            ldd = _out_matrix(out, "out", (rows, cols), dev)
            if out.data_ptr() == dY.data_ptr() and rows and (out.dtype != dY.dtype or ldd != ldg):
                raise ValueError("out may be dY itself, not another view of its memory")
        dp, ddt = out.data_ptr(), _DTYPE_CODE[out.dtype]
    else:
        out = None
    dw = torch.empty(cols, dtype=torch.float32, device=dev) if want_dw else None
    db = torch.empty(cols, dtype=torch.float32, device=dev) if want_db else None
    args = (dY.data_ptr(), _DTYPE_CODE[dY.dtype], rows, cols, ldg, xp, xdt, ldx, sp,
            mean.data_ptr() if rows else None, rstd.data_ptr() if rows else None, w, wdt, dp, ddt, ldd,
            None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr())
    # The workspace is this call's alone (two threads may call at once); it stays
    # with the stream's allocator, or with the graph that captures the call.  The
    # size last asked for with these sizes is tried first: types and alignments may
    # need more, which the library refuses before anything is launched.
    fn = lib().metis_layer_norm_bwd
    key = (dev.index, rows, cols)
    need = _norm_ws.get(key, 256)
    for last in (False, True):
        size = ctypes.c_size_t(need)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        status = _status_on(dev, fn, *args, ws.data_ptr(), ctypes.byref(size))
        if status != ERR_WORKSPACE or last:
            _check(status, "metis_layer_norm_bwd")
            break
        _check(_status_on(dev, fn, *args, None, ctypes.byref(size)), "metis_layer_norm_bwd (workspace query)")
        need = size.value
        if len(_norm_ws) >= 4096:
            _norm_ws.clear()
        _norm_ws[key] = need
    return out, dw, db


def selftest_wait_timeout(limit_ns=1_000_000, device="cuda"):
    """Run the library's bounded device wait on a barrier that never
    completes (metis_selftest_wait_timeout); returns the device status word
    after the launch finished (DEV_TIMEOUT set when the wait ended itself)."""
    st = torch.zeros(1, dtype=torch.int32, device=device)
    _check(lib().metis_selftest_wait_timeout(int(limit_ns), _ptr(st), _stream()), "metis_selftest_wait_timeout")
    torch.cuda.synchronize()
    return int(st.item())
