"""A small synthetic MLP trained with W4A4G4 linear layers on the GPU.

Source: "Metis: Training LLMs with FP4 Quantization" abstract (W4A4G4: the
forward product and both backward products of every linear layer run on FP4
operands, and the spectral split keeps the FP4 training loss close to the
higher-precision run); SII release section 2.4 item 1 (the dominant low-rank
part and the long-tail residual are quantized independently).

The workload (reading R31): a two-layer ReLU regression Y = relu(X W1) W2 with
loss ||Y - T||^2 / (2 n d_out), trained by plain SGD.  Every product of every
layer goes through the library's C ABI under one policy:

  "fp4"    each operand quantized along the product's contraction axis
           (forward: X and W along K; dX = dZ W^T: dZ and W along N;
           dW = X^T dZ: X and dZ along M);
  "metis"  as "fp4", but the weight and the output gradient enter as spectral
           split operands (metis_split: R_q + U_q diag(S) V_q^T), in the
           operand roles of metis_linear_fwd / metis_linear_bwd.

With ``Policy(saved="mxint8")`` (or "mxfp8") every layer's input is kept in 8
bits between the forward and the backward pass, and the operand X^T of dW is
quantized from those.  ``norm_step`` is the same network with a layer norm
behind the first layer, Y = relu(norm(X W1) g + b) W2, whose backward pass takes
its input from the 8 bits too.

The products, quantizations, splits, norms and 8-bit copies all run in the
library's kernels; the ReLU, its mask, the loss and the SGD update are the
workload around the layer and run as float32 torch operations.  ``step`` returns every product's FP4
operands and output, so that a test can hold each product to the oracle's
float64 product of exactly those operands.
"""
import torch

from . import api


class Policy:
    def __init__(self, kind="fp4", fmt="nv", k=8, p=8, q=1, seed=0, saved=None):
        if kind not in ("fp4", "metis"):
            raise ValueError("policy is fp4 or metis")
        if saved is not None and saved not in api.ACT8_FMT:
            raise ValueError("saved is None, mxint8 or mxfp8")
        self.kind, self.fmt, self.k, self.p, self.q, self.seed = kind, fmt, k, p, q, seed
        self.saved = saved


def _split(A, pol, salt):
    return api.split(A.contiguous(), pol.k, pol.p, pol.q, pol.seed + salt, pol.fmt, rows=True, cols=True)


def keep(X, pol):
    """What stays of a layer's input for its backward pass."""
    return X if pol.saved is None else api.save_act8(X, pol.saved)


def forward(X, W, pol, salt, record):
    """Z = X W (X: n x K, W: K x N, float32 CUDA tensors)."""
    M, K = X.shape
    N = W.shape[1]
    xop = api.Operand(api.quantize_fp4(X.contiguous(), pol.fmt, 1))          # X along K
    if pol.kind == "fp4":
        wop = api.Operand(api.quantize_fp4(W.contiguous(), pol.fmt, 0))      # W along K
    else:
        wop = _split(W, pol, salt).operand("right")
    Z = api.linear_fwd(xop, wop, M, N, K)
    record.append(("fwd", xop, wop, Z))
    return Z


def backward(dZ, X, W, pol, salt, record, need_dx=True):
    """(dX, dW) of Z = X W: dX = dZ W^T (contraction over N), dW = X^T dZ
    (contraction over the batch M).  X: the layer's input, or what ``keep`` made
    of it."""
    M, (K, N) = dZ.shape[0], W.shape
    if pol.kind == "fp4":
        dz_n = api.Operand(api.quantize_fp4(dZ.contiguous(), pol.fmt, 1))    # dZ along N
        dz_m = api.Operand(api.quantize_fp4(dZ.contiguous(), pol.fmt, 0))    # dZ along M
        wt = api.Operand(api.quantize_fp4(W.contiguous(), pol.fmt, 1)) if need_dx else None   # W^T along N
    else:
        sd = _split(dZ, pol, salt + 1)
        dz_n, dz_m = sd.operand("left"), sd.operand("right")
        wt = None
        if need_dx:
            sw = _split(W, pol, salt)
            wt = api.Operand(sw.R_rows, pol.k, sw.V_q, sw.U_q, sw.S)
    xt = api.Operand(api.quantize_fp4_act8(X, pol.fmt, 0) if isinstance(X, api.Act8)
                     else api.quantize_fp4(X.contiguous(), pol.fmt, 0))       # X^T along M
    dX, dW = api.linear_bwd(dz_n if need_dx else None, wt, xt, dz_m, M, N, K, want_dx=need_dx)
    if need_dx:
        record.append(("dx", dz_n, wt, dX))
    record.append(("dw", xt, dz_m, dW))
    return dX, dW


def step(params, X, T, pol, t=0):
    """Loss and (dW1, dW2) at ``params``; also the record of every product:
    (name, left operand, right operand, output)."""
    W1, W2 = params
    record = []
    Z1 = forward(X, W1, pol, 8 * t, record)
    A1 = torch.relu(Z1)
    x_kept, a_kept = keep(X, pol), keep(A1, pol)
    Y = forward(A1, W2, pol, 8 * t + 2, record)
    D = Y - T
    loss = 0.5 * float((D * D).sum()) / D.numel()
    dY = D / D.numel()
    dA1, dW2 = backward(dY, a_kept, W2, pol, 8 * t + 4, record)
    dZ1 = dA1 * (Z1 > 0)
    _, dW1 = backward(dZ1, x_kept, W1, pol, 8 * t + 6, record, need_dx=False)
    return loss, (dW1, dW2), record


def norm_step(params, X, T, pol, t=0):
    """Loss and (dW1, dW2, dg, db) of the network with a layer norm at ``params``
    = (W1, W2, g, b); also the record of every product and, as ("norm", input,
    norm, dN, gradients), of the norm."""
    W1, W2, g, b = params
    record = []
    Z1 = forward(X, W1, pol, 8 * t, record)
    norm = api.layer_norm_fwd(Z1, g, b, save=pol.saved)
    A1 = torch.relu(norm.Y)
    x_kept, a_kept = keep(X, pol), keep(A1, pol)
    Y = forward(A1, W2, pol, 8 * t + 2, record)
    D = Y - T
    loss = 0.5 * float((D * D).sum()) / D.numel()
    dY = D / D.numel()
    dA1, dW2 = backward(dY, a_kept, W2, pol, 8 * t + 4, record)
    dN = dA1 * (norm.Y > 0)
    z_kept = Z1 if norm.saved is None else norm.saved
    grads = api.layer_norm_bwd(dN, z_kept, norm.mean, norm.rstd, g)
    record.append(("norm", Z1, norm, dN, grads))
    dZ1, dg, db = grads
    _, dW1 = backward(dZ1, x_kept, W1, pol, 8 * t + 6, record, need_dx=False)
    return loss, (dW1, dW2, dg, db), record


def train(params, X, T, pol, lr, steps):
    """Plain SGD of ``step``, or of ``norm_step`` for four parameters; returns the
    loss before every step and the final params."""
    one = step if len(params) == 2 else norm_step
    losses = []
    for t in range(steps):
        loss, grads, _ = one(params, X, T, pol, t)
        losses.append(loss)
        params = tuple(w - lr * d for w, d in zip(params, grads))
    return losses, params
