"""The training step with inputs kept in 8 bits and a layer norm
(spectral_domain_quantization_b200.mlp): the calls together, as a training loop
makes them.

Every product is held to the oracle's float64 product of the FP4 operands the
library used (2e-3, the product tolerance); the operand X^T of each dW is the
oracle's quantization of what the 8 bits hold, byte for byte; the norm's outputs
and gradients are held to float64 on the tensors the step used, with the bounds of
tests/test_gpu_layer_norm.py."""
import numpy as np
import pytest
import torch

from oracle import act8, fp4, gemm
from oracle import mlp as omlp
from spectral_domain_quantization_b200 import api, mlp

from gpu_helpers import assert_fp4_equal, read_fp4, rel_fro
from test_gpu_layer_norm import check_bwd, check_fwd, np64

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.float32(a))).cuda()


def operand(op):
    R = read_fp4(op.R)
    if op.k == 0:
        return gemm.Operand(R)
    return gemm.Operand(R, op.k, read_fp4(op.P), read_fp4(op.F), op.S.cpu().numpy().astype(np.float64))


def held(x, fmt):
    """The float32 values that 8 bits hold of a tensor."""
    return np.float32(act8.load(*act8.save(np64(x), fmt), x.shape[1], fmt))


@pytest.mark.parametrize("kind,fmt", [("fp4", "nv"), ("fp4", "mx"), ("metis", "nv")])
@pytest.mark.parametrize("saved", [None, "mxint8", "mxfp8"])
def test_norm_step(kind, fmt, saved):
    X, T, (W1, W2) = omlp.problem()
    rng = np.random.default_rng(5)
    g, b = dev(1 + 0.2 * rng.standard_normal(W1.shape[1])), dev(0.1 * rng.standard_normal(W1.shape[1]))
    Xd = dev(X)
    loss, grads, record = mlp.norm_step((dev(W1), dev(W2), g, b), Xd, dev(T), mlp.Policy(kind, fmt, saved=saved))
    torch.cuda.synchronize()
    assert [r[0] for r in record] == ["fwd", "fwd", "dx", "dw", "norm", "dw"]
    assert np.isfinite(loss) and all(torch.isfinite(t).all() for t in grads)
    for r in record:
        if r[0] != "norm":
            assert rel_fro(r[3].cpu().numpy(), gemm.gemm(operand(r[1]), operand(r[2]))) < 2e-3, r[0]
    _, Z1, norm, dN, ngrads = record[4]
    check_fwd(norm, Z1, g, b)
    z = np64(Z1) if saved is None else np.float64(held(Z1, saved))
    check_bwd(ngrads, dN, z, norm.mean, norm.rstd, g)
    assert grads[2] is ngrads[1] and grads[3] is ngrads[2]
    if saved is not None:
        A1 = torch.relu(norm.Y)
        assert_fp4_equal(record[3][1].R, fp4.quantize(held(A1, saved), fmt, 0))
        assert_fp4_equal(record[5][1].R, fp4.quantize(held(Xd, saved), fmt, 0))


@pytest.mark.parametrize("saved", ["mxint8", "mxfp8"])
def test_step_from_8_bits(saved):
    # the same step: only X^T of each dW comes from the 8 bits
    X, T, (W1, W2) = omlp.problem()
    Xd = dev(X)
    loss0, _, rec0 = mlp.step((dev(W1), dev(W2)), Xd, dev(T), mlp.Policy("fp4", "nv"))
    loss, grads, rec = mlp.step((dev(W1), dev(W2)), Xd, dev(T), mlp.Policy("fp4", "nv", saved=saved))
    assert loss == loss0 and torch.equal(rec[0][3], rec0[0][3]) and torch.equal(rec[2][3], rec0[2][3])
    assert_fp4_equal(rec[4][1].R, fp4.quantize(held(Xd, saved), "nv", 0))
    for name, left, right, out in rec:
        assert rel_fro(out.cpu().numpy(), gemm.gemm(operand(left), operand(right))) < 2e-3, name


def test_training_runs():
    X, T, (W1, W2) = omlp.problem()
    n = W1.shape[1]
    params = (dev(W1), dev(W2), torch.ones(n, device="cuda"), torch.zeros(n, device="cuda"))
    losses, out = mlp.train(params, dev(X), dev(T), mlp.Policy("fp4", "nv", saved="mxint8"), 0.1, 5)
    assert len(losses) == 5 and np.all(np.isfinite(losses)) and len(out) == 4
    assert not any(torch.equal(p, q) for p, q in zip(params, out))
    with pytest.raises(ValueError):
        mlp.Policy(saved="int8")


def test_captured_step():
    # norm, 8-bit copy and dW in one graph, replayed on new inputs
    g0 = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn((256, 192), generator=g0, device="cuda").bfloat16()
    dY = (0.1 * torch.randn((256, 320), generator=g0, device="cuda")).bfloat16()
    w, b = torch.ones(192, device="cuda"), torch.zeros(192, device="cuda")

    def step():
        r = api.layer_norm_fwd(X, w, b)
        a = api.save_act8(r.Y)
        xt, dy = api.Operand(api.quantize_fp4_act8(a, "nv", 0)), api.Operand(api.quantize_fp4(dY, "nv", 0))
        return r.Y, api.linear_bwd(None, None, xt, dy, 256, 320, 192, want_dx=False)[1]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, dW = step()
    for k in range(3):
        X.normal_(generator=g0)
        dY.normal_(generator=g0)
        graph.replay()
        torch.cuda.synchronize()
        Y2, dW2 = step()
        assert torch.equal(Y, Y2) and torch.equal(dW, dW2)
