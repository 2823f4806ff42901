"""Two threads that call on one stream: every result is the one a call alone gives."""
import threading

import pytest
import torch

from spectral_domain_quantization_b200 import api

pytestmark = pytest.mark.gpu


def run_two(calls, rounds=100):
    """Each call in a thread of its own, `rounds` times; their results."""
    got = [[], []]

    def work(k):
        for _ in range(rounds):
            got[k].append(calls[k]())

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [len(g) for g in got] == [rounds, rounds]
    return got


@pytest.mark.parametrize("axis", [0, 1])
def test_quantize(axis):
    # tensors of very different maxima: NVFP4's is in the scratch memory between kernels
    gen = torch.Generator(device="cuda").manual_seed(80)
    X = [torch.randn((1024, 2048), generator=gen, device="cuda").mul_(s) for s in (1.0, 1e4)]
    calls = [lambda k=k: api.quantize_fp4(X[k], "nv", axis) for k in range(2)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    for w, got in zip(want, run_two(calls)):
        for q in got:
            assert torch.equal(q.tensor_scale, w.tensor_scale)
            assert torch.equal(q.scales, w.scales) and torch.equal(q.codes, w.codes)


def test_products_with_low_rank_terms():
    # the low-rank terms of both operands are put together in scratch memory
    M, K, N = 512, 384, 256
    gen = torch.Generator(device="cuda").manual_seed(81)
    calls = []
    for s in (1.0, 50.0):
        dy = torch.randn((M, N), generator=gen, device="cuda").mul_(s)
        x = torch.randn((M, K), generator=gen, device="cuda")
        d = api.split(dy, 8, 8, 1, 0, "nv", rows=True, cols=True)
        w = api.split(torch.randn((K, N), generator=gen, device="cuda"), 8, 8, 1, 0, "nv", rows=True, cols=True)
        xt = api.Operand(api.quantize_fp4(x, "nv", 0))
        left = api.Operand(d.R_rows, 8, d.V_q, d.U_q, d.S)
        right = api.Operand(w.R_rows, 8, w.V_q, w.U_q, w.S)
        dm = api.Operand(d.R_cols, 8, d.U_q, d.V_q, d.S)
        calls.append(lambda a=left, b=right, c=xt, e=dm: api.linear_bwd(a, b, c, e, M, N, K))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    for w, got in zip(want, run_two(calls)):
        assert all(torch.equal(p, q) for pair in got for p, q in zip(pair, w))
