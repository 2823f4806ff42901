"""The tensor scale of an MXFP4 result: 1 from the call on, whenever and wherever it is
first read, and the result's own."""
import pytest
import torch

from spectral_domain_quantization_b200 import api

pytestmark = pytest.mark.gpu


def results():
    X = torch.randn((64, 96), device="cuda")
    return [api.quantize_fp4(X, "mx", 1), api.quantize_fp4(X, "mx", 0),
            api.quantize_fp4_act8(api.save_act8(X), "mx", 0)]


def test_first_read_in_a_capture():
    # a capture runs nothing: what is read there is the value that was there before
    qs = results()
    torch.cuda.synchronize()
    sums = [torch.empty(1, device="cuda") for _ in qs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fill = torch.full((1 << 16,), 7.0, device="cuda")     # the graph's own memory
        for q, s in zip(qs, sums):
            torch.add(q.tensor_scale, fill[:1], out=s)
    assert [float(q.tensor_scale) for q in qs] == [1.0] * 3
    g.replay()
    torch.cuda.synchronize()
    assert [float(s) for s in sums] == [8.0] * 3
    del g, fill
    torch.cuda.empty_cache()
    torch.full((1 << 22,), 3.0, device="cuda")
    assert [float(q.tensor_scale) for q in qs] == [1.0] * 3


def test_result_of_a_capture():
    X = torch.randn((64, 96), device="cuda")
    api.quantize_fp4(X, "mx", 1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = api.quantize_fp4(X, "mx", 1)
        a = api.quantize_fp4_act8(api.save_act8(X), "mx", 0)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert float(q.tensor_scale) == 1.0 and float(a.tensor_scale) == 1.0


def test_many_results_and_streams():
    # more results than are made ready at once, on two streams in turn; each one's own
    X = torch.randn((32, 32), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qs = []
    for k in range(2500):
        with torch.cuda.stream(side if k % 3 == 0 else torch.cuda.current_stream()):
            qs.append(api.quantize_fp4(X, "mx", k % 2))
    torch.cuda.synchronize()
    assert len({q.tensor_scale.data_ptr() for q in qs}) == len(qs)
    assert float(torch.cat([q.tensor_scale for q in qs]).min()) == 1.0
    for k, q in enumerate(qs[:40]):
        q.tensor_scale.fill_(k + 2)
    assert float(torch.cat([q.tensor_scale for q in qs[40:]]).max()) == 1.0
    assert [float(q.tensor_scale) for q in qs[:40]] == [k + 2 for k in range(40)]


def test_given_result():
    # a result passed back in keeps the value it has (MXFP4's is not written)
    X = torch.randn((64, 96), device="cuda")
    q = api.quantize_fp4(X, "mx", 1)
    assert api.quantize_fp4(2 * X, "mx", 1, out=q) is q and float(q.tensor_scale) == 1.0
    own = api.QTensor("mx", 64, 96)
    assert api.quantize_fp4(X, "mx", 1, out=own) is own and float(own.tensor_scale) == 1.0
