"""Two threads that call on one stream: the scratch memory of their calls (host
side, with a stand-in for the library's function; ctypes lets the other thread run
during a call)."""
import ctypes
import threading

import pytest
import torch

from spectral_domain_quantization_b200 import api

CPU = torch.device("cpu", 0)


@pytest.fixture
def one_stream(monkeypatch):
    monkeypatch.setattr(api, "_stream_of", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


def sized(need, during):
    """A library function that needs `need` bytes, and calls during(workspace address) once it has them."""
    def fn(ws, size, stream):
        if ws is None:
            size._obj.value = need
            return api.OK
        if size._obj.value < need:
            return api.ERR_WORKSPACE
        during(ws.value if isinstance(ws, ctypes.c_void_p) else ws)
        return api.OK
    return fn


def test_calls_of_two_threads_share_no_scratch(one_stream):
    barrier = threading.Barrier(2, timeout=20)
    seen = {}

    def work(k):
        def during(at):
            barrier.wait()                        # both calls are under way
            seen.setdefault(k, []).append(at)
            barrier.wait()
        for need in (1000, 1000, 5000, 2000):     # a first buffer, one that is held, a larger one
            api._call_with_workspace(sized(need, during), (), (0,), CPU, "stand-in")

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(seen[0]) == len(seen[1]) == 4
    assert all(a != b for a, b in zip(seen[0], seen[1]))


def test_one_thread_keeps_its_buffer(one_stream):
    at = []
    for need in (1 << 12, 300, 1 << 12):
        api._call_with_workspace(sized(need, at.append), (), (0,), CPU, "stand-in")
    assert at[0] == at[1] == at[2]
