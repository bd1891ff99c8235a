"""Paged key-value cache on the CPU, at the edges of what its Python calls allow."""
import ctypes
import types

import pytest
import torch

from decode_kv_cache_gb300 import longflow as lf


def cache_on(index):
    """A cache's Python side without its pools."""
    c = lf.LFPagedCache.__new__(lf.LFPagedCache)
    c.device, c._index = torch.device("cuda", index), index
    return c


@pytest.mark.parametrize("stream", [types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77),
                                    types.SimpleNamespace(device=torch.device("cpu")), "side", 1.5],
                         ids=["another device", "cpu", "text", "number"])
def test_streams_that_are_not_of_the_device_are_refused(monkeypatch, stream):
    """A call on a stream of another device would run on the cache's device, on a stream that nobody named."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    called = []
    with pytest.raises(lf.LFError, match="stream: expected a stream of cuda:0"):
        cache_on(0)._run(stream, called.append)
    assert not called


def test_taking_errors_from_nowhere_is_refused():
    from decode_kv_cache_gb300 import build as b
    b.build()
    lib, p = lf.load_library(), lf.LFPages()
    call = lambda: lib.lf_paged_take_errors(ctypes.byref(p), taken, None)  # noqa: E731
    taken = 0x10000
    assert lib.lf_paged_take_errors(None, taken, None) == lf.LF_ERR_ARG and "null" in lf.lf_last_error()
    assert call() == lf.LF_ERR_ARG and "error word" in lf.lf_last_error()
    p.err, taken = 0x20000, None
    assert call() == lf.LF_ERR_ARG and "taken" in lf.lf_last_error()
    taken = 0x10002
    assert call() == lf.LF_ERR_ARG and "aligned" in lf.lf_last_error()
    p.err, taken = 0x20001, 0x10000
    assert call() == lf.LF_ERR_ARG and "aligned" in lf.lf_last_error()


def test_pools_are_made_on_the_device_that_is_named(monkeypatch):
    """"cuda" is the current device, as torch has it, and no other kind of device turns into cuda:0."""
    made = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: made.append(device))
    monkeypatch.setattr(lf.LFPagedCache, "_take", lambda self, k, v: None)
    for device, want in ((None, 3), ("cuda", 3), ("cuda:1", 1), (torch.device("cuda", 0), 0), (2, 2)):
        lf.LFPagedCache(1, 4, 16, 8, 128, device=device)
        assert made.pop() == made.pop() == torch.device("cuda", want)
    for device in ("cpu", torch.device("meta")):
        with pytest.raises(lf.LFError, match="expected a CUDA device"):
            lf.LFPagedCache(1, 4, 16, 8, 128, device=device)
    assert not made
