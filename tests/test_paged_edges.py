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


def test_addresses_that_are_not_aligned_are_refused():
    """Before any launch: an int or a float read from such an address would end the caller's context."""
    from decode_kv_cache_gb300 import build as b
    b.build()
    lib = lf.load_library()
    at = lambda i, off=0: 0x10000 * i + off  # noqa: E731

    def pages(err=None):
        return ctypes.byref(lf.LFPages(lf.LF_BF16, 8, 128, 16, 100, 8 * 16 * 128, 16 * 128, 128, at(1), at(2), err))

    for off in (1, 2, 3):
        for err, table, lens in ((at(9, off), at(3), at(4)), (None, at(3, off), at(4)), (None, at(3), at(4, off))):
            for code in (lib.lf_paged_append(pages(err), 4, table, 10, lens, at(5), at(5), at(6), 7, None),
                         lib.lf_paged_decode(pages(err), 4, table, 1000, lens, 32, at(5), None, None, at(5), None, 0, 0,
                                             at(7), 1 << 40, None),
                         lib.lf_paged_prompt(pages(err), 4, table, 10, lens, 32, at(5), at(6), 7, 3, at(5), None, 0, 0,
                                             at(7), 1 << 40, None)):
                assert code == lf.LF_ERR_ARG and "4-byte aligned" in lf.lf_last_error()
        for code, name in (
                (lib.lf_paged_append(pages(), 4, at(3), 10, at(4), at(5), at(5), at(6, off), 7, None), "new_start"),
                (lib.lf_paged_decode(pages(), 4, at(3), 1000, at(4), 32, at(5), None, None, at(5), at(8, off), 0, 0, at(7),
                                     1 << 40, None), "lse"),
                (lib.lf_paged_prompt(pages(), 4, at(3), 10, at(4), 32, at(5), at(6, off), 7, 3, at(5), None, 0, 0, at(7),
                                     1 << 40, None), "q_start"),
                (lib.lf_paged_prompt(pages(), 4, at(3), 10, at(4), 32, at(5), at(6), 7, 3, at(5), at(8, off), 0, 0, at(7),
                                     1 << 40, None), "lse")):
            assert code == lf.LF_ERR_ARG and "4-byte aligned" in lf.lf_last_error(), name
