"""Paged key-value cache on the CPU: its oracle against library attention, and every refusal of
the C entry points, which come before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest
import torch

from decode_kv_cache_gb300 import longflow as lf
from oracle import paged_oracle

A, B, C, D, E = (0x10000 * i for i in range(1, 6))   # aligned addresses that nothing reads


@pytest.fixture(scope="module")
def lib():
    from decode_kv_cache_gb300 import build as b
    b.build()
    return lf.load_library()


def pages(**kw):
    p = dict(dtype=lf.LF_BF16, kv_heads=8, head_dim=128, page_size=16, num_pages=100,
             page_stride=8 * 16 * 128, head_stride=16 * 128, token_stride=128, k=A, v=B, err=None)
    p.update(kw)
    s = lf.LFPages()
    for n, x in p.items():
        setattr(s, n, x)
    return s


# ---- the oracle ---------------------------------------------------------------------------------

@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (5, 3), (1, 2), (100, 4)])
def test_oracle_against_library_attention(window, sinks):
    g = torch.Generator().manual_seed(3)
    n, rows, hq, hkv, d = 23, 9, 4, 2, 16
    q = torch.randn(rows, hq, d, generator=g, dtype=torch.float64)
    k, v = (torch.randn(hkv, n, d, generator=g, dtype=torch.float64) for _ in range(2))
    see = paged_oracle.visible(np.arange(n - rows, n), n, window, sinks)
    out, lse, size, _ = paged_oracle.attend(q, k, v, see)
    rep = lambda x: x.repeat_interleave(hq // hkv, 0)  # noqa: E731
    ref = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), rep(k), rep(v), attn_mask=torch.from_numpy(see)[None]).transpose(0, 1)
    np.testing.assert_allclose(out, ref.numpy(), rtol=1e-12, atol=1e-12)
    z = torch.einsum("rhd,hnd->rhn", q, rep(k)) / math.sqrt(d)
    z = z.masked_fill(~torch.from_numpy(see)[:, None], -math.inf)
    np.testing.assert_allclose(lse, torch.logsumexp(z, -1).numpy(), rtol=1e-12)
    assert (size >= np.abs(out) - 1e-12).all()


def test_oracle_window_and_sinks_by_hand():
    see = paged_oracle.visible([0, 3, 9], 10, 3, 2)
    assert np.flatnonzero(see[0]).tolist() == [0]
    assert np.flatnonzero(see[1]).tolist() == [0, 1, 2, 3]
    assert np.flatnonzero(see[2]).tolist() == [0, 1, 7, 8, 9]
    assert paged_oracle.visible([-1], 4, 0, 0).sum() == 0
    out, lse, _, _ = paged_oracle.attend(np.ones((1, 1, 4)), np.ones((1, 4, 4)), np.ones((1, 4, 4)),
                                         paged_oracle.visible([-1], 4, 0, 0))
    assert (out == 0).all() and np.isneginf(lse).all()


def test_oracle_append_and_gather_are_inverse():
    rng = np.random.default_rng(1)
    table, lens, start = [[3, 0, 6], [5, 2, 9]], [5, 4], [0, 2, 6]
    pool, new = rng.normal(size=(7, 2, 2, 4)), rng.normal(size=(6, 2, 4))
    after = paged_oracle.append(pool, table, lens, new, start, 2)
    for b in range(2):
        n = start[b + 1] - start[b]
        got = paged_oracle.gather(after, table[b], lens[b], 2)
        np.testing.assert_array_equal(got[:, lens[b] - n:], new[start[b]:start[b + 1]].swapaxes(0, 1))
    changed = (after != pool).any(axis=(1, 3))
    assert changed.sum() == 6


# ---- refusals -------------------------------------------------------------------------------------

def append(lib, p, batch=4, table=C, width=10, lens=D, k=E, v=E, start=D, total=7):
    return lib.lf_paged_append(None if p is None else ctypes.byref(p), batch, table, width, lens, k, v,
                               start, total, None)


def decode(lib, p, batch=4, table=C, width=1000, lens=D, hq=32, q=E, k=E, v=E, out=E, lse=None, window=0,
           sinks=0, ws=E, nbytes=1 << 40):
    return lib.lf_paged_decode(None if p is None else ctypes.byref(p), batch, table, width, lens, hq, q, k,
                               v, out, lse, window, sinks, ws, nbytes, None)


def prompt(lib, p, batch=4, table=C, width=10, lens=D, hq=32, q=E, start=D, total=7, most=3, out=E, lse=None,
           window=0, sinks=0, ws=E, nbytes=1 << 40):
    return lib.lf_paged_prompt(None if p is None else ctypes.byref(p), batch, table, width, lens, hq, q,
                               start, total, most, out, lse, window, sinks, ws, nbytes, None)


BAD_POOLS = [
    (dict(dtype=2), "dtype"), (dict(head_dim=96), "head_dim 96"), (dict(kv_heads=0), "kv_heads"),
    (dict(page_size=0), "page_size"), (dict(num_pages=0), "num_pages"), (dict(k=None), "pools"),
    (dict(v=None), "pools"), (dict(k=A + 8), "16-byte aligned"), (dict(page_stride=-128), "strides"),
    (dict(token_stride=129), "multiples of 16 bytes"), (dict(head_stride=1 << 41), "strides"),
]


@pytest.mark.parametrize("call", [append, decode, prompt], ids=lambda f: f.__name__)
@pytest.mark.parametrize("bad,msg", BAD_POOLS, ids=lambda x: str(x))
def test_bad_pools_are_refused(lib, call, bad, msg):
    assert call(lib, pages(**bad)) in (lf.LF_ERR_ARG, lf.LF_ERR_UNSUPPORTED)
    assert msg in lf.lf_last_error()


@pytest.mark.parametrize("call", [append, decode, prompt], ids=lambda f: f.__name__)
def test_bad_sequences_are_refused(lib, call):
    assert call(lib, None) == lf.LF_ERR_ARG
    for kw, msg in [(dict(batch=0), "batch"), (dict(batch=65536), "batch"), (dict(width=0), "max_pages"),
                    (dict(width=1 << 28), "max_pages"), (dict(table=None), "null page_table"),
                    (dict(lens=None), "null page_table or lens")]:
        assert call(lib, pages(), **kw) == lf.LF_ERR_ARG, kw
        assert msg in lf.lf_last_error(), kw
    assert call(lib, pages(kv_heads=65535), batch=65535) == lf.LF_ERR_ARG
    assert "batch * kv_heads" in lf.lf_last_error()


@pytest.mark.parametrize("call", [decode, prompt], ids=lambda f: f.__name__)
def test_bad_heads_and_windows_are_refused(lib, call):
    for kw, msg, code in [(dict(hq=0), "multiple of kv_heads", lf.LF_ERR_ARG),
                          (dict(hq=12), "multiple of kv_heads", lf.LF_ERR_ARG),
                          (dict(hq=24), "group size 3", lf.LF_ERR_UNSUPPORTED),
                          (dict(hq=128), "group size 16", lf.LF_ERR_UNSUPPORTED),
                          (dict(window=-1), "window", lf.LF_ERR_ARG),
                          (dict(sinks=-1, window=4), "sinks", lf.LF_ERR_ARG),
                          (dict(sinks=4), "sinks need a window", lf.LF_ERR_ARG),
                          (dict(q=None), "q and out", lf.LF_ERR_ARG),
                          (dict(out=E + 2), "16-byte aligned", lf.LF_ERR_ARG)]:
        assert call(lib, pages(), **kw) == code, kw
        assert msg in lf.lf_last_error(), kw
    assert lf.lf_last_status() == lf.LF_ERR_ARG


def test_bad_append_calls_are_refused(lib):
    for kw, msg in [(dict(total=-1), "total_new"), (dict(start=None), "one token"), (dict(k=None), "k_new"),
                    (dict(v=E + 4), "16-byte aligned")]:
        assert append(lib, pages(), **kw) == lf.LF_ERR_ARG, kw
        assert msg in lf.lf_last_error(), kw
    assert append(lib, pages(), total=0) == lf.LF_OK      # nothing to do, nothing launched


def test_bad_prompt_calls_are_refused(lib):
    for kw, msg in [(dict(total=-1), "total_q"), (dict(most=8), "max_q <= total_q"), (dict(most=-1), "max_q"),
                    (dict(start=None), "q_start"), (dict(total=2**31 - 1, most=2**31 - 1), "must be below 2^31")]:
        assert prompt(lib, pages(), **kw) == lf.LF_ERR_ARG, kw
        assert msg in lf.lf_last_error(), kw
    assert prompt(lib, pages(), total=0, most=0) == lf.LF_OK
    assert prompt(lib, pages(), most=0) == lf.LF_OK
    n = ctypes.c_size_t(7)
    call = lib.lf_paged_prompt_workspace
    assert call(None, 1, 1, 8, 1, 1, 0, 0, ctypes.byref(n)) == lf.LF_ERR_ARG
    assert call(ctypes.byref(pages()), 1, 1, 8, 1, 1, 0, 0, None) == lf.LF_ERR_ARG
    assert call(ctypes.byref(pages()), 1, 1, 8, 1, -1, 0, 0, ctypes.byref(n)) == lf.LF_ERR_ARG
    assert call(ctypes.byref(pages()), 1, 1, 8, 1, 2, 0, 0, ctypes.byref(n)) == lf.LF_ERR_ARG
    assert call(ctypes.byref(pages()), 1, 1, 24, 1, 1, 0, 0, ctypes.byref(n)) == lf.LF_ERR_UNSUPPORTED
    assert call(ctypes.byref(pages()), 1, 1, 8, 1, 0, 0, 0, ctypes.byref(n)) == lf.LF_OK and n.value == 0


def test_bad_decode_calls_are_refused(lib):
    for kw, msg in [(dict(k=None), "come together"), (dict(v=None), "come together"),
                    (dict(k=E + 2), "16-byte aligned")]:
        assert decode(lib, pages(), **kw) == lf.LF_ERR_ARG, kw
        assert msg in lf.lf_last_error(), kw
    n = ctypes.c_size_t(7)
    assert lib.lf_paged_decode_workspace(None, 1, 1, 8, 0, 0, ctypes.byref(n)) == lf.LF_ERR_ARG
    assert lib.lf_paged_decode_workspace(ctypes.byref(pages()), 1, 1, 8, 0, 0, None) == lf.LF_ERR_ARG
    assert lib.lf_paged_decode_workspace(ctypes.byref(pages()), 1, 1, 24, 0, 0, ctypes.byref(n)) == \
        lf.LF_ERR_UNSUPPORTED


def test_cache_refuses_what_is_no_pool():
    with pytest.raises(lf.LFError, match="CUDA tensor"):
        lf.LFPagedCache.over(torch.zeros(1, 2, 2, 16, 16), torch.zeros(1, 2, 2, 16, 16))
    with pytest.raises(lf.LFError, match=">= 1"):
        lf.LFPagedCache(1, 0, 16, 8, 128, device="cuda:0")
    with pytest.raises(lf.LFError, match="dtype"):
        lf.LFPagedCache(1, 4, 16, 8, 128, dtype="f16", device="cuda:0")


def test_pages_struct_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in lf.LFPages._fields_]
    src = tmp_path / "pages.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "longflow.h"\nint main(void){\n' +
                   'printf("%zu ", sizeof(lf_pages));\n' +
                   "".join(f'printf("%zu ", offsetof(lf_pages, {f}));\n' for f in fields) + "return 0; }")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-I", include, str(src), "-o", str(tmp_path / "x")],
                   check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "x")], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(lf.LFPages)] + [getattr(lf.LFPages, f).offset for f in fields]
