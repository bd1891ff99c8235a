"""Decoding behind shared prefixes on the CPU: every refusal of the C entry points, which come before any CUDA call."""
import ctypes

import pytest

from decode_kv_cache_gb300 import longflow as lf

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


def decode(lib, p, batch=4, table=C, width=1000, lens=D, hq=32, q=E, start=D, groups=2, prefix=C, k=E, v=E, out=E,
           lse=None, ws=E, nbytes=1 << 50):
    return lib.lf_paged_decode_shared(None if p is None else ctypes.byref(p), batch, table, width, lens, hq, q, start,
                                      groups, prefix, k, v, out, lse, ws, nbytes, None)


@pytest.mark.parametrize("bad,msg", [
    (dict(dtype=2), "dtype"), (dict(head_dim=96), "head_dim 96"), (dict(kv_heads=0), "kv_heads"), (dict(page_size=0), "page_size"),
    (dict(num_pages=0), "num_pages"), (dict(k=None), "pools"), (dict(v=B + 8), "16-byte aligned"), (dict(page_stride=-128), "strides"),
    (dict(err=A + 2), "error word")], ids=lambda x: str(x))
def test_bad_pools_are_refused(lib, bad, msg):
    assert decode(lib, pages(**bad)) in (lf.LF_ERR_ARG, lf.LF_ERR_UNSUPPORTED)
    assert msg in lf.lf_last_error()


def test_bad_calls_are_refused(lib):
    assert decode(lib, None) == lf.LF_ERR_ARG
    for kw, msg, code in [(dict(batch=0), "batch", lf.LF_ERR_ARG), (dict(batch=65536), "batch", lf.LF_ERR_ARG),
                          (dict(width=0), "max_pages", lf.LF_ERR_ARG), (dict(width=1 << 28), "max_pages", lf.LF_ERR_ARG),
                          (dict(table=None), "page_table", lf.LF_ERR_ARG), (dict(lens=D + 1), "4-byte", lf.LF_ERR_ARG),
                          (dict(hq=12), "multiple of kv_heads", lf.LF_ERR_ARG), (dict(hq=24), "group size 3", lf.LF_ERR_UNSUPPORTED),
                          (dict(q=None), "q and out", lf.LF_ERR_ARG), (dict(out=E + 2), "16-byte", lf.LF_ERR_ARG),
                          (dict(start=None), "group_start", lf.LF_ERR_ARG), (dict(prefix=None), "prefix_lens", lf.LF_ERR_ARG),
                          (dict(start=D + 2), "4-byte", lf.LF_ERR_ARG), (dict(prefix=C + 1), "4-byte", lf.LF_ERR_ARG),
                          (dict(groups=0), "groups", lf.LF_ERR_ARG), (dict(groups=5), "groups", lf.LF_ERR_ARG),
                          (dict(groups=-1), "groups", lf.LF_ERR_ARG), (dict(k=None), "come together", lf.LF_ERR_ARG),
                          (dict(v=None), "come together", lf.LF_ERR_ARG), (dict(k=E + 4), "16-byte", lf.LF_ERR_ARG),
                          (dict(lse=E + 2), "lse", lf.LF_ERR_ARG)]:
        assert decode(lib, pages(), **kw) == code, kw
        assert msg in lf.lf_last_error(), kw


def test_bad_workspace_questions_are_refused(lib):
    n = ctypes.c_size_t(7)
    call = lib.lf_paged_decode_shared_workspace
    assert call(None, 4, 10, 8, 1, ctypes.byref(n)) == lf.LF_ERR_ARG
    assert call(ctypes.byref(pages()), 4, 10, 8, 1, None) == lf.LF_ERR_ARG
    assert call(ctypes.byref(pages()), 4, 10, 24, 1, ctypes.byref(n)) == lf.LF_ERR_UNSUPPORTED
    assert call(ctypes.byref(pages()), 4, 10, 8, 0, ctypes.byref(n)) == lf.LF_ERR_ARG
    assert call(ctypes.byref(pages()), 4, 10, 8, 5, ctypes.byref(n)) == lf.LF_ERR_ARG
    assert call(ctypes.byref(pages()), 0, 10, 8, 1, ctypes.byref(n)) == lf.LF_ERR_ARG


RANGES = r"""
#define __device__
#define __forceinline__ inline
#include <cstdio>
#include "lf_ranges.h"
int main() {
  unsigned p, c, i, x;
  while (scanf("%u %u %u %u", &p, &c, &i, &x) == 4) {
    const lf::Ranges r(p, c);
    printf("%u %u %u %d\n", r.first(i), r.first(i + 1), r.owner(x), (int)r.small);
  }
}
"""


def test_ranges_are_exact_at_every_size(tmp_path):
    """Where a CTA's range starts and whose a place is, against whole numbers of any size: on both sides of where products
    leave 32 bits, up to the most places that a call may have."""
    import os
    import random
    import shutil
    import subprocess
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_kv_cache_gb300", "csrc")
    src = tmp_path / "ranges.cpp"
    src.write_text(RANGES)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(tmp_path / "x")], check=True)
    rng, cases = random.Random(1), []
    for _ in range(20000):
        c = rng.choice((1, 2, 7, 63, 128, 151, rng.randint(1, 303)))
        edge = 0xffffffff // (c + 1)
        p = rng.choice((rng.randint(c, 5000), rng.randint(c, 2**31 - 1), edge + rng.randint(-3, 3), 2**31 - 1 - rng.randint(0, 9)))
        p = max(c, min(p, 2**31 - 1))
        i = rng.choice((0, c - 1, rng.randrange(c)))
        x = rng.choice((0, p - 1, rng.randrange(p), p * i // c, max(0, p * i // c - 1)))
        cases.append((p, c, i, x))
    text = "\n".join(" ".join(map(str, t)) for t in cases)
    got = subprocess.run([str(tmp_path / "x")], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    sides = set()
    for (p, c, i, x), line in zip(cases, got):
        first, end, owner, small = map(int, line.split())
        sides.add(small)
        assert first == p * i // c and end == p * (i + 1) // c, (p, c, i)
        assert 0 <= owner < c and p * owner // c <= x < p * (owner + 1) // c, (p, c, x)
    assert sides == {0, 1}
