"""Rotary positions on the CPU: the oracle, the conversion of frequencies, and every refusal of the C entry
points, which come before any CUDA call."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from decode_kv_cache_gb300 import longflow as lf
from oracle import rotary_oracle

A, B, C, D, E = (0x10000 * i for i in range(1, 6))   # aligned addresses that nothing reads


@pytest.fixture(scope="module")
def lib():
    from decode_kv_cache_gb300 import build as b
    b.build()
    return lf.load_library()


# ---- the oracle ---------------------------------------------------------------------------------

@pytest.mark.parametrize("adjacent", [False, True])
def test_oracle_turns_pairs_as_complex_numbers(adjacent):
    rng = np.random.default_rng(1)
    x, pos, f = rng.normal(size=(7, 3, 32)), rng.integers(-9, 9, size=(1, 7)), rotary_oracle.frequencies(16, 100.0)
    y, size = rotary_oracle.rotate(x, pos, f, adjacent=adjacent)
    a, b = rotary_oracle.pairs(16, adjacent)
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[0][:, None, None] * f)
    np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, rtol=1e-13, atol=1e-13)
    np.testing.assert_array_equal(y[..., 16:], x[..., 16:])
    back, _ = rotary_oracle.rotate(y, pos, f, adjacent=adjacent, inverse=True)
    np.testing.assert_allclose(back, x, rtol=1e-12, atol=1e-12)
    assert (size[..., :16] >= np.abs(y[..., :16]) - 1e-12).all() and (size[..., 16:] == 0).all()


def test_oracle_axes_and_relative_positions():
    rng = np.random.default_rng(2)
    f, axis = rotary_oracle.frequencies(8), [0, 1, 1, 2]
    q, k = rng.normal(size=(2, 1, 1, 8))
    at = lambda x, p: rotary_oracle.rotate(x, np.array(p).reshape(3, 1), f, axis)[0].ravel()  # noqa: E731
    # a product of two rotated rows depends on the differences of their positions alone
    want = at(q, (5, 7, 2)) @ at(k, (1, 9, 2))
    np.testing.assert_allclose(at(q, (14, 3, 0)) @ at(k, (10, 5, 0)), want, rtol=1e-12)
    only = at(q, (0, 4, 0)) - q.ravel()
    assert np.flatnonzero(np.abs(only) > 1e-9).tolist() == [1, 2, 5, 6]   # pairs 1 and 2


# ---- frequencies --------------------------------------------------------------------------------

def one_over_two_pi(bits=260):
    """floor(2^bits / (2 pi)) by Machin's formula in whole numbers."""
    def arctan_of_inverse(n):
        term, total, k, sign = (1 << (bits + 60)) // n, 0, 1, 1
        while term:
            total += sign * (term // k)
            term, k, sign = term // (n * n), k + 2, -sign
        return total
    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))   # 2^(bits + 60) pi
    return (1 << (2 * bits + 60)) // (2 * pi)


def test_turns_are_the_nearest_64_bit_fractions(lib):
    rng = np.random.default_rng(3)
    freq = [0.0, 1.0, -1.0, 1024.0, -1024.0, 1e-4, 5e-324, 1e-30, 2.0**-60, 6.283185307179586]
    freq += rotary_oracle.frequencies(128, 1e6).tolist() + (rng.uniform(-1, 1, 300) * 10.0 ** rng.uniform(-12, 3, 300)).tolist()
    inverse = Fraction(one_over_two_pi(), 1 << 260)
    for f, got in zip(freq, lf.lf_rotary_turns(freq)):
        off = (Fraction(got) - Fraction(f) * inverse * 2**64) % 2**64
        assert min(off, 2**64 - off) <= Fraction(1, 2) + Fraction(1, 1000), f


def test_turns_are_the_nearest_where_two_are_almost_as_near(lib):
    """Within 2^-24 of halfway between two of them the fourth word of 1 / (2 pi) decides.  192 bits of it, cut, are off by up
    to 2^-192; times up to 2^10 radians in units of 2^-64 of a turn that is 2^-118."""
    inverse = Fraction(one_over_two_pi(), 1 << 260)
    assert lf.lf_rotary_turns([512.0000040903037]) == [8989679718594790752]
    near = [512.0000040903037, 512.0, 1023.9999999999999, 1.0, 3e-5] + rotary_oracle.frequencies(128, 1e6).tolist()
    for f, got in zip(near, lf.lf_rotary_turns(near)):
        off = (Fraction(got) - Fraction(f) * inverse * 2**64) % 2**64
        assert min(off, 2**64 - off) <= Fraction(1, 2) + Fraction(1, 2**100), f


def test_bad_frequencies_are_refused(lib):
    for f in (float("nan"), float("inf"), 1025.0, -1e9):
        with pytest.raises(lf.LFError, match="frequency 1"):
            lf.lf_rotary_turns([1.0, f])
    assert lib.lf_rotary_turns(None, 0, None) == lf.LF_ERR_ARG
    assert lf.lf_rotary_turns([]) == []


# ---- refusals -----------------------------------------------------------------------------------

def pages(**kw):
    p = dict(dtype=lf.LF_BF16, kv_heads=8, head_dim=128, page_size=16, num_pages=100,
             page_stride=8 * 16 * 128, head_stride=16 * 128, token_stride=128, k=A, v=B, err=None)
    p.update(kw)
    s = lf.LFPages()
    for n, x in p.items():
        setattr(s, n, x)
    return s


def table(**kw):
    p = dict(rotary_dim=64, axes=3, adjacent=0, scale=1.0, turns=A, axis=B)
    p.update(kw)
    return lf.LFRotaryTable(*(p[n] for n, _ in lf.LFRotaryTable._fields_))


def rows(**kw):
    p = dict(x=A, y=B, heads=8, x_seq=0, x_token=1024, x_head=128, y_seq=0, y_token=1024, y_head=128)
    p.update(kw)
    return lf.LFRows(*(p[n] for n, _ in lf.LFRows._fields_))


def rotate(lib, r, dtype=lf.LF_BF16, dim=128, seqs=1, tokens=4, q=None, k=None, positions=C, stride=4, inverse=0):
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    return lib.lf_rotate(ref(r), dtype, dim, seqs, tokens, ref(rows() if q is None else q), ref(k), positions, stride,
                         inverse, None)


def append(lib, r, p=None, batch=4, tab=C, width=10, lens=D, k=E, v=E, start=D, total=7, positions=C, stride=7, hq=32,
           q=A, out=B):
    return lib.lf_paged_append_rotated(ctypes.byref(pages() if p is None else p), batch, tab, width, lens, k, v, start,
                                       total, None if r is None else ctypes.byref(r), positions, stride, hq, q, out, None)


@pytest.mark.parametrize("call", [rotate, append], ids=lambda f: f.__name__)
def test_bad_rotaries_are_refused(lib, call):
    assert call(lib, None) == lf.LF_ERR_ARG and "null rotary" in lf.lf_last_error()
    for kw, msg in [(dict(rotary_dim=0), "rotary_dim"), (dict(rotary_dim=24), "multiple of 16"),
                    (dict(rotary_dim=144), "at most the rows' 128"), (dict(rotary_dim=-16), "rotary_dim"),
                    (dict(axes=0), "axes"), (dict(axes=5), "axes"), (dict(adjacent=2), "adjacent"),
                    (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"), (dict(turns=None), "turns"),
                    (dict(turns=A + 4), "8-byte aligned"), (dict(axis=B + 2), "4-byte aligned")]:
        assert call(lib, table(**kw)) == lf.LF_ERR_ARG, kw
        assert msg in lf.lf_last_error(), kw
    assert call(lib, table(), positions=C + 1) == lf.LF_ERR_ARG
    assert call(lib, table(), stride=-1) == lf.LF_ERR_ARG and "axis_stride" in lf.lf_last_error()


def test_bad_rotate_calls_are_refused(lib):
    for kw, msg in [(dict(dtype=2), "dtype"), (dict(dim=120), "row_dim"), (dict(dim=528), "row_dim"), (dict(dim=0), "row_dim"),
                    (dict(seqs=-1), "seqs"), (dict(tokens=-1), "tokens"), (dict(seqs=65536, tokens=32768), "below 2^31"),
                    (dict(inverse=2), "inverse"), (dict(positions=None), "null positions")]:
        assert rotate(lib, table(), **kw) == lf.LF_ERR_ARG, kw
        assert msg in lf.lf_last_error(), kw
    for kw, msg in [(dict(heads=0), "heads"), (dict(heads=65536), "heads"), (dict(x=None), "non-null"), (dict(y=None), "non-null"),
                    (dict(x=A + 8), "16-byte aligned"), (dict(x_head=-8), "strides"), (dict(y_token=4), "multiples of 16 bytes"),
                    (dict(x_seq=1 << 41), "strides")]:
        assert rotate(lib, table(), q=rows(**kw)) == lf.LF_ERR_ARG, kw
        assert msg in lf.lf_last_error() and lf.lf_last_error().startswith("q:"), kw
        assert rotate(lib, table(), k=rows(**kw)) == lf.LF_ERR_ARG, kw
        assert msg in lf.lf_last_error() and lf.lf_last_error().startswith("k:"), kw
    assert lib.lf_rotate(ctypes.byref(table()), 0, 128, 1, 4, None, None, C, 4, 0, None) == lf.LF_ERR_ARG
    assert rotate(lib, table(), tokens=0) == lf.LF_OK and rotate(lib, table(), seqs=0) == lf.LF_OK


def test_bad_rotated_appends_are_refused(lib):
    for kw, msg in [(dict(p=pages(dtype=2)), "dtype"), (dict(p=pages(head_dim=96)), "head_dim 96"), (dict(batch=0), "batch"),
                    (dict(tab=None), "page_table"), (dict(width=0), "max_pages"), (dict(total=-1), "total_new"),
                    (dict(start=None), "one token"), (dict(k=None), "k_new"), (dict(v=E + 4), "16-byte aligned"),
                    (dict(q=None), "come together"), (dict(out=None), "come together"), (dict(hq=0), "q_heads"),
                    (dict(out=B + 8), "16-byte aligned"), (dict(start=D + 2), "new_start")]:
        code = append(lib, table(), **kw)
        assert code in (lf.LF_ERR_ARG, lf.LF_ERR_UNSUPPORTED), kw
        assert msg in lf.lf_last_error(), kw
    assert append(lib, table(), total=0) == lf.LF_OK


def test_outputs_that_overlap_are_refused(lib):
    """Rows are read ahead of the writes: an output is its own input's rows or lies apart from everything."""
    for kw, msg in [(dict(y_head=0), "rows of y overlap"), (dict(y_token=0), "rows of y overlap"), (dict(y_token=896), "rows of y overlap"),
                    (dict(y_head=64), "rows of y overlap"), (dict(x_token=0, y_token=0, y=A), "rows of y overlap"),
                    (dict(y=A + 16), "q's x"), (dict(y=A - 256), "q's x"), (dict(y=A + 256), "q's x"), (dict(y=A + 3 * 2048 + 1792), "q's x"),
                    (dict(y=A, y_token=2048), "q's x"), (dict(y=A + 2048, x_token=2048, y_token=2048, y_head=136), "q's x")]:
        assert rotate(lib, table(), q=rows(**kw)) == lf.LF_ERR_ARG, kw
        assert msg in lf.lf_last_error(), (kw, lf.lf_last_error())
    # in place, in sequences of more columns; keys in the queries' place, and keys' output in the queries'
    assert rotate(lib, table(), q=rows(y=A), k=rows(x=C, y=C + 2 * 2048)) == lf.LF_ERR_ARG and "k's x" in lf.lf_last_error()
    assert rotate(lib, table(), q=rows(y=A), k=rows(x=C, y=A + 2 * 2048)) == lf.LF_ERR_ARG and "q's x" in lf.lf_last_error()
    assert rotate(lib, table(), q=rows(), k=rows(x=C, y=B + 2048)) == lf.LF_ERR_ARG and "k: y overlaps q's y" in lf.lf_last_error()
    assert rotate(lib, table(), q=rows(y=C), k=rows(x=C + 4 * 2048 - 256, y=D)) == lf.LF_ERR_ARG and "k's x" in lf.lf_last_error()
    # seven tokens of 32 heads of 256 bytes, 8 of keys
    for kw in (dict(out=A + 16), dict(out=A + 7 * 32 * 256 - 16), dict(out=A - 7 * 32 * 256 + 16), dict(q=A, out=E), dict(q=A, k=D, out=D + 7 * 8 * 256 - 16),
               dict(q=A, v=C, out=C + 16)):
        assert append(lib, table(), **kw) == lf.LF_ERR_ARG, kw
        assert "q_out may be q" in lf.lf_last_error(), kw


OVERLAP = r"""
#include <cstdio>
#include "lf_overlap.h"
using namespace lf;
int main() {
  RowSet a, b;
  long long v[14];
  for (;;) {
    for (int i = 0; i < 14; ++i)
      if (scanf("%lld", v + i) != 1) return 0;
    a = RowSet{(uintptr_t)v[0], {v[1], v[2], v[3]}, {v[4], v[5], v[6]}, 2};
    b = RowSet{(uintptr_t)v[7], {v[8], v[9], v[10]}, {v[11], v[12], v[13]}, 2};
    printf("%d %d %d\n", (int)rows_overlap_themselves(a), (int)rows_overlap(a, b), (int)same_rows(a, b));
  }
}
"""


def test_overlaps_are_found_as_by_looking_at_every_byte(tmp_path):
    """Every answer against the bytes that the rows have, over small layouts of all kinds; large ones that are views of a
    tensor are told apart, and sizes times strides past 64 bits do no harm."""
    import os
    import random
    import shutil
    import subprocess
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_kv_cache_gb300", "csrc")
    src = tmp_path / "overlap.cpp"
    src.write_text(OVERLAP)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(tmp_path / "x")], check=True)
    rng, cases, want = random.Random(1), [], []

    def row_starts(at, n, st):
        return [at + i * st[0] + j * st[1] + k * st[2] for i in range(n[0]) for j in range(n[1]) for k in range(n[2])]

    for _ in range(6000):
        def layout(like=None):
            n = [rng.choice((1, 1, 2, 3, 4)) for _ in range(3)]
            if like and rng.random() < 0.6:
                return rng.randrange(200, 260), (like[1] if rng.random() < 0.5 else n), like[2]
            st = [rng.choice((0, 1, 2, 3, 4, 6, 8, 12, 16, 24, 48)) for _ in range(3)]
            return rng.randrange(200, 260), n, st
        a = layout()
        b = layout(a)
        if rng.random() < 0.2:
            b = (a[0], *b[1:])
        own = [x for s in row_starts(*a) for x in (s, s + 1)]
        other = {x for s in row_starts(*b) for x in (s, s + 1)}
        cases.append((a, b))
        want.append((len(own) != len(set(own)), bool(other.intersection(own)),
                     a[0] == b[0] and a[1] == b[1] and all(n == 1 or x == y for n, x, y in zip(a[1], a[2], b[2]))))
    big = 2**31 - 1
    views = [((10**9, [3, 70000, 32], [70000 * 96, 96, 2]), (10**9 + 64, [3, 70000, 8], [70000 * 96, 96, 2]), (0, 0, 0)),    # of one wide row
             ((10**9, [3, 70000, 32], [70000 * 96, 96, 2]), (10**9 + 62, [3, 70000, 8], [70000 * 96, 96, 2]), (0, 1, 0)),
             ((10**9, [8, 5000, 4], [40000, 2, 10000]), (10**9, [8, 5000, 4], [40000, 2, 10000]), (0, 1, 1)),                # a slab
             ((10**9, [1, big, 65535], [0, 2**44, 2]), (10**9 + 2**20, [1, big, 65535], [0, 2**44, 2]), (0, 0, 0)),
             ((10**9, [big, 1, 1], [2**44, 0, 0]), (10**9 + 2**44 * 1000 + 1, [big, 1, 1], [2**44, 0, 0]), (0, 1, 0))]
    for a, b, w in views:
        cases.append((a, b))
        want.append(w)
    text = "\n".join(" ".join(str(x) for s in c for x in (s[0], *s[1], *s[2])) for c in cases)
    got = subprocess.run([str(tmp_path / "x")], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    for c, w, g in zip(cases, want, got):
        assert tuple(int(x) for x in w) == tuple(int(x) for x in g.split()), (c, w, g)


def test_rotary_refuses_what_is_none():
    for kw, msg in [(dict(rotary_dim=24), "multiple of 16"), (dict(rotary_dim=64.0), "multiple of 16"), (dict(rotary_dim=528), "multiple of 16"),
                    (dict(base=0), "base"), (dict(sections=[16, 15]), "sum to 32"), (dict(sections=[8, 8, 8, 4, 4]), "sections"),
                    (dict(sections=[33, -1]), "sections"), (dict(sections=[32], axis=[0] * 32), "at most one"),
                    (dict(axis=[0] * 31), "32 frequencies and axes"), (dict(axis=[4] * 32), "axis"), (dict(axis=[-1] * 32), "axis"),
                    (dict(inv_freq=[1.0] * 16), "32 frequencies"), (dict(inv_freq=[2000.0] * 32), "frequency 0"),
                    (dict(scale=float("nan")), "scale"), (dict(device="cpu"), "CUDA device")]:
        with pytest.raises(lf.LFError, match=msg):
            lf.LFRotary(**{"rotary_dim": 64, **kw})


def test_gradients_are_not_lost_unseen():
    """A result without a graph is refused where gradients are recorded, before anything runs."""
    r = object.__new__(lf.LFRotary)          # (a CPU tensor's index; no GPU)
    r._index, r.device, r.axes = -1, torch.device("cpu"), 1
    x, pos = torch.randn(4, 2, 16), torch.zeros(4, dtype=torch.int32)
    leaf = torch.randn(4, 2, 16, requires_grad=True)
    for kw in (dict(q=leaf), dict(q=x, k=leaf), dict(q=x, q_out=leaf), dict(q=x, k=x, k_out=leaf), dict(q=leaf * 2)):
        with pytest.raises(lf.LFError, match="gradient"):
            r.rotate(positions=pos, **kw)
    ran = []
    r._lib = type("Lib", (), {"lf_rotate": staticmethod(lambda *a: ran.append(a) or 0)})
    r._table = table()
    r._rotate(0, leaf.detach(), pos, None, None, None, 0, 0)
    assert len(ran) == 1


def test_outputs_that_autograd_has_saved_are_known_to_have_changed(monkeypatch):
    """A tensor that is rotated in place after autograd saved it: backward says so instead of using what it holds now."""
    r = object.__new__(lf.LFRotary)
    r._index, r.device, r.axes = -1, torch.device("cpu"), 1
    monkeypatch.setattr(lf, "_run_on", lambda *a: None)
    pos = torch.zeros(4, dtype=torch.int32)
    for kw in (lambda x: dict(q=x, q_out=x), lambda x: dict(q=torch.zeros(4, 2, 16), k=x, k_out=x)):
        x, w = torch.randn(4, 2, 16), torch.ones((), requires_grad=True)
        y = (w * x).sum()
        r.rotate(positions=pos, **kw(x))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    with torch.inference_mode():
        x = torch.randn(4, 2, 16)
        r.rotate(x, pos, q_out=x)


def test_structs_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    lines, want = [], []
    for c, s in (("lf_rotary", lf.LFRotaryTable), ("lf_rows", lf.LFRows)):
        lines.append(f'printf("%zu ", sizeof({c}));')
        want.append(ctypes.sizeof(s))
        for f, _ in s._fields_:
            lines.append(f'printf("%zu ", offsetof({c}, {f}));')
            want.append(getattr(s, f).offset)
    src = tmp_path / "rotary.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "longflow.h"\nint main(void){\n' + "\n".join(lines) +
                   'printf("%d", LF_ROTARY_MAX_AXES); return 0; }')
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-I", include, str(src), "-o", str(tmp_path / "x")], check=True)
    got = subprocess.run([str(tmp_path / "x")], capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == want + [lf._MAX_AXES]
