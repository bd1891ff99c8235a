"""Paged key-value cache on the GPU, at the edges of what its calls allow: row starts, windows whose
pages are given back, bounds that are wider than the call, streams, and the error word."""
import math

import numpy as np
import pytest
import torch

from decode_kv_cache_gb300 import longflow as lf
from oracle import paged_oracle
from paged_harness import Paged, starts

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def weight_step(kind):
    """Prompt: a bf16 cache's weights are rounded to bf16 before the product with V."""
    return 2.0 ** -8 if kind == "bf16" else 0.0


# ---- append: row starts -----------------------------------------------------------------------------

def append_and_compare(p, st, total, stored):
    """Rows st[b] .. st[b + 1] - 1 of the sequences in `stored` reach their pages, and nothing else does."""
    kn, vn = p.randn(total, p.kv_heads, p.d), p.randn(total, p.kv_heads, p.d)
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    want = []
    for pool, rows in ((p.k, kn), (p.v, vn)):
        pool = f(pool)
        for b in stored:
            pool = paged_oracle.append(pool, [p.np_table[b]], [p.lens[b]], f(rows), [st[b], st[b + 1]], p.page)
        want.append(pool)
    p.cache.append(0, kn, vn, p.table, p.t_lens, ints(st))
    for pool, x in zip((p.k, p.v), want):
        np.testing.assert_array_equal(f(pool), x)
    return p.cache.check()


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("f32", 16)])
def test_append_row_starts(kind, d):
    """Rows in front of the first sequence are left.  A sequence whose starts lie outside the rows is
    reported and not stored; the others are."""
    p = Paged(kind, 2, d, 16, [200, 90, 150], seed=d)
    assert append_and_compare(p, [300, 500, 560, 700], 700, [0, 1, 2]) == 0
    assert append_and_compare(p, [-1000, 100, 160, 300], 700, [1, 2]) == lf.LF_DEVERR_STATE
    assert append_and_compare(p, [-50, 100, 160, 300], 700, [1, 2]) == lf.LF_DEVERR_STATE
    assert append_and_compare(p, [0, 200, 260, 401], 400, [0, 1]) == lf.LF_DEVERR_STATE
    assert append_and_compare(p, [0, 200, 260, 2**31 - 1], 400, [0, 1]) == lf.LF_DEVERR_STATE


def test_append_row_starts_that_decrease():
    p = Paged("bf16", 2, 64, 16, [200, 90, 150], seed=3)
    kn = p.randn(250, 2, 64)
    p.cache.append(0, kn, kn, p.table, p.t_lens, ints([0, 150, 100, 250]))
    assert p.cache.check() == lf.LF_DEVERR_STATE


def test_append_row_starts_of_more_sequences_than_threads():
    """Four rows, 1000 sequences: the last one's end lies behind the rows."""
    p = Paged("bf16", 1, 16, 4, [9] * 1000, seed=4)
    assert append_and_compare(p, [0] * 1000 + [5], 4, []) == lf.LF_DEVERR_STATE
    assert append_and_compare(p, [0] * 1000 + [4], 4, [999]) == 0


# ---- prompt: pages behind the window --------------------------------------------------------------

@pytest.mark.parametrize("window,sinks", [(100, 4), (1, 0), (64, 0), (130, 140), (700, 1)])
@pytest.mark.parametrize("kind,d,page", [("bf16", 128, 16), ("bf16", 64, 64), ("bf16", 128, 256), ("bf16", 128, 8),
                                         ("bf16", 32, 16), ("bf16", 128, 24), ("f32", 64, 16), ("f32", 128, 16)])
def test_prompt_positions_that_no_query_sees(kind, d, page, window, sinks):
    """A caller gives the pages behind the window back: their entries are no pages any more, and the
    places that are left behind in pages that it keeps hold NaN.  The results do not change by a bit (so
    nothing was computed again because of a NaN), and there is no error."""
    old, new = [900, 0, 1000, 300, 1500], [60, 20, 1, 150, 300]
    lens = [a + b for a, b in zip(old, new)]
    p = Paged(kind, 2, d, page, lens, seed=page + window)
    st = starts(new)
    q = p.randn(st[-1], 4, d)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    args = (p.table, p.t_lens, ints(st), max(new), window, sinks)
    before = p.cache.prompt(0, q, *args, lse=lse)
    before_lse = lse.clone()
    gone = 0
    for b in range(len(lens)):
        lo, hi = sinks, old[b] - window + 1          # positions lo .. hi - 1: seen by none
        if lo < hi:
            p.hide(b, lo, hi)
        for i in range(p.width):
            if lo <= i * page and (i + 1) * page <= hi:
                p.table[b, i] = -1
                gone += 1
    assert gone > 0
    out = p.cache.prompt(0, q, *args, lse=lse)
    assert p.cache.check() == 0
    assert torch.equal(out, before) and torch.equal(lse, before_lse)
    for b in range(len(lens)):
        rows = slice(st[b], st[b + 1])
        p.check(b, q[rows], old[b], out[rows], lse[rows], window, sinks, weight_step(kind))


@pytest.mark.parametrize("kind,d,page", [("bf16", 128, 16), ("bf16", 32, 16), ("f32", 64, 16)])
def test_prompt_positions_that_no_query_sees_with_shared_keys(kind, d, page):
    """The same where several blocks share the keys of few rows."""
    n, rows, window, sinks = 6000, 5, 3000, 20
    p = Paged(kind, 1, d, page, [n], seed=d)
    assert lf.lf_paged_prompt_workspace(p.cache._pages[0], 1, p.width, 2, rows, rows, window, sinks) > 0
    q, st = p.randn(rows, 2, d), ints([0, rows])
    before = p.cache.prompt(0, q, p.table, p.t_lens, st, rows, window, sinks)
    hi = n - rows - window + 1
    p.hide(0, sinks, hi)
    for i in range(p.width):
        if sinks <= i * page and (i + 1) * page <= hi:
            p.table[0, i] = -1
    out = p.cache.prompt(0, q, p.table, p.t_lens, st, rows, window, sinks)
    assert p.cache.check() == 0 and torch.equal(out, before)
    p.check(0, q, n - rows, out, None, window, sinks, weight_step(kind))


# ---- prompt: the bound on a sequence's rows ------------------------------------------------------

@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("others", [2, 20, 50])
def test_prompt_rows_behind_the_bound_are_left(kind, d, others):
    """A sequence with more rows than max_q: the rows up to max_q are computed, the rest is left and
    reported.  (2, 20 and 50 other sequences: the three ways in which pieces are numbered.)"""
    most = 201
    new = [300] + [1] * others + [201]
    old = [0] + [i % 30 for i in range(others)] + [5]
    lens = [a + b for a, b in zip(old, new)]
    p = Paged(kind, 2, d, 16, lens, seed=d + others)
    st = starts(new)
    q = p.randn(st[-1], 8, d)
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:2], 3.0, dtype=torch.float32, device="cuda")
    p.cache.prompt(0, q, p.table, p.t_lens, ints(st), most, out=out, lse=lse)
    assert p.cache.check() == lf.LF_DEVERR_STATE
    assert (out[most:300] == 3).all() and (lse[most:300] == 3).all()
    for b in range(len(lens)):
        rows = slice(st[b], min(st[b] + most, st[b + 1]))
        p.check(b, q[rows], old[b], out[rows], lse[rows], weight_step=weight_step(kind))


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 32), ("f32", 64)])
def test_prompt_rows_behind_the_bound_with_shared_keys(kind, d):
    p = Paged(kind, 2, d, 16, [5000, 4000], seed=d)
    assert lf.lf_paged_prompt_workspace(p.cache._pages[0], 2, p.width, 8, 8, 3) > 0
    q, st = p.randn(8, 8, d), ints([0, 5, 8])
    out = torch.full_like(q, 3.0)
    p.cache.prompt(0, q, p.table, p.t_lens, st, 3, out=out)
    assert p.cache.check() == lf.LF_DEVERR_STATE
    assert (out[3:5] == 3).all()
    p.check(0, q[:3], 4995, out[:3], None, weight_step=weight_step(kind))
    p.check(1, q[5:], 3997, out[5:], None, weight_step=weight_step(kind))


def test_prompt_takes_a_bound_that_is_wider_than_the_call():
    """max_q is a bound: one that is larger than the call's rows, as a chunk limit is, changes nothing."""
    p = Paged("bf16", 2, 128, 16, [90, 40], seed=8)
    q, st = p.randn(50, 8, 128), ints([0, 30, 50])
    a = p.cache.prompt(0, q, p.table, p.t_lens, st, 30)
    for most in (50, 51, 512, 2**31 - 1, 2**40):
        b = p.cache.prompt(0, q, p.table, p.t_lens, st, most)
        p.check(0, q[:30], 60, b[:30], None, weight_step=2.0 ** -8)
        p.check(1, q[30:], 20, b[30:], None, weight_step=2.0 ** -8)
        assert torch.equal(a, b)
    assert p.cache.check() == 0
    none = p.cache.prompt(0, q[:0], p.table, p.t_lens, ints([0, 0, 0]), 512)
    assert none.shape == (0, 8, 128)


# ---- streams ------------------------------------------------------------------------------------

def busy(stream=None, clocks=100_000_000):
    """About 50 ms of work in front of what follows on the stream."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(clocks)


def test_a_stream_handle_of_zero_is_the_default_stream():
    """torch.cuda.default_stream().cuda_stream is 0: a call with it comes behind the default stream's work."""
    side = torch.cuda.Stream()      # (the first one makes torch's pool of them, which waits for the device)
    p = Paged("bf16", 8, 128, 16, [3000, 50], seed=60)
    real, st = p.randn(2, 32, 128), ints([0, 1, 2])
    want = p.cache.decode(0, real, p.table, p.t_lens)
    want_prompt = p.cache.prompt(0, real, p.table, p.t_lens, st, 1)
    q = torch.zeros_like(real)
    torch.cuda.synchronize()
    assert torch.cuda.default_stream().cuda_stream == 0
    busy()
    q.copy_(real)
    got = p.cache.decode(0, q, p.table, p.t_lens, stream=torch.cuda.default_stream().cuda_stream)
    got_prompt = p.cache.prompt(0, q, p.table, p.t_lens, st, 1, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_prompt, want_prompt)
    with torch.cuda.stream(side):      # and not the current one
        busy()
        q.zero_()
        got = p.cache.decode(0, real, p.table, p.t_lens, stream=0)
    torch.cuda.default_stream().synchronize()
    assert torch.equal(got.clone(), want)
    torch.cuda.synchronize()


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_tensors_that_are_let_go_while_another_stream_reads_them(handle):
    """A call on a stream of the caller's, with tensors that the caller drops as soon as it returns: memory
    that the stream still has to read is not handed out again."""
    p = Paged("bf16", 8, 128, 16, [3000, 50], seed=61)
    real, st = p.randn(2, 32, 128), ints([0, 1, 2])
    kn, vn = p.randn(2, 8, 128), p.randn(2, 8, 128)
    want_d = p.cache.decode(0, real, p.table, p.t_lens, kn, vn)
    want_p = p.cache.prompt(0, real, p.table, p.t_lens, st, 1)
    want_k = p.k.clone()
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side

    def dropped(call):
        """call's inputs as copies that nobody holds afterwards; their places are overwritten."""
        torch.cuda.synchronize()
        busy(side)
        mine = [x.clone() for x in (real, kn, vn, p.table, p.t_lens, st)]
        torch.cuda.current_stream().synchronize()     # the copies are made; the side stream has not begun
        shapes = [(x.shape, x.dtype) for x in mine]
        got = call(*mine)
        del mine
        junk = [torch.full(shape, 1, dtype=t, device="cuda") for shape, t in shapes for _ in range(3)]
        torch.cuda.synchronize()
        del junk
        return got

    got = dropped(lambda q, k, v, t, n, i: p.cache.decode(0, q, t, n, k, v, stream=s))
    assert torch.equal(got, want_d)
    got = dropped(lambda q, k, v, t, n, i: p.cache.prompt(0, q, t, n, i, 1, stream=s))
    assert torch.equal(got, want_p)
    dropped(lambda q, k, v, t, n, i: p.cache.append(0, k, v, t, n, i, stream=s))
    assert torch.equal(torch.nan_to_num(p.k, 77.0), torch.nan_to_num(want_k, 77.0))
    assert p.cache.check() == 0


def test_a_cache_that_is_let_go_while_another_stream_uses_it():
    p = Paged("bf16", 8, 128, 16, [3000, 50], seed=65)
    q = p.randn(2, 32, 128)
    want = p.cache.decode(0, q, p.table, p.t_lens)
    side = torch.cuda.Stream()
    k, v = p.k.clone(), p.v.clone()
    cache = lf.LFPagedCache.over(k[None], v[None])
    torch.cuda.synchronize()
    busy(side)
    got = cache.decode(0, q, p.table, p.t_lens, stream=side)
    shape = k.shape
    del k, v, cache
    junk = [torch.full(shape, 1, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    del junk
    assert torch.equal(got, want)


def test_a_named_stream_under_capture():
    """A call that names the stream on which a graph is captured, replayed after its inputs' makers are gone."""
    p = Paged("bf16", 2, 128, 16, [3000, 50], seed=66)
    q, st = p.randn(2, 8, 128), ints([0, 1, 2])
    want = p.cache.decode(0, q, p.table, p.t_lens), p.cache.prompt(0, q, p.table, p.t_lens, st, 1)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        a = p.cache.decode(0, q, p.table, p.t_lens, stream=side)
        b = p.cache.prompt(0, q, p.table, p.t_lens, st, 1, stream=side)
    for _ in range(3):
        a.zero_(), b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


# ---- the error word ---------------------------------------------------------------------------------

def test_the_error_word_is_clear_before_any_stream_reads_it():
    """A cache made on a busy stream and used on another one starts without errors and keeps its own."""
    k = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    v, table, lens = torch.zeros_like(k), ints([[-5]]), ints([3])
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    junk = [torch.full((1,), 0x7fff, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del junk                               # the allocator hands their places out again
    side = torch.cuda.Stream()
    busy()
    cache = lf.LFPagedCache.over(k, v)
    assert cache.check(side) == 0
    busy()
    cache = lf.LFPagedCache.over(k, v)
    cache.decode(0, q, table, lens, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert cache.check() == lf.LF_DEVERR_STATE


def test_errors_that_come_during_a_check_are_kept():
    """While one stream's errors are read and cleared, another stream reports its own: each is seen once."""
    p = Paged("bf16", 1, 64, 16, [40], seed=62)
    q = p.randn(1, 4, 64)
    bad_table, bad_q = p.table.clone(), q.clone()
    bad_table[0, 1] = -1
    bad_q[0, 0, 0] = math.nan
    side, lost = torch.cuda.Stream(), 0
    torch.cuda.synchronize()
    for i in range(400):
        p.cache.decode(0, q, bad_table, p.t_lens)                 # LF_DEVERR_STATE
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(500 * (i % 200))                    # up to some 50 us
            p.cache.decode(0, bad_q, p.table, p.t_lens)           # LF_DEVERR_NONFINITE
        bits = p.cache.check()
        torch.cuda.synchronize()
        bits |= p.cache.check()
        lost += bits != lf.LF_DEVERR_STATE | lf.LF_DEVERR_NONFINITE
    assert lost == 0 and p.cache.check() == 0


# ---- numbers that the C calls cannot take ------------------------------------------------------------

def test_numbers_that_do_not_fit_the_c_calls_are_refused():
    """ctypes takes the low 32 bits of a number without a word: a window of 2^32 + 1 would be one of 1."""
    p = Paged("bf16", 2, 128, 16, [100, 50], seed=63)
    q, st = p.randn(2, 8, 128), ints([0, 1, 2])
    c = p.cache
    for bad in (2**31, 2**32, 2**32 + 1, -1, -2**32 + 1):
        with pytest.raises(lf.LFError, match="window"):
            c.decode(0, q, p.table, p.t_lens, window=bad)
        with pytest.raises(lf.LFError, match="window"):
            c.prompt(0, q, p.table, p.t_lens, st, 1, window=bad)
        with pytest.raises(lf.LFError, match="sinks"):
            c.decode(0, q, p.table, p.t_lens, window=4, sinks=bad)
        with pytest.raises(lf.LFError, match="sinks"):
            c.prompt(0, q, p.table, p.t_lens, st, 1, window=4, sinks=bad)
    with pytest.raises(lf.LFError, match="max_q"):
        c.prompt(0, q, p.table, p.t_lens, st, -2**32 + 1)
    whole = c.decode(0, q, p.table, p.t_lens)
    assert torch.equal(whole, c.decode(0, q, p.table, p.t_lens, window=2**31 - 1, sinks=2**31 - 1))


def test_pools_with_more_pages_than_an_int_are_refused():
    """2^32 + 1 pages (all the same one here) would be one page."""
    k = torch.zeros(1, 1, 1, 1, 16, dtype=torch.bfloat16, device="cuda")
    for n in (2**31, 2**32 + 1):
        big = k.expand(1, n, 1, 1, 16)
        with pytest.raises(lf.LFError, match="2\\^31 - 1"):
            lf.LFPagedCache.over(big, big)
    lf.LFPagedCache.over(k.expand(1, 2**31 - 1, 1, 1, 16), k.expand(1, 2**31 - 1, 1, 1, 16))


# ---- a table that is much wider than its sequences, and company ----------------------------------------

@pytest.mark.parametrize("kind,d,page", [("bf16", 128, 16), ("bf16", 64, 128), ("bf16", 32, 16), ("bf16", 128, 24),
                                         ("f32", 64, 16), ("f32", 128, 64)])
def test_tables_that_are_much_wider_than_their_sequences(kind, d, page):
    """A table row is as wide as the longest context that a server allows.  The host sees the width alone, so
    that it cuts units and shares keys that are not there: blocks whose share is empty, and their joins."""
    lens, new = [5, 300, 0, 129, 700], [5, 2, 0, 129, 40]
    st = starts(new)
    p = Paged(kind, 2, d, page, lens, seed=d, width=8192)
    q = p.randn(5, 8, d)
    lse = torch.empty(5, 8, dtype=torch.float32, device="cuda")
    for window, sinks in ((0, 0), (50, 3), (20000, 4)):
        out = p.cache.decode(0, q, p.table, p.t_lens, window=window, sinks=sinks, lse=lse)
        for b, n in enumerate(lens):
            p.check(b, q[b:b + 1], n - 1, out[b:b + 1], lse[b:b + 1], window, sinks, 2.0 ** -17 if kind == "bf16" else 0.0)
    for some in ([0, 1, 2, 3, 4], [0, 2], [1]):      # fewer pieces, more shares of each
        count = [new[b] for b in some]
        at = starts(count)
        qq = p.randn(at[-1], 8, d)
        ls = torch.empty(at[-1], 8, dtype=torch.float32, device="cuda")
        assert lf.lf_paged_prompt_workspace(p.cache._pages[0], len(some), 8192, 8, at[-1], max(count)) > 0
        for window, sinks in ((0, 0), (50, 3), (20000, 4)):
            out = p.cache.prompt(0, qq, p.table[some], p.t_lens[some], ints(at), max(count), window, sinks, lse=ls)
            for i, b in enumerate(some):
                rows = slice(at[i], at[i + 1])
                p.check(b, qq[rows], lens[b] - new[b], out[rows], ls[rows], window, sinks, weight_step(kind))
    kn = p.randn(st[-1], 2, d)
    want = paged_oracle.append(p.k.double().cpu().numpy(), p.np_table, lens, kn.double().cpu().numpy(), st, page)
    p.cache.append(0, kn, kn, p.table, p.t_lens, ints(st))
    np.testing.assert_array_equal(p.k.double().cpu().numpy(), want)
    assert p.cache.check() == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_decode_alone_in_a_batch_and_under_a_wider_table(kind):
    """Where a sequence's keys are cut follows its company and its table's width, and with it the last bits of its
    sums: each result is within the bounds of rounding, and the same call gives the same bits again."""
    p = Paged(kind, 8, 128, 16, [3000, 50, 1777, 2999], seed=9, width=1024)
    q = p.randn(4, 32, 128)
    step = 2.0 ** -17 if kind == "bf16" else 0.0
    batch = p.cache.decode(0, q, p.table, p.t_lens)
    assert torch.equal(batch, p.cache.decode(0, q, p.table, p.t_lens))
    for b, n in enumerate(p.lens):
        p.check(b, q[b:b + 1], n - 1, batch[b:b + 1], None, weight_step=step)
        for width in (-(-n // 16), 200, 1024):
            if width * 16 < n:
                continue
            one = [x[b:b + 1].contiguous() for x in (q, p.table[:, :width], p.t_lens)]
            alone = p.cache.decode(0, *one)
            assert torch.equal(alone, p.cache.decode(0, *one))
            p.check(b, q[b:b + 1], n - 1, alone, None, weight_step=step)


def test_the_c_named_calls_do_what_the_cache_does():
    p = Paged("bf16", 2, 128, 16, [70, 33], seed=64)
    pages, st, q = p.cache._pages[0], ints([0, 70, 103]), p.randn(103, 8, 128)
    kn, vn = p.randn(103, 2, 128), p.randn(103, 2, 128)
    lf.lf_paged_append(pages, 2, p.table, p.width, p.t_lens, kn, vn, st, 103)
    got = [x.clone() for x in (p.k, p.v)]
    p.cache.append(0, vn, kn, p.table, p.t_lens, st)
    p.cache.append(0, kn, vn, p.table, p.t_lens, st)
    assert all(torch.equal(torch.nan_to_num(a, 7.0), torch.nan_to_num(b, 7.0)) for a, b in zip(got, (p.k, p.v)))
    out = torch.empty_like(q)
    need = lf.lf_paged_prompt_workspace(pages, 2, p.width, 8, 103, 70)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    lf.lf_paged_prompt(pages, 2, p.table, p.width, p.t_lens, 8, q, st, 103, 70, out, None, 0, 0, ws, need)
    assert torch.equal(out, p.cache.prompt(0, q, p.table, p.t_lens, st, 70))


# ---- logits that are large and close to one another ----------------------------------------------------

def large_logits(kind, heads, d, page, n, seed):
    """A sequence and a maker of queries whose logits are about 2^19 / sqrt(d), differ by some tens, and are
    exact in fp32 in any order of summation: whole numbers, their sums below 2^24."""
    p = Paged(kind, heads, d, page, [n], seed=seed)
    whole = lambda *s: torch.randint(-3, 4, s, generator=p.g, device="cuda")  # noqa: E731
    k = torch.zeros(heads, n, d, device="cuda")
    k[..., 0], k[..., 1:9] = 2048.0, whole(heads, n, 8).float()
    p.rows_k[0] = k.to(p.k.dtype)
    for i in range(-(-n // page)):
        m = min(page, n - i * page)
        p.k[int(p.np_table[0, i]), :, :m] = p.rows_k[0][:, i * page:i * page + m]

    def queries(rows, q_heads):
        q = torch.zeros(rows, q_heads, d, device="cuda")
        q[..., 0], q[..., 1:9] = 256.0, whole(rows, q_heads, 8).float()
        return q.to(p.k.dtype)

    return p, queries


def check_large_logits(p, q, first_pos, out, step):
    """Against fp64, with bounds that know nothing of the logits' size: an exponent is a difference of at most 64
    in log2 (8 products of at most 9, twice, times log2(e) / 4), rounded once, with a factor that is rounded
    once; 2^x, thrice where parts are joined, is good to 2^-21; a sum over n keys and its rescalings adds
    n + 64 roundings; numerator and denominator alike.  (A logit rounded before the maximum is taken from it
    would be off by 2^-24 of its size: 2^-24 * 2^19 / 8 * log2(e) * ln 2, 0.4 %.)"""
    n = p.lens[0]
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    see = paged_oracle.visible(first_pos + np.arange(q.shape[0]), n, 0, 0)
    ref, _, size, _ = paged_oracle.attend(f(q), f(p.rows_k[0]), f(p.rows_v[0]), see)
    rel = 2 * (3 * 2.0 ** -21 + 2 * 64 * 2.0 ** -24 + (n + 64) * 2.0 ** -24)
    half = 2.0 ** -8 if p.kind == "bf16" else 2.0 ** -24
    err = (rel + step) * size
    assert (np.abs(f(out) - ref) <= err + half * (np.abs(ref) + err)).all()


@pytest.mark.parametrize("kind,d,group", [("f32", 64, 1), ("f32", 128, 4), ("f32", 16, 8), ("bf16", 128, 4),
                                          ("bf16", 64, 1), ("bf16", 16, 2)])
@pytest.mark.parametrize("n", [12, 300, 3000])
def test_decode_large_logits(kind, d, group, n):
    p, queries = large_logits(kind, 2, d, 16, n, d + n)
    q = queries(1, 2 * group)
    check_large_logits(p, q, n - 1, p.cache.decode(0, q, p.table, p.t_lens), 2.0 ** -17 if kind == "bf16" else 0.0)


@pytest.mark.parametrize("kind,d,page", [("f32", 16, 16), ("f32", 64, 16), ("f32", 128, 16), ("bf16", 128, 16),
                                         ("bf16", 64, 64), ("bf16", 128, 24), ("bf16", 32, 16)])
@pytest.mark.parametrize("n,rows", [(12, 12), (200, 150), (3000, 3)])
def test_prompt_large_logits(kind, d, page, n, rows):
    p, queries = large_logits(kind, 2, d, page, n, d + n)
    q = queries(rows, 8)
    out = p.cache.prompt(0, q, p.table, p.t_lens, ints([0, rows]), rows)
    check_large_logits(p, q, n - rows, out, weight_step(kind))


def test_prompt_large_logits_in_pieces_of_64_rows():
    """fp32, heads of 128, enough rows for the kernel that takes 64 of them at a time; the last ones are compared."""
    n = 1300
    p, queries = large_logits("f32", 16, 128, 16, n, 7)
    q = queries(n, 32)
    out = p.cache.prompt(0, q, p.table, p.t_lens, ints([0, n]), n)
    check_large_logits(p, q[-2:], n - 2, out[-2:], 0.0)


@pytest.mark.parametrize("d,page", [(128, 16), (32, 16)])
def test_prompt_large_logits_beside_values_that_are_not_finite(d, page):
    """The rows that are computed again, one by one."""
    n = 100
    p, queries = large_logits("bf16", 2, d, page, n, d)
    q = queries(n, 4)
    p.v[int(p.np_table[0, 99 // page]), :, 99 % page] = math.inf     # seen by the last row only
    out = p.cache.prompt(0, q, p.table, p.t_lens, ints([0, n]), n)
    p.lens[0] = 99
    p.rows_k[0], p.rows_v[0] = p.rows_k[0][:, :99], p.rows_v[0][:, :99]
    # Blocks take 32 tokens or more here: 96 .. 98 are computed again with 99, their weights not rounded to bf16.
    # Blocks that do not read position 99 keep the products of the others, with weights that are.
    check_large_logits(p, q[96:99], 96, out[96:99], 0.0)
    check_large_logits(p, q[:96], 0, out[:96], weight_step("bf16"))


@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_decode_products_of_a_logit_are_no_single_chain(d):
    """fp32.  One product of 1 and d - 1 of less than half a step of it: a chain of sums loses each that comes
    behind the 1 in it.  With chains of at most 8, and at most 2 + 2 additions that join them, the logit is off by
    12 halves of a step; its scaling, m and the log-sum-exp's factor are a rounding each, and the factors are
    rounded themselves: 5 more."""
    n = 2
    for at in range(0, d, 3):
        p = Paged("f32", 1, d, 16, [n], seed=d)
        k = torch.full((1, n, d), 0.98 * 2.0 ** -24, device="cuda")
        k[..., at] = 1.0
        k[:, 1] = -1000.0      # the other key weighs nothing
        p.rows_k[0] = k
        p.k[int(p.np_table[0, 0]), :, :n] = k
        q = torch.ones(1, 1, d, device="cuda")
        lse = torch.empty(1, 1, dtype=torch.float32, device="cuda")
        p.cache.decode(0, q, p.table, p.t_lens, lse=lse)
        want = float(k[0, 0].double().sum()) / math.sqrt(d)
        assert abs(float(lse) - want) <= 17 * 2.0 ** -24 * want, at


# ---- calls that the header allows -------------------------------------------------------------------------

def attend(q, k, v, n):
    """fp64 attention of one query per sequence on the GPU: q [b][H][d], k, v [b][H][most][d], n [b]."""
    q, k, v = q.double(), k.double(), v.double()
    z = torch.einsum("bhd,bhnd->bhn", q, k) / math.sqrt(q.shape[-1])
    z = z.masked_fill(torch.arange(k.shape[2], device="cuda")[None, None] >= n[:, None, None], -math.inf)
    w = torch.softmax(z, -1)
    dots = (torch.einsum("bhd,bhnd->bhn", q.abs(), k.abs()) / math.sqrt(q.shape[-1])).amax(-1)
    return torch.einsum("bhn,bhnd->bhd", w, v), torch.einsum("bhn,bhnd->bhd", w, v.abs()), dots


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_the_largest_batch(kind):
    """65535 sequences of one to four tokens: append, decode and a prompt of one token each."""
    from paged_harness import TYPES, bounds
    b, d, page = 65535, 16, 4
    g = torch.Generator(device="cuda").manual_seed(70)
    t = TYPES[kind]
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    k, v = rnd(b, 1, page, d), rnd(b, 1, page, d)
    cache = lf.LFPagedCache.over(k[None], v[None])
    table = torch.randperm(b, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    lens = (1 + torch.arange(b, device="cuda") % 4).to(torch.int32)
    kn, vn, q = rnd(b, 1, d), rnd(b, 1, d), rnd(b, 1, d)
    want = k.clone()
    want[table[:, 0].long(), :, lens.long() - 1] = kn
    start = torch.arange(b + 1, dtype=torch.int32, device="cuda")
    cache.append(0, kn, vn, table, lens, start)
    assert torch.equal(k, want)
    ref, size, dots = attend(q, k[table[:, 0].long()], v[table[:, 0].long()], lens)
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    k.zero_()
    cache.append(0, want[table[:, 0].long(), :, lens.long() - 1].contiguous(), vn, table, lens)
    assert torch.equal(k.sum((1, 2)), want[table[:, 0].long(), 0, lens.long() - 1][torch.argsort(table[:, 0])])
    k.copy_(want)
    for out, step in ((cache.decode(0, q, table, lens, kn, vn), 2.0 ** -17), (cache.decode(0, q, table, lens), 2.0 ** -17),
                      (cache.prompt(0, q, table, lens, start, 1), 2.0 ** -8)):
        tol, _ = bounds(kind, d, 4, f(ref), f(size), f(dots), step if kind == "bf16" else 0.0)
        assert (np.abs(f(out) - f(ref)) <= tol).all()
    assert torch.equal(k, want) and cache.check() == 0


@pytest.mark.parametrize("kind,d", [("bf16", 64), ("bf16", 16), ("f32", 32)])
def test_many_heads(kind, d):
    p = Paged(kind, 700, d, 16, [37, 0, 5], seed=71)
    q = p.randn(3, 700, d)
    out = p.cache.decode(0, q, p.table, p.t_lens)
    for b in (0, 2):
        p.check(b, q[b:b + 1], p.lens[b] - 1, out[b:b + 1], None, weight_step=2.0 ** -17 if kind == "bf16" else 0.0)
    q, st = p.randn(5, 700, d), ints([0, 3, 3, 5])
    out = p.cache.prompt(0, q, p.table, p.t_lens, st, 3)
    p.check(0, q[:3], 34, out[:3], None, weight_step=weight_step(kind))
    p.check(2, q[3:], 3, out[3:], None, weight_step=weight_step(kind))
    assert p.cache.check() == 0


@pytest.mark.parametrize("page", [1000, 1024, 300])
@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_a_page_that_holds_a_whole_sequence(kind, d, page):
    p = Paged(kind, 2, d, page, [300, 257, 1], seed=page + d, spare=0)
    for window, sinks in ((0, 0), (100, 3)):
        q, st = p.randn(300 + 57 + 1, 4, d), ints([0, 300, 357, 358])
        out = p.cache.prompt(0, q, p.table, p.t_lens, st, 300, window, sinks)
        for b, (lo, hi) in enumerate([(0, 300), (300, 357), (357, 358)]):
            p.check(b, q[lo:hi], p.lens[b] - (hi - lo), out[lo:hi], None, window, sinks, weight_step(kind))
        out = p.cache.decode(0, q[:3].contiguous(), p.table, p.t_lens, window=window, sinks=sinks)
        for b in range(3):
            p.check(b, q[b:b + 1], p.lens[b] - 1, out[b:b + 1], None, window, sinks, 2.0 ** -17 if kind == "bf16" else 0.0)
    assert p.cache.check() == 0


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 32), ("f32", 64)])
def test_pages_that_sequences_share(kind, d):
    """A prefix that three sequences have in common, one of them twice in the batch."""
    p = Paged(kind, 2, d, 16, [200, 150, 96], seed=72)
    table, rows_k, rows_v = p.table.clone(), p.rows_k, p.rows_v
    table[1, :6] = table[2, :6] = table[0, :6]      # 96 tokens
    for r in (rows_k, rows_v):
        r[1][:, :96], r[2][:, :96] = r[0][:, :96], r[0][:, :96]
    twice = table[[0, 1, 2, 1]].contiguous()
    p.lens = [200, 150, 96, 150]
    p.rows_k, p.rows_v = rows_k + [rows_k[1]], rows_v + [rows_v[1]]
    lens, q = ints(p.lens), p.randn(4 * 20, 4, d)
    out = p.cache.prompt(0, q, twice, lens, ints([0, 20, 40, 60, 80]), 20)
    one = p.cache.decode(0, q[:4].contiguous(), twice, lens)
    for b in range(4):
        p.check(b, q[20 * b:20 * b + 20], p.lens[b] - 20, out[20 * b:20 * b + 20], None, weight_step=weight_step(kind))
        p.check(b, q[b:b + 1], p.lens[b] - 1, one[b:b + 1], None, weight_step=2.0 ** -17 if kind == "bf16" else 0.0)


@pytest.mark.parametrize("kind,d,batch", [("bf16", 128, 5), ("bf16", 128, 40), ("bf16", 32, 40), ("f32", 64, 5)])
def test_a_captured_prompt_follows_its_starts_lengths_and_table(kind, d, batch):
    """One graph of append and prompt for up to 300 rows, replayed for other chunks of other sequences."""
    rows, most = 300, 120
    rng = np.random.default_rng(d + batch)
    p = Paged(kind, 2, d, 16, [400] * batch, seed=73)
    q, kn, vn = p.randn(rows, 4, d), p.randn(rows, 2, d), p.randn(rows, 2, d)
    table, lens, st = p.table.clone(), p.t_lens.clone(), ints([0] * (batch + 1))
    out = torch.full_like(q, 3.0)
    p.cache.append(0, kn, vn, table, lens, st)
    p.cache.prompt(0, q, table, lens, st, most, 90, 4, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.cache.append(0, kn, vn, table, lens, st)
        p.cache.prompt(0, q, table, lens, st, most, 90, 4, out=out)
    whole_k, whole_v = p.rows_k, p.rows_v
    for _ in range(4):
        new = np.minimum(rng.integers(0, most + 1, batch), 0 if batch > 5 else most)
        new[rng.integers(batch)] = most
        new[rng.integers(batch)] = rng.integers(1, most)
        if new.sum() > rows:
            new[2:] = 0
        old = rng.integers(0, 400 - most, batch)
        order = rng.permutation(batch)
        at = starts(new.tolist())
        p.lens = (old + new).tolist()
        table.copy_(p.table[ints(order.tolist()).long()])
        lens.copy_(ints(p.lens)), st.copy_(ints(at)), out.fill_(3.0)
        p.rows_k, p.rows_v = [], []
        graph.replay()
        torch.cuda.synchronize()
        assert p.cache.check() == 0
        for b in range(batch):
            for mine, whole, fresh in ((p.rows_k, whole_k, kn), (p.rows_v, whole_v, vn)):
                whole[order[b]][:, old[b]:old[b] + new[b]] = fresh[at[b]:at[b + 1]].transpose(0, 1)
                mine.append(whole[order[b]][:, :p.lens[b]])
        for b in range(batch):
            r = slice(at[b], at[b + 1])
            p.check(b, q[r], int(old[b]), out[r], None, 90, 4, weight_step(kind))
        assert (out[at[-1]:] == 3).all()


def test_a_cache_made_during_a_capture_is_refused():
    """Before anything that would end the capture: the graph that is captured around it works."""
    p = Paged("bf16", 2, 128, 16, [100, 50], seed=74)
    q = p.randn(2, 8, 128)
    want = p.cache.decode(0, q, p.table, p.t_lens)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        with pytest.raises(lf.LFError, match="before the capture"):
            lf.LFPagedCache.over(p.k[None], p.v[None])
        out = p.cache.decode(0, q, p.table, p.t_lens)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
