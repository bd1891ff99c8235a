"""Paged key-value cache on the GPU against the fp64 oracle: append, decode, prompt, and a run of
them together."""
import math

import numpy as np
import pytest
import torch

from decode_kv_cache_gb300 import longflow as lf
from oracle import paged_oracle
from paged_harness import TYPES, Paged, starts

pytestmark = pytest.mark.gpu


# ---- append -------------------------------------------------------------------------------------

@pytest.mark.parametrize("order", ["hnd", "nhd", "interleaved"])
@pytest.mark.parametrize("kind,heads,d,page", [("bf16", 8, 128, 16), ("f32", 3, 16, 5), ("bf16", 1, 16, 1),
                                               ("f32", 8, 64, 128), ("bf16", 2, 32, 24)])
def test_append(kind, heads, d, page, order):
    lens, new = [40, 7, 0, 1, 130, 33], [40, 3, 0, 1, 2, 0]
    p = Paged(kind, heads, d, page, lens, seed=5, order=order)
    st = starts(new)
    kn, vn = p.randn(st[-1] + 4, heads, d), p.randn(st[-1] + 4, heads, d)   # four rows behind the last
    before = [x.double().cpu().numpy() for x in (p.k, p.v)]
    p.cache.append(0, kn, vn, p.table, p.t_lens, torch.tensor(st, dtype=torch.int32, device="cuda"))
    for pool, rows, was in ((p.k, kn, before[0]), (p.v, vn, before[1])):
        want = paged_oracle.append(was, p.np_table, lens, rows.double().cpu().numpy(), st, page)
        np.testing.assert_array_equal(pool.double().cpu().numpy(), want)
    assert p.cache.check() == 0


def test_append_one_token_each_and_many_sequences():
    lens = [1 + (i * 7) % 50 for i in range(300)]
    p = Paged("bf16", 2, 64, 8, lens, seed=6)
    kn, vn = p.randn(300, 2, 64), p.randn(300, 2, 64)
    was = p.k.double().cpu().numpy()
    p.cache.append(0, kn, vn, p.table, p.t_lens)
    want = paged_oracle.append(was, p.np_table, lens, kn.double().cpu().numpy(), starts([1] * 300), 8)
    np.testing.assert_array_equal(p.k.double().cpu().numpy(), want)


def test_append_skips_bad_places_and_says_so():
    """Pages outside the pool, a length above the row and more tokens than the length: those tokens
    are left out, all others stored."""
    lens = [20, 20, 20, 20]
    p = Paged("f32", 2, 16, 8, lens, seed=7)
    table = p.np_table.copy()
    table[0, 1] = p.k.shape[0]       # positions 8..15 of sequence 0
    table[1, 0] = -1                 # positions 0..7 of sequence 1
    t = torch.from_numpy(table).cuda()
    claimed = torch.tensor([20, 20, 8 * p.width + 3, 2], dtype=torch.int32, device="cuda")
    new = [20, 20, 4, 4]             # sequence 2: only position 8 * width - 1 fits; 3: two before 0
    st = starts(new)
    kn, vn = p.randn(st[-1], 2, 16), p.randn(st[-1], 2, 16)
    table[2, p.width - 1] = table[3, 2]   # a page of sequence 3 that it does not write here
    t = torch.from_numpy(table).cuda()
    want = p.k.cpu().clone()
    for b in range(4):
        for i in range(new[b]):
            pos = int(claimed[b]) - new[b] + i
            if not 0 <= pos < 8 * p.width or not 0 <= table[b, pos // 8] < p.k.shape[0]:
                continue
            want[table[b, pos // 8], :, pos % 8] = kn[st[b] + i].cpu()
    p.cache.append(0, kn, vn, t, claimed, torch.tensor(st, dtype=torch.int32, device="cuda"))
    got = p.k.cpu()
    assert torch.equal(torch.nan_to_num(got, 77.0), torch.nan_to_num(want, 77.0))
    assert p.cache.check() == lf.LF_DEVERR_STATE
    assert p.cache.check() == 0


# ---- decode -------------------------------------------------------------------------------------

def run_decode(kind, heads, group, d, page, lens, window=0, sinks=0, writes=False, order="hnd", seed=0, scale=1.0):
    p = Paged(kind, heads, d, page, lens, seed=seed, order=order, scale=scale)
    b = len(lens)
    q = p.randn(b, heads * group, d)
    kn = vn = None
    if writes:
        kn, vn = p.randn(b, heads, d), p.randn(b, heads, d)
        for i, n in enumerate(lens):
            if n:
                p.hide(i, n - 1, n)       # the call brings it
                p.rows_k[i][:, n - 1] = kn[i]
                p.rows_v[i][:, n - 1] = vn[i]
    if window:                            # what no query sees may hold anything
        for i, n in enumerate(lens):
            p.hide(i, min(sinks, n), max(min(sinks, n), n - window))
    was = [x.double().cpu().numpy() for x in (p.k, p.v)]
    lse = torch.empty(b, heads * group, dtype=torch.float32, device="cuda")
    out = p.cache.decode(0, q, p.table, p.t_lens, kn, vn, window=window, sinks=sinks, lse=lse)
    worst = 0.0
    for i, n in enumerate(lens):
        # p is split into two bf16 for the product with V (bf16 caches): half a step of the second, 2^-17
        worst = max(worst, p.check(i, q[i:i + 1], n - 1, out[i:i + 1], lse[i:i + 1], window, sinks,
                                   2.0 ** -17 if kind == "bf16" else 0.0))
    if writes:
        for pool, new, old in ((p.k, kn, was[0]), (p.v, vn, was[1])):
            st = starts([1 if n else 0 for n in lens])
            rows = new[[i for i, n in enumerate(lens) if n]].double().cpu().numpy()
            np.testing.assert_array_equal(pool.double().cpu().numpy(),
                                          paged_oracle.append(old, p.np_table, lens, rows, st, page))
    else:
        for pool, old in ((p.k, was[0]), (p.v, was[1])):
            np.testing.assert_array_equal(pool.double().cpu().numpy(), old)
    assert p.cache.check() == 0
    return worst


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_decode_every_head_layout(kind, d, group):
    run_decode(kind, 2, group, d, 16, [1, 2, 15, 16, 17, 0, 100, 257], seed=d + group)
    # long enough for ranges that cut units, and joins
    run_decode(kind, 2, group, d, 16, [700, 0, 1, 2500], seed=d + group + 1, writes=True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 64, 128, 256])
def test_decode_page_sizes(kind, page):
    run_decode(kind, 3, 4, 128, page, [5, 1300, 640, 129, 1], seed=page, writes=True)


@pytest.mark.parametrize("order", ["nhd", "interleaved"])
def test_decode_memory_orders(order):
    run_decode("bf16", 4, 2, 128, 16, [333, 1, 1999], order=order, writes=True)
    run_decode("f32", 4, 2, 64, 16, [333, 1, 1999], order=order, writes=True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (100, 4), (64, 0), (1500, 4), (3000, 5),
                                          (2**31 - 1, 2**31 - 1)])
def test_decode_windows(kind, window, sinks):
    run_decode(kind, 2, 4, 128, 16, [1, 3, 8, 11, 12, 104, 105, 1504, 2400, 0], window, sinks, writes=True)


def test_decode_one_long_sequence_and_many_short():
    run_decode("bf16", 1, 8, 128, 16, [40001], seed=1, writes=True)
    run_decode("bf16", 8, 4, 128, 32, [(i * 37) % 90 for i in range(300)] + [3000], seed=2, writes=True)
    run_decode("f32", 1, 1, 64, 16, [30011], seed=3)


def test_decode_sharp_and_flat_logits():
    run_decode("bf16", 2, 4, 128, 16, [900, 1200], scale=6.0)       # one key takes nearly all
    run_decode("f32", 2, 4, 128, 16, [900, 1200], scale=6.0)
    run_decode("bf16", 2, 4, 128, 16, [900, 1200], scale=0.0)       # all alike


def test_decode_does_not_depend_on_its_company():
    """A sequence gives the same bits alone, in a batch, and again."""
    p = Paged("bf16", 8, 128, 16, [3000, 50, 1777, 2999], seed=9)
    q = p.randn(4, 32, 128)
    a = p.cache.decode(0, q, p.table, p.t_lens)
    for _ in range(3):
        assert torch.equal(a, p.cache.decode(0, q, p.table, p.t_lens))


def test_decode_not_finite_sets_the_error_word():
    p = Paged("bf16", 2, 128, 16, [100, 50], seed=10)
    q = p.randn(2, 8, 128)
    q[1, 3, 5] = math.nan
    out = p.cache.decode(0, q, p.table, p.t_lens)
    assert p.cache.check() == lf.LF_DEVERR_NONFINITE
    assert torch.isnan(out[1, 3]).all()
    p.check(0, q[:1], 99, out[:1], None, weight_step=2.0 ** -17)
    rest = [h for h in range(8) if h != 3]
    assert torch.isfinite(out[1, rest].float()).all()


def test_decode_bad_pages_and_lengths_set_the_error_word():
    p = Paged("bf16", 2, 128, 16, [100, 50, 200], seed=11)
    q = p.randn(3, 8, 128)
    p.table[1, 1] = p.k.shape[0] + 5
    p.t_lens[2] = 16 * p.width + 1
    out = p.cache.decode(0, q, p.table, p.t_lens)
    assert p.cache.check() & lf.LF_DEVERR_STATE
    p.check(0, q[:1], 99, out[:1], None, weight_step=2.0 ** -17)
    # a token past its row of the table is stored nowhere
    was, kn = p.k.clone(), p.randn(3, 2, 128)
    p.cache.decode(0, q, p.table, p.t_lens, kn, kn)
    assert p.cache.check() & lf.LF_DEVERR_STATE
    changed = (torch.nan_to_num(p.k, 77.0) != torch.nan_to_num(was, 77.0)).any(-1).any(1).nonzero().tolist()
    x = int(p.np_table[0, 99 // 16])
    y = int(p.np_table[1, 49 // 16])
    assert sorted(changed) == sorted([[x, 99 % 16], [y, 49 % 16]])
    p.t_lens[2] = -3
    out = p.cache.decode(0, q, p.table, p.t_lens)
    assert p.cache.check() & lf.LF_DEVERR_STATE
    assert (out[2] == 0).all()


def test_offsets_beyond_32_bits():
    """Pages whose elements lie past 2^32 bytes and 2^31 elements of the pools."""
    free, _ = torch.cuda.mem_get_info()
    if free < 24e9:
        pytest.skip("needs ~20 GB of free device memory")
    pages, heads, d, page = 1_200_000, 2, 128, 16
    k, v = (torch.empty(pages, heads, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2**31
    small = Paged("bf16", heads, d, page, [700], seed=12)
    far = pages - 1 - np.arange(small.width, dtype=np.int64) * 7
    for i in range(-(-700 // page)):
        k[far[i]], v[far[i]] = small.k[small.np_table[0, i]], small.v[small.np_table[0, i]]
    big = lf.LFPagedCache.over(k[None], v[None])
    table = torch.from_numpy(far.astype(np.int32))[None].cuda()
    q, kn, vn = small.randn(1, 8, d), small.randn(1, heads, d), small.randn(1, heads, d)
    a = small.cache.decode(0, q, small.table, small.t_lens, kn, vn)
    b = big.decode(0, q, table, small.t_lens, kn, vn)
    assert torch.equal(a, b)
    last = 699 // page
    assert torch.equal(k[far[last], :, 699 % page], kn[0])
    qq, st = small.randn(70, 8, d), torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    a = small.cache.prompt(0, qq, small.table, small.t_lens, st, 70)
    assert torch.equal(a, big.prompt(0, qq, table, small.t_lens, st, 70))
    kn, vn = small.randn(70, heads, d), small.randn(70, heads, d)
    big.append(0, kn, vn, table, small.t_lens, st)
    assert torch.equal(k[far[last], :, 699 % page], kn[-1])


# ---- prompt -------------------------------------------------------------------------------------

def run_prompt(kind, heads, group, d, page, old, new, window=0, sinks=0, order="hnd", seed=0, scale=1.0,
               behind=5, weight_step=None):
    lens = [a + b for a, b in zip(old, new)]
    p = Paged(kind, heads, d, page, lens, seed=seed, order=order, scale=scale)
    st = starts(new)
    q = p.randn(st[-1] + behind, heads * group, d)
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:2], 3.0, dtype=torch.float32, device="cuda")
    p.cache.prompt(0, q, p.table, p.t_lens, torch.tensor(st, dtype=torch.int32, device="cuda"), max(new),
                   window=window, sinks=sinks, out=out, lse=lse)
    # a bf16 cache's weights may be rounded to bf16 before the product with V
    step = weight_step if weight_step is not None else (2.0 ** -8 if kind == "bf16" else 0.0)
    worst = 0.0
    for b in range(len(lens)):
        rows = slice(st[b], st[b + 1])
        worst = max(worst, p.check(b, q[rows], old[b], out[rows], lse[rows], window, sinks, step))
    assert (out[st[-1]:] == 3).all() and (lse[st[-1]:] == 3).all()   # rows behind the last are left
    assert p.cache.check() == 0
    return worst


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_prompt_every_head_layout(kind, d, group):
    run_prompt(kind, 2, group, d, 16, [0, 0, 5, 130, 0], [1, 70, 3, 40, 0], seed=d + group)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 64, 128, 256])
def test_prompt_page_sizes(kind, page):
    run_prompt(kind, 2, 4, 128, page, [0, 300, 127], [129, 33, 1], seed=page)


@pytest.mark.parametrize("order", ["nhd", "interleaved"])
def test_prompt_memory_orders(order):
    run_prompt("bf16", 2, 2, 128, 16, [0, 200], [150, 20], order=order)
    run_prompt("f32", 2, 2, 64, 16, [0, 200], [150, 20], order=order)


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (100, 4), (128, 130), (300, 1),
                                          (2**31 - 1, 2**31 - 1)])
def test_prompt_windows(kind, d, window, sinks):
    run_prompt(kind, 2, 2, d, 16, [0, 400, 0], [390, 60, 9], window, sinks)


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("f32", 128)])
def test_prompt_longer(kind, d):
    run_prompt(kind, 1, 2, d, 64, [0], [1100], seed=3)
    run_prompt(kind, 1, 8, d, 32, [1500], [37], seed=4)


@pytest.mark.parametrize("kind,d,page", [("bf16", 128, 16), ("bf16", 64, 128), ("bf16", 32, 16), ("bf16", 128, 24),
                                         ("f32", 64, 16), ("f32", 128, 64)])
def test_prompt_few_rows_over_a_long_axis(kind, d, page):
    """Several blocks share the keys of few rows, and their parts are joined."""
    assert lf.lf_paged_prompt_workspace(Paged(kind, 2, d, page, [1]).cache._pages[0], 3, 6000 // page, 8, 9, 5) > 0
    run_prompt(kind, 2, 4, d, page, [5000, 0, 77], [3, 1, 5], seed=d)
    run_prompt(kind, 1, 8, d, page, [6000], [1], seed=d + 1)
    run_prompt(kind, 2, 1, d, page, [5000, 300], [40, 0], 3000, 200, seed=d + 2)
    run_prompt(kind, 1, 2, d, page, [0, 4000], [140, 130], seed=d + 3)


@pytest.mark.parametrize("kind,d,group", [("bf16", 128, 4), ("bf16", 64, 1), ("bf16", 32, 8), ("f32", 64, 2)])
def test_prompt_mixed_batches(kind, d, group):
    """One long chunk among sequences of a token or none: pieces are numbered by the rows before them."""
    new = [1, 0, 1, 130, 1, 0, 64, 1, 256, 0] + [1] * 30
    old = [i * 7 % 90 for i in range(len(new))]
    run_prompt(kind, 2, group, d, 16, old, new, seed=d + group)
    run_prompt(kind, 1, group, d, 16, old, new[::-1], 20, 2, seed=d + group + 1)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("batch", [32, 33, 1024, 1025])
def test_prompt_many_sequences(kind, batch):
    """The sequence of a piece is found 32 at a time: one, two and three rounds of it."""
    new = [3 if i % 97 == 5 else i % 2 for i in range(batch)]
    new[batch // 2], new[-1] = 90, 70
    run_prompt(kind, 1, 4, 64, 8, [i % 5 for i in range(batch)], new, seed=batch)


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 32), ("f32", 64)])
def test_prompt_row_starts(kind, d):
    """Rows in front of the first sequence are left; starts outside the rows spoil no other sequence."""
    p = Paged(kind, 2, d, 16, [200, 90, 150], seed=d)
    q = p.randn(700, 8, d)
    step = 2.0 ** -8 if kind == "bf16" else 0.0

    def run(st, most):
        out = torch.full_like(q, 3.0)
        p.cache.prompt(0, q, p.table, p.t_lens, torch.tensor(st, dtype=torch.int32, device="cuda"), most, out=out)
        return out

    out = run([300, 500, 560, 700], 200)
    for b, (lo, hi) in enumerate([(300, 500), (500, 560), (560, 700)]):
        p.check(b, q[lo:hi], p.lens[b] - (hi - lo), out[lo:hi], None, weight_step=step)
    assert (out[:300] == 3).all() and p.cache.check() == 0
    out = run([-1000, 100, 160, 300], 140)       # the first sequence starts in front of the rows
    p.check(1, q[100:160], 30, out[100:160], None, weight_step=step)
    p.check(2, q[160:300], 10, out[160:300], None, weight_step=step)
    assert (out[300:] == 3).all() and p.cache.check() == lf.LF_DEVERR_STATE
    out = run([0, 200, 260, 2**31 - 1], 200)     # the last one ends behind them
    p.check(0, q[:200], 0, out[:200], None, weight_step=step)
    p.check(1, q[200:260], 30, out[200:260], None, weight_step=step)
    assert (out[260:] == 3).all() and p.cache.check() == lf.LF_DEVERR_STATE
    run([0, 400, 100, 300], 200)                 # they decrease: reported, nothing more is said
    assert p.cache.check() & lf.LF_DEVERR_STATE


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 32), ("f32", 64)])
def test_prompt_shared_keys_and_values_that_are_not_finite(kind, d):
    """As below, where blocks share the keys: a block whose keys hold a NaN computes its share by hand."""
    p = Paged(kind, 1, d, 16, [4100], seed=23)
    q = p.randn(60, 2, d)
    st = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    x, s = int(p.np_table[0, 4070 // 16]), 4070 % 16
    p.v[x, 0, s] = math.nan
    out = p.cache.prompt(0, q, p.table, p.t_lens, st, 60)
    assert torch.isnan(out[30:].float()).all()
    p.check(0, q[:30], 4040, out[:30], None, weight_step=2.0 ** -8 if kind == "bf16" else 0.0)


def test_prompt_sharp_and_flat_logits():
    run_prompt("bf16", 2, 4, 128, 16, [0], [300], scale=6.0)
    run_prompt("f32", 2, 4, 128, 16, [0], [300], scale=6.0)
    run_prompt("bf16", 2, 4, 128, 16, [0], [300], scale=0.0)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_prompt_rows_before_position_zero_see_nothing(kind):
    """More queries than the sequence is long: the first ones sit before position 0."""
    p = Paged(kind, 2, 128, 16, [10, 40], seed=20)
    q = p.randn(14 + 40, 8, 128)
    st = torch.tensor([0, 14, 54], dtype=torch.int32, device="cuda")
    lse = torch.empty(54, 8, dtype=torch.float32, device="cuda")
    out = p.cache.prompt(0, q, p.table, p.t_lens, st, 40, lse=lse)
    assert (out[:4] == 0).all() and torch.isneginf(lse[:4]).all()
    step = 2.0 ** -8 if kind == "bf16" else 0.0
    p.check(0, q[4:14], 0, out[4:14], lse[4:14], weight_step=step)
    p.check(1, q[14:], 0, out[14:], lse[14:], weight_step=step)
    assert p.cache.check() == lf.LF_DEVERR_STATE


@pytest.mark.parametrize("kind,page", [("bf16", 16), ("bf16", 24), ("f32", 16)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_prompt_what_a_query_does_not_see_does_not_reach_it(kind, page, bad):
    """A token with values that are not finite changes only the queries that see it."""
    p = Paged(kind, 2, 128, page, [200], seed=21)
    q = p.randn(200, 4, 128)
    st = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    x, s = int(p.np_table[0, 150 // page]), 150 % page
    p.v[x, 1, s] = bad
    for window, sinks, clean in ((0, 0, range(150)), (20, 0, [*range(150), *range(170, 200)])):
        good = [int(i) for i in clean]
        out = p.cache.prompt(0, q, p.table, p.t_lens, st, 200, window=window, sinks=sinks)
        assert not torch.isfinite(out[150, 2:].float()).any()
        assert torch.isfinite(out[:, :2].float()).all()          # the other head
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        see = paged_oracle.visible(good, 200, window, sinks)
        vv = f(p.rows_v[0]).copy()
        vv[1, 150] = 0.0
        ref, _, size, dots = paged_oracle.attend(f(q[good]), f(p.rows_k[0]), vv, see)
        from paged_harness import bounds
        tol, _ = bounds(kind, 128, 200, ref, size, dots, 2.0 ** -8 if kind == "bf16" else 0.0)
        assert (np.abs(f(out[good]) - ref) <= tol).all()


def test_prompt_bad_rows_pages_and_lengths_set_the_error_word():
    p = Paged("bf16", 2, 128, 16, [100, 50, 60], seed=22)
    q = p.randn(210, 8, 128)
    st = torch.tensor([0, 100, 150, 300], dtype=torch.int32, device="cuda")   # the last one's end: past q
    p.table[1, 1] = -1
    out = torch.full_like(q, 3.0)
    p.cache.prompt(0, q, p.table, p.t_lens, st, 100, out=out)
    assert p.cache.check() & lf.LF_DEVERR_STATE
    p.check(0, q[:100], 0, out[:100], None, weight_step=2.0 ** -8)
    assert (out[150:] == 3).all()
    # more rows than max_q: the rest is left
    st = torch.tensor([0, 100, 150, 210], dtype=torch.int32, device="cuda")
    p = Paged("bf16", 2, 128, 16, [100, 50, 60], seed=22)
    p.cache.prompt(0, q, p.table, p.t_lens, st, 60)
    assert p.cache.check() == lf.LF_DEVERR_STATE


# ---- together -------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind,d,group,window,sinks", [("bf16", 128, 4, 0, 0), ("bf16", 64, 2, 40, 4),
                                                       ("f32", 32, 1, 0, 0)])
def test_a_conversation(kind, d, group, window, sinks):
    """Prompts enter in two chunks, then tokens one by one (the decode steps as one captured graph that
    advances the lengths itself): every output equals attention over the tokens so far."""
    heads, page, steps = 2, 16, 20
    chunk1, chunk2 = [30, 1, 17], [11, 45, 0]
    total = [a + b + steps for a, b in zip(chunk1, chunk2)]
    t = TYPES[kind]
    g = torch.Generator(device="cuda").manual_seed(31)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    k, v = ([rnd(n, heads, d) for n in total] for _ in range(2))
    q = [rnd(n, heads * group, d) for n in total]
    width = max(-(-n // page) for n in total)
    cache = lf.LFPagedCache(2, 3 * width, page, heads, d, dtype=kind)
    table = torch.randperm(3 * width, generator=g, device="cuda").to(torch.int32).view(3, width)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    outs = [[] for _ in total]
    at = [0, 0, 0]
    for chunk in (chunk1, chunk2):
        st = torch.tensor(starts(chunk), dtype=torch.int32, device="cuda")
        lens += torch.tensor(chunk, dtype=torch.int32, device="cuda")
        cut = lambda x: torch.cat([x[b][at[b]:at[b] + chunk[b]] for b in range(3)])  # noqa: E731
        cache.append(1, cut(k), cut(v), table, lens, st)
        o = cache.prompt(1, cut(q), table, lens, st, max(chunk), window=window, sinks=sinks)
        for b in range(3):
            outs[b].append(o[int(st[b]):int(st[b + 1])].clone())
            at[b] += chunk[b]
    qi, ki, vi = (torch.empty(3, h, d, dtype=t, device="cuda") for h in (heads * group, heads, heads))
    out = torch.empty_like(qi)

    def step():
        lens.add_(1)
        cache.decode(1, qi, table, lens, ki, vi, window=window, sinks=sinks, out=out)

    graph = None
    for i in range(steps):
        for dst, src in ((qi, q), (ki, k), (vi, v)):
            dst.copy_(torch.stack([src[b][at[b] + i] for b in range(3)]))
        if i < 2:
            step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        for b in range(3):
            outs[b].append(out[b:b + 1].clone())
    assert cache.check() == 0
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    from paged_harness import bounds
    for b, n in enumerate(total):
        see = paged_oracle.visible(np.arange(n), n, window, sinks)
        ref, _, size, dots = paged_oracle.attend(f(q[b]), f(k[b]).swapaxes(0, 1), f(v[b]).swapaxes(0, 1), see)
        tol, _ = bounds(kind, d, n, ref, size, dots, 2.0 ** -8 if kind == "bf16" else 0.0)
        got = f(torch.cat(outs[b]))
        assert (np.abs(got - ref) <= tol).all(), b


def test_streams_and_graphs_do_not_meet():
    """Long calls on two side streams at once, and two graphs replayed at once, give what they give alone."""
    a = Paged("bf16", 8, 128, 16, [5000, 3000, 70], seed=41)
    b = Paged("bf16", 8, 128, 16, [2000, 6000, 1], seed=42)
    qa, qb = a.randn(3, 32, 128), b.randn(3, 32, 128)
    ref_a, ref_b = a.cache.decode(0, qa, a.table, a.t_lens), b.cache.decode(0, qb, b.table, b.t_lens)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(a.cache.decode(0, qa, a.table, a.t_lens, stream=s1), b.cache.decode(0, qb, b.table, b.t_lens, stream=s2))
           for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref_a) and torch.equal(y, ref_b) for x, y in got)
    graphs = []
    for p, q in ((a, qa), (b, qb)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = p.cache.decode(0, q, p.table, p.t_lens)
        graphs.append((g, o))
    for p, q in ((a, qa), (b, qb)):           # few rows: prompts that share keys and join
        st = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
        ref = p.cache.prompt(0, q, p.table, p.t_lens, st, 1)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = p.cache.prompt(0, q, p.table, p.t_lens, st, 1)
        graphs.append((g, o, ref, st))
    for _ in range(10):
        for (g, *_), s in zip(graphs, (s1, s2, s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], ref_a) and torch.equal(graphs[1][1], ref_b)
    assert torch.equal(graphs[2][1], graphs[2][2]) and torch.equal(graphs[3][1], graphs[3][2])


def test_workspaces_are_asked_for():
    p = Paged("bf16", 2, 128, 16, [4000, 5000], seed=51)
    pages, q = p.cache._pages[0], p.randn(2, 8, 128)
    out, st = torch.empty_like(q), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    n = lf.lf_paged_decode_workspace(pages, 2, p.width, 8)
    m = lf.lf_paged_prompt_workspace(pages, 2, p.width, 8, 2, 1)
    assert n > 0 and m > 0
    # few short sequences need none, by the table's width or by the window
    assert lf.lf_paged_decode_workspace(pages, 2, 4, 8) == 0
    assert lf.lf_paged_decode_workspace(pages, 2, 1000, 8, window=60, sinks=4) == 0
    ws = torch.empty(max(n, m) + 16, dtype=torch.uint8, device="cuda")
    for w, size in ((None, n), (ws, n - 1), (ws.data_ptr() + 8, n)):
        with pytest.raises(lf.LFError, match="workspace"):
            lf.lf_paged_decode(pages, 2, p.table, p.width, p.t_lens, 8, q, None, None, out, None, 0, 0, w, size)
    for w, size in ((None, m), (ws, m - 1), (ws.data_ptr() + 8, m)):
        with pytest.raises(lf.LFError, match="workspace"):
            lf.lf_paged_prompt(pages, 2, p.table, p.width, p.t_lens, 8, q, st, 2, 1, out, None, 0, 0, w, size)
    lf.lf_paged_decode(pages, 2, p.table, p.width, p.t_lens, 8, q, None, None, out, None, 0, 0, ws, n)
    p.check(0, q[:1], 3999, out[:1], None, weight_step=2.0 ** -17)
    lf.lf_paged_prompt(pages, 2, p.table, p.width, p.t_lens, 8, q, st, 2, 1, out, None, 0, 0, ws, m)
    p.check(1, q[1:], 4999, out[1:], None, weight_step=2.0 ** -8)


def test_bad_tensors_are_refused():
    p = Paged("bf16", 2, 128, 16, [100, 50], seed=50)
    q = p.randn(2, 8, 128)
    c = p.cache
    for call, msg in [
        (lambda: c.decode(1, q, p.table, p.t_lens), "layer 1 outside"),
        (lambda: c.decode(-1, q, p.table, p.t_lens), "layer -1 outside"),
        (lambda: c.decode(0, q.float(), p.table, p.t_lens), "q: expected"),
        (lambda: c.decode(0, q[:, :, :64], p.table, p.t_lens), "q: expected"),
        (lambda: c.decode(0, q[:1], p.table, p.t_lens), "q: expected"),
        (lambda: c.decode(0, q, p.table.long(), p.t_lens), "page_table: expected"),
        (lambda: c.decode(0, q, p.table[:, ::2], p.t_lens), "page_table: expected"),
        (lambda: c.decode(0, q, p.table, p.t_lens.cpu()), "lens: expected"),
        (lambda: c.decode(0, q, p.table, p.t_lens, q[:, :2]), "k_new: expected"),
        (lambda: c.decode(0, q, p.table, p.t_lens, q[:, :2].contiguous()), "v_new: expected"),
        (lambda: c.decode(0, q, p.table, p.t_lens, sinks=3), "sinks need a window"),
        (lambda: c.decode(0, q, p.table, p.t_lens, out=q.float()), "out: expected"),
        (lambda: c.decode(0, q, p.table, p.t_lens, lse=q), "lse: expected"),
        (lambda: c.prompt(0, q, p.table, p.t_lens, p.t_lens, 2), "q_start: expected"),
        (lambda: c.append(0, q[:, :2].contiguous(), q[:, :1].contiguous(), p.table, p.t_lens), "v_new: expected"),
        (lambda: lf.LFPagedCache.over(p.k[None], p.v[None].float()), "must agree"),
        (lambda: lf.LFPagedCache.over(p.k[None].transpose(3, 4), p.v[None].transpose(3, 4)), "contiguous"),
    ]:
        with pytest.raises(lf.LFError, match=msg):
            call()
    p.check(0, q[:1], 99, c.decode(0, q, p.table, p.t_lens)[:1], None, weight_step=2.0 ** -17)
