"""Rotary positions on the GPU against the fp64 oracle: rows where they lie, and on their way to a paged cache."""
import math

import numpy as np
import pytest
import torch

from decode_kv_cache_gb300 import longflow as lf
from oracle import paged_oracle, rotary_oracle
from paged_harness import HALF_STEP, TYPES, Paged, starts

pytestmark = pytest.mark.gpu

f64 = lambda x: x.detach().double().cpu().numpy()  # noqa: E731


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def close(kind, got, want, size):
    """A cosine is off by 3.5 x 2^-24 (its angle by 2^-34 of a turn and 2^-25 of at most pi / 4, sincospif by two
    units of at most 2^-24 each), a product with it, a sum and the scale by 2^-24 more each: 7 x 2^-24 of the two
    terms; the result is rounded once."""
    err = 7 * 2.0 ** -24 * size
    tol = err + HALF_STEP[kind] * (np.abs(want) + err) * (size > 0)   # what does not turn is copied
    assert got.shape == want.shape
    off = np.abs(got - want)
    assert (off <= tol).all(), f"off by {off.max()}, {np.nanmax(off / np.maximum(tol, 1e-300)):.3g} of the bound"


def values(kind, *shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(TYPES[kind])


def position_set(rng, *shape):
    p = rng.integers(-200000, 200000, size=shape)
    p.ravel()[:6] = [0, 1, -1, 2**31 - 1, -2**31, 131071][:p.size]
    return p


SECTIONS = {1: None, 2: lambda p: [p - p // 3, p // 3], 3: lambda p: [p // 4, p // 2, p - p // 4 - p // 2],
            4: lambda p: [1, 0, p - 2, 1]}


@pytest.mark.parametrize("axes", [1, 3, 4])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("kind,dim,rotary", [("bf16", 128, 128), ("bf16", 64, 32), ("bf16", 16, 16), ("bf16", 80, 48),
                                             ("bf16", 512, 512), ("f32", 128, 128), ("f32", 48, 16), ("f32", 256, 64),
                                             ("f32", 16, 16)])
def test_rows(kind, dim, rotary, adjacent, axes):
    rng = np.random.default_rng(dim + axes)
    sections = SECTIONS[axes] and SECTIONS[axes](rotary // 2)
    r = lf.LFRotary(rotary, base=1e6, sections=sections, adjacent=adjacent, scale=0.75)
    axis = None if sections is None else np.repeat(np.arange(axes), sections)
    freq = rotary_oracle.frequencies(rotary, 1e6)
    for tokens, hq, hk in ((1, 1, 0), (1, 32, 8), (7, 3, 1), (301, 5, 2), (9000, 2, 1)):
        pos = position_set(rng, axes, tokens)
        q = values(kind, tokens, hq, dim, seed=tokens)
        k = values(kind, tokens, hk, dim, seed=tokens + 1) if hk else None
        p = ints(pos if axes > 1 else pos[0])
        for inverse in (False, True):
            out = r.rotate(q, p, k=k, inverse=inverse)
            for x, y in zip((q, k), out if hk else (out,)):
                want, size = rotary_oracle.rotate(f64(x), pos, freq, axis, adjacent, 0.75, inverse)
                close(kind, f64(y), want, size)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_of_a_slab_and_of_other_orders(kind):
    """Prompts as LFCache.prefill takes them, [batch][heads][tokens][dim], rotated in place through a transposed
    view; rows inside wider ones; the same row for every token; one position set for all axes."""
    b, h, n, d = 3, 4, 50, 64
    r = lf.LFRotary(64, sections=[8, 12, 12])
    freq, axis = rotary_oracle.frequencies(64), np.repeat([0, 1, 2], [8, 12, 12])
    rng = np.random.default_rng(5)
    pos = position_set(rng, 3, b, n)
    slab = values(kind, b, h, n, d, seed=1)
    before = f64(slab.transpose(1, 2))
    x = slab.transpose(1, 2)
    assert r.rotate(x, ints(pos), q_out=x) is x
    want, size = rotary_oracle.rotate(before, pos, freq, axis)
    close(kind, f64(slab.transpose(1, 2)), want, size)

    wide = values(kind, b * n, h + 3, d + 32, seed=2)
    keep = wide.clone()
    x, p = wide[:, 2:2 + h, 16:16 + d], ints(pos.reshape(3, -1))
    want, size = rotary_oracle.rotate(f64(x), pos.reshape(3, -1), freq, axis)
    y = r.rotate(x, p)
    close(kind, f64(y), want, size)
    assert torch.equal(wide, keep)
    r.rotate(x, p, q_out=x)
    assert torch.equal(x, y)
    keep[:, 2:2 + h, 16:16 + d] = y
    assert torch.equal(wide, keep)          # nothing around the rows has changed

    one = values(kind, 1, h, d, seed=3).expand(b * n, h, d)
    want, size = rotary_oracle.rotate(f64(one), np.broadcast_to(pos[1].reshape(1, -1), (3, b * n)), freq, axis)
    close(kind, f64(r.rotate(one, ints(pos[1].reshape(-1)))), want, size)


def test_far_positions_keep_their_angles():
    """Frequency 1 at positions up to 2^31: fp32 angles would be off by a hundred radians."""
    r = lf.LFRotary(16, inv_freq=[1.0, -1.0, 0.1, 3e-9, 0.0, 1024.0, 1e-4, 6.25])
    pos = np.array([[2**31 - 1, -2**31, 10**9 + 7, 123456789, 1]])
    x = values("f32", 5, 1, 16)
    want, size = rotary_oracle.rotate(f64(x), pos, [1.0, -1.0, 0.1, 3e-9, 0.0, 1024.0, 1e-4, 6.25])
    # The expectation's own angles are products in 64 bits, off by 2^-53 of up to 2^41 radians at frequency 1024: 2^-12,
    # too rough, and that pair is left out; at 6.25, 2^34 radians, by 2^-19, which the rest is given for.
    got = f64(r.rotate(x, ints(pos[0])))
    keep = [i for i in range(16) if i % 8 != 5]
    err = 7 * 2.0 ** -24 * size + 2.0 ** -19 * size
    assert (np.abs(got - want) <= err + 2.0 ** -24 * (np.abs(want) + err))[..., keep].all()
    near, size = rotary_oracle.rotate(f64(x), pos * 0 + 3, [1.0, -1.0, 0.1, 3e-9, 0.0, 1024.0, 1e-4, 6.25])
    close("f32", f64(r.rotate(x, ints(pos[0] * 0 + 3))), near, size)


def test_a_gradient_goes_back_by_the_inverse():
    """d <w, rotate(x)> / dx = rotate(w, inverse), by the formula and, the rotation being linear, by the difference
    that each unit of x makes."""
    d, rotary = 64, 32
    r = lf.LFRotary(rotary, sections=[4, 6, 6], scale=1.25)
    freq, axis = rotary_oracle.frequencies(rotary), np.repeat([0, 1, 2], [4, 6, 6])
    pos = np.array([[5], [77], [-300]])
    w = values("f32", 1, 1, d)
    got = f64(r.rotate(w, ints(pos), inverse=True)).ravel()
    want, size = rotary_oracle.rotate(f64(w), pos, freq, axis, scale=1.25, inverse=True)
    close("f32", got.reshape(1, 1, d), want, size)
    units = torch.eye(d, device="cuda").view(d, 1, d)
    y = f64(r.rotate(units, ints(np.repeat(pos, d, 1))))[:, 0]     # row i: what unit i of x does to y
    by_difference = y @ f64(w).ravel()
    assert (np.abs(got - by_difference) <= 2 * 7 * 2.0 ** -24 * (size.ravel() + np.abs(got)) + 2.0 ** -23 * np.abs(got)).all()
    q = values("f32", 40, 3, d, seed=4)
    p = ints(np.repeat(pos, 40, 1))
    x = q.double().requires_grad_()
    a, b = rotary_oracle.pairs(rotary, False)
    ang = torch.tensor(pos[axis, 0] * freq, device="cuda")
    y = torch.cat(((x[..., a] * ang.cos() - x[..., b] * ang.sin()) * 1.25, (x[..., b] * ang.cos() + x[..., a] * ang.sin()) * 1.25,
                   x[..., rotary:]), -1)
    g = values("f32", 40, 3, d, seed=5)
    y.backward(g.double())
    _, size = rotary_oracle.rotate(f64(g), np.repeat(pos, 40, 1), freq, axis, scale=1.25)
    close("f32", f64(r.rotate(g, p, inverse=True)), f64(x.grad), size)


def test_values_that_are_not_finite_stay_in_their_pairs():
    r = lf.LFRotary(32)
    x = values("bf16", 3, 2, 64)
    clean = r.rotate(x, ints([3, 4, 5]))
    x[1, 0, 7], x[2, 1, 40] = math.nan, math.inf
    y = r.rotate(x, ints([3, 4, 5]))
    same = torch.ones_like(x, dtype=torch.bool)
    same[1, 0, 7] = same[1, 0, 7 + 16] = same[2, 1, 40] = False
    assert torch.equal(y[same], clean[same]) and torch.isnan(y[1, 0, 7]) and torch.isnan(y[1, 0, 23]) and y[2, 1, 40] == math.inf


def test_no_tokens_and_streams_and_capture():
    r = lf.LFRotary(64, sections=[16, 8, 8])
    none = values("bf16", 0, 4, 64)
    assert r.rotate(none, ints([])).shape == (0, 4, 64)
    x, pos = values("bf16", 60, 4, 64), ints(np.random.default_rng(1).integers(0, 999, (3, 60)))
    want = r.rotate(x, pos)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    mine, at = x.clone(), pos.clone()
    torch.cuda.current_stream().synchronize()
    got = r.rotate(mine, at, stream=side)
    del mine, at
    junk = [torch.full_like(x, 7.0) for _ in range(4)] + [torch.full_like(pos, 1) for _ in range(4)]
    torch.cuda.synchronize()
    del junk
    assert torch.equal(got, want)
    y = torch.empty_like(x)
    with torch.cuda.graph(graph):
        r.rotate(x, pos, q_out=y)
    for i in range(3):
        pos.add_(1)
        graph.replay()
        assert torch.equal(y, r.rotate(x, pos))


def test_refusals():
    r = lf.LFRotary(64, sections=[16, 8, 8])
    x, pos = values("bf16", 6, 4, 64), ints(np.zeros((3, 6)))
    for args, kw, msg in [((x, pos.cpu()), {}, "positions"), ((x, pos.long()), {}, "positions"), ((x, pos[:2]), {}, "positions"),
                          ((x, pos[:, :5]), {}, "positions"), ((x, pos.t().contiguous().t()), {}, "positions"),
                          ((x[0], pos), {}, "q:"), ((x.half(), pos), {}, "q:"), ((x.cpu(), pos), {}, "q:"),
                          ((x.transpose(1, 2), pos), {}, "q:"), ((x, pos), dict(q_out=x[:5]), "q_out"),
                          ((x, pos), dict(k=x.float()), "k:"), ((x, pos), dict(k=x[:5]), "k:"),
                          ((x, pos), dict(k=torch.zeros(6, 4, 128, dtype=x.dtype, device="cuda")), "columns"),
                          ((values("f32", 6, 4, 272), pos), {}, "row_dim"),
                          ((x, pos), dict(k_out=x), "k_out without k"), ((x[:, :0], pos), {}, "heads"),
                          ((x[..., :48], pos), {}, "rotary_dim"), ((values("bf16", 6, 4, 72), pos), {}, "row_dim"),
                          ((values("bf16", 6, 4, 72)[..., 4:68], pos), {}, "aligned")]:
        with pytest.raises(lf.LFError, match=msg):
            r.rotate(*args, **kw)
    torch.cuda.synchronize()


# ---- on the way to a paged cache ------------------------------------------------------------------

def append_and_compare(p, r, freq, counts, pos=None, axis=None, q_heads=4, st=None, total=None, stored=None, adjacent=False,
                       stream=None):
    """The call's rows against the oracle; everything else in the pools keeps its bits.  -> error bits"""
    st = starts(counts) if st is None else st
    total = st[-1] if total is None else total
    stored = range(len(p.lens)) if stored is None else stored
    kn, vn, q = p.randn(total, p.kv_heads, p.d), p.randn(total, p.kv_heads, p.d), p.randn(total, q_heads, p.d)
    out = torch.full_like(q, 3.0)
    cache_pos, mine = np.zeros(total, int), np.zeros(total, bool)
    for b in stored:
        lo, hi = st[b], st[b + 1]
        cache_pos[lo:hi], mine[lo:hi] = np.arange(p.lens[b] - (hi - lo), p.lens[b]), True
    at = np.broadcast_to(cache_pos, (4, total)) if pos is None else np.asarray(pos)
    want_k, size_k = rotary_oracle.rotate(f64(kn), at, freq, axis, adjacent)
    want_q, size_q = rotary_oracle.rotate(f64(q), at, freq, axis, adjacent)
    bits = torch.int16 if p.kind == "bf16" else torch.int32
    before = [x.clone().view(bits) for x in (p.k, p.v)]
    got = p.cache.append_rotated(0, kn, vn, p.table, p.t_lens, r, new_start=ints(st), positions=None if pos is None else ints(pos),
                                 q=q, q_out=out, stream=stream)
    torch.cuda.synchronize()
    assert got is out
    where = []
    for b in stored:
        for i in range(st[b], st[b + 1]):
            where.append((i, p.np_table[b, cache_pos[i] // p.page], cache_pos[i] % p.page))
    i, x, s = (torch.tensor([w[j] for w in where], dtype=torch.long, device="cuda") for j in range(3))
    n = i.cpu().numpy()
    close(p.kind, f64(p.k[x, :, s]), want_k[n], size_k[n])
    assert torch.equal(p.v[x, :, s], vn[i])
    close(p.kind, f64(out)[mine], want_q[mine], size_q[mine])
    assert (out[torch.from_numpy(~mine).cuda()] == 3).all()
    for pool, old in zip((p.k, p.v), before):
        now = pool.clone().view(bits)
        now[x, :, s] = old[x, :, s]
        assert torch.equal(now, old)
    return p.cache.check()


@pytest.mark.parametrize("order", ["hnd", "nhd", "interleaved"])
@pytest.mark.parametrize("kind,d,page,rotary", [("bf16", 128, 16, 128), ("bf16", 64, 24, 32), ("bf16", 16, 5, 16), ("bf16", 32, 64, 32),
                                                ("f32", 128, 1, 64), ("f32", 16, 7, 16), ("f32", 64, 16, 64)])
def test_append(kind, d, page, rotary, order):
    freq = rotary_oracle.frequencies(rotary, 5e5)
    for adjacent in (False, True):
        r = lf.LFRotary(rotary, base=5e5, adjacent=adjacent)
        for counts, old in (([1], [0]), ([5, 0, 300, 1], [0, 17, 1000, 40]), ([1] * 70, [i * 13 % 90 for i in range(70)])):
            p = Paged(kind, 3, d, page, [a + b for a, b in zip(counts, old)], seed=d + page, order=order)
            assert append_and_compare(p, r, freq, counts, adjacent=adjacent) == 0
            for hq in (1, 12):
                assert append_and_compare(p, r, freq, counts, adjacent=adjacent, q_heads=hq) == 0


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("f32", 64)])
def test_append_with_positions_on_three_axes(kind, d):
    sections = [d // 8, d // 4 - d // 16, d // 2 - d // 8 - d // 4 + d // 16]
    r = lf.LFRotary(d, base=1e6, sections=sections)
    freq, axis = rotary_oracle.frequencies(d, 1e6), np.repeat([0, 1, 2], sections)
    counts = [200, 31, 1]
    p = Paged(kind, 2, d, 16, [260, 31, 900], seed=d)
    pos = position_set(np.random.default_rng(7), 3, sum(counts))
    assert append_and_compare(p, r, freq, counts, pos, axis) == 0
    assert append_and_compare(p, r, freq, counts, None, axis) == 0       # text: the cache's position on every axis
    one = np.broadcast_to(pos[0], (3, sum(counts)))
    kn = p.randn(sum(counts), 2, d)
    a = p.cache.append_rotated(0, kn, kn, p.table, p.t_lens, r, ints(starts(counts)), ints(one), q=kn)
    b = p.cache.append_rotated(0, kn, kn, p.table, p.t_lens, r, ints(starts(counts)), ints(pos[0]), q=kn)
    assert torch.equal(a, b)


def test_append_is_the_plain_one_at_position_zero():
    """At position 0 nothing turns: append_rotated stores the bits that append does; without q it returns none."""
    p = Paged("bf16", 2, 128, 16, [100, 9], seed=1)
    r = lf.LFRotary(128)
    kn, vn, st = p.randn(60, 2, 128), p.randn(60, 2, 128), ints([0, 51, 60])
    vn.view(torch.int16)[3, 1, 5] = 0x7fb1                       # a NaN keeps its bits
    p.cache.append(0, kn, vn, p.table, p.t_lens, st)
    k, v = p.k.clone(), p.v.clone()
    p.k.zero_(), p.v.zero_()
    assert p.cache.append_rotated(0, kn, vn, p.table, p.t_lens, r, st, ints(np.zeros(60))) is None
    mine = p.k != 0
    assert torch.equal(p.k[mine], k[mine]) and int(mine.sum()) > 60 * 2 * 127
    seen = p.v.view(torch.int16) != 0
    assert torch.equal(p.v.view(torch.int16)[seen], v.view(torch.int16)[seen]) and (p.v.view(torch.int16) == 0x7fb1).sum() == 1


@pytest.mark.parametrize("batch", [1, 31, 32, 33, 1000, 2500])
def test_append_finds_sequences(batch):
    """One warp's search over 1, 2 and 3 rounds, with empty sequences among them."""
    rng = np.random.default_rng(batch)
    counts = rng.integers(0, 4, batch)
    counts[-1] = 2
    r = lf.LFRotary(16)
    p = Paged("bf16", 1, 16, 4, (counts + rng.integers(0, 6, batch)).tolist(), seed=batch)
    assert append_and_compare(p, r, rotary_oracle.frequencies(16), counts.tolist(), q_heads=2) == 0


def test_append_row_starts():
    """As append: rows of no sequence are left, in q_out too; wrong starts are reported and nothing of the sequence stored."""
    p = Paged("bf16", 2, 128, 16, [200, 90, 150], seed=3)
    r, f = lf.LFRotary(128), rotary_oracle.frequencies(128)
    assert append_and_compare(p, r, f, None, st=[300, 500, 560, 700], total=760) == 0
    bad = lf.LF_DEVERR_STATE
    assert append_and_compare(p, r, f, None, st=[-50, 100, 160, 300], total=700, stored=[1, 2]) == bad
    assert append_and_compare(p, r, f, None, st=[0, 200, 260, 401], total=400, stored=[0, 1]) == bad
    assert append_and_compare(p, r, f, None, st=[0, 200, 260, 2**31 - 1], total=400, stored=[0, 1]) == bad
    kn = p.randn(250, 2, 128)
    p.cache.append_rotated(0, kn, kn, p.table, p.t_lens, r, ints([0, 150, 100, 250]))
    assert p.cache.check() == bad
    p = Paged("bf16", 1, 16, 4, [9] * 1000, seed=4)
    kn = p.randn(4, 1, 16)
    p.cache.append_rotated(0, kn, kn, p.table, p.t_lens, lf.LFRotary(16), ints([0] * 1000 + [5]))
    assert p.cache.check() == bad


def test_append_reports_bad_pages_and_lengths():
    p = Paged("f32", 2, 64, 16, [40, 20], seed=5)
    r, kn = lf.LFRotary(64), p.randn(2, 2, 64)
    keep = p.k.clone()
    for table, lens in ((ints([[-1] * p.width, [p.k.shape[0]] * p.width]), p.t_lens), (p.table, ints([0, -3])),
                        (p.table, ints([p.width * 16 + 1, 2**31 - 1]))):
        q = p.randn(2, 4, 64)
        p.cache.append_rotated(0, kn, kn, table, lens, r, q=q)
        assert p.cache.check() == lf.LF_DEVERR_STATE
        assert torch.equal(torch.nan_to_num(p.k, 7.0), torch.nan_to_num(keep, 7.0))


def test_append_in_place_on_a_stream_and_captured():
    p = Paged("bf16", 2, 128, 16, [700, 40], seed=6)
    r, st = lf.LFRotary(128, base=1e6), ints([0, 600, 630])
    kn, vn, q = p.randn(630, 2, 128), p.randn(630, 2, 128), p.randn(630, 8, 128)
    want = p.cache.append_rotated(0, kn, vn, p.table, p.t_lens, r, st, q=q)
    want_k = torch.nan_to_num(p.k.clone(), 7.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mine = [x.clone() for x in (kn, vn, p.table, p.t_lens, st, q)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = p.cache.append_rotated(0, mine[0], mine[1], mine[2], mine[3], r, mine[4], q=mine[5], stream=side.cuda_stream)
    del mine
    junk = [torch.full_like(x, 1) for x in (kn, vn, p.table, p.t_lens, st, q) for _ in range(3)]
    torch.cuda.synchronize()
    del junk
    assert torch.equal(got, want) and torch.equal(torch.nan_to_num(p.k, 7.0), want_k)
    y = q.clone()
    assert p.cache.append_rotated(0, kn, vn, p.table, p.t_lens, r, st, q=y, q_out=y) is y and torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = p.cache.append_rotated(0, kn, vn, p.table, p.t_lens, r, st, q=q)
    p.t_lens.sub_(3)                              # the graph follows the lengths
    graph.replay()
    assert torch.equal(a, p.cache.append_rotated(0, kn, vn, p.table, p.t_lens, r, st, q=q)) and not torch.equal(a, want)
    with pytest.raises(lf.LFError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            lf.LFRotary(64)
    assert p.cache.check() == 0


def test_append_refusals():
    p = Paged("bf16", 2, 128, 16, [70, 40], seed=7)
    r, st = lf.LFRotary(64), ints([0, 20, 30])
    kn, q = p.randn(30, 2, 128), p.randn(30, 8, 128)
    ok = dict(k_new=kn, v_new=kn, page_table=p.table, lens=p.t_lens, rotary=r, new_start=st, q=q)
    for kw, msg in [(dict(rotary=None), "rotary"), (dict(rotary=r._table), "rotary"), (dict(k_new=kn[:29]), "v_new"),
                    (dict(v_new=kn.float()), "v_new"), (dict(new_start=None), "k_new"), (dict(new_start=st[:2]), "new_start"),
                    (dict(q=q[:29]), "q:"), (dict(q=q.float()), "q:"), (dict(q_out=q[:, :4]), "q_out"), (dict(q=None, q_out=q), "without q"),
                    (dict(positions=st), "positions"), (dict(positions=ints(np.zeros((2, 30)))), "positions"),
                    (dict(positions=torch.zeros(30, device="cuda")), "positions"), (dict(rotary=lf.LFRotary(256)), "rotary_dim")]:
        with pytest.raises(lf.LFError, match=msg):
            p.cache.append_rotated(0, **{**ok, **kw})
    with pytest.raises(lf.LFError, match="layer"):
        p.cache.append_rotated(1, **ok)
    assert p.cache.check() == 0


def test_rotated_prompt_and_step_attend_by_relative_positions():
    """A prompt appended with rotation and attended, then a step: the fp64 oracle's attention over rotated rows."""
    d, hkv, hq, lens = 128, 2, 8, [150, 40]
    p = Paged("bf16", hkv, d, 16, [n + 1 for n in lens], seed=9)
    r, freq = lf.LFRotary(d, base=1e4), rotary_oracle.frequencies(d, 1e4)
    st = starts(lens)
    kn, vn, q = p.randn(st[-1], hkv, d, scale=1.0), p.randn(st[-1], hkv, d), p.randn(st[-1], hq, d, scale=1.0)
    t_lens = ints(lens)
    qr = p.cache.append_rotated(0, kn, vn, p.table, t_lens, r, ints(st), q=q)
    out = p.cache.prompt(0, qr, p.table, t_lens, ints(st), max(lens))
    k1, v1, q1 = p.randn(2, hkv, d, scale=1.0), p.randn(2, hkv, d), p.randn(2, hq, d, scale=1.0)
    t_lens.add_(1)
    qr1 = p.cache.append_rotated(0, k1, v1, p.table, t_lens, r, q=q1)
    step = p.cache.decode(0, qr1, p.table, t_lens)
    for b, n in enumerate(lens):
        pos = np.arange(n + 1)[None]
        raw = np.concatenate((f64(kn)[st[b]:st[b + 1]], f64(k1)[b:b + 1]))
        kk = rotary_oracle.rotate(raw, pos, freq)[0].swapaxes(0, 1)
        vv = np.concatenate((f64(vn)[st[b]:st[b + 1]], f64(v1)[b:b + 1])).swapaxes(0, 1)
        qq = rotary_oracle.rotate(np.concatenate((f64(q)[st[b]:st[b + 1]], f64(q1)[b:b + 1])), pos, freq)[0]
        want, _, size, dots = paged_oracle.attend(qq, kk, vv, paged_oracle.visible(np.arange(n + 1), n + 1, 0, 0))
        got = np.concatenate((f64(out)[st[b]:st[b + 1]], f64(step)[b:b + 1]))
        # rotated keys and queries are rounded to bf16: 2 x 2^-8 of every product of a logit, and as much of a weight
        rel = 2 * (2 * 2.0 ** -8) * dots + 2.0 ** -8
        assert (np.abs(got - want) <= (rel[..., None] + 2.0 ** -8) * size + 2.0 ** -8 * np.abs(want)).all()
    assert p.cache.check() == 0


# ---- small angles, and calls that could go wrong unseen ---------------------------------------------

def test_small_angles_keep_their_sines():
    """(x, 0) becomes (x cos w, x sin w): the sine of a small angle to its own size.  The angle is rounded by 2^-24 of itself
    and, its frequency being held in 2^-64 of a turn, off by 2^-65 x 2 pi / frequency of itself; sincospif by two units, at most
    2^-23 each, of the sine; the product by 2^-24 of it.  Opposite positions turn by opposite angles, and turning back is
    turning by the opposite position: the same bits."""
    freq = [1e-9, 1.1547e-6, 3e-5, 1e-3, -2e-8, 4.7e-5, 1e-12, 0.01]
    r = lf.LFRotary(16, inv_freq=freq)
    pos = np.array([1, 3, -1, -3, 17, -500])
    x = values("f32", len(pos), 1, 16)
    x[..., 8:] = 0
    y = r.rotate(x, ints(pos))
    f = np.array(freq)
    want = f64(x)[..., :8] * np.sin(pos[:, None, None] * f)
    rel = 2.0 ** -24 + 2.0 ** -65 * 2 * math.pi / np.abs(f) + 2 * 2.0 ** -23 + 2.0 ** -24 + 2.0 ** -40
    assert (np.abs(f64(y)[..., 8:] - want) <= rel * np.abs(want)).all()
    mirror = r.rotate(x, ints(-pos))
    assert torch.equal(mirror[..., :8], y[..., :8]) and torch.equal(mirror[..., 8:], -y[..., 8:])
    x = values("f32", 400, 2, 128, seed=1)
    r = lf.LFRotary(128, base=1e6)
    far = ints(position_set(np.random.default_rng(3), 400))
    far[4] = -2**31 + 1                    # (the least number has no opposite)
    assert torch.equal(r.rotate(x, far, inverse=True), r.rotate(x, -far))


def test_gradients_are_refused_where_they_are_recorded():
    """Refused where a gradient would be lost; under no_grad, and inside an autograd function, the call runs."""
    r = lf.LFRotary(64)
    x, pos = values("f32", 6, 4, 64).requires_grad_(), ints([5, 0, -7, 300, 1, 2])
    plain = x.detach().clone()
    for call in (lambda: r.rotate(x, pos), lambda: r.rotate(x * 2, pos), lambda: r.rotate(plain, pos, k=x),
                 lambda: r.rotate(plain, pos, q_out=x)):
        with pytest.raises(lf.LFError, match="gradient"):
            call()
    assert torch.equal(x, plain)
    p = Paged("f32", 4, 64, 16, [3, 3], seed=8)
    for kw in (dict(k_new=x), dict(v_new=x), dict(q=x), dict(q=plain, q_out=x)):
        with pytest.raises(lf.LFError, match="gradient"):
            p.cache.append_rotated(0, **{**dict(k_new=plain, v_new=plain, page_table=p.table, lens=p.t_lens, rotary=r,
                                                new_start=ints([0, 3, 6])), **kw})

    class Rotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, pos):
            ctx.save_for_backward(pos)
            return r.rotate(x, pos)

        @staticmethod
        def backward(ctx, g):
            return r.rotate(g, *ctx.saved_tensors, inverse=True), None

    g = values("f32", 6, 4, 64, seed=1)
    y = Rotate.apply(x, pos)
    y.backward(g)
    with torch.no_grad():
        assert torch.equal(y, r.rotate(x, pos)) and torch.equal(x.grad, r.rotate(g, pos, inverse=True))


def test_what_autograd_has_saved_is_not_overwritten_unseen():
    """Outputs that the caller gives count as changed in place, in every call that writes to them; new ones do not matter."""
    p = Paged("bf16", 2, 128, 16, [20, 9], seed=10)
    r, kn, q, pos = lf.LFRotary(128), p.randn(2, 2, 128), p.randn(2, 4, 128), ints([3, 4])
    lse = torch.zeros(2, 4, device="cuda")
    start, none = ints([0, 1, 2]), ints([0, 0])
    for call in (lambda o: r.rotate(q, pos, q_out=o), lambda o: r.rotate(o, pos, q_out=o), lambda o: r.rotate(kn, pos, k=o, k_out=o),
                 lambda o: p.cache.append_rotated(0, kn, kn, p.table, p.t_lens, r, q=q, q_out=o),
                 lambda o: p.cache.decode(0, q, p.table, p.t_lens, out=o, lse=lse),
                 lambda o: p.cache.decode_shared(0, q, p.table, p.t_lens, start, none, out=o, lse=lse),
                 lambda o: p.cache.prompt(0, q, p.table, p.t_lens, start, 1, out=o, lse=lse)):
        out, w, before = q.clone(), torch.ones((), device="cuda", dtype=q.dtype, requires_grad=True), lse._version
        y = (w * out).sum()
        call(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    assert lse._version == before + 1
    w, x = torch.ones((), device="cuda", dtype=q.dtype, requires_grad=True), q.clone()
    y = (w * x).sum()
    r.rotate(x, pos)
    y.backward()
    with torch.inference_mode():
        x = q.clone()
        assert r.rotate(x, pos, q_out=x) is x
    assert p.cache.check() == 0


def test_views_of_one_tensor_in_place_and_side_by_side():
    """Queries and keys of one wide projection, rotated in place and into the values' columns; outputs that overlap are refused."""
    r, pos = lf.LFRotary(64), ints(np.arange(50) * 7)
    wide = values("bf16", 50, 4 + 2 + 4 + 2, 64)
    q, k, q2, k2 = wide[:, :4], wide[:, 4:6], wide[:, 6:10], wide[:, 10:]
    want_q, want_k = r.rotate(q.contiguous(), pos, k=k.contiguous())
    r.rotate(q, pos, k=k, q_out=q2, k_out=k2)
    assert torch.equal(q2, want_q) and torch.equal(k2, want_k)
    r.rotate(q, pos, k=k, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    keep = wide.clone()
    one = torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda").expand(50, 4, 64)
    rolling = torch.empty(53 * 64, dtype=torch.bfloat16, device="cuda").as_strided((50, 4, 64), (64, 64, 1))
    for args, kw, msg in [((q, pos), dict(q_out=one), "rows of y overlap"), ((q, pos), dict(q_out=rolling), "rows of y overlap"),
                          ((q, pos), dict(q_out=wide[:, 1:5]), "q's x"), ((q[1:], pos[1:].contiguous()), dict(q_out=q[:-1]), "q's x"),
                          ((q, pos), dict(k=k, k_out=q[:, 1:3]), "q's x"), ((q, pos), dict(k=k, q_out=wide[:, 2:6], k_out=k), "q's x"),
                          ((q, pos), dict(k=k, q_out=q2, k_out=q2[:, :2]), "q's y"), ((q, pos), dict(k=k, q_out=wide[:, 5:9], k_out=k2), "k's x")]:
        with pytest.raises(lf.LFError, match=msg):
            r.rotate(*args, **kw)
    p = Paged("bf16", 2, 128, 16, [30, 9], seed=11)
    flat = p.randn(40, 4, 128)
    with pytest.raises(lf.LFError, match="q_out may be q"):
        p.cache.append_rotated(0, p.randn(30, 2, 128), p.randn(30, 2, 128), p.table, p.t_lens, lf.LFRotary(128), ints([0, 25, 30]),
                               q=flat[:30], q_out=flat[1:31])
    torch.cuda.synchronize()
    assert torch.equal(wide, keep)


@pytest.mark.parametrize("kind,d,hkv,hq,axes", [("bf16", 16, 1, 2, 1), ("bf16", 128, 2, 1, 3), ("f32", 64, 1, 4, 1), ("f32", 16, 2, 2, 4),
                                                ("f32", 128, 8, 32, 1)])
def test_append_of_so_many_tokens_that_a_warp_takes_several(kind, d, hkv, hq, axes):
    """Tokens of several sequences in one warp, empty ones between them, the last warp's not all there; fp32 prompts of 40
    heads, where a token is several steps."""
    rng = np.random.default_rng(d + axes)
    n = 30 if hq == 32 else 1400
    counts = rng.integers(0, 300 if hq == 32 else 17, n)
    counts[rng.integers(0, n, n // 5)] = 0
    counts[-1] = 3
    sections = SECTIONS[axes] and SECTIONS[axes](d // 2)
    axis = None if sections is None else np.repeat(np.arange(axes), sections)
    r = lf.LFRotary(d, base=1e5, sections=sections)
    p = Paged(kind, hkv, d, 16, (counts + rng.integers(0, 20, n)).tolist(), seed=d)
    pos = None if axes == 1 else position_set(rng, axes, int(counts.sum()))
    assert append_and_compare(p, r, rotary_oracle.frequencies(d, 1e5), counts.tolist(), pos, axis, q_heads=hq) == 0
    if axes == 1 and hq < 32:      # a sequence with wrong starts among a warp's tokens: reported, and nothing of it stored
        st = starts(counts.tolist())
        b = n // 2
        st[b] = st[b + 1] + 1
        kn, q = p.randn(st[-1], hkv, d), p.randn(st[-1], hq, d)
        out = torch.full_like(q, 3.0)
        p.cache.append_rotated(0, kn, kn, p.table, p.t_lens, r, ints(st), q=q, q_out=out)
        assert p.cache.check() == lf.LF_DEVERR_STATE


def test_rows_of_slabs_so_many_that_a_warp_takes_several():
    """Tokens of two sequences in one warp, the second's rows far from the first's; in place and back."""
    r = lf.LFRotary(32, sections=[4, 6, 6], adjacent=True)
    freq, axis = rotary_oracle.frequencies(32), np.repeat([0, 1, 2], [4, 6, 6])
    pos = position_set(np.random.default_rng(1), 3, 33, 301)
    for kind in ("bf16", "f32"):
        slab = values(kind, 33, 2, 301, 64, seed=3)
        before, x = f64(slab.transpose(1, 2)), slab.transpose(1, 2)
        want, size = rotary_oracle.rotate(before, pos, freq, axis, True)
        y = r.rotate(x, ints(pos))
        close(kind, f64(y), want, size)
        r.rotate(x, ints(pos), q_out=x)
        assert torch.equal(x, y)
