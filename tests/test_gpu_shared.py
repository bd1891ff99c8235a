"""Decoding behind shared prefixes on the GPU against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from decode_kv_cache_gb300 import longflow as lf
from shared_harness import Family

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def run(f, q_heads, fresh=False):
    """One call, checked: every row, the log-sum-exp, the same bits again."""
    batch = len(f.lens)
    q = f.randn(batch, q_heads, f.d)
    lse = torch.empty(batch, q_heads, dtype=torch.float32, device="cuda")
    kn = f.randn(batch, f.kv_heads, f.d) if fresh else None
    vn = f.randn(batch, f.kv_heads, f.d) if fresh else None
    out = f.decode(q, kn, vn, lse=lse)
    again_lse = torch.empty_like(lse)
    again = f.decode(q, kn, vn, lse=again_lse)
    assert f.cache.check() == 0
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    if fresh:
        f.write_new(kn, vn)
    worst = f.check(q, out, lse, fresh=fresh)
    return q, out, lse, worst


# One group; groups of one; sequences that share nothing, that share a part, that are all prefix, that are
# empty; a group's first that is shorter than its prefix, or empty; prefixes of one token and of whole pages.
SHAPES = [
    [[(100, 130), (100, 101), (100, 250)]],
    [[(0, 40)], [(33, 90), (0, 20), (32, 60), (1, 2), (33, 33)], [(7, 7)]],
    [[(64, 0), (64, 100), (10, 65), (64, 64)], [(300, 3), (300, 420), (128, 200)], [(0, 0), (0, 5)]],
    [[(500, 501 + i) for i in range(9)], [(1, 1 + i) for i in range(4)]],
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("kind,d,page", [("bf16", 128, 16), ("bf16", 64, 32), ("bf16", 32, 16), ("bf16", 16, 8), ("bf16", 128, 24),
                                         ("bf16", 64, 256), ("bf16", 128, 5), ("f32", 128, 16), ("f32", 64, 7), ("f32", 32, 64),
                                         ("f32", 16, 16)])
def test_against_the_oracle(kind, d, page, shape):
    for group, hkv, order in ((1, 2, "hnd"), (2, 1, "nhd"), (4, 2, "hnd"), (8, 1, "nhd")):
        f = Family(kind, hkv, d, page, SHAPES[shape], seed=d + page + group, order=order)
        run(f, hkv * group)


@pytest.mark.parametrize("kind,d,page", [("bf16", 128, 16), ("bf16", 64, 64), ("bf16", 32, 16), ("bf16", 128, 24), ("f32", 128, 16),
                                         ("f32", 64, 16)])
def test_with_new_tokens(kind, d, page):
    """The call's own tokens, written to their pages: right behind the prefix, in its last page, far behind it."""
    shape = [[(100, 101), (100, 130), (96, 97), (100, 100), (40, 41)], [(0, 1), (0, 77)], [(257, 300), (256, 257)], [(3, 1)]]
    for group, hkv in ((4, 2), (1, 3)):
        f = Family(kind, hkv, d, page, shape, seed=d + group)
        before_k, before_v = f.k.clone(), f.v.clone()
        batch = len(f.lens)
        q, kn, vn = f.randn(batch, hkv * group, d), f.randn(batch, hkv, d), f.randn(batch, hkv, d)
        for b, n in enumerate(f.lens):      # (the first of the last group has no page of its own behind its prefix's)
            x = int(f.np_table[b, (n - 1) // page])
            if x < 0:
                f.np_table[b, (n - 1) // page] = x = f.k.shape[0] - 1
                f.table[b, (n - 1) // page] = x
            before_k[x, :, (n - 1) % page], before_v[x, :, (n - 1) % page] = kn[b], vn[b]
        out = f.decode(q, kn, vn)
        assert f.cache.check() == 0
        f.write_new(kn, vn)
        for pool, want in ((f.k, before_k), (f.v, before_v)):
            assert torch.equal(torch.nan_to_num(pool, 77.0), torch.nan_to_num(want, 77.0))
        f.check(q, out, fresh=True)


@pytest.mark.parametrize("kind,d,page,group,members,prefix", [
    ("bf16", 128, 16, 4, 64, 3000), ("bf16", 128, 16, 4, 65, 500), ("bf16", 128, 64, 8, 100, 1000), ("bf16", 128, 128, 1, 300, 2000),
    ("bf16", 64, 16, 2, 130, 1500), ("bf16", 32, 16, 8, 40, 700), ("bf16", 128, 24, 4, 33, 900), ("f32", 64, 16, 1, 50, 1000),
    ("f32", 128, 16, 8, 20, 600), ("f32", 16, 16, 2, 70, 400), ("bf16", 128, 16, 2, 3, 40000), ("f32", 128, 32, 1, 2, 9000)])
def test_more_rows_and_longer_prefixes(kind, d, page, group, members, prefix):
    """More rows than a block takes, and prefixes that many blocks share."""
    rng = np.random.default_rng(members)
    f = Family(kind, 1, d, page, [[(prefix, prefix + int(t)) for t in rng.integers(0, 90, members)]], seed=members)
    q = f.randn(members, group, d)
    lse = torch.empty(members, group, dtype=torch.float32, device="cuda")
    out = f.decode(q, lse=lse)
    assert f.cache.check() == 0
    f.check(q, out, lse, which=sorted({0, 1, members // 2, members - 2, members - 1}))
    plain_table = f.table.clone()       # and all of them against lf_paged_decode on whole rows
    whole = prefix // page
    plain_table[:, :whole] = f.table[0, :whole]
    if prefix % page:
        for b in range(1, members):
            x = int(f.np_table[b, whole])
            if x >= 0:
                for pool in (f.k, f.v):
                    pool[x, :, :prefix % page] = pool[int(f.np_table[0, whole]), :, :prefix % page]
            else:
                plain_table[b, whole] = f.table[0, whole]
    ref = f.cache.decode(0, q, plain_table, f.t_lens)
    assert f.cache.check() == 0
    step = 2.0 ** -7 if kind == "bf16" else 2.0 ** -18
    assert ((out.float() - ref.float()).abs() <= step * (ref.float().abs() + 1)).all()


@pytest.mark.parametrize("kind,d,groups", [("bf16", 128, 50), ("bf16", 128, 700), ("bf16", 32, 300), ("f32", 64, 260), ("f32", 128, 40)])
def test_many_groups(kind, d, groups):
    """More units than blocks that run at once, and more groups than a block has threads."""
    rng = np.random.default_rng(groups)
    shape = []
    for i in range(groups):
        p = int(rng.integers(0, 400)) if i % 5 else int(rng.integers(0, 3))
        shape.append([(p, p + int(rng.integers(0, 40)))] + [(int(q), int(q + rng.integers(0, 30)))
                                                           for q in rng.integers(0, p + 1, int(rng.integers(0, 3)))])
    f = Family(kind, 2, d, 16, shape, seed=groups)
    batch = len(f.lens)
    q = f.randn(batch, 8, d)
    out = f.decode(q)
    assert f.cache.check() == 0
    f.check(q, out, which=range(0, batch, max(1, batch // 40)))


def test_a_wide_table_and_one_head():
    f = Family("bf16", 1, 128, 16, [[(100, 140), (100, 120)]], seed=3, width=20000)
    run(f, 1)


@pytest.mark.parametrize("kind,d,page", [("bf16", 128, 16), ("bf16", 64, 128), ("bf16", 32, 16), ("bf16", 128, 24), ("f32", 64, 16),
                                         ("f32", 128, 16)])
def test_what_a_shorter_prefix_does_not_see(kind, d, page):
    """NaN and infinities in the leader's positions behind a member's prefix reach the members that see them, no other."""
    shape = [[(400, 410), (150, 180), (399, 400), (0, 30), (151, 200)]]
    f = Family(kind, 2, d, page, shape, seed=5)
    q = f.randn(5, 8, d)
    f.check(q, f.decode(q))
    for pool, what, pos in ((f.v, math.nan, 200), (f.k, math.inf, 350), (f.v, -math.inf, 399)):
        pool[int(f.np_table[0, pos // page]), 1, pos % page, 3] = what
    lse = torch.empty(5, 8, dtype=torch.float32, device="cuda")
    out = f.decode(q, lse=lse)
    f.check(q, out, lse, which=[1, 3, 4])
    assert torch.isfinite(out[:, :4]).all() and not torch.isfinite(out[[0, 2], 4:]).all()
    assert f.cache.check() in (0, lf.LF_DEVERR_NONFINITE)


def test_weights_are_the_decodes_where_nothing_is_shared():
    """prefix_lens of zero: lf_paged_decode's own arithmetic, up to where its ranges are cut."""
    f = Family("bf16", 2, 128, 16, [[(0, 900), (0, 31)], [(0, 1), (0, 0)]], seed=6)
    q = f.randn(4, 8, 128)
    a, b = f.decode(q), f.cache.decode(0, q, f.table, f.t_lens)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -8 * b.float().abs().max()
    f.check(q, a)


def test_large_logits_keep_their_weights():
    """Logits of thousands: shares are joined by maxima, not by log-sum-exps rounded at the logits' size."""
    f = Family("f32", 1, 64, 16, [[(700, 800), (700, 701), (200, 333)]], seed=7, scale=40.0)
    run(f, 4)


def test_padded_batches():
    """Rows without a sequence, their prefixes left from another step; one group of them alone."""
    f = Family("bf16", 2, 128, 16, [[(200, 250), (200, 201)], [(64, 0), (64, 0)], [(90, 0)]], seed=8)
    q, _, lse, _ = run(f, 8)
    assert (f.decode(q)[2:] == 0).all() and torch.isneginf(lse[2:]).all()


# ---- what is reported -----------------------------------------------------------------------------

def test_wrong_groups_are_reported_and_others_computed():
    f = Family("bf16", 2, 128, 16, [[(100, 130), (100, 120)], [(50, 60), (50, 70)], [(0, 40)]], seed=9)
    q = f.randn(5, 8, 128)
    def call(start, prefix=None):
        out = torch.full_like(q, 3.0)
        f.cache.decode_shared(0, q, f.table, f.t_lens, ints(start), f.t_prefix if prefix is None else ints(prefix), out=out)
        return out, f.cache.check()
    bad = lf.LF_DEVERR_STATE
    out, bits = call([0, 2, 4])                       # sequence 4 is in no group
    assert bits == bad and (out[4] == 3).all()
    f.check(q, out, which=[0, 1, 2, 3])
    out, bits = call([2, 4, 5])                       # 0 and 1 are in none
    assert bits == bad and (out[:2] == 3).all()
    f.check(q, out, which=[2, 3, 4])
    for start in ([0, 2, 6], [0, 2, 2**31 - 1]):      # a group that ends behind the batch
        out, bits = call(start)
        assert bits == bad and (out[2:] == 3).all()
        f.check(q, out, which=[0, 1])
    out, bits = call([-3, 2, 5])
    assert bits == bad and (out[:2] == 3).all()
    call_bits = call([0, 4, 2, 5])[1]                 # starts that decrease
    assert call_bits == bad
    out, bits = call([0, 2, 4, 5], [100, 101, 50, 50, 0])   # longer than its group's first
    assert bits == bad and (out[1] == 3).all()
    f.check(q, out, which=[0, 2, 3, 4])
    out, bits = call([0, 2, 4, 5])
    assert bits == 0
    f.check(q, out)


def test_negative_prefixes_count_as_none_and_long_ones_as_the_length():
    f = Family("f32", 1, 64, 16, [[(300, 40), (300, 290), (300, 300)], [(-5, 20), (-2**31, 7)]], seed=10)
    run(f, 2)


def test_bad_pages_and_lengths_are_reported():
    f = Family("bf16", 2, 128, 16, [[(100, 130), (100, 120)], [(0, 60)]], seed=11)
    q = f.randn(3, 8, 128)
    for b, i in ((0, 2), (1, 7), (2, 0)):
        for x in (-1, f.k.shape[0], 2**31 - 1):
            t = f.table.clone()
            t[b, i] = x
            out = f.cache.decode_shared(0, q, t, f.t_lens, f.t_start, f.t_prefix)
            assert f.cache.check() == lf.LF_DEVERR_STATE
            f.check(q, out, which=[2] if b < 2 else [0, 1])
    for n in (-1, f.width * 16 + 1, 2**31 - 1):
        out = f.cache.decode_shared(0, q, f.table, ints([130, 120, n]), f.t_start, f.t_prefix)
        assert f.cache.check() & lf.LF_DEVERR_STATE     # (a length behind the tokens reads the NaN there, too)
        f.check(q, out, which=[0, 1])
    bad = q.clone()
    bad[1, 3, 5] = math.nan
    out = f.cache.decode_shared(0, bad, f.table, f.t_lens, f.t_start, f.t_prefix)
    assert f.cache.check() == lf.LF_DEVERR_NONFINITE
    f.check(q, out, which=[0, 2])


def test_refusals():
    f = Family("bf16", 2, 128, 16, [[(100, 130), (100, 120)], [(0, 60)]], seed=12)
    q = f.randn(3, 8, 128)
    ok = dict(q=q, page_table=f.table, lens=f.t_lens, group_start=f.t_start, prefix_lens=f.t_prefix)
    kn = f.randn(3, 2, 128)
    for kw, msg in [(dict(q=q[:2]), "q:"), (dict(q=q.float()), "q:"), (dict(group_start=f.t_start[:1]), "groups"),
                    (dict(group_start=ints([0] * 6)), "groups"), (dict(group_start=f.t_start.long()), "group_start"),
                    (dict(group_start=f.t_start.cpu()), "group_start"), (dict(prefix_lens=f.t_prefix[:2]), "prefix_lens"),
                    (dict(prefix_lens=f.t_prefix.float()), "prefix_lens"), (dict(k_new=kn), "v_new"), (dict(k_new=kn[:2], v_new=kn), "k_new"),
                    (dict(out=q[:, :4]), "out"), (dict(lse=q), "lse"), (dict(q=q[:, :6].contiguous()), "group size 3")]:
        with pytest.raises(lf.LFError, match=msg):
            f.cache.decode_shared(0, **{**ok, **kw})
    p, need = f.cache._pages[0], lf.lf_paged_decode_shared_workspace(f.cache._pages[0], 3, f.width, 8, 2)
    ws, out = torch.empty(need + 16, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    args = (p, 3, f.table, f.width, f.t_lens, 8, q, f.t_start, 2, f.t_prefix, None, None, out, None)
    for w, n in ((ws, need - 1), (None, need), (ws[8:], need)):
        with pytest.raises(lf.LFError, match="workspace"):
            lf.lf_paged_decode_shared(*args, w, n)
    wide = lf.LFPages.from_buffer_copy(p)
    wide.page_size = 2**30
    with pytest.raises(lf.LFError, match="too large for one call"):
        lf.lf_paged_decode_shared_workspace(wide, 4096, 1, 8, 4096)
    lf.lf_paged_decode_shared(*args, ws, need)
    assert torch.equal(out, f.decode(q)) and f.cache.check() == 0


# ---- streams, graphs, company -----------------------------------------------------------------------

def test_a_captured_call_follows_its_inputs():
    f = Family("bf16", 2, 128, 16, [[(300, 350), (300, 310), (120, 330)], [(0, 50), (0, 20)]], seed=13)
    q, kn, vn = f.randn(5, 8, 128), f.randn(5, 2, 128), f.randn(5, 2, 128)
    f.decode(q, kn, vn)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f.decode(q, kn, vn)
        two = f.decode(q)                     # (a second call of the graph: workspaces of their own)
    for start, prefix, lens in (([0, 3, 5], [300, 300, 120, 0, 0], [350, 310, 330, 50, 20]),
                                ([0, 3, 5], [300, 300, 120, 0, 0], [349, 301, 300, 1, 0]),
                                ([0, 1, 5], [0, 0, 0, 0, 0], [340, 0, 0, 50, 20]),
                                ([0, 3, 5], [16, 15, 1, 0, 0], [17, 0, 0, 20, 20])):
        f.t_start.copy_(ints(start)), f.t_prefix.copy_(ints(prefix)), f.t_lens.copy_(ints(lens))
        q.copy_(f.randn(5, 8, 128))
        k = f.k.clone(), f.v.clone()
        out.zero_(), two.zero_()
        graph.replay()
        got = out.clone(), two.clone()
        f.k.copy_(k[0]), f.v.copy_(k[1])
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
        assert torch.equal(got[0], f.decode(q, kn, vn)) and torch.equal(got[1], f.decode(q))
    assert f.cache.check() == 0


def test_other_streams():
    """A call on a stream of the caller's, whose tensors are let go at once; two streams side by side; the error word's
    stream."""
    f = Family("bf16", 8, 128, 16, [[(2000, 2100)] * 6, [(600, 700)] * 5], seed=14)
    q = f.randn(11, 32, 128)
    want = f.decode(q)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        mine = [x.clone() for x in (q, f.table, f.t_lens, f.t_start, f.t_prefix)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        got = f.cache.decode_shared(0, *mine, stream=s)
        shapes = [(x.shape, x.dtype) for x in mine]
        del mine
        junk = [torch.full(shape, 1, dtype=t, device="cuda") for shape, t in shapes for _ in range(3)]
        torch.cuda.synchronize()
        del junk
        assert torch.equal(got, want)
    outs = []
    for i in range(20):
        outs.append(f.decode(q, stream=side))
        outs.append(f.decode(q, stream=other))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)
    assert f.cache.check(side) == 0


def test_calls_in_a_row_do_not_meet():
    """Each launch of a call starts while the one before it drains: calls with other inputs right behind one another, the
    appends of one the keys of the next."""
    f = Family("bf16", 2, 128, 16, [[(1000, 1001 + i) for i in range(8)]], seed=15, width=80)
    steps, batch = 12, 8
    spare = f.k.shape[0]
    for b in range(batch):                # room for the steps' tokens: pages behind the pool's own
        for i in range(f.width):
            if f.np_table[b, i] < 0 and i * 16 >= 1000:
                f.np_table[b, i] = spare
                spare += 1
    pools = [torch.cat((x, torch.full((spare - x.shape[0], *x.shape[1:]), math.nan, dtype=x.dtype, device="cuda"))) for x in (f.k, f.v)]
    f.k, f.v = pools
    f.cache = lf.LFPagedCache.over(f.k[None], f.v[None])
    f.table = torch.from_numpy(f.np_table).cuda()
    qs, ks, vs = f.randn(steps, batch, 8, 128), f.randn(steps, batch, 2, 128), f.randn(steps, batch, 2, 128)
    lens = [ints([n + 1 + s for n in f.lens]) for s in range(steps)]
    torch.cuda.synchronize()
    outs = [f.cache.decode_shared(0, qs[s], f.table, lens[s], f.t_start, f.t_prefix, ks[s], vs[s]) for s in range(steps)]
    assert f.cache.check() == 0
    for s in range(steps):
        f.lens = [n + 1 for n in f.lens]
        f.own = [tuple(torch.cat((x, new[s, b][:, None]), 1) if x.shape[1] < f.lens[b] else x for x, new in zip(f.own[b], (ks, vs)))
                 for b in range(batch)]
        f.check(qs[s], outs[s], which=[0, 3, 7], fresh=True)


def test_pages_behind_four_gigabytes():
    """Offsets of pages and rows past 32 bits."""
    n = 150000
    k = torch.empty(1, n, 8, 16, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    f = Family("bf16", 8, 128, 16, [[(200, 210), (200, 230)]], seed=16)
    table = np.where(f.np_table >= 0, n - 1 - f.np_table, -7).astype(np.int32)
    for x in range(f.k.shape[0]):
        k[0, n - 1 - x], v[0, n - 1 - x] = f.k[x], f.v[x]
    cache = lf.LFPagedCache.over(k, v)
    q = f.randn(2, 32, 128)
    assert torch.equal(cache.decode_shared(0, q, ints(table), f.t_lens, f.t_start, f.t_prefix), f.decode(q))
    assert cache.check() == 0


def test_rotated_steps_behind_a_shared_prompt():
    """A run as a server makes it: a prompt is appended with rotation once, its pages are listed by every answer's row, each
    step appends with rotation and decodes behind the prompt: as attention over each whole sequence."""
    d, hkv, hq, n, answers, steps, page = 128, 2, 8, 100, 5, 6, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    cache = lf.LFPagedCache(1, 40, page, hkv, d)
    cache.k.fill_(math.nan), cache.v.fill_(math.nan)
    r = lf.LFRotary(d, base=1e6)
    prompt = ints([[0, 1, 2, 3, 4, 5, 6]])
    k0, v0, q0 = randn(n, hkv, d), randn(n, hkv, d), randn(n, hq, d)
    cache.append_rotated(0, k0, v0, prompt, ints([n]), r, ints([0, n]), q=q0)
    table = np.full((answers, 8), -1, dtype=np.int32)
    table[0, :7] = range(7)               # the first answer owns the prompt's last page
    table[:, 7] = [10 + b for b in range(answers)]
    for b in range(1, answers):
        table[b, 6] = 20 + b              # the others' places behind the prompt
    table = ints(table)
    lens = ints([n] * answers)
    keys = [[] for _ in range(answers)]
    for s in range(steps):
        lens.add_(1)
        k, v, q = randn(answers, hkv, d), randn(answers, hkv, d), randn(answers, hq, d)
        qr = cache.append_rotated(0, k, v, table, lens, r, q=q)
        out = cache.decode_shared(0, qr, table, lens, ints([0, answers]), ints([n] * answers))
        pos = torch.arange(n + steps, dtype=torch.int32, device="cuda")
        for b in range(answers):
            keys[b].append((k[b], v[b]))
            kk = torch.cat((k0, torch.stack([x for x, _ in keys[b]])))
            vv = torch.cat((v0, torch.stack([x for _, x in keys[b]]))).double()
            kk = r.rotate(kk, pos[:n + s + 1]).double()
            z = torch.einsum("ghd,ngd->ghn", qr[b].view(hkv, hq // hkv, d).double(), kk) / math.sqrt(d)
            want = torch.einsum("ghn,ngd->ghd", torch.softmax(z, -1), vv).reshape(hq, d)
            size = torch.einsum("ghn,ngd->ghd", torch.softmax(z, -1), vv.abs()).reshape(hq, d)
            assert ((out[b].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -13) * size + 2.0 ** -8 * want.abs()).all()
    assert cache.check() == 0


# ---- found by looking for what the tests above do not reach ----------------------------------------

@pytest.mark.parametrize("kind,d,page,group", [("bf16", 128, 16, 4), ("bf16", 64, 32, 8), ("bf16", 128, 24, 2), ("f32", 64, 16, 1)])
def test_branches_in_all_rows_of_a_block(kind, d, page, group):
    """Members that leave the prefix everywhere, in both query tiles and in several pieces, behind groups of other lengths, so
    that ranges end inside units; with new tokens."""
    rng = np.random.default_rng(page)
    shape = [[(700, 720)] + [(int(p), int(p) + 1 + int(t)) for p, t in zip(rng.integers(0, 701, 99), rng.integers(0, 60, 99))],
             [(2000, 2001)] + [(int(p), int(p) + 1 + int(t)) for p, t in zip(rng.integers(1900, 2001, 9), rng.integers(0, 300, 9))],
             [(130, 150)] * 3, [(0, 1500)], [(5, 6), (5, 700)]]
    f = Family(kind, 2, d, page, shape, seed=group)
    batch = len(f.lens)
    q, kn, vn = f.randn(batch, 2 * group, d), f.randn(batch, 2, d), f.randn(batch, 2, d)
    lse = torch.empty(batch, 2 * group, dtype=torch.float32, device="cuda")
    out = f.decode(q, kn, vn, lse=lse)
    again = f.decode(q, kn, vn)
    assert torch.equal(out, again) and f.cache.check() == 0
    f.write_new(kn, vn)
    f.check(q, out, lse, which=list(range(0, batch, 7)) + [99, 100, 109, 110, 113, batch - 2, batch - 1], fresh=True)


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 32), ("f32", 64)])
def test_prefixes_behind_every_length(kind, d):
    """The largest number there is as a prefix: every sequence is all prefix, whatever the table holds behind it."""
    f = Family(kind, 2, d, 16, [[(333, 333), (333, 200), (333, 0), (333, 1)], [(64, 64)]], seed=17)
    q = f.randn(5, 8, d)
    want = f.decode(q)
    f.check(q, want)
    top = ints([2**31 - 1] * 5)
    out = f.cache.decode_shared(0, q, f.table, f.t_lens, f.t_start, top)
    assert f.cache.check() == 0
    f.check(q, out)


@pytest.mark.parametrize("kind,d,batch", [("bf16", 64, 3000), ("f32", 16, 2000)])
def test_large_batches(kind, d, batch):
    """More sequences and groups than a block has threads, one KV head, a page for each."""
    rng = np.random.default_rng(batch)
    shape = [[(int(p), int(p) + int(t)) for t in rng.integers(0, 9, int(rng.integers(1, 4)))]
             for p in rng.integers(0, 20, batch // 2)]
    f = Family(kind, 1, d, 16, shape, seed=batch)
    q = f.randn(len(f.lens), 2, d)
    out = f.decode(q)
    assert f.cache.check() == 0
    f.check(q, out, which=range(0, len(f.lens), 61))


def test_layers_and_strides():
    """Another layer's pools, K and V of a token side by side."""
    f = Family("bf16", 2, 128, 16, [[(100, 130), (100, 120)]], seed=18)
    pages = f.k.shape[0]
    both = torch.full((2, pages, 2, 16, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    both[1, :, :, :, 0], both[1, :, :, :, 1] = f.k, f.v
    cache = lf.LFPagedCache.over(both[:, :, :, :, 0], both[:, :, :, :, 1])
    q = f.randn(2, 8, 128)
    assert torch.equal(cache.decode_shared(1, q, f.table, f.t_lens, f.t_start, f.t_prefix), f.decode(q))
    assert cache.check() == 0


def test_neighbours_of_the_call_keep_their_bits():
    """What lies around out and lse is not written."""
    f = Family("bf16", 2, 128, 16, [[(100, 130), (100, 120), (40, 0)]], seed=19)
    q = f.randn(3, 8, 128)
    wide, flat = torch.full((5, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((5, 8), 3.0, device="cuda")
    f.decode(q, out=wide[1:4], lse=flat[1:4])
    assert (wide[[0, 4]] == 3).all() and (flat[[0, 4]] == 3).all()
    f.check(q, wide[1:4], flat[1:4])


# ---- prefixes that no sequence sees to their end ----------------------------------------------------

@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("kind,d,page", [("bf16", 128, 16), ("bf16", 64, 32), ("bf16", 32, 16), ("bf16", 128, 24), ("f32", 64, 16),
                                         ("f32", 128, 16)])
def test_prefixes_left_from_another_step_change_nothing(kind, d, page, fresh):
    """Prefixes of padded rows, and prefixes above the lengths, under a wide table: work is laid out by what is seen, so that
    every row has the bits that it has with prefixes of just that."""
    shape = [[(500, 520), (500, 505), (300, 420)], [(333, 333), (200, 200)], [(0, 0)], [(0, 0), (0, 0)], [(0, 40)]] + [[(0, 0)]] * 9
    f = Family(kind, 2, d, page, shape, seed=d, width=131072 // page)
    batch = len(f.lens)
    q = f.randn(batch, 8, d)
    kn, vn = (f.randn(batch, 2, d), f.randn(batch, 2, d)) if fresh else (None, None)
    top, lse = 2**31 - 1, torch.empty(batch, 8, device="cuda")
    want = f.decode(q, kn, vn, lse=lse)
    assert f.cache.check() == 0
    for stale in ([500, 500, 300, top, top, 60000, 60000, 100, 0] + [60000] * 9,
                  [500, 500, 300, 333, 200, top, top, top, 0] + [top, 1, 131072] * 3,
                  [500, 500, 300, 100000, 400, 0, 1, 1, 0] + [0] * 8 + [120000]):
        other = torch.empty_like(lse)
        got = f.cache.decode_shared(0, q, f.table, f.t_lens, f.t_start, ints(stale), kn, vn, lse=other)
        assert f.cache.check() == 0
        assert torch.equal(got, want) and torch.equal(other, lse), stale
    if not fresh:
        f.check(q, want, lse)


@pytest.mark.parametrize("kind,d,groups", [("bf16", 64, 2500), ("bf16", 128, 4200), ("bf16", 32, 1100), ("f32", 16, 600)])
def test_more_groups_than_a_block_looks_at_together(kind, d, groups):
    """Groups in several tables, their ends in the middle of a group of many; empty groups and rows without a sequence."""
    rng = np.random.default_rng(groups)
    shape = []
    for i in range(groups):
        p = int(rng.integers(1, 60))
        n = 300 if i == groups // 2 else int(rng.integers(1, 3))
        shape.append([(p, p + int(t)) if rng.random() < 0.9 else (p, 0) for t in rng.integers(0, 9, n)])
    f = Family(kind, 1, d, 16, shape, seed=groups)
    batch = len(f.lens)
    q = f.randn(batch, 2, d)
    out = f.decode(q)
    assert f.cache.check() == 0
    f.check(q, out, which=list(range(0, batch, 97)) + [batch - 1])
    empty = np.sort(np.concatenate((f.start, rng.choice(f.start, min(batch - groups, 200)))))   # some groups of none
    assert torch.equal(f.cache.decode_shared(0, q, f.table, f.t_lens, ints(empty), f.t_prefix), out)
    graph = torch.cuda.CUDAGraph()              # captured, it follows its inputs: the launch that looks at the groups too
    with torch.cuda.graph(graph):
        got = f.decode(q)
    graph.replay()
    assert torch.equal(got, out)
    f.t_prefix.copy_(torch.where(f.t_lens > 0, f.t_prefix, 2**31 - 1))
    f.t_prefix[f.t_start[:-1].long()] = 2**31 - 1
    graph.replay()
    assert torch.equal(got, f.decode(q)) and f.cache.check() == 0


@pytest.mark.parametrize("d,members", [(16, 2), (32, 2), (64, 2), (128, 2), (128, 70), (128, 300)])
def test_products_of_a_prefix_are_summed_in_short_chains(d, members):
    """fp32: the log-sum-exp of a prefix of one key is its logit.  One large product first, all others just below half a unit of
    its last place: each is lost where it is added alone.  Products are added in twos to two sums, d / 4 roundings each at
    the sum's size, 2^-24 of it, with one of the twos; then the two sums' own, the scale, the product with it, and ln 2 and
    the product with that."""
    f = Family("f32", 1, d, 16, [[(1, 1)] * members], seed=d)
    for small in (0.49, 0.245, 0.3, -0.24):
        q, k = torch.ones(members, 1, d, device="cuda"), torch.full((d,), small * 2.0 ** -23, device="cuda")
        k[0] = 1.0
        f.k[int(f.np_table[0, 0]), 0, 0] = k
        lse = torch.empty(members, 1, device="cuda")
        f.decode(q, lse=lse)
        want = float(k.double().sum()) / math.sqrt(d)
        size = float(k.double().abs().sum()) / math.sqrt(d)
        assert abs(lse.double() - want).max() <= (d / 4 + 1 + 1 + 4) * 2.0 ** -24 * size, small
    assert f.cache.check() == 0


@pytest.mark.parametrize("kind,d,page_size", [("bf16", 128, 16), ("bf16", 64, 2**30), ("bf16", 128, 24), ("bf16", 16, 16), ("f32", 64, 128)])
def test_no_call_below_the_header_s_limit_is_refused(kind, d, page_size):
    """batch * kv_heads * (max_pages * page_size / 128 + 9) below 2^31, at any number of groups; what the tensor cores' kernel
    would have to count past 32 bits for is refused."""
    f = Family(kind, 1, d, 16, [[(0, 1)]])
    p = lf.LFPages.from_buffer_copy(f.cache._pages[0])
    p.page_size = page_size
    for tokens in (page_size, 2**20 // page_size * page_size, 2**28 // page_size * page_size, (2**31 - 257) // page_size * page_size):
        if tokens == 0:
            continue
        for kv_heads in (1, 8, 64):
            p.kv_heads = kv_heads
            batch = min(65535, (2**31 - 1) * 128 // (kv_heads * (tokens + 9 * 128)))
            assert batch * kv_heads * (tokens + 9 * 128) < 2**31 * 128
            for groups in {1, max(1, batch // 3), batch} if batch else ():
                assert lf.lf_paged_decode_shared_workspace(p, batch, tokens // page_size, kv_heads, groups) > 0
    if kind == "bf16" and d >= 64 and page_size != 24:
        p.kv_heads = 64
        with pytest.raises(lf.LFError, match="too large for one call"):
            lf.lf_paged_decode_shared_workspace(p, 65535, (2**31 - 257) // page_size, 64, 65535)


@pytest.mark.parametrize("group,members,prefix", [(8, 32, 700), (8, 33, 130), (4, 100, 64), (1, 256, 1000), (2, 129, 63)])
def test_fp32_groups_of_many_rows(group, members, prefix):
    """Heads of 128, 256 rows and more of a KV head, where blocks take 64 rows; some leave the prefix early."""
    rng = np.random.default_rng(members)
    shape = [[(prefix, prefix + 20)] + [(int(p), int(p) + 1 + int(t)) for p, t in
                                        zip(rng.integers(0, prefix + 1, members - 1), rng.integers(0, 40, members - 1))]]
    f = Family("f32", 2, 128, 16, shape, seed=members)
    q, kn, vn = f.randn(members, 2 * group, 128), f.randn(members, 2, 128), f.randn(members, 2, 128)
    lse = torch.empty(members, 2 * group, device="cuda")
    out = f.decode(q, kn, vn, lse=lse)
    assert torch.equal(out, f.decode(q, kn, vn)) and f.cache.check() == 0
    f.write_new(kn, vn)
    f.check(q, out, lse, which=list(range(0, members, 13)) + [members - 1], fresh=True)


@pytest.mark.parametrize("kind,d,page,hkv,group,members,prefix", [("bf16", 64, 16, 8, 8, 64, 8192), ("bf16", 64, 64, 4, 4, 150, 4000),
                                                                  ("bf16", 32, 16, 8, 4, 64, 3000), ("bf16", 128, 24, 8, 4, 32, 4000),
                                                                  ("f32", 64, 16, 8, 1, 64, 3000)])
def test_sizes_that_keep_every_block_busy(kind, d, page, hkv, group, members, prefix):
    """Heads of 64 on the tensor cores, and the other kernels, with all blocks at work on several tiles each."""
    rng = np.random.default_rng(members)
    f = Family(kind, hkv, d, page, [[(prefix, prefix + int(t)) for t in rng.integers(1, 400, members)]], seed=members)
    q, kn, vn = f.randn(members, hkv * group, d), f.randn(members, hkv, d), f.randn(members, hkv, d)
    lse = torch.empty(members, hkv * group, device="cuda")
    out = f.decode(q, kn, vn, lse=lse)
    assert torch.equal(out, f.decode(q, kn, vn)) and f.cache.check() == 0
    f.write_new(kn, vn)
    f.check(q, out, lse, which=[0, members // 2, members - 1], fresh=True)
