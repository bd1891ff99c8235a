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
