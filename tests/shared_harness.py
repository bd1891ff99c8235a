"""Inputs for the tests of decoding behind shared prefixes (GPU side; the expected values are the fp64 oracle's)."""
import math

import numpy as np
import torch

from decode_kv_cache_gb300 import longflow as lf
from oracle import paged_oracle
from paged_harness import TYPES, bounds


class Family:
    """Groups of sequences: groups is a list of lists of (prefix, length).  A group's first sequence has the pages of the
    longest prefix, whatever its own length.  What no sequence may read is NaN, or an entry that is no page: a member's
    entries wholly below its prefix, the places below it in its first own page, and everything behind the ends."""

    def __init__(self, kind, kv_heads, d, page, groups, seed=0, width=None, scale=1.0, q_heads=None, order="hnd"):
        self.kind, self.kv_heads, self.d, self.page = kind, kv_heads, d, page
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        t = TYPES[kind]
        self.prefix = [max(0, p) for m in groups for p, _ in m]
        self.lens = [n for m in groups for _, n in m]
        self.start = [0] + list(np.cumsum([len(m) for m in groups]))
        self.first = [self.start[i] for i, m in enumerate(groups) for _ in m]
        batch = len(self.lens)
        held = [max(n, self.prefix[b]) if self.first[b] == b else n for b, n in enumerate(self.lens)]
        skip = [0 if self.first[b] == b else min(self.prefix[b], held[b]) for b in range(batch)]
        need = [-(-held[b] // page) - skip[b] // page for b in range(batch)]
        pages = sum(need) + 3
        self.width = width or max(1, max(-(-n // page) for n in held) + 1)
        if order == "hnd":
            both = torch.full((2, pages, kv_heads, page, d), math.nan, dtype=t, device="cuda")
            k, v = both[0], both[1]
        else:   # tokens outside heads
            both = torch.full((2, pages, page, kv_heads, d), math.nan, dtype=t, device="cuda")
            k, v = both[0].transpose(1, 2), both[1].transpose(1, 2)
        self.k, self.v = k, v
        perm = torch.randperm(pages, generator=g, device="cuda").tolist()
        table = np.full((batch, self.width), -7, dtype=np.int32)
        own = []
        for b in range(batch):
            at = skip[b] // page
            mine = [perm.pop() for _ in range(need[b])]
            table[b, at:at + len(mine)] = mine
            kk = (scale * torch.randn(kv_heads, held[b], d, generator=g, device="cuda")).to(t)
            vv = (torch.randn(kv_heads, held[b], d, generator=g, device="cuda") *
                  torch.exp(0.5 * torch.randn(1, held[b], 1, generator=g, device="cuda"))).to(t)
            for i, x in enumerate(mine):
                lo, hi = max((at + i) * page, skip[b]), min((at + i + 1) * page, held[b])
                if lo < hi:
                    s = slice(lo - (at + i) * page, hi - (at + i) * page)
                    k[x, :, s] = kk[:, lo:hi]
                    v[x, :, s] = vv[:, lo:hi]
            own.append((kk, vv))
        self.np_table, self.table = table, torch.from_numpy(table).cuda()
        self.t_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.t_prefix = torch.tensor([p for m in groups for p, _ in m], dtype=torch.int32, device="cuda")
        self.t_start = torch.tensor(self.start, dtype=torch.int32, device="cuda")
        self.own = own
        self.cache = lf.LFPagedCache.over(k[None], v[None])

    def randn(self, *shape, scale=1.5):
        return (scale * torch.randn(*shape, generator=self.g, device="cuda")).to(TYPES[self.kind])

    def rows(self, b, fresh=False):
        """Keys and values that sequence b sees, [kv_heads][len][d]."""
        n = self.lens[b]
        p = max(0, min(self.prefix[b], n - (1 if fresh else 0)))
        return [torch.cat((x[:, :p], y[:, p:n]), 1) for x, y in zip(self.own[self.first[b]], self.own[b])]

    def write_new(self, k_new, v_new):
        """What the call's new tokens make of the sequences."""
        for b, n in enumerate(self.lens):
            if n > 0:
                for x, new in zip(self.own[b], (k_new, v_new)):
                    x[:, n - 1] = new[b]

    def decode(self, q, k_new=None, v_new=None, **kw):
        return self.cache.decode_shared(0, q, self.table, self.t_lens, self.t_start, self.t_prefix, k_new, v_new, **kw)

    def check(self, q, out, lse=None, which=None, fresh=False):
        """Against the oracle; -> the worst share of the bound."""
        f = lambda x: x.detach().double().cpu().numpy()  # noqa: E731
        worst = 0.0
        for b in range(len(self.lens)) if which is None else which:
            n = self.lens[b]
            kk, vv = self.rows(b, fresh)
            ref, ref_lse, size, dots = paged_oracle.attend(f(q[b:b + 1]), f(kk), f(vv), paged_oracle.visible([n - 1], n, 0, 0))
            # the prefix's weights are rounded to bf16 before the product with the values
            tol, tol_lse = bounds(self.kind, self.d, n, ref, size, dots, 2.0 ** -8 if self.kind == "bf16" else 0.0)
            err = np.abs(f(out[b:b + 1]) - ref)
            assert np.isfinite(err).all(), f"sequence {b}: not finite"
            w = float((err / tol).max())
            assert w <= 1, f"sequence {b} ({self.prefix[b]} of {n}): {w:.3g} of the bound"
            worst = max(worst, w)
            if lse is not None:
                got = f(lse[b:b + 1])
                if n == 0:
                    assert np.isneginf(got).all()
                else:
                    assert (np.abs(got - ref_lse) <= tol_lse).all(), f"sequence {b}: lse"
        return worst
