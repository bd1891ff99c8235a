"""Inputs and bounds for the paged cache's tests (GPU side; the expected values are the fp64
oracle's)."""
import math

import numpy as np
import torch

from decode_kv_cache_gb300 import longflow as lf
from oracle import paged_oracle

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def bounds(kind, d, n, out, size, dots, weight_step=0.0):
    """How far a right kernel's out and lse may be from the fp64 values.

    A logit in units of log2 carries the products' sums in fp32, at most d + 4 roundings of terms
    that sum to `dots` log2(e) in size; its weight moves by that times ln 2, numerator and
    denominator alike; 2^x itself is good to 2^-21; sums over n keys and their rescalings add n + 64
    roundings; `weight_step` is the rounding of the weights before the product with the values.
    The output is rounded once."""
    logit = (d + 4) * 2.0 ** -24 * dots * math.log2(math.e)
    rel = 2 * math.log(2) * logit + 2.0 ** -20 + 2 * (n + 64) * 2.0 ** -24
    err = (rel[..., None] + weight_step) * size
    tol = err + HALF_STEP[kind] * (np.abs(out) + err) + 1e-30
    return tol, rel + 2.0 ** -22 * (1 + dots)


class Paged:
    """A cache with random contents: tables of shuffled pages, `lens` tokens per sequence, and NaN in
    every place of the pools that no token holds."""

    def __init__(self, kind, kv_heads, d, page, lens, seed=0, order="hnd", spare=3, width=None, scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.kv_heads, self.d, self.page, self.lens = kind, kv_heads, d, page, list(lens)
        t = TYPES[kind]
        need = [-(-n // page) for n in lens]
        self.width = width or max(1, max(need) + 1)
        pages = sum(need) + spare
        # [pages][kv_heads][page][d] in memory orders that a caller may have
        if order == "hnd":
            both = torch.full((2, pages, kv_heads, page, d), math.nan, dtype=t, device="cuda")
            k, v = both[0], both[1]
        elif order == "nhd":        # tokens outside heads
            both = torch.full((2, pages, page, kv_heads, d), math.nan, dtype=t, device="cuda")
            k, v = both[0].transpose(1, 2), both[1].transpose(1, 2)
        elif order == "interleaved":  # K and V of a token side by side
            both = torch.full((pages, kv_heads, page, 2, d), math.nan, dtype=t, device="cuda")
            k, v = both[:, :, :, 0], both[:, :, :, 1]
        self.k, self.v = k, v
        perm = torch.randperm(pages, generator=g, device="cuda").tolist()
        table = np.full((len(lens), self.width), -7, dtype=np.int32)   # never read past the end
        self.rows_k, self.rows_v = [], []
        for b, n in enumerate(lens):
            mine = [perm.pop() for _ in range(need[b])]
            table[b, :len(mine)] = mine
            kk = (scale * torch.randn(kv_heads, n, d, generator=g, device="cuda")).to(t)
            vv = (torch.randn(kv_heads, n, d, generator=g, device="cuda") *
                  torch.exp(0.5 * torch.randn(1, n, 1, generator=g, device="cuda"))).to(t)
            for i, x in enumerate(mine):
                m = min(page, n - i * page)
                k[x, :, :m] = kk[:, i * page:i * page + m]
                v[x, :, :m] = vv[:, i * page:i * page + m]
            self.rows_k.append(kk)
            self.rows_v.append(vv)
        self.np_table = table
        self.table = torch.from_numpy(table).cuda()
        self.t_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.cache = lf.LFPagedCache.over(k[None], v[None])
        self.g = g

    def randn(self, *shape, scale=1.5):
        return (scale * torch.randn(*shape, generator=self.g, device="cuda")).to(TYPES[self.kind])

    def hide(self, b, lo, hi):
        """Positions lo .. hi - 1 of sequence b become NaN in the pools."""
        for p in range(lo, hi):
            x = int(self.np_table[b, p // self.page])
            self.k[x, :, p % self.page] = math.nan
            self.v[x, :, p % self.page] = math.nan

    def check(self, b, q, first_pos, out, lse, window=0, sinks=0, weight_step=0.0):
        """One sequence's rows of out / lse against the oracle; returns the worst share of the bound."""
        n = self.lens[b]
        pos = first_pos + np.arange(q.shape[0])
        see = paged_oracle.visible(pos, n, window, sinks)
        f = lambda x: x.detach().double().cpu().numpy()  # noqa: E731
        kk, vv = f(self.rows_k[b]), f(self.rows_v[b])
        ref, ref_lse, size, dots = paged_oracle.attend(f(q), kk, vv, see)
        tol, tol_lse = bounds(self.kind, self.d, n, ref, size, dots, weight_step)
        err = np.abs(f(out) - ref)
        assert np.isfinite(err).all(), f"sequence {b}: not finite"
        worst = float((err / tol).max()) if err.size else 0.0
        assert worst <= 1, f"sequence {b}: {worst:.3g} of the bound at {np.unravel_index((err / tol).argmax(), err.shape)}"
        if lse is not None:
            got = f(lse)
            none = ~see.any(axis=1)
            assert np.isneginf(got[none]).all()
            e = np.abs(got[~none] - ref_lse[~none])
            assert (e <= tol_lse[~none]).all(), f"sequence {b}: lse off by {e.max()}"
        return worst


def starts(counts):
    return [0] + list(np.cumsum(counts))
