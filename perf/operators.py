"""The paged key-value cache's operators as they are measured: append, decode, prompt.

A layer's keys and values live in pages of `page` tokens, `[pages][kv_heads][page][dim]`.  Row b of
the page table lists sequence b's pages in order of position, `lens[b]` is its length after this
call's tokens.  Query head h reads KV head h // group; logits are scaled by 1 / sqrt(dim).

- append: this call's tokens (sequence b's are rows new_start[b] .. new_start[b + 1] - 1, the last
  ones by position) are written to their pages.
- decode: one new token per sequence.  Its key and value are written to its page ("writes"), and its
  query attends to every position of the sequence, itself included.
- prompt: the last tokens of every sequence, their keys and values already in the pages, attend
  causally: to their own position and everything before it.

With a window W > 0 the query at position p sees the positions p - W + 1 .. p and, besides them, the
first `sinks` positions.  A query that sees nothing gives zeros.

`own` false: plain torch operations in 32 bits.  `own` true: the calls of LFPagedCache.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FIELDS = ("op", "type", "kv_heads", "group", "dim", "page", "seqs", "old_min", "old_max", "new_min",
          "new_max", "window", "sinks", "writes", "pick")


def _case(name, *values):
    return dict(zip(FIELDS, values), **({"name": name} if name else {}))


def listed():
    return [
        # append ------------------------------------------------------------------------------
        # The prompts of 32 requests, 64 to 2048 tokens each, enter a bf16 cache (8 KV heads of 128).
        _case("append-prompts", "append", "bf16", 8, 4, 128, 16, 32, 0, 0, 64, 2048, 0, 0, True, 1),
        # One token for each of 256 running sequences of an fp32 cache, heads of 64.
        _case("append-step-f32", "append", "f32", 8, 1, 64, 16, 256, 10, 3000, 1, 1, 0, 0, True, 2),
        # decode ------------------------------------------------------------------------------
        # One conversation of 300 tokens, 16 query / 8 KV heads: the latency of a single call.
        _case("decode-one-short", "decode", "bf16", 8, 2, 128, 16, 1, 299, 299, 1, 1, 0, 0, True, 3),
        # 64 sequences at 3276 tokens, 32 / 8 heads: the steady batch of the slab's own benchmark.
        _case("decode-steady", "decode", "bf16", 8, 4, 128, 16, 64, 3275, 3275, 1, 1, 0, 0, True, 4),
        # 256 sequences of 64 to 3276 tokens, as a server holds them.
        _case("decode-ragged", "decode", "bf16", 8, 4, 128, 32, 256, 63, 3275, 1, 1, 0, 0, True, 5),
        # Two long documents, 100 to 130 thousand tokens: few rows, a long axis.
        _case("decode-long", "decode", "bf16", 8, 4, 128, 128, 2, 100000, 130000, 1, 1, 0, 0, True, 6),
        # 64 sequences of up to 16384 tokens that keep 4 sinks and a window of 1000.
        _case("decode-window", "decode", "bf16", 8, 4, 128, 64, 64, 500, 16383, 1, 1, 1000, 4, True, 7),
        # fp32, 8 heads of 64 without groups, 1000-token buffers, 17 sequences.
        _case("decode-f32", "decode", "f32", 8, 1, 64, 16, 17, 700, 999, 1, 1, 0, 0, True, 8),
        # prompt ------------------------------------------------------------------------------
        # Chunks of 1 to 512 tokens of 24 requests, each behind 0 to 2048 tokens it had already.
        _case("prompt-chunks", "prompt", "bf16", 8, 4, 128, 16, 24, 0, 2048, 1, 512, 0, 0, False, 9),
        # One prompt of 8192 tokens, 32 / 8 heads.
        _case("prompt-long", "prompt", "bf16", 8, 4, 128, 64, 1, 0, 0, 8192, 8192, 0, 0, False, 10),
        # One prompt of 12000 tokens with a window of 1000 and 4 sinks, 16 / 8 heads.
        _case("prompt-window", "prompt", "bf16", 8, 2, 128, 32, 1, 0, 0, 12000, 12000, 1000, 4, False, 11),
        # fp32, 8 heads of 64 without groups, three prompts of up to 1000 tokens.
        _case("prompt-f32", "prompt", "f32", 8, 1, 64, 16, 3, 0, 0, 500, 1000, 0, 0, False, 12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prompt", "prompt"])
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    dim = 128 if rng.random() < 0.5 else rng.choice([16, 32, 64])
    page = rng.choice([8, 16, 32, 64, 128])
    window = _log(rng, 16, 4096) if rng.random() < 0.4 else 0
    sinks = rng.choice([0, 1, 4, 16]) if window else 0
    row = kv_heads * dim * (2 if kind == "bf16" else 4)  # bytes of one token's keys
    if op == "append":
        seqs, new = _log(rng, 1, 256), _log(rng, 1, 2048)
        new = max(1, min(new, 128 * 2**20 // (row * seqs)))
        old = rng.randrange(0, 1024)
        return _case(None, op, kind, kv_heads, group, dim, page, seqs, 0, old, max(1, new // 8), new, 0, 0,
                     True, rng.randrange(1 << 20))
    if op == "decode":
        seqs = _log(rng, 1, 256)
        most = _log(rng, 2, max(3, min(130000, 400 * 2**20 // (row * seqs))))
        least = rng.choice([0, most // 2, most - 1])
        return _case(None, op, kind, kv_heads, group, dim, page, seqs, least, most - 1, 1, 1, window, sinks,
                     rng.random() < 0.7, rng.randrange(1 << 20))
    seqs = _log(rng, 1, 32)
    heads = kv_heads * group
    # Pairs of a query and a key over all padded sequences: a plain form holds them all.
    pairs = (2**30 if kind == "bf16" else 2**28) // heads // seqs
    new = _log(rng, 1, max(2, min(8192, math.isqrt(pairs))))
    old = rng.choice([0, 0, _log(rng, 1, max(2, min(16384, pairs // new - new if pairs // new > new else 1)))])
    return _case(None, op, kind, kv_heads, group, dim, page, seqs, 0, old, max(1, new // 4), new, window,
                 sinks, False, rng.randrange(1 << 20))


def _lengths(case):
    """([tokens already cached], [tokens of this call]) of every sequence: the case's own numbers."""
    r = random.Random(case["pick"])
    n = case["seqs"]
    old = [r.randint(case["old_min"], case["old_max"]) for _ in range(n)]
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(n)]
    return old, new


def prepare(case, seed):
    dev, t = "cuda", TYPES[case["type"]]
    g = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + case["pick"])
    hkv, hq, d, page = case["kv_heads"], case["kv_heads"] * case["group"], case["dim"], case["page"]
    old, new = _lengths(case)
    lens = [a + b for a, b in zip(old, new)]
    need = [-(-n // page) for n in lens]
    width, pages = max(need), sum(need) + 3
    # A pool that has served other requests: every page holds values, handed out in no order.
    def values(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def keys(n):
        x = values(n, hkv, page, d)
        far = torch.rand(n, 1, page, 1, generator=g, device=dev) < 0.01  # keys that many queries like
        u = torch.nn.functional.normalize(values(hkv, 1, d), dim=-1)
        return (x + far * (3 * math.sqrt(d)) * u).to(t)

    k = keys(pages)
    v = (values(pages, hkv, page, d) * torch.exp(0.5 * values(pages, 1, page, 1))).to(t)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = dict(case, k=k, v=v, table=table, max_new=max(new), max_len=max(lens), total=start[-1],
             lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             new_start=torch.tensor(start, dtype=torch.int32, device=dev))
    if case["writes"]:
        s["k_new"] = values(start[-1], hkv, d).to(t)
        s["v_new"] = values(start[-1], hkv, d).to(t)
    if case["op"] != "append":
        s["q"] = (1.5 * values(start[-1], hq, d)).to(t)
    if own:  # the handle that a program keeps for its pools
        from decode_kv_cache_gb300.longflow import LFPagedCache
        s["cache"] = LFPagedCache.over(k[None], v[None])
    return s


def _owners(s):
    """Sequence and position of every row of this call's tokens."""
    n = torch.arange(s["total"], device=s["lens"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["new_start"], n, right=True) - 1
    fresh = s["new_start"][1:] - s["new_start"][:-1]
    return seq, (s["lens"] - fresh)[seq] + n - s["new_start"][seq]


def _plain_append(s):
    seq, pos = _owners(s)
    page, slot = s["table"][seq, pos // s["page"]].long(), (pos % s["page"]).long()
    s["k"][page, :, slot] = s["k_new"]
    s["v"][page, :, slot] = s["v_new"]
    return s["k"], s["v"]


def _seen(s, q_pos, keys):
    """Which of `keys` (positions) the queries at q_pos[..., None] see."""
    see = keys <= q_pos
    if s["window"]:
        see = see & ((keys > q_pos - s["window"]) | (keys < s["sinks"]))
    return see


def _rows(s, pool):
    """A pool's tokens by sequence and position, [seqs][kv_heads][max_len][dim], in 32 bits."""
    x = pool[s["table"].long()].float()  # [seqs][width][kv_heads][page][dim]
    return x.transpose(1, 2).flatten(2, 3)[:, :, : s["max_len"]]


def _softmax_times(logits, see, v):
    logits = logits.masked_fill_(~see, -math.inf)
    top = logits.amax(-1, keepdim=True).clamp_min(-1e30)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, (p @ v) / total, 0.0)


def _plain_decode(s):
    if s["writes"]:
        _plain_append(s)
    b, hkv, gr, d = s["seqs"], s["kv_heads"], s["group"], s["dim"]
    q = s["q"].float().view(b, hkv, gr, d)
    logits = (q @ _rows(s, s["k"]).transpose(-1, -2)) / math.sqrt(d)
    keys = torch.arange(s["max_len"], device=q.device)
    see = _seen(s, s["lens"].view(-1, 1, 1, 1) - 1, keys)
    out = _softmax_times(logits, see, _rows(s, s["v"])).view(b, hkv * gr, d).to(s["q"].dtype)
    return (out, s["k"], s["v"]) if s["writes"] else out


def _plain_prompt(s):
    b, hkv, gr, d, n = s["seqs"], s["kv_heads"], s["group"], s["dim"], s["max_new"]
    row = (s["new_start"][:-1, None] + torch.arange(n, device=s["lens"].device)).clamp_max(s["total"] - 1)
    fresh = s["new_start"][1:] - s["new_start"][:-1]
    pos = (s["lens"] - fresh)[:, None] + torch.arange(n, device=s["lens"].device)
    q = s["q"][row].float().view(b, n, hkv, gr, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, gr * n, d)
    logits = (q @ _rows(s, s["k"]).transpose(-1, -2)).view(b, hkv, gr, n, -1).div_(math.sqrt(d))
    keys = torch.arange(s["max_len"], device=q.device)
    see = _seen(s, pos[..., None], keys)[:, None, None]
    out = _softmax_times(logits, see, _rows(s, s["v"])[:, :, None])
    seq, _ = _owners(s)
    at = torch.arange(s["total"], device=q.device) - s["new_start"][seq]
    return out[seq, :, :, at].reshape(s["total"], hkv * gr, d).to(s["q"].dtype)


def run(s):
    if own:
        c = s["cache"]
        if s["op"] == "append":
            c.append(0, s["k_new"], s["v_new"], s["table"], s["lens"], new_start=s["new_start"])
            return s["k"], s["v"]
        if s["op"] == "decode":
            out = c.decode(0, s["q"], s["table"], s["lens"], s.get("k_new"), s.get("v_new"),
                           window=s["window"], sinks=s["sinks"])
            return (out, s["k"], s["v"]) if s["writes"] else out
        return c.prompt(0, s["q"], s["table"], s["lens"], s["new_start"], s["max_new"],
                        window=s["window"], sinks=s["sinks"])
    return {"append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt}[s["op"]](s)


def _pairs(case):
    """Pairs of a query token and a key token that it sees, and keys that any query sees."""
    old, new = _lengths(case)
    w, sinks = case["window"], case["sinks"]
    pairs = keys = 0
    for o, n in zip(old, new):
        if not w:
            pairs += n * o + n * (n + 1) // 2
            keys += o + n
            continue
        for p in range(o, o + n):
            pairs += min(p + 1, w) + min(sinks, max(0, p + 1 - w))
        first = max(0, o + 1 - w)
        keys += o + n - first + min(sinks, first)
    return pairs, keys


def work(case):
    e = 2 if case["type"] == "bf16" else 4
    token = case["kv_heads"] * case["dim"] * e
    _, new = _lengths(case)
    if case["op"] == "append":
        return {"bytes": 4 * token * sum(new), "flops": 0}
    pairs, keys = _pairs(case)
    query = token * case["group"]
    wrote = 4 * token * sum(new) if case["writes"] else 0
    read = keys - (sum(new) if case["writes"] else 0)  # a written token's own key comes from the call
    return {"bytes": 2 * token * read + wrote + 2 * query * sum(new),
            "flops": 4 * case["dim"] * case["kv_heads"] * case["group"] * pairs}


def exact(case, seed):
    """The definition in 64 bits, one sequence and one KV head at a time."""
    s = prepare(case, seed)
    old, new = _lengths(case)
    dev, page, gr, d = s["k"].device, case["page"], case["group"], case["dim"]
    if case["writes"]:
        spots = []
        table = s["table"].cpu()
        for b in range(case["seqs"]):
            for p in range(old[b], old[b] + new[b]):
                spots.append(int(table[b, p // page]) * page + p % page)
        spots = torch.tensor(spots, device=dev)
        for pool, fresh in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
            flat = pool.permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], d)
            flat = flat.index_copy(0, spots, fresh)
            pool.copy_(flat.view(-1, page, case["kv_heads"], d).permute(0, 2, 1, 3))
    if case["op"] == "append":
        return s["k"], s["v"]
    out = torch.zeros(s["total"], case["kv_heads"] * gr, d, dtype=torch.float64, device=dev)
    row = 0
    for b in range(case["seqs"]):
        o, n = old[b], new[b]
        which = s["table"][b, : -(-(o + n) // page)].long()
        at = torch.arange(o + n, device=dev)
        me = torch.arange(o, o + n, device=dev)[:, None]
        hidden = at[None] > me
        if case["window"]:
            hidden |= (at[None] <= me - case["window"]) & (at[None] >= case["sinks"])
        for h in range(case["kv_heads"]):
            kk = s["k"][which, h].reshape(-1, d)[: o + n].double()
            vv = s["v"][which, h].reshape(-1, d)[: o + n].double()
            for j in range(h * gr, (h + 1) * gr):
                z = s["q"][row:row + n, j].double() @ kk.t() * d ** -0.5
                out[row:row + n, j] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ vv
        row += n
    return (out, s["k"], s["v"]) if case["op"] == "decode" and case["writes"] else out
