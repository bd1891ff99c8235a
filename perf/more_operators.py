"""Position rotation and attention behind shared prefixes as they are measured: rotate, append, shared.

Rotation.  Of a head's first `rotary` columns the two of pair i turn by the angle w_i p, where p is the
token's position on the axis that pair i belongs to and w_i = base^(-2 i / rotary); the other columns
stay.  Pair i is columns (i, i + rotary / 2), or (2 i, 2 i + 1) where `adjacent`.  Tokens of text have one
position; those of a video have three (time, height, width), and `sections` says how many pairs each axis
takes.  `inverse` turns back: the rotation's transpose, which also takes gradients to where they came from.

- rotate: the queries (and keys) of a call's tokens, each with its positions.  `slab` says that the keys
  lie as `[sequence][head][token][dim]`, as a slab's prefill takes them.
- append: keys are rotated and written with their values to the pages of a paged cache,
  `[pages][kv_heads][page][dim]`: row b of the page table lists sequence b's pages, `lens[b]` is its length
  after the call's tokens, which are its last ones.  The queries of the same tokens are rotated on the way.
  Positions are those in the cache, or the caller's.
- shared: one new token per sequence of a paged cache, written to its page, attends to its whole sequence.
  The sequences come in groups; the first prefix_lens[b] positions of sequence b are those of its
  group's first one, in that one's pages.  Logits are scaled by 1 / sqrt(dim).

`own` false: plain torch operations in 32 bits, angles in 64.  `own` true: LFRotary and LFPagedCache.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _turn(name, op, type, heads, kv_heads, dim, rotary, sections, adjacent, base, seqs, tokens, **more):
    case = dict(op=op, type=type, heads=heads, kv_heads=kv_heads, dim=dim, rotary=rotary, sections=sections,
                adjacent=adjacent, base=base, seqs=seqs, tokens_min=tokens[0], tokens_max=tokens[1],
                far=0, inverse=False, slab=False, page=16, pick=0)
    case.update(more, **({"name": name} if name else {}))
    return case


def _behind(name, type, kv_heads, group, dim, page, groups, members, prefix, tail, branch, pick):
    case = dict(op="shared", type=type, kv_heads=kv_heads, group=group, dim=dim, page=page, groups=groups,
                members_min=members[0], members_max=members[1], prefix_min=prefix[0], prefix_max=prefix[1],
                tail_min=tail[0], tail_max=tail[1], branch=branch, pick=pick)
    case.update(**({"name": name} if name else {}))
    return case


def listed():
    return [
        # rotate ------------------------------------------------------------------------------
        # One decode step of 64 sequences somewhere within 16384 tokens: the latency of a single call.
        _turn("rotate-step", "rotate", "bf16", 32, 8, 128, 128, "", False, 1e6, 64, (1, 1), far=16384, pick=1),
        # A prompt with a video of 16000 tokens: three axes, 16 / 24 / 24 pairs, 32 / 8 heads of 128.
        _turn("rotate-video", "rotate", "bf16", 32, 8, 128, 128, "16,24,24", False, 1e6, 1, (16000, 16000), pick=2),
        # fp32 keys of 17 prompts of 1000 tokens as a slab takes them, heads of 64 of which a half turns,
        # adjacent pairs, turned back.
        _turn("rotate-slab-f32", "rotate", "f32", 8, 0, 64, 32, "", True, 1e4, 17, (1000, 1000), inverse=True,
              slab=True, pick=3),
        # append ------------------------------------------------------------------------------
        # The prompts of 32 requests, 64 to 2048 tokens each, with their queries, 32 / 8 heads of 128.
        _turn("append-prompts", "append", "bf16", 32, 8, 128, 128, "", False, 1e6, 32, (64, 2048), pick=4),
        # A video of 6000 tokens for each of two requests behind 100000 positions of text.
        _turn("append-video", "append", "bf16", 16, 8, 128, 128, "16,24,24", False, 1e6, 2, (6000, 6000),
              far=100000, pick=5),
        # One token for each of 256 running sequences, fp32, heads of 64 without groups, adjacent pairs.
        _turn("append-step-f32", "append", "f32", 8, 8, 64, 64, "", True, 1e4, 256, (1, 1), far=3000, pick=6),
        # shared ------------------------------------------------------------------------------
        # Eight short answers to one prompt of 2000 tokens, 16 / 8 heads: the latency of a single call.
        _behind("shared-few", "bf16", 8, 2, 128, 16, 1, (8, 8), (2000, 2000), (1, 64), False, 7),
        # 64 samples of one prompt of 8192 tokens, 100 to 1000 tokens into their answers.
        _behind("shared-samples", "bf16", 8, 4, 128, 16, 1, (64, 64), (8192, 8192), (100, 1000), False, 8),
        # 32 questions about one document of 60000 tokens.
        _behind("shared-long", "bf16", 8, 4, 128, 64, 1, (32, 32), (60000, 60000), (50, 500), False, 9),
        # 256 requests in 16 groups by their instructions, which some of them share only in part.
        _behind("shared-groups", "bf16", 8, 4, 128, 32, 16, (8, 24), (500, 4000), (16, 700), True, 10),
        # 256 sequences behind 16384 tokens: the products count as much as the bytes.
        _behind("shared-wide", "bf16", 8, 4, 128, 128, 1, (256, 256), (16384, 16384), (64, 512), False, 11),
        # fp32, 8 heads of 64 without groups, 24 sequences behind 3000 tokens.
        _behind("shared-f32", "f32", 8, 1, 64, 16, 1, (24, 24), (3000, 3000), (1, 200), False, 12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "shared", "shared"])
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    dim = 128 if rng.random() < 0.5 else rng.choice([16, 32, 64])
    page, pick = rng.choice([8, 16, 24, 32, 64, 128]), rng.randrange(1 << 20)
    row = kv_heads * dim * (2 if kind == "bf16" else 4)  # bytes of one token's keys
    if op == "shared":
        groups = _log(rng, 1, 24)
        members = _log(rng, 1, max(2, 256 // groups))
        # products and rows of the pools within those of the largest listed cases
        per = kv_heads * group * dim * groups * members * (1 if kind == "bf16" else 4)
        most = max(2, min(65536, 2**34 // per, 400 * 2**20 // (row * groups)))
        prefix = _log(rng, 1, most)
        tail = _log(rng, 1, max(2, min(1500, 400 * 2**20 // (row * groups * members))))
        return _behind(None, kind, kv_heads, group, dim, page, groups, (max(1, members // 2), members),
                       (max(1, prefix // 4), prefix), (1, tail), rng.random() < 0.4, pick)
    rotary = rng.choice([x for x in (16, 32, 64, 96, 128) if x <= dim])
    pairs = rotary // 2
    sections = ""
    if rng.random() < 0.4:
        a = rng.randrange(1, pairs - 1)
        b = rng.randrange(1, pairs - a)
        sections = f"{a},{b},{pairs - a - b}"
    seqs = _log(rng, 1, 256)
    tokens = _log(rng, 1, max(2, min(16000, 65536 // seqs, 150 * 2**20 // (row * (group + 1) * seqs))))
    slab = op == "rotate" and rng.random() < 0.3
    heads = kv_heads if slab else kv_heads * group
    least = tokens if op == "rotate" else max(1, tokens // 4)
    return _turn(None, op, kind, heads, 0 if slab else kv_heads, dim, rotary, sections, rng.random() < 0.4,
                 rng.choice([1e4, 5e5, 1e6]), seqs, (least, tokens), far=_log(rng, 1, 120000),
                 inverse=op == "rotate" and rng.random() < 0.4, slab=slab, page=page, pick=pick)


# ---- inputs -------------------------------------------------------------------------------------------

def _counts(case):
    """Tokens of every sequence of a rotate or append call: the case's own numbers."""
    r = random.Random(case["pick"])
    return [r.randint(case["tokens_min"], case["tokens_max"]) for _ in range(case["seqs"])]


def _family(case):
    """[members of each group], [shared length of each sequence], [its whole length]."""
    r = random.Random(case["pick"])
    members, shared, lens = [], [], []
    for _ in range(case["groups"]):
        n, p = r.randint(case["members_min"], case["members_max"]), r.randint(case["prefix_min"], case["prefix_max"])
        members.append(n)
        for i in range(n):
            mine = p if i == 0 or not case["branch"] or r.random() < 0.7 else r.randint(0, p)
            shared.append(mine)
            lens.append(mine + r.randint(case["tail_min"], case["tail_max"]))
    return members, shared, lens


def _video(n, start):
    """Positions on three axes of n tokens: a fifth of text, frames of 14 x 18, text behind them."""
    text, rows, cols = n // 5, 14, 18
    pos, at = [(start + i,) * 3 for i in range(text)], start + text
    for i in range(n - text - n // 10):
        frame, cell = divmod(i, rows * cols)
        pos.append((at + frame, at + cell // cols, at + cell % cols))
    at = max(max(p) for p in pos) + 1 if pos else start
    while len(pos) < n:
        pos.append((at,) * 3)
        at += 1
    return pos


def _frequencies(case):
    i = torch.arange(case["rotary"] // 2, dtype=torch.float64)
    return float(case["base"]) ** (-2 * i / case["rotary"])


def prepare(case, seed):
    dev, t = "cuda", TYPES[case["type"]]
    g = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + case["pick"])
    d, page = case["dim"], case["page"]

    def values(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def pool(pages):
        k = values(pages, case["kv_heads"], page, d).to(t)
        v = (values(pages, case["kv_heads"], page, d) * torch.exp(0.5 * values(pages, 1, page, 1))).to(t)
        return k, v

    def pages_of(n):
        return torch.randperm(n, generator=g, device=dev).to(torch.int32), n

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = dict(case)
    if case["op"] == "shared":
        members, shared, lens = _family(case)
        n, group = len(lens), case["group"]
        # own pages of every sequence, from the page its shared part ends in; the group's first, which shares
        # the most, has them all
        first, starts = [], [0]
        for m in members:
            first += [starts[-1]] * m
            starts.append(starts[-1] + m)
        need = [-(-lens[b] // page) - (0 if first[b] == b else shared[b] // page) for b in range(n)]
        order, pages = pages_of(sum(need) + 3)
        k, v = pool(pages)
        far = torch.rand(pages, 1, page, 1, generator=g, device=dev) < 0.01  # keys that many queries like
        u = torch.nn.functional.normalize(values(case["kv_heads"], 1, d), dim=-1)
        k = (k.float() + far * (3 * math.sqrt(d)) * u).to(t)
        table = torch.zeros(n, -(-max(lens) // page), dtype=torch.int32, device=dev)
        at = 0
        for b in range(n):
            mine = order[at:at + need[b]]
            at += need[b]
            if first[b] == b:
                table[b, :need[b]] = mine
                continue
            whole = shared[b] // page
            table[b, :whole] = table[first[b], :whole]
            table[b, whole:whole + need[b]] = mine
            rest = shared[b] - whole * page
            if rest:  # the page that the shared part ends in is a copy of its own
                src = table[first[b], whole].long()
                k[mine[0].long(), :, :rest] = k[src, :, :rest]
                v[mine[0].long(), :, :rest] = v[src, :, :rest]
        s.update(k=k, v=v, table=table, lens=ints(lens), prefix_lens=ints(shared), group_start=ints(starts),
                 host_lens=lens, host_shared=shared, host_first=first,
                 q=(1.5 * values(n, case["kv_heads"] * group, d)).to(t),
                 k_new=values(n, case["kv_heads"], d).to(t), v_new=values(n, case["kv_heads"], d).to(t))
        if own:  # the handle that a program keeps for its pools
            from decode_kv_cache_gb300.longflow import LFPagedCache
            s["cache"] = LFPagedCache.over(k[None], v[None])
        return s

    counts = _counts(case)
    total, axes = sum(counts), 3 if case["sections"] else 1
    r = random.Random(case["pick"] + int(seed))
    behind = [r.randrange(case["far"]) if case["far"] else 0 for _ in counts]
    if axes == 3:
        positions = ints([p for n, o in zip(counts, behind) for p in _video(n, o)]).t().contiguous()
    else:
        positions = ints([o + i for n, o in zip(counts, behind) for i in range(n)])
    s["freq"] = _frequencies(case).to(dev)
    s["axis"] = torch.repeat_interleave(torch.arange(axes), torch.tensor(
        [int(x) for x in case["sections"].split(",")] if case["sections"] else [case["rotary"] // 2])).to(dev)
    if own:
        from decode_kv_cache_gb300.longflow import LFRotary
        s["rotary_handle"] = LFRotary(
            case["rotary"], base=case["base"], adjacent=case["adjacent"],
            sections=[int(x) for x in case["sections"].split(",")] if case["sections"] else None)
    if case["op"] == "rotate":
        if case["slab"]:
            x = values(case["seqs"], case["heads"], counts[0], d).to(t).transpose(1, 2)
            s.update(q=x, positions=positions.view(*positions.shape[:-1], case["seqs"], counts[0]))
        else:
            s.update(q=values(total, case["heads"], d).to(t), positions=positions)
        if case["kv_heads"]:
            s["k_new"] = values(total, case["kv_heads"], d).to(t)
        return s
    # The pages that the tokens go to, and what was there before: three axes do not count as the cache
    # does, so these tokens come behind few others there; one axis follows the cache's positions.
    old = [min(o, 300) for o in behind] if axes == 3 else behind
    lens = [o + n for o, n in zip(old, counts)]
    width = -(-max(lens) // page)
    need = [-(-n // page) - o // page for n, o in zip(lens, old)]  # (pages of earlier tokens are not touched)
    order, pages = pages_of(sum(-(-n // page) + 1 for n in counts) + 3)
    k, v = pool(pages)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, old[b] // page:old[b] // page + n] = order[at:at + n]
        at += n
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    s.update(k=k, v=v, table=table, lens=ints(lens), new_start=ints(starts), positions=positions, total=total,
             q=values(total, case["heads"], d).to(t), k_new=values(total, case["kv_heads"], d).to(t),
             v_new=values(total, case["kv_heads"], d).to(t))
    if own:
        from decode_kv_cache_gb300.longflow import LFPagedCache
        s["cache"] = LFPagedCache.over(k[None], v[None])
    return s


# ---- the plain forms ------------------------------------------------------------------------------------

def _plain_rotated(s, x, positions):
    """x [..., heads, dim] with positions [...], or [axes, ...]."""
    if s["sections"]:
        p = torch.movedim(positions, 0, -1)[..., s["axis"]].double()
    else:
        p = positions.double()[..., None]
    angle = p * s["freq"]
    if s["inverse"]:
        angle = -angle
    cos, sin = angle.cos().float()[..., None, :], angle.sin().float()[..., None, :]
    n, half = s["rotary"], s["rotary"] // 2
    f = x.float()
    one, two = (f[..., 0:n:2], f[..., 1:n:2]) if s["adjacent"] else (f[..., :half], f[..., half:n])
    a, b = one * cos - two * sin, two * cos + one * sin
    turned = torch.stack((a, b), -1).flatten(-2) if s["adjacent"] else torch.cat((a, b), -1)
    return torch.cat((turned, f[..., n:]), -1).to(x.dtype)


def _plain_rotate(s):
    q = _plain_rotated(s, s["q"], s["positions"])
    return (q, _plain_rotated(s, s["k_new"], s["positions"])) if "k_new" in s else q


def _plain_append(s):
    n = torch.arange(s["total"], device=s["lens"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["new_start"], n, right=True) - 1
    fresh = s["new_start"][1:] - s["new_start"][:-1]
    pos = (s["lens"] - fresh)[seq] + n - s["new_start"][seq]
    turn = s["positions"] if s["sections"] else pos
    page, slot = s["table"][seq, pos // s["page"]].long(), (pos % s["page"]).long()
    s["k"][page, :, slot] = _plain_rotated(s, s["k_new"], turn)
    s["v"][page, :, slot] = s["v_new"]
    return _plain_rotated(s, s["q"], turn), s["k"], s["v"]


def _plain_shared(s):
    """One sequence after another, over its own whole length."""
    hkv, gr, d, page = s["kv_heads"], s["group"], s["dim"], s["page"]
    last = (s["lens"] - 1).long()
    spot = s["table"].gather(1, (last // page)[:, None])[:, 0].long()
    s["k"][spot, :, last % page] = s["k_new"]
    s["v"][spot, :, last % page] = s["v_new"]
    out = torch.empty_like(s["q"])
    for b, n in enumerate(s["host_lens"]):
        which = s["table"][b, :-(-n // page)].long()
        whole = s["host_shared"][b] // page
        which[:whole] = s["table"][s["host_first"][b], :whole].long()
        k, v = (pool[which].float().transpose(0, 1).flatten(1, 2)[:, :n] for pool in (s["k"], s["v"]))
        logits = s["q"][b].float().view(hkv, gr, d) @ k.transpose(-1, -2) / math.sqrt(d)
        p = (logits - logits.amax(-1, keepdim=True)).exp()
        out[b] = ((p @ v) / p.sum(-1, keepdim=True)).view(hkv * gr, d).to(out.dtype)
    return out, s["k"], s["v"]


def run(s):
    if own:
        if s["op"] == "rotate":
            return s["rotary_handle"].rotate(s["q"], s["positions"], k=s.get("k_new"), inverse=s["inverse"])
        c = s["cache"]
        if s["op"] == "append":
            q = c.append_rotated(0, s["k_new"], s["v_new"], s["table"], s["lens"], s["rotary_handle"],
                                 new_start=s["new_start"], positions=s["positions"] if s["sections"] else None,
                                 q=s["q"])
            return q, s["k"], s["v"]
        out = c.decode_shared(0, s["q"], s["table"], s["lens"], s["group_start"], s["prefix_lens"], s["k_new"],
                              s["v_new"])
        return out, s["k"], s["v"]
    return {"rotate": _plain_rotate, "append": _plain_append, "shared": _plain_shared}[s["op"]](s)


def work(case):
    e = 2 if case["type"] == "bf16" else 4
    d = case["dim"]
    if case["op"] == "shared":
        token = case["kv_heads"] * d * e
        members, shared, lens = _family(case)
        prefixes = [max(shared[sum(members[:i]):][:m]) for i, m in enumerate(members)]
        keys = sum(prefixes) + sum(n - 1 - p for n, p in zip(lens, shared))  # the new token's come from the call
        return {"bytes": 2 * token * keys + 4 * token * len(lens) + 2 * token * case["group"] * len(lens),
                "flops": 4 * d * case["kv_heads"] * case["group"] * sum(lens)}
    n = sum(_counts(case))
    heads = case["heads"] + case["kv_heads"] * (2 if case["op"] == "append" else 1)
    given = case["op"] == "rotate" or bool(case["sections"])
    positions = 4 * n * (3 if case["sections"] else 1) if given else 0
    return {"bytes": 2 * n * heads * d * e + positions,
            "flops": 3 * n * (case["heads"] + case["kv_heads"]) * case["rotary"]}


# ---- the definition in 64 bits --------------------------------------------------------------------------

def _exactly_turned(case, x, positions):
    """Each pair as a complex number times e^(i w p), a head at a time."""
    n = case["rotary"]
    w = torch.exp(torch.arange(0, n, 2, dtype=torch.float64, device=x.device) * (-math.log(case["base"]) / n))
    if case["sections"]:
        parts, at = [], 0
        for axis, size in enumerate(int(c) for c in case["sections"].split(",")):
            parts.append(positions[axis].double().unsqueeze(-1) * w[at:at + size])
            at += size
        angle = torch.cat(parts, -1)
    else:
        angle = positions.double().unsqueeze(-1) * w
    turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)
    out = x.double().clone(memory_format=torch.contiguous_format)
    for h in range(x.shape[-2]):
        y = out[..., h, :n]
        if case["adjacent"]:
            z = torch.view_as_complex(y.reshape(*y.shape[:-1], n // 2, 2).contiguous()) * turn
            y.copy_(torch.view_as_real(z).reshape(y.shape))
        else:
            z = torch.complex(y[..., :n // 2].contiguous(), y[..., n // 2:].contiguous()) * turn
            y[..., :n // 2] = z.real
            y[..., n // 2:] = z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        q = _exactly_turned(case, s["q"], s["positions"])
        return (q, _exactly_turned(case, s["k_new"], s["positions"])) if "k_new" in s else q
    page, hkv, d = case["page"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        counts, lens, table = _counts(case), s["lens"].tolist(), s["table"].cpu()
        at = [(b, lens[b] - n + i) for b, n in enumerate(counts) for i in range(n)]
        spots = torch.tensor([int(table[b, p // page]) * page + p % page for b, p in at], device="cuda")
        turn = s["positions"] if case["sections"] else torch.tensor([p for _, p in at], device="cuda")
        pools = []
        for pool, fresh in ((s["k"].double(), _exactly_turned(case, s["k_new"], turn)),
                            (s["v"].double(), s["v_new"].double())):
            flat = pool.permute(0, 2, 1, 3).reshape(-1, hkv, d).index_copy(0, spots, fresh)
            pools.append(flat.view(-1, page, hkv, d).permute(0, 2, 1, 3).contiguous())
        return _exactly_turned(case, s["q"], turn), *pools
    members, shared, lens = _family(case)
    out = torch.zeros(len(lens), hkv * case["group"], d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):   # the new tokens first: they may lie in a page that others read
        x, slot = int(s["table"][b, (n - 1) // page]), (n - 1) % page
        s["k"][x, :, slot], s["v"][x, :, slot] = s["k_new"][b], s["v_new"][b]
    leader = [i for i, m in enumerate(members) for _ in range(m)]
    begin = [sum(members[:i]) for i in range(len(members))]
    for b, n in enumerate(lens):
        p = torch.arange(n, device="cuda")
        row = torch.where(p < shared[b], begin[leader[b]], b)
        x = s["table"][row, p // page].long()
        for h in range(hkv):
            k, v = s["k"][x, h, p % page].double(), s["v"][x, h, p % page].double()
            for j in range(h * case["group"], (h + 1) * case["group"]):
                out[b, j] = torch.softmax(k @ s["q"][b, j].double() * d ** -0.5, 0) @ v
    return out, s["k"], s["v"]
