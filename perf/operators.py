"""Timed cases of the paged key-value cache operators: rows written to a cache and read back, attention
of new tokens over it, and the KL divergence of two attentions over it.

A cache holds fixed-size pages [pages, Hkv, page, d] of keys and of values; a sequence's keys lie in the
pages that its row of the page table names, in order.  It is bf16, or e4m3 with one power-of-two scale per
row (a byte per token and head: the scale's exponent plus 127).  `own` false: elementary torch operations in 32 bits.  `own`
true: the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LEAST = -96            # smallest exponent of a row's scale
NONE = -1              # page table entry behind a sequence's last page


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One token of each running sequence of a serving batch, written and read back: launch latency.
        dict(name="write-decode", op="write", B=64, Hkv=8, NT=1, ctx=2000, ragged=True, d=128, page=64,
             kind="e4m3", back="new"),
        # A ragged batch of short prompts behind cached prefixes, small heads, unquantised; the whole
        # context read back for the dense kernels.
        dict(name="write-ragged", op="write", B=4, Hkv=8, NT=777, ctx=1300, ragged=True, d=64, page=16,
             kind="bf16", back="all"),
        # A whole 16K prompt of 32 heads quantised into the cache and read back.
        dict(name="write-prompt", op="write", B=1, Hkv=32, NT=16384, ctx=0, ragged=False, d=128, page=64,
             kind="e4m3", back="all"),
        # One short sequence, one new token: the call's latency.
        dict(name="attn-short", op="attn", B=1, Hq=32, Hkv=8, NQ=1, len=300, ragged=False, d=128, page=16,
             kind="bf16"),
        # The decode workload's shape: one token of 16 heads against 131072 cached keys.
        dict(name="attn-long", op="attn", B=1, Hq=16, Hkv=16, NQ=1, len=131072, ragged=False, d=128, page=64,
             kind="bf16"),
        # A serving batch: 64 sequences of uneven length, four query heads to a key head, quantised.
        dict(name="attn-batch", op="attn", B=64, Hq=32, Hkv=8, NQ=1, len=8192, ragged=True, d=128, page=64,
             kind="e4m3"),
        # The grouped-query workload's heads (d = 64) with one new token for each of its sequences.
        dict(name="attn-gqa", op="attn", B=4, Hq=32, Hkv=8, NQ=1, len=32768, ragged=False, d=64, page=32,
             kind="bf16"),
        # Several tokens checked at once (drafts), causal among themselves: 20 query rows to a key head.
        dict(name="attn-drafts", op="attn", B=7, Hq=32, Hkv=8, NQ=5, len=12345, ragged=True, d=128, page=128,
             kind="e4m3"),
        # Divergence of two queries' attentions for one short sequence: latency.
        dict(name="kl-short", op="kl", B=1, Hq=16, Hkv=16, NQ=1, len=1000, ragged=False, d=64, page=16,
             kind="bf16", kind2="same"),
        # The decode workload itself, over pages.
        dict(name="kl-long", op="kl", B=1, Hq=16, Hkv=16, NQ=1, len=131072, ragged=False, d=128, page=64,
             kind="bf16", kind2="same"),
        # A student over a quantised cache against its teacher over the unquantised one, serving batch.
        dict(name="kl-drift", op="kl", B=16, Hq=32, Hkv=8, NQ=1, len=8192, ragged=True, d=128, page=64,
             kind="bf16", kind2="e4m3"),
        # The same, both quantised, a few new tokens, small heads, odd sizes.
        dict(name="kl-drafts", op="kl", B=5, Hq=24, Hkv=8, NQ=3, len=9999, ragged=True, d=64, page=32,
             kind="e4m3", kind2="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "attn", "attn", "kl", "kl"])
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    kind = rng.choice(["bf16", "e4m3"])
    Hkv = rng.choice([1, 2, 4, 8, 16, 32])
    if op == "write":
        B = _log(rng, 1, 64)
        NT = _log(rng, 1, max(1, (1 << 24) // (d * Hkv * B)))
        ctx = _log(rng, 1, 4000) if rng.random() < 0.5 else 0
        back = "all" if Hkv * B * (NT + ctx) * d <= 1 << 25 and rng.random() < 0.5 else "new"
        return dict(op=op, B=B, Hkv=Hkv, NT=NT, ctx=ctx, ragged=rng.random() < 0.7, d=d, page=page, kind=kind,
                    back=back)
    group = rng.choice([1, 2, 3, 4, 7, 8])
    NQ = min(rng.choice([1, 1, 1, 2, 3, 5, 8]), 32 // group)
    B = _log(rng, 1, 64)
    most = max(64, min(131072, (1 << 27) // (d * Hkv * B)))
    case = dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, NQ=NQ, len=_log(rng, 40, most), ragged=rng.random() < 0.6,
                d=d, page=page, kind=kind)
    if op == "kl":
        case["kind2"] = rng.choice(["same", "bf16", "e4m3"])
    return case


def _lengths(case):
    """Tokens of each sequence: in the cache for attention, to be written otherwise."""
    most, B = case["NT"] if case["op"] == "write" else case["len"], case["B"]
    if not case["ragged"] or B == 1:
        return [most] * B
    r = random.Random(most * 1009 + B)
    got = [r.randint(max(1, most // 16), most) for _ in range(B)]
    got[0] = most
    if B >= 4:
        got[B // 2] = 0    # a sequence that is finished: nothing to do for it
    return got


def _before(case):
    """Tokens of each sequence in the cache before the new ones are written."""
    ctx, B = case["ctx"], case["B"]
    if not case["ragged"] or ctx == 0:
        return [ctx] * B
    r = random.Random(ctx * 1013 + B)
    return [r.randint(0, ctx) for _ in range(B)]


def work(case):
    es = 2 if case["kind"] == "bf16" else 1 + 1 / case["d"]
    row = case["Hkv"] * case["d"]
    if case["op"] == "write":
        n = _lengths(case)
        back = n if case["back"] == "new" else [a + b for a, b in zip(n, _before(case))]
        return {"bytes": 2 * row * (sum(n) * (2 + es) + sum(back) * (es + 2)), "flops": 2 * row * (sum(n) + sum(back))}
    n, rows = sum(_lengths(case)), case["Hq"] * case["NQ"]
    small = case["B"] * rows * case["d"]
    if case["op"] == "attn":
        return {"bytes": 2 * row * es * n + 4 * small + 4 * case["B"] * rows, "flops": 4 * rows * case["d"] * n}
    es2 = 0 if case["kind2"] == "same" else 2 if case["kind2"] == "bf16" else 1 + 1 / case["d"]
    return {"bytes": row * (es + es2) * n + 4 * small + 12 * case["B"] * rows, "flops": 4 * rows * case["d"] * n}


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """Rows of fp32 in e4m3 with a power-of-two scale each: the largest finite value fits 448."""
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, e - 9 + (m > 0.875), LEAST).clamp(min=LEAST).to(torch.int32)
    inverse = ((127 - e) << 23).view(torch.float32)
    codes = (x * inverse.unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _values(codes, exp):
    return codes.to(torch.float32) * (exp.to(torch.int32) << 23).view(torch.float32).unsqueeze(-1)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _rows(g, *shape):
    """Keys or values: normal, with a few strong channels."""
    strong = 1 + 2 * (torch.rand(shape[-1], generator=g, device=DEV) < 0.05).float()
    return (_randn(g, *shape) * strong).to(torch.bfloat16)


def _cache(rows, kind):
    """[codes or bf16, exponents or None] of bf16 pages."""
    if kind == "bf16":
        return [rows, None]
    return list(_quantise(rows.float()))


def _table(g, lengths, page):
    """A page table over shuffled pages, and the number of pages (one more than it names)."""
    need = [-(-n // page) for n in lengths]
    total = sum(need)
    order = torch.randperm(total, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    width = max(1, max(need))
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)
    count = torch.tensor(need, device=DEV)
    at = torch.arange(width, device=DEV)
    inside = at[None] < count[:, None]
    table = torch.where(inside, order[(first[:, None] + at[None]).clamp(max=max(0, total - 1))] if total else NONE, NONE)
    return table.to(torch.int32).contiguous(), total + 1


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    s = dict(case)
    if case["op"] == "write":
        new, before = _lengths(case), _before(case)
        after = [a + b for a, b in zip(new, before)]
        s["table"], pages = _table(g, after, page)
        s["k_new"], s["v_new"] = _rows(g, B, Hkv, case["NT"], d), _rows(g, B, Hkv, case["NT"], d)
        s["start"], s["count"] = _ints(before), _ints(new)
        s["from"], s["back_count"] = (s["start"], s["count"]) if case["back"] == "new" else (_ints([0] * B), _ints(after))
        rows = case["NT"] if case["back"] == "new" else max(1, max(after))
        s["out"] = tuple(torch.zeros(B, Hkv, rows, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        s["k"], s["v"] = (_cache(_rows(g, pages, Hkv, page, d), case["kind"]) for _ in range(2))
        pairs = [("cache", s["k"], s["v"])]
    else:
        Hq, NQ = case["Hq"], case["NQ"]
        lengths = _lengths(case)
        s["table"], pages = _table(g, lengths, page)
        s["lengths"] = _ints(lengths)
        s["scale"] = 1.0 / math.sqrt(d)
        keys = _rows(g, pages, Hkv, page, d)
        s["k"] = _cache(keys, case["kind"])
        q = _randn(g, B, Hq, NQ, d)
        s["q"] = q.to(torch.bfloat16)
        if case["op"] == "attn":
            s["v"] = _cache(_rows(g, pages, Hkv, page, d), case["kind"])
            pairs = [("cache", s["k"], s["v"])]
        else:
            s["q2"] = (q + 0.5 * _randn(g, B, Hq, NQ, d)).to(torch.bfloat16)
            s["k2"] = s["k"] if case["kind2"] == "same" else _cache(keys, case["kind2"])
            pairs = [("cache", s["k"], [None, None]), ("cache2", s["k2"], [None, None])]
            if case["kind2"] != "same" and case["kind2"] == case["kind"]:
                # two caches of one kind: the second holds other keys, near the first's
                near = (keys.float() + 0.1 * _randn(g, pages, Hkv, page, d)).to(torch.bfloat16)
                s["k2"] = _cache(near, case["kind2"])
                pairs[1] = ("cache2", s["k2"], [None, None])
    if own:
        from attention_kl_divergence_02_b200 import binding
        for name, k, v in pairs:
            s[name] = s["cache"] if name == "cache2" and s["k2"] is s["k"] else binding.PagedCache(
                k[0], v[0], k_exp=k[1], v_exp=v[1])
        if case["op"] != "write":
            s["workspace"] = binding.paged_workspace(B, case["Hq"], Hkv, case["NQ"], d, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"write": _write, "attn": _attn, "kl": _kl}[s["op"]](s)


def _run_own(s):
    from attention_kl_divergence_02_b200 import binding
    if s["op"] == "write":
        binding.cache_append(s["cache"], s["k_new"], s["v_new"], s["table"], s["start"], count=s["count"])
        return binding.cache_gather(s["cache"], s["table"], s["back_count"], start=s["from"], out=s["out"])
    if s["op"] == "attn":
        return binding.paged_attn(s["q"], s["cache"], s["table"], s["lengths"], scale=s["scale"],
                                  workspace=s["workspace"])
    return binding.paged_kl(s["q"], s["cache"], s["q2"], s["cache2"], s["table"], s["lengths"], scale=s["scale"],
                            workspace=s["workspace"])


def _put(cache, rows, page, slot):
    """Writes rows [B, Hkv, NT, d] to (page, head, slot)."""
    rows = rows.permute(0, 2, 1, 3)      # [B, NT, Hkv, d]
    if cache[1] is None:
        cache[0][page, :, slot] = rows
    else:
        codes, exp = _quantise(rows.float())
        cache[0].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
        cache[1][page, :, slot] = exp


def _get(cache, page, slot):
    """Rows [B, Hkv, N, d] at (page, slot) [B, N], in fp32."""
    if cache[1] is None:
        return cache[0][page, :, slot].permute(0, 2, 1, 3).float()
    codes = cache[0].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
    return _values(codes, cache[1][page, :, slot]).permute(0, 2, 1, 3)


def _places(s, start, count, n):
    """(page, slot, valid) [B, n] of rows start .. start + n - 1; rows that count leaves out lie in the spare page."""
    i = torch.arange(n, device=DEV)
    pos = start[:, None].long() + i[None]
    valid = i[None] < count[:, None]
    at = (pos // s["page"]).clamp(max=s["table"].shape[1] - 1)
    page = torch.where(valid, torch.gather(s["table"].long(), 1, at), s["k"][0].shape[0] - 1)
    return page, pos % s["page"], valid


def _write(s):
    page, slot, _ = _places(s, s["start"], s["count"], s["NT"])
    _put(s["k"], s["k_new"], page, slot)
    _put(s["v"], s["v_new"], page, slot)
    page, slot, valid = _places(s, s["from"], s["back_count"], s["out"][0].shape[2])
    keep = valid[:, None, :, None]
    for cache, out in zip((s["k"], s["v"]), s["out"]):
        out.copy_(torch.where(keep, _get(cache, page, slot), out.float()))
    return s["out"]


def _seen(s):
    """[B, 1, rows, n]: whether a query row sees a key; the new tokens are a sequence's last."""
    n = s["table"].shape[1] * s["page"]
    i = torch.arange(s["Hq"] // s["Hkv"] * s["NQ"], device=DEV) % s["NQ"]
    last = s["lengths"][:, None] - (s["NQ"] - 1 - i)[None]
    return torch.arange(n, device=DEV)[None, None, None] < last[:, None, :, None]


def _all(s, cache):
    """Every sequence's rows [B, Hkv, n, d] in fp32, the table's whole width."""
    page = s["table"].clamp(min=0).long()
    rows = cache[0][page] if cache[1] is None else cache[0].view(torch.uint8)[page].view(torch.float8_e4m3fn)
    rows = rows.float() if cache[1] is None else _values(rows, cache[1][page])
    return rows.transpose(1, 2).flatten(2, 3)


def _scores(s, q, keys):
    q = q.float().view(s["B"], s["Hkv"], -1, s["d"])
    return (q @ keys.transpose(-1, -2)) * s["scale"]


def _softmax(x, seen):
    """(weights' numerators, their sums, log of the sums of exponentials); nothing seen: 0, 0 and -inf."""
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    return e, total, torch.log(total) + top


def _attn(s):
    seen = _seen(s)
    e, total, lse = _softmax(_scores(s, s["q"], _all(s, s["k"])), seen)
    values = _all(s, s["v"]) * (torch.arange(seen.shape[-1], device=DEV)[None] < s["lengths"][:, None])[:, None, :, None]
    out = (e @ values) / torch.where(total > 0, total, 1.0)
    shape = (s["B"], s["Hq"], s["NQ"])
    return out.view(*shape, s["d"]).to(torch.bfloat16), lse.view(shape)


def _kl(s):
    seen = _seen(s)
    x1 = _scores(s, s["q"], _all(s, s["k"]))
    x2 = _scores(s, s["q2"], _all(s, s["k2"]))
    e1, total, lse1 = _softmax(x1, seen)
    _, _, lse2 = _softmax(x2, seen)
    some = total > 0
    shift = torch.where(some, lse2 - lse1, 0.0)
    part = (e1 * torch.where(seen, x1 - x2 + shift, 0.0)).sum(-1, keepdim=True)
    kl = torch.where(some, part / torch.where(some, total, 1.0), 0.0)
    shape = (s["B"], s["Hq"], s["NQ"])
    return kl.view(shape), lse1.view(shape), lse2.view(shape)


# ------------------------------------------------------------------ 64 bits, from the definition
def _coarse(x):
    """What a row's values are after e4m3 with its power-of-two scale, in 64 bits."""
    size = x.abs().where(torch.isfinite(x), torch.zeros_like(x)).amax(-1, keepdim=True)
    e = torch.full_like(size, float(LEAST))
    for k in range(LEAST, 121):     # the smallest exponent with size <= 448 * 2^k
        e = torch.where((size > 448.0 * 2.0 ** (k - 1)) & (k > LEAST), float(k), e)
    unit = torch.exp2(e)
    y = (x / unit).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * unit


def _wide(cache):
    rows = cache[0].double()
    return rows if cache[1] is None else rows * torch.exp2(cache[1].double() - 127).unsqueeze(-1)


def _sequence(wide, table, n, page):
    """One sequence's rows [Hkv, n, d]."""
    got = wide[table[: -(-n // page)].long()]
    return got.transpose(0, 1).reshape(wide.shape[1], -1, wide.shape[3])[:, :n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        outs = [torch.zeros(o.shape, dtype=torch.float64, device=DEV) for o in s["out"]]
        for b, (c, n) in enumerate(zip(_before(case), _lengths(case))):
            for out, new, old in zip(outs, (s["k_new"], s["v_new"]), (s["k"], s["v"])):
                fresh = new[b, :, :n].double()
                if n and case["kind"] == "e4m3":
                    fresh = _coarse(fresh)
                if case["back"] == "new":
                    out[b, :, :n] = fresh
                else:
                    if c:
                        out[b, :, :c] = _sequence(_wide(old), s["table"][b], c, case["page"])
                    out[b, :, c:c + n] = fresh
        return tuple(outs)
    B, Hq, NQ, d, group = case["B"], case["Hq"], case["NQ"], case["d"], case["Hq"] // case["Hkv"]
    like = dict(dtype=torch.float64, device=DEV)
    lse = [torch.full((B, Hq, NQ), -math.inf, **like) for _ in range(2)]
    kl, out = torch.zeros(B, Hq, NQ, **like), torch.zeros(B, Hq, NQ, d, **like)
    caches = [s["k"], s["v"] if case["op"] == "attn" else s["k2"]]
    for b, n in enumerate(_lengths(case)):
        if not n:
            continue
        pages = s["table"][b, : -(-n // case["page"])].long()
        rows = [_sequence(_wide([c[0].view(torch.uint8)[pages].view(c[0].dtype) if c[1] is not None else c[0][pages],
                                 None if c[1] is None else c[1][pages]]),
                          torch.arange(len(pages), device=DEV), n, case["page"]).repeat_interleave(group, 0) for c in caches]
        for i in range(NQ):
            m = n - (NQ - 1 - i)
            if m < 1:
                continue
            a = torch.einsum("hd,hkd->hk", s["q"][b, :, i].double(), rows[0][:, :m]) * s["scale"]
            lse[0][b, :, i] = torch.logsumexp(a, -1)
            p = torch.log_softmax(a, -1)
            if case["op"] == "attn":
                out[b, :, i] = torch.einsum("hk,hkd->hd", p.exp(), rows[1][:, :m])
            else:
                c = torch.einsum("hd,hkd->hk", s["q2"][b, :, i].double(), rows[1][:, :m]) * s["scale"]
                lse[1][b, :, i] = torch.logsumexp(c, -1)
                kl[b, :, i] = (p.exp() * (p - torch.log_softmax(c, -1))).sum(-1)
    return (out, lse[0]) if case["op"] == "attn" else (kl, lse[0], lse[1])
