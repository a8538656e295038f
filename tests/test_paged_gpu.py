"""Paged key-value cache: append and read back, attention of new tokens, KL divergence over pages, each
against its 64-bit form on poisoned caches (NaN in everything no sequence owns)."""
import math

import pytest
import torch

from attention_kl_divergence_02_b200 import binding

import paged_ref as ref

pytestmark = pytest.mark.gpu


def status():
    return binding.streamkl_device_status()


def workspace(B, Hq, Hkv, NQ, d):
    """NaN behind the counters."""
    ws = binding.paged_workspace(B, Hq, Hkv, NQ, d)
    ws[binding.PAGED_COUNTER_BYTES // 4:] = float("nan")
    return ws


def counters_are_zero(ws):
    return not bool(ws[:binding.PAGED_COUNTER_BYTES // 4].view(torch.int32).any())


def rows(lengths):
    """New rows [B, Hkv, NT, d] as the calls take them."""
    return max(1, max(lengths))


# ------------------------------------------------------------------ append and read back
WRITE = [
    # Hkv, d, page, kind, starts, counts
    (2, 128, 64, "e4m3", [0], [1]),
    (2, 64, 16, "e4m3", [0, 15, 16, 17, 100], [33, 1, 0, 50, 16]),
    (3, 128, 16, "bf16", [5, 0, 31], [64, 7, 1]),
    (1, 64, 256, "bf16", [255, 256, 1], [2, 300, 1000]),
    (8, 128, 32, "e4m3", [0, 77], [777, 3]),
]


@pytest.mark.parametrize("case", WRITE, ids=lambda c: "h%dd%dp%d%s" % c[:4])
def test_append_and_gather(case):
    Hkv, d, page, kind, starts, counts = case
    B, NT = len(starts), max(counts) + 2        # rows behind every count, NaN: never used
    after = [s + c for s, c in zip(starts, counts)]
    c = ref.Case(after, Hkv, d, page, kind, seed=3)
    old = [x.clone() for x in c.kc], [x.clone() for x in c.vc]
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    new = []
    for _ in range(2):
        x = torch.randn((B, Hkv, NT, d), generator=g, device="cuda")
        x = x * torch.exp2(torch.randint(-20, 21, (B, Hkv, NT, 1), generator=g, device="cuda").float())
        for b in range(B):
            x[b, :, counts[b]:] = float("nan")
        new.append(x.to(torch.bfloat16))
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    bits = torch.int16 if kind == "bf16" else torch.uint8
    before = c.cache.k.view(bits).clone()
    binding.cache_append(c.cache, new[0], new[1], c.table, start, count=count)
    rows_back = max(after) + 1
    out = tuple(torch.full((B, Hkv, rows_back, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = binding.cache_gather(c.cache, c.table, c.len, out=out)
    assert status() == binding.OK
    for x, fresh, kept in zip(got, new, old):
        for b in range(B):
            s, n = starts[b], counts[b]
            want = kept[b].clone()
            if n:
                want[:, s:s + n] = ref.dequantise(*ref.quantise(fresh[b, :, :n])) if kind == "e4m3" else fresh[b, :, :n].double()
            assert torch.equal(x[b, :, :after[b]].double(), want), b
            assert bool((x[b, :, after[b]:] == 7.0).all()), b
    # nothing but the new rows was written
    touched = torch.zeros(c.cache.k.shape[:3], dtype=torch.bool, device="cuda")
    for b in range(B):
        for i in range(starts[b], after[b]):
            touched[int(c.table[b, i // page]), :, i % page] = True
    assert torch.equal(c.cache.k.view(bits)[~touched], before[~touched])
    # from a position, into rows of its own
    part = binding.cache_gather(c.cache, c.table, count, start=start, rows=NT)
    for b in range(B):
        assert torch.equal(part[0][b, :, :counts[b]], got[0][b, :, starts[b]:after[b]])
        assert not bool(part[1][b, :, counts[b]:].any())


def test_quantised_rows_at_the_edges_of_the_types():
    """Zeros, the largest and smallest bf16 values, values at rounding ties, infinities and NaN."""
    d = 64
    x = torch.zeros((16, d))
    top = torch.finfo(torch.bfloat16).max
    x[1] = top
    x[2, 0], x[2, 1] = top, 1.0
    x[3] = 2.0 ** -133                      # smallest subnormal
    x[4] = torch.linspace(-448, 448, d)
    x[5, :4] = torch.tensor([448.0, 450.0, -2.0 ** -9, 2.0 ** -10])
    x[6, :4] = torch.tensor([448.0, 17.0, 19.0, -21.0])      # ties between codes
    x[7, :3] = torch.tensor([math.inf, -math.inf, 3.0])
    x[8, :2] = torch.tensor([math.nan, 5.0])
    x[9] = math.inf
    x[10] = 2.0 ** -96 * 448
    x[11] = 2.0 ** -106
    x[12, :2] = torch.tensor([448.0 * 2.0 ** 3, 449.0 * 2 ** -20])
    x[13] = 1.0 / 3
    x = x.to(torch.bfloat16).cuda().view(1, 1, 16, d)
    cache = binding.PagedCache.empty(2, 1, 16, d, quantised=True)
    table = torch.ones((1, 1), dtype=torch.int32, device="cuda")
    zero, n = (torch.full((1,), v, dtype=torch.int32, device="cuda") for v in (0, 16))
    binding.cache_append(cache, x, -x, table, zero)
    k, v = binding.cache_gather(cache, table, n, rows=16)
    codes, e = ref.quantise(x[0])
    want = ref.dequantise(codes, e)
    assert torch.equal(cache.k_exp[1].double() - 127, e)
    assert bool((cache.k_exp[0] == 127).all()) and not bool(cache.k[0].view(torch.uint8).any())
    assert torch.equal(torch.isnan(k[0].double()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(k[0].double(), nan=0.5), torch.nan_to_num(want, nan=0.5))
    assert torch.equal(torch.nan_to_num(-v[0].double(), nan=0.5), torch.nan_to_num(want, nan=0.5))


# ------------------------------------------------------------------ attention
ATTN = [
    # Hq, Hkv, NQ, d, page, kind, causal, lengths
    (8, 8, 1, 128, 64, "bf16", True, [1]),
    (8, 2, 1, 128, 16, "bf16", True, [0, 1, 15, 16, 17, 63, 64, 65, 300]),
    (8, 2, 1, 64, 16, "e4m3", True, [0, 1, 15, 16, 17, 63, 64, 65, 300]),
    (4, 4, 1, 128, 128, "e4m3", True, [5000]),                 # cut over many CTAs
    (2, 1, 1, 64, 32, "bf16", True, [20000, 3, 0, 129]),
    (32, 8, 1, 128, 64, "e4m3", True, [1000, 0, 77, 2048, 1, 640, 63, 64]),
    (9, 1, 1, 128, 16, "bf16", True, [333, 1]),                # 9 rows: two blocks of 8
    (4, 1, 4, 64, 64, "bf16", True, [1, 2, 3, 4, 5, 17, 700]),  # fewer keys than new tokens
    (4, 1, 4, 64, 64, "e4m3", False, [1, 2, 3, 4, 5, 17, 700]),
    (14, 2, 5, 128, 32, "e4m3", True, [40, 4, 3000]),          # 35 rows: two blocks of 32
    (6, 2, 5, 128, 16, "bf16", True, [40, 4, 0, 2000]),        # 15 rows
    (8, 1, 4, 128, 16, "bf16", True, [100, 31, 1601]),         # 32 rows
    (1, 1, 33, 64, 1024, "bf16", True, [10, 33, 1025]),
    (3, 1, 1, 64, 16, "e4m3", True, list(range(200))),         # many sequences, each whole
    (4, 2, 1, 64, 16, "bf16", True, [37 * i % 1500 for i in range(70)]),   # many, in shares
    (8, 1, 2, 128, 16, "e4m3", True, [513, 1, 130]),           # 16 rows
    (8, 1, 3, 128, 32, "bf16", True, [513, 2, 130]),           # 24 rows
    (8, 1, 4, 64, 32, "e4m3", True, [900, 3, 131]),            # 32 rows
    (8, 1, 4, 128, 32, "e4m3", False, [900, 3, 131]),
    (16, 16, 1, 64, 1024, "e4m3", True, [65600]),              # more turns than a batch of page entries
    (16, 16, 1, 128, 1024, "bf16", True, [62001]),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "q%dkv%dn%dd%dp%d%s%sB%d" % (*c[:6], "c" if c[6] else "", len(c[7])))
def test_attention(case):
    Hq, Hkv, NQ, d, page, kind, causal, lengths = case
    c = ref.Case(lengths, Hkv, d, page, kind, seed=11)
    q = ref.queries(len(lengths), Hq, NQ, d, seed=12)
    scale = 0.9 / math.sqrt(d)
    ws = workspace(len(lengths), Hq, Hkv, NQ, d)
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len, scale=scale, causal=causal, workspace=ws)
    assert status() == binding.OK
    assert counters_are_zero(ws)
    want, want_lse, tol, tol_lse = ref.attention(c, q, scale, causal)
    ref.close(out, want, tol, "out")
    ref.close(lse, want_lse, tol_lse, "lse")
    again = binding.paged_attn(q, c.cache, c.table, c.len, scale=scale, causal=causal)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)     # the same bits


def test_attention_over_rows_of_very_different_size():
    """e4m3 scales between 2^-70 and 2^70 in one sequence: the weights carry them."""
    c = ref.Case([700, 45], 2, 128, 16, "e4m3", seed=4)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    for b, n in enumerate(c.lengths):
        e = torch.randint(-60, 61, (1, n, 1), generator=g, device="cuda").float()
        c.v[b] = (c.v[b].float() * torch.exp2(e)).to(torch.bfloat16)
    c.fill()
    q = ref.queries(2, 8, 1, 128, seed=5)
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len)
    want, want_lse, tol, tol_lse = ref.attention(c, q, 128 ** -0.5, True)
    ref.close(out, want, tol, "out")
    ref.close(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_of_large_and_tiny_queries(kind):
    """Query rows of sizes 2^-60 to 2^6, one of zeros; scores of one row far apart (weights underflow)."""
    c = ref.Case([500], 2, 64, 32, kind, seed=6)
    q = ref.queries(1, 8, 1, 64, seed=7).float()
    q[0, 0], q[0, 1], q[0, 2] = q[0, 0] * 2.0 ** -60, q[0, 1] * 2.0 ** 6, 0.0
    q = q.to(torch.bfloat16)
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len)
    want, want_lse, tol, tol_lse = ref.attention(c, q, 0.125, True)
    ref.close(out, want, tol, "out")
    ref.close(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("kind,NQ", [("bf16", 4), ("e4m3", 4), ("bf16", 40), ("e4m3", 40)])
def test_values_behind_a_rows_limit_do_not_reach_it(kind, NQ):
    """The newest tokens' keys and values are NaN (bf16: and infinite): rows that do not see them keep
    their results, rows that see them are NaN."""
    n = 85                        # the limits lie inside a tile
    blind = NQ - 2                # the rows before do not see token n - 2
    c = ref.Case([n], 2, 128, 16, kind, seed=8)
    q = ref.queries(1, 4, NQ, 128, seed=9)
    want = binding.paged_attn(q, c.cache, c.table, c.len)
    page, slot = int(c.table[0, (n - 2) // 16]), (n - 2) % 16
    if kind == "bf16":
        c.cache.v[page, :, slot, ::3] = math.inf
        c.cache.v[page, :, slot, 1::3] = math.nan
        c.cache.k[page, 1, slot, 5] = math.nan
    else:
        c.cache.v.view(torch.uint8)[page, :, slot] = 0x7f
        c.cache.k.view(torch.uint8)[page, 1, slot, 5] = 0xff
    got = binding.paged_attn(q, c.cache, c.table, c.len)
    assert status() == binding.OK
    assert torch.equal(got[0][:, :, :blind], want[0][:, :, :blind])
    assert torch.equal(got[1][:, :, :blind], want[1][:, :, :blind])
    seen = got[0][:, :, blind:]
    assert not bool(torch.isfinite(seen[..., 1::3]).any()) and not bool(torch.isfinite(seen[..., ::3]).any())
    assert bool(torch.isnan(got[1][0, 2:, blind:]).all()) and torch.equal(got[1][0, :2], want[1][0, :2])


def test_pages_and_lengths_outside_the_cache():
    """Recorded, and no memory is touched: such keys count as masked, lengths are clamped."""
    c = ref.Case([100, 64, 50], 2, 64, 16, "bf16", seed=10)
    q = ref.queries(3, 4, 1, 64, seed=11)
    good = c.table.clone()
    c.table[0, 2], c.table[0, 4] = c.pages, -7          # keys 32..47 and 64..79 of sequence 0
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len)
    assert status() == binding.ERR_PAGE and status() == binding.OK
    for pool in (c.kc, c.vc):
        pool[0] = torch.cat([pool[0][:, :32], pool[0][:, 48:64], pool[0][:, 80:]], 1)
    c.lengths[0] = 68
    want, want_lse, tol, tol_lse = ref.attention(c, q, 0.125, True)
    ref.close(out, want, tol, "out")
    ref.close(lse, want_lse, tol_lse, "lse")
    kl = binding.paged_kl(q, c.cache, q, c.cache, c.table, c.len)
    assert status() == binding.ERR_PAGE
    ref.close(kl[1], want_lse, tol_lse, "lse")
    # a length beyond the table, and a negative one
    wide = torch.tensor([10 ** 9, 64, -5], dtype=torch.int32, device="cuda")
    full = torch.tensor([c.table.shape[1] * 16, 64, 0], dtype=torch.int32, device="cuda")
    good[0, :] = good[1, 0]
    a = binding.paged_attn(q, c.cache, good, wide)
    assert status() == binding.ERR_PAGE
    b = binding.paged_attn(q, c.cache, good, full)
    assert status() == binding.OK
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # append and gather: nothing written, nothing read
    new = torch.ones((3, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    kept = c.cache.k.view(torch.int16).clone()
    for start in ([98, -1, 10 ** 9], [33, 2 ** 31 - 2, -2 ** 31]):
        s = torch.tensor(start, dtype=torch.int32, device="cuda")
        table = torch.full_like(c.table, c.pages)
        binding.cache_append(c.cache, new, new, table, s)
        assert status() == binding.ERR_PAGE
        assert torch.equal(c.cache.k.view(torch.int16), kept)
        n = torch.full((3,), 4, dtype=torch.int32, device="cuda")
        k, _ = binding.cache_gather(c.cache, table, n, start=s, rows=4)
        assert status() == binding.ERR_PAGE and not bool(k.any())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_beyond_32_bits(kind):
    """A pool of more than 2^32 elements (and bytes): a sequence in its last pages."""
    Hkv, page, d = 8, 1024, 128
    pages = (1 << 32) // (Hkv * page * d) + 3
    c = ref.Case([2500], Hkv, d, page, kind, seed=13)
    dtype = c.cache.k.dtype
    pools = [torch.empty((pages, Hkv, page, d), dtype=dtype, device="cuda") for _ in range(2)]
    exps = [None, None]
    if kind == "e4m3":
        exps = [torch.empty((pages, Hkv, page), dtype=torch.uint8, device="cuda") for _ in range(2)]
    shift = pages - c.pages
    bits = torch.int16 if kind == "bf16" else torch.uint8
    for pool, old in zip(pools, (c.cache.k, c.cache.v)):
        pool[shift:].view(bits).copy_(old.view(bits))
    if kind == "e4m3":
        exps[0][shift:], exps[1][shift:] = c.cache.k_exp, c.cache.v_exp
    big = binding.PagedCache(pools[0], pools[1], k_exp=exps[0], v_exp=exps[1])
    q = ref.queries(1, 16, 1, d, seed=14)
    far = torch.where(c.table >= 0, c.table + shift, c.table)
    a, b = binding.paged_attn(q, c.cache, c.table, c.len), binding.paged_attn(q, big, far, c.len)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q2 = ref.queries(1, 16, 1, d, seed=15, near=q)
    a, b = binding.paged_kl(q, c.cache, q2, c.cache, c.table, c.len), binding.paged_kl(q, big, q2, big, far, c.len)
    assert torch.equal(a[0], b[0])
    x = binding.cache_gather(c.cache, c.table, c.len, rows=2500)
    binding.cache_append(big, x[1], x[0], far, torch.zeros(1, dtype=torch.int32, device="cuda"))
    y = binding.cache_gather(big, far, c.len, rows=2500)
    assert torch.equal(x[0], y[1]) and torch.equal(x[1], y[0])
    assert status() == binding.OK


# ------------------------------------------------------------------ divergence
KL = [
    # Hq, Hkv, NQ, d, page, kind1, kind2, causal, lengths
    (8, 8, 1, 128, 64, "bf16", "same", True, [1]),
    (8, 2, 1, 128, 16, "bf16", "same", True, [0, 1, 15, 16, 17, 63, 64, 65, 300]),
    (8, 2, 1, 64, 16, "e4m3", "same", True, [0, 1, 15, 16, 17, 63, 64, 65, 300]),
    (4, 4, 1, 128, 128, "bf16", "e4m3", True, [5000, 3]),
    (4, 4, 1, 64, 64, "e4m3", "bf16", True, [700, 0, 64]),
    (4, 2, 1, 128, 32, "e4m3", "e4m3", True, [9000]),
    (4, 2, 1, 64, 32, "bf16", "bf16", True, [20000, 3, 0, 129]),
    (9, 1, 1, 128, 16, "bf16", "bf16", True, [333, 1]),
    (4, 1, 4, 64, 64, "bf16", "e4m3", True, [1, 2, 3, 4, 5, 17, 700]),
    (4, 1, 4, 64, 64, "e4m3", "same", False, [1, 2, 3, 4, 5, 17, 700]),
    (14, 2, 5, 128, 32, "e4m3", "bf16", True, [40, 4, 3000]),
    (8, 1, 4, 128, 16, "bf16", "same", True, [100, 31, 1601]),
    (3, 1, 1, 64, 16, "bf16", "e4m3", True, list(range(200))),
    (4, 2, 1, 64, 16, "bf16", "same", True, [37 * i % 1500 for i in range(70)]),
    (8, 1, 5, 128, 32, "bf16", "bf16", True, [900, 3, 131]),   # 40 rows: blocks of 16
    (16, 16, 1, 64, 1024, "e4m3", "bf16", True, [65600]),
    (16, 16, 1, 128, 1024, "bf16", "same", True, [62001]),
]


def pair(lengths, Hkv, d, page, kind1, kind2, seed):
    """Two cases over one table; the second's keys near the first's."""
    c1 = ref.Case(lengths, Hkv, d, page, kind1, seed)
    if kind2 == "same":
        return c1, c1
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    keys = c1.k if kind1 != kind2 else [
        (k.float() + 0.2 * torch.randn(k.shape, generator=g, device="cuda")).to(torch.bfloat16) for k in c1.k]
    return c1, ref.Case(lengths, Hkv, d, page, kind2, seed + 2, keys=keys, table=c1.table)


@pytest.mark.parametrize("case", KL, ids=lambda c: "q%dkv%dn%dd%dp%d%s_%s%sB%d" % (*c[:7], "c" if c[7] else "", len(c[8])))
def test_divergence(case):
    Hq, Hkv, NQ, d, page, kind1, kind2, causal, lengths = case
    c1, c2 = pair(lengths, Hkv, d, page, kind1, kind2, seed=21)
    q1 = ref.queries(len(lengths), Hq, NQ, d, seed=22)
    q2 = ref.queries(len(lengths), Hq, NQ, d, seed=23, near=q1)
    scale = 0.9 / math.sqrt(d)
    ws = workspace(len(lengths), Hq, Hkv, NQ, d)
    got = binding.paged_kl(q1, c1.cache, q2, c2.cache, c1.table, c1.len, scale=scale, causal=causal, workspace=ws)
    assert status() == binding.OK
    assert counters_are_zero(ws)
    kl, lse1, lse2, tol, tol_lse = ref.divergence(c1, q1, c2, q2, scale, causal)
    ref.close(got[0], kl, tol, "kl")
    ref.close(got[1], lse1, tol_lse, "lse1")
    ref.close(got[2], lse2, tol_lse, "lse2")
    again = binding.paged_kl(q1, c1.cache, q2, c2.cache, c1.table, c1.len, scale=scale, causal=causal)
    assert all(torch.equal(a, b) for a, b in zip(again, got))


def test_divergence_of_equal_attentions_is_zero():
    """The same queries over one cache, d log2 units of acc cancel exactly."""
    c = ref.Case([3000, 17], 2, 128, 64, "bf16", seed=24)
    q = ref.queries(2, 8, 1, 128, seed=25)
    kl, lse1, lse2 = binding.paged_kl(q, c.cache, q, c.cache, c.table, c.len)
    assert not bool(kl.any()) and torch.equal(lse1, lse2)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("quantised", [False, True])
def test_a_run_of_them_together(quantised):
    """A teacher's and a student's caches filled token by token behind their prompts; each step's
    attention and divergence agree with the 64-bit forms, and the read-back keys give the dense
    forward the same divergence."""
    B, Hq, Hkv, d, page, steps = 3, 8, 2, 128, 16, 4
    prompt = [37, 1, 64]
    final = [n + steps for n in prompt]
    kind = "e4m3" if quantised else "bf16"
    c1, c2 = pair(final, Hkv, d, page, "bf16", kind, seed=31)
    caches = [binding.PagedCache.empty(c1.pages, Hkv, page, d, quantised=x) for x in (False, quantised)]
    width = rows(prompt)
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    count = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    for c, cache in zip((c1, c2), caches):
        k = torch.zeros((B, Hkv, width, d), dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        for b in range(B):
            k[b, :, :prompt[b]], v[b, :, :prompt[b]] = c.k[b][:, :prompt[b]], c.v[b][:, :prompt[b]]
        binding.cache_append(cache, k, v, c1.table, start, count=count)
    lengths = count.clone()
    ws = binding.paged_workspace(B, Hq, Hkv, 1, d)
    scale = d ** -0.5
    for step in range(steps):
        q1 = ref.queries(B, Hq, 1, d, seed=40 + step)
        q2 = ref.queries(B, Hq, 1, d, seed=50 + step, near=q1)
        for c, cache in zip((c1, c2), caches):
            k = torch.stack([c.k[b][:, prompt[b] + step] for b in range(B)]).unsqueeze(2).contiguous()
            v = torch.stack([c.v[b][:, prompt[b] + step] for b in range(B)]).unsqueeze(2).contiguous()
            binding.cache_append(cache, k, v, c1.table, lengths)
        lengths += 1
        out, lse = binding.paged_attn(q2, caches[1], c1.table, lengths, workspace=ws)
        got = binding.paged_kl(q1, caches[0], q2, caches[1], c1.table, lengths, workspace=ws)
        now = [n + step + 1 for n in prompt]
        c1.lengths = c2.lengths = now
        want, want_lse, tol, tol_lse = ref.attention(c2, q2, scale, True)
        ref.close(out, want, tol, "out")
        ref.close(lse, want_lse, tol_lse, "lse")
        kl, lse1, lse2, tol, tol_lse = ref.divergence(c1, q1, c2, q2, scale, True)
        ref.close(got[0], kl, tol, "kl")
        ref.close(got[2], lse, tol_lse * 2, "lse of both calls")
    assert status() == binding.OK
    # the dense forward over one sequence's read-back keys, without padding
    for b in range(B):
        one = c1.table[b:b + 1].contiguous()
        n = lengths[b:b + 1].contiguous()
        k1 = binding.cache_gather(caches[0], one, n, rows=final[b])[0]
        k2 = binding.cache_gather(caches[1], one, n, rows=final[b])[0]
        dense = binding.fwd(q1[b:b + 1].contiguous(), k1, q2[b:b + 1].contiguous(), k2)
        assert float((dense[0] - got[0][b:b + 1]).abs().max()) <= 1e-4      # the dense kernel's own 2.7e-6 exp2
        assert float((dense[1] - got[1][b:b + 1]).abs().max()) <= 1e-4


def test_graph_replays_on_new_lengths_pages_and_rows():
    """One captured step (append, attention, divergence), replayed while lengths and tables change in
    place; two graphs share a workspace."""
    B, Hq, Hkv, d, page = 2, 4, 2, 64, 16
    c = ref.Case([300, 41], Hkv, d, page, "e4m3", seed=61)
    q = ref.queries(B, Hq, 1, d, seed=62)
    q2 = ref.queries(B, Hq, 1, d, seed=63, near=q)
    lengths = torch.tensor([120, 7], dtype=torch.int32, device="cuda")
    table = c.table.clone()
    ws = binding.paged_workspace(B, Hq, Hkv, 1, d)
    out = (torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda"))
    kls = tuple(torch.empty((B, Hq, 1), device="cuda") for _ in range(3))

    def attn():
        binding.paged_attn(q, c.cache, table, lengths, out=out, workspace=ws)

    def kl():
        binding.paged_kl(q, c.cache, q2, c.cache, table, lengths, out=kls, workspace=ws)

    graphs = []
    for f in (attn, kl):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            f()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for now in ([120, 7], [300, 41], [0, 1], [64, 0]):
        lengths.copy_(torch.tensor(now, dtype=torch.int32))
        for t in (*out, *kls):
            t.fill_(float("nan"))
        for g in graphs:
            g.replay()
        c.lengths = now
        want, want_lse, tol, tol_lse = ref.attention(c, q, d ** -0.5, True)
        ref.close(out[0], want, tol, "out")
        ref.close(out[1], want_lse, tol_lse, "lse")
        want, lse1, lse2, tol, tol_lse = ref.divergence(c, q, c, q2, d ** -0.5, True)
        ref.close(kls[0], want, tol, "kl")
    table.copy_(table.flip(0))           # the sequences change places
    lengths.copy_(torch.tensor([41, 300], dtype=torch.int32))
    graphs[0].replay()
    eager = binding.paged_attn(q, c.cache, table, lengths)
    assert torch.equal(out[0], eager[0]) and status() == binding.OK


def test_on_another_stream():
    """Allocations and launches belong to the stream that is named, by object or by handle."""
    c = ref.Case([2000, 33], 2, 128, 16, "bf16", seed=71)
    q = ref.queries(2, 8, 1, 128, seed=72)
    want = binding.paged_attn(q, c.cache, c.table, c.len)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        for _ in range(3):
            got = binding.paged_attn(q, c.cache, c.table, c.len, stream=handle)
            kl = binding.paged_kl(q, c.cache, q, c.cache, c.table, c.len, stream=handle)
            back = binding.cache_gather(c.cache, c.table, c.len, rows=2000, stream=handle)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not bool(kl[0].any()) and float((kl[1] - want[1]).abs().max()) <= 1e-5
        assert torch.equal(back[0][1, :, :33], c.k[1])


def test_two_streams_at_once():
    """Two calls that overlap, each with its own workspace."""
    c = ref.Case([9000, 300, 4000], 4, 128, 64, "e4m3", seed=81)
    q = [ref.queries(3, 8, 1, 128, seed=82 + i) for i in range(2)]
    want = [binding.paged_attn(x, c.cache, c.table, c.len) for x in q]
    spaces = [workspace(3, 8, 4, 1, 128) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = binding.paged_attn(q[i], c.cache, c.table, c.len, workspace=spaces[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])
        assert counters_are_zero(spaces[i])


def test_sequences_share_pages():
    """Two sequences with a common prefix of pages, one twice in the batch."""
    c = ref.Case([200, 200, 90], 2, 64, 16, "bf16", seed=91)
    table = c.table.clone()
    table[1] = table[0]                       # the same 200 keys
    table[2, :3] = table[0, :3]               # 48 keys of the first, then its own
    c.kc[1], c.vc[1] = c.kc[0], c.vc[0]
    for pool in (c.kc, c.vc):
        pool[2] = torch.cat([pool[0][:, :48], pool[2][:, 48:]], 1)
    q = ref.queries(3, 4, 1, 64, seed=92)
    out, lse = binding.paged_attn(q, c.cache, table, c.len)
    want, want_lse, tol, tol_lse = ref.attention(c, q, 0.125, True)
    ref.close(out, want, tol, "out")
    ref.close(lse, want_lse, tol_lse, "lse")


def test_one_workspace_for_calls_of_any_size():
    big = workspace(8, 64, 2, 1, 128)
    for Hq, Hkv, d, lengths, seed in ((64, 2, 128, [3000] * 8, 1), (2, 2, 64, [5000], 2), (8, 2, 128, [700, 64], 3),
                                      (64, 2, 128, [3000] * 8, 1)):
        c = ref.Case(lengths, Hkv, d, 64, "bf16", seed=100 + seed)
        q = ref.queries(len(lengths), Hq, 1, d, seed=110 + seed)
        own = binding.paged_attn(q, c.cache, c.table, c.len)
        got = binding.paged_attn(q, c.cache, c.table, c.len, workspace=big)
        kl = binding.paged_kl(q, c.cache, q, c.cache, c.table, c.len, workspace=big)
        assert torch.equal(got[0], own[0]) and torch.equal(got[1], own[1]) and not bool(kl[0].any())
        assert counters_are_zero(big)


@pytest.mark.parametrize("fast", [True, False])
def test_refusals(fast, monkeypatch):
    """Tensors that the kernels would misread, by the extension's path and by the plain one."""
    if not fast:
        monkeypatch.setattr(binding, "_fast", None)
    c = ref.Case([40, 20], 2, 64, 16, "bf16", seed=120)
    q = ref.queries(2, 4, 1, 64, seed=121)
    ws = workspace(2, 4, 2, 1, 64)
    new = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    want = binding.paged_attn(q, c.cache, c.table, c.len)
    got = binding.paged_attn(q, c.cache, c.table, c.len, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for bad in (q.float(), q[:1], q[..., :32], q.transpose(1, 2), q[:, :3].contiguous(), q.cpu(), q[0]):
        with pytest.raises(ValueError):
            binding.paged_attn(bad, c.cache, c.table, c.len, workspace=ws)
        with pytest.raises(ValueError):
            binding.paged_kl(q, c.cache, bad, c.cache, c.table, c.len, workspace=ws)
    for table in (c.table.long(), c.table[:1], c.table.t().contiguous().t(), c.table[0], c.table.cpu()):
        with pytest.raises(ValueError):
            binding.paged_attn(q, c.cache, table, c.len, workspace=ws)
        with pytest.raises(ValueError):
            binding.cache_append(c.cache, new, new, table, zero)
        with pytest.raises(ValueError):
            binding.cache_gather(c.cache, table, c.len, out=(new, new))
    for lengths in (c.len.long(), c.len[:1], c.len.cpu()):
        with pytest.raises(ValueError):
            binding.paged_attn(q, c.cache, c.table, lengths, workspace=ws)
        with pytest.raises(ValueError):
            binding.cache_append(c.cache, new, new, c.table, lengths)
    for space in (ws[::2], ws.half(), ws.cpu()):
        with pytest.raises(ValueError):
            binding.paged_attn(q, c.cache, c.table, c.len, workspace=space)
    with pytest.raises(binding.StreamKLError):        # too small: the library's own check
        binding.paged_attn(q, c.cache, c.table, c.len, workspace=ws[:64].contiguous())
    with pytest.raises(binding.StreamKLError):
        binding.paged_attn(q, c.cache, c.table, c.len, scale=-1.0, workspace=ws)
    for rows_ in (new[:, :1].contiguous(), new.float(), new[..., :32].contiguous(), new.transpose(2, 3)):
        with pytest.raises(ValueError):
            binding.cache_append(c.cache, rows_, rows_, c.table, zero)
    keys = binding.PagedCache(c.cache.k)
    with pytest.raises(ValueError):
        binding.paged_attn(q, keys, c.table, c.len, workspace=ws)
    with pytest.raises(ValueError):
        binding.cache_append(keys, new, new, c.table, zero)
    kl = binding.paged_kl(q, keys, q, keys, c.table, c.len, workspace=ws)
    assert not bool(kl[0].any()) and status() == binding.OK
    other = binding.PagedCache.empty(c.pages + 1, 2, 16, 64)
    with pytest.raises((ValueError, binding.StreamKLError)):
        binding.paged_kl(q, c.cache, q, other, c.table, c.len, workspace=ws)
