"""Paged attention and divergence where a small error would not show among random keys: many small weights
beside a large one, scores far beyond the usual, keys and queries of extreme and opposite size, and every value
tile of a long sequence accounted for."""
import math

import pytest
import torch

from attention_kl_divergence_02_b200 import binding

import paged_ref as ref

pytestmark = pytest.mark.gpu


def shared_rows(case, B):
    """Table and lengths of B sequences that all are the case's only one."""
    return case.table.expand(B, -1).contiguous(), case.len.expand(B).contiguous()


# ------------------------------------------------------------------ one strong key, many weak ones
@pytest.mark.parametrize("d,Hq,n,B", [(64, 1, 1 << 20, 448), (128, 20, 1 << 18, 300)])
def test_many_weak_keys_beside_a_strong_one(d, Hq, n, B):
    """One key outweighs each of the others by 2^25.2, their values are 16 times its own, and enough
    sequences share the pages that a CTA folds a whole one: what one warp leaves out of the weighted
    sum, but not of the sum of weights, shows as a bias."""
    c = ref.Case([n], 1, d, 1024, "e4m3", seed=1)
    c.k[0].zero_()
    # 25.157 octaves = 17.4375 in natural units, of which every column gives 1 / d; 2.25 is an e4m3 number
    c.k[0][:, 5] = 2.25
    scale = 0.125 * 64 / d
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    v = torch.randint(8, 16, (1, n, d), generator=g, device="cuda").float()      # 4 bits: exact
    v[:, 5] /= 16
    c.v[0] = v.to(torch.bfloat16)
    c.fill()
    q = torch.full((B, Hq, 1, d), 0.96875, dtype=torch.bfloat16, device="cuda")
    table, lengths = shared_rows(c, B)
    out, lse = binding.paged_attn(q, c.cache, table, lengths, scale=scale)
    s = torch.zeros(n, dtype=torch.float64, device="cuda")
    s[5] = 0.96875 * 2.25 * d * scale
    p = torch.softmax(s, 0)
    want = p @ c.vc[0][0]
    # the output's rounding; one fp16 rounding of each weight (2^-11) and what exp2 and the rescalings leave;
    # a warp's fp32 sums: at most every fourth tile of 16 keys is its own
    tol = want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20 + (n / 64) * 2.0 ** -23)
    # weights below fp16's normal numbers: half its smallest step, 2^-25, of a reference that lies at most
    # 2^4 (a bound) / 2^7 above the largest p_j 2^e_j, for each of a warp's n / 4 codes of at most 448
    row = c.vc[0][0].abs().amax(-1)
    unit = torch.exp2(torch.ceil(torch.log2(row / 448)))
    tol = tol + n / 4 * 2.0 ** -28 * 448 * float((p * unit).max())
    assert float((tol / want).max()) < 0.012         # the test means something: a quarter of the weak keys are 2.3 to 7.6 %
    ref.close(out, want.expand_as(out), tol.expand_as(out), "out")
    want_lse = torch.logsumexp(s, 0).expand_as(lse)
    # scores are exact products of a few bits each but for the scale's factor log2(e)
    ref.close(lse, want_lse, want_lse * 2.0 ** -21 + 2.0 ** -21 + (n / 64) * 2.0 ** -23, "lse")


# ------------------------------------------------------------------ large scores
def aligned(lengths, Hkv, d, kind, seed, gain=0):
    """A case whose key `at[b]` of every sequence and head is four times the direction that all its queries have,
    and so wins by far; (case, directions [Hkv, d], at)."""
    c = ref.Case(lengths, Hkv, d, 16, kind, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    u = torch.randn((Hkv, d), generator=g, device="cuda")
    at = [n * 2 // 3 for n in lengths]
    for b in range(len(lengths)):
        k = c.k[b].float()
        k[:, at[b]] = 4 * u
        c.k[b] = (k * 2.0 ** gain).to(torch.bfloat16)
    c.fill()
    return c, u, at


def along(u, B, group, NQ, gain, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    Hkv, d = u.shape
    q = u.repeat_interleave(group, 0)[None, :, None] + 0.1 * torch.randn((B, Hkv * group, NQ, d), generator=g, device="cuda")
    return (q * 2.0 ** gain).to(torch.bfloat16)


@pytest.mark.parametrize("gain,key_gain", [(15, 0), (20, 0), (24, 0), (28, 0), (35, 0), (60, 0), (-96, 112), (118, -90)])
@pytest.mark.parametrize("kind,d,NQ", [("bf16", 64, 1), ("bf16", 128, 5), ("e4m3", 64, 5), ("e4m3", 128, 1)])
def test_large_scores_pick_one_key(kind, d, NQ, gain, key_gain):
    """Scores near 2^(gain + key_gain + 5) with one key far above the rest: exactly its values."""
    lengths = [700, 45, 3000]
    c, u, at = aligned(lengths, 2, d, kind, seed=20, gain=key_gain)
    q = along(u, 3, 4, NQ, gain, seed=22)
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len, causal=False)
    scale = d ** -0.5
    for b in range(3):
        k, v = (x[b].repeat_interleave(4, 0) for x in (c.kc, c.vc))
        s = torch.einsum("hid,hkd->hik", q[b].double(), k) * scale
        top = s[..., at[b]]
        rest = s.clone()
        rest[..., at[b]] = -math.inf
        assert float((top - rest.amax(-1)).min()) > 2.0 ** (gain + key_gain + 1)
        assert torch.equal(out[b].double(), v[:, at[b]].unsqueeze(1).expand(-1, NQ, -1)), b
        e = ref.score_error(q[b].reshape(-1, d), k.repeat_interleave(NQ, 0), scale)
        ref.close(lse[b], top, top.abs() * 2.0 ** -22 + e, "lse")


@pytest.mark.parametrize("kinds", [("bf16", "same"), ("e4m3", "same"), ("bf16", "e4m3")])
@pytest.mark.parametrize("gain,key_gain", [(28, 0), (60, 0), (120, -88), (-96, 112)])
def test_large_scores_in_the_divergence(kinds, gain, key_gain):
    """Both rows on the same key: divergence 0, whatever the scores are."""
    c1, u, at = aligned([700, 45, 3000], 2, 64, kinds[0], seed=25, gain=key_gain)
    c2 = c1
    if kinds[1] != "same":
        c2 = ref.Case(c1.lengths, 2, 64, 16, kinds[1], 26, keys=[x.to(torch.bfloat16) for x in c1.k], table=c1.table)
    q1 = along(u, 3, 4, 1, gain, seed=27)
    q2 = (q1.float() * 2).to(torch.bfloat16)
    kl, lse1, lse2 = binding.paged_kl(q1, c1.cache, q2, c2.cache, c1.table, c1.len)
    for b in range(3):
        tops = []
        for c, q, lse in ((c1, q1, lse1), (c2, q2, lse2)):
            k = c.kc[b].repeat_interleave(4, 0)
            s = torch.einsum("hid,hkd->hik", q[b].double(), k) * 0.125
            assert bool((s.argmax(-1) == at[b]).all())
            e = ref.score_error(q[b].reshape(-1, 64), k, 0.125)
            ref.close(lse[b], s.amax(-1), s.amax(-1).abs() * 2.0 ** -22 + e, "lse")
            tops.append(s.amax(-1))
        # y - z is rounded once (half a step of their difference)
        ref.close(kl[b], torch.zeros_like(tops[0]), (tops[0] - tops[1]).abs() * 2.0 ** -23, "kl")


# ------------------------------------------------------------------ keys and queries of opposite extreme size
OPPOSITE = [
    # exponents of the keys' size, of the queries', of the scale beside 1 / sqrt(d)
    ((112, 118), -117, 0), ((-95, -88), 92, 0), ((-90, 110), -110, 0), ((108, 114), -94, -20), ((-95, -88), 118, -26),
    ((60, 64), -20, -44),
]


@pytest.mark.parametrize("keys,gain,by", OPPOSITE, ids=lambda x: str(x))
@pytest.mark.parametrize("kind,d,NQ", [("bf16", 128, 1), ("e4m3", 128, 1), ("e4m3", 64, 5)])
def test_attention_of_keys_and_queries_of_opposite_size(kind, d, NQ, keys, gain, by):
    """Ordinary scores from keys of 2^-95 to 2^118 and queries that make up for it."""
    c = ref.Case([500, 77], 2, d, 32, kind, seed=30, gain=keys)
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    c.v = [torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16) for x in c.v]
    c.fill()
    q = (ref.queries(2, 8, NQ, d, seed=32).float() * 2.0 ** gain).to(torch.bfloat16)
    scale = d ** -0.5 * 2.0 ** by
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len, scale=scale)
    want, want_lse, tol, tol_lse = ref.attention(c, q, scale, True)
    assert bool(torch.isfinite(want_lse).all())
    ref.close(out, want, tol, "out")
    ref.close(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("keys,gain,by", OPPOSITE, ids=lambda x: str(x))
@pytest.mark.parametrize("kinds", [("e4m3", "same"), ("bf16", "e4m3"), ("e4m3", "bf16")])
def test_divergence_of_keys_and_queries_of_opposite_size(kinds, keys, gain, by):
    c1 = ref.Case([500, 77], 2, 64, 32, kinds[0], seed=33, gain=keys)
    c2 = c1 if kinds[1] == "same" else ref.Case([500, 77], 2, 64, 32, kinds[1], 34, keys=c1.k, table=c1.table)
    q1 = ref.queries(2, 8, 1, 64, seed=35)
    q2 = ref.queries(2, 8, 1, 64, seed=36, near=q1)
    q1, q2 = ((x.float() * 2.0 ** gain).to(torch.bfloat16) for x in (q1, q2))
    scale = 0.125 * 2.0 ** by
    got = binding.paged_kl(q1, c1.cache, q2, c2.cache, c1.table, c1.len, scale=scale)
    kl, lse1, lse2, tol, tol_lse = ref.divergence(c1, q1, c2, q2, scale, True)
    ref.close(got[0], kl, tol, "kl")
    ref.close(got[1], lse1, tol_lse, "lse1")
    ref.close(got[2], lse2, tol_lse, "lse2")


# ------------------------------------------------------------------ every tile of a long sequence
LONG = [
    # Hq, Hkv, NQ, d, page, kind, causal, lengths
    (16, 16, 1, 64, 1024, "e4m3", True, [65600]),
    (16, 16, 1, 128, 1024, "bf16", True, [62001]),
    (4, 1, 5, 128, 16, "e4m3", True, [20011, 3000, 0, 17, 9999]),      # 20 rows
    (4, 1, 8, 128, 32, "bf16", True, [30003, 511]),                    # 32 rows
    (8, 2, 3, 64, 16, "bf16", True, [33333, 64, 2049]),                # 12 rows
    (7, 1, 1, 128, 64, "e4m3", True, [131072 - 15]),
    (2, 1, 1, 64, 16, "e4m3", True, [900] * 150),                      # dealt out whole
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "q%dkv%dn%dd%dp%d%sB%d" % (*c[:6], len(c[7])))
def test_every_value_counts_once(case):
    """Keys of zeros weigh every value alike, and the values are small whole numbers: all sums are exact, so a
    tile that is lost, doubled, or taken from another place changes the mean beyond its rounding."""
    Hq, Hkv, NQ, d, page, kind, causal, lengths = case
    c = ref.Case(lengths, Hkv, d, page, kind, seed=40)
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    for b, n in enumerate(lengths):
        c.k[b].zero_()
        c.v[b] = torch.randint(-16, 17, (Hkv, n, d), generator=g, device="cuda").to(torch.bfloat16)
    c.fill()
    q = ref.queries(len(lengths), Hq, NQ, d, seed=42)
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len, causal=causal)
    for b, n in enumerate(lengths):
        upto = torch.cat([torch.zeros((Hkv, 1, d), dtype=torch.float64, device="cuda"), c.vc[b].cumsum(1)], 1)
        for i in range(NQ):
            m = max(0, n - (NQ - 1 - i))
            want = upto[:, m].repeat_interleave(Hq // Hkv, 0) / max(1, m)
            # one rounding to bf16, half a step; 1 / l and two products in fp32
            ref.close(out[b, :, i], want, want.abs() * (2.0 ** -8 + 2.0 ** -22), "sequence %d, token %d" % (b, i))
            if m:
                assert float((lse[b, :, i].double() - math.log(m)).abs().max()) <= 2.0 ** -21 + math.log(m) * 2.0 ** -22
            else:
                assert bool((lse[b, :, i] == -math.inf).all())


@pytest.mark.parametrize("kind,d,n", [("e4m3", 64, 65600), ("bf16", 128, 62001), ("bf16", 64, 65551), ("e4m3", 128, 40000)])
def test_a_key_meets_its_own_values(kind, d, n):
    """Single keys at the borders of tiles, units, pages and batches of page entries (and elsewhere) win a row each:
    the row is that key's values."""
    Hkv, R = 16, 8
    c = ref.Case([n], Hkv, d, 1024, kind, seed=50)
    g = torch.Generator(device="cuda")
    g.manual_seed(51)
    border = [0, 15, 16, 31, 32, 47, 48, 63, 64, 127, 128, 511, 512, 1007, 1008, 1023, 1024, 1025, 2031, 2032, 2047, 2048,
              2049, 4095, 4096, 8191, 8192, 16383, 16384, 32767, 32768, n - 17, n - 16, n - 2, n - 1]
    other = torch.randperm(n, generator=g, device="cuda").tolist()
    at = (border + [x for x in other if x not in border])[:Hkv * R]
    u = torch.where(torch.rand((Hkv, R, d), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    at = torch.tensor(at, device="cuda").view(R, Hkv).t()                  # [Hkv, R]
    k = 0.1 * torch.randn((Hkv, n, d), generator=g, device="cuda")
    for h in range(Hkv):
        k[h, at[h]] = u[h] * 512 / d                                       # score 512 / sqrt(d) of its own row
    c.k[0] = k.to(torch.bfloat16)
    c.fill()
    q = u.unsqueeze(0).to(torch.bfloat16)                                  # [1, Hkv, R, d]
    scale = d ** -0.5
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len, scale=scale, causal=False)
    for h in range(Hkv):
        s = q[0, h].double() @ c.kc[0][h].t() * scale
        own = s.gather(1, at[h][:, None])
        p = torch.softmax(s, -1)
        assert float(p.gather(1, at[h][:, None]).min()) > 1 - 2.0 ** -12
        want = p @ c.vc[0][h]
        # the output's and the weight's rounding; the others, together under 2^-12, half off at most
        tol = want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20) + (1 - p.gather(1, at[h][:, None])) * float(c.vc[0][h].abs().max())
        ref.close(out[0, h], want, tol, "head %d" % h)
        ref.close(lse[0, h], own[:, 0], own[:, 0].abs() * 2.0 ** -20 + 2.0 ** -12, "lse")
