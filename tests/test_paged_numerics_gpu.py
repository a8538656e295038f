"""Paged attention and divergence of scores far beyond the usual, and of keys and queries of extreme and
opposite size."""
import math

import pytest
import torch

from attention_kl_divergence_02_b200 import binding

import paged_ref as ref

pytestmark = pytest.mark.gpu


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
