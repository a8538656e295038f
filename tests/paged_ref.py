"""Plain 64-bit forms of the paged-cache operators for the tests, and caches to run them on.

Every cache made here is poisoned: what no sequence owns (pages outside the tables, slots behind a
length) holds NaN, so a kernel that lets it reach a result fails."""
import math

import torch

from attention_kl_divergence_02_b200 import binding

LEAST = -96


def quantise(x):
    """bf16 rows -> (codes as float64 multiples of the scale, exponent): the definition, in 64 bits."""
    x = x.double()
    a = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    e = torch.full_like(a, float(LEAST))
    for k in range(120, LEAST - 1, -1):       # the least exponent >= LEAST with a <= 448 * 2^e
        e = torch.where(a <= 448.0 * 2.0 ** k, float(k), e)
    top = torch.where(e == 120, 240.0, 448.0).unsqueeze(-1)      # 256 * 2^120 is no bf16 number
    y = torch.minimum(torch.maximum(x / torch.exp2(e).unsqueeze(-1), -top), top)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, e


def dequantise(codes, e):
    return codes * torch.exp2(e).unsqueeze(-1)


class Case:
    """Pages and a table for sequences of the given lengths, and their rows in order."""

    def __init__(self, lengths, Hkv, d, page, kind, seed, spare=3, keys=None, table=None, width=None, gain=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.lengths, self.Hkv, self.d, self.page, self.kind = lengths, Hkv, d, page, kind
        B = len(lengths)
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + spare
        if table is None:
            order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
            table = torch.full((B, width or max(1, max(need))), -1, dtype=torch.int32, device="cuda")
            at = 0
            for b, n in enumerate(need):
                table[b, :n] = order[at:at + n]
                at += n
        self.table, self.pages = table, pages
        self.len = torch.tensor(lengths, dtype=torch.int32, device="cuda")

        def draw(n):
            x = torch.randn((Hkv, n, d), generator=g, device="cuda")
            if gain is not None:                    # rows of very different size
                x = x * torch.exp2(torch.randint(gain[0], gain[1] + 1, (1, n, 1), generator=g, device="cuda").float())
            return x.to(torch.bfloat16)

        self.k = [draw(n) for n in lengths] if keys is None else keys
        self.v = [draw(n) for n in lengths]
        self.fill()

    def fill(self):
        """Writes self.k and self.v into a poisoned cache, by the definition; keeps the cached values."""
        B = len(self.lengths)
        pools, self.kc, self.vc, exps = [], [], [], []
        for rows, kept in ((self.k, self.kc), (self.v, self.vc)):
            shape = (self.pages, self.Hkv, self.page, self.d)
            if self.kind == "bf16":
                pool, exp = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda"), None
            else:
                pool = torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                exp = torch.full(shape[:3], 255, dtype=torch.uint8, device="cuda")
            for b in range(B):
                n = self.lengths[b]
                x, e = rows[b], None
                if self.kind != "bf16":
                    x, e = quantise(rows[b])
                    kept.append(dequantise(x, e))
                else:
                    kept.append(x.double())
                for j in range(-(-n // self.page)):
                    m = min(self.page, n - j * self.page)
                    p = int(self.table[b, j])
                    s = slice(j * self.page, j * self.page + m)
                    if e is None:
                        pool[p, :, :m] = x[:, s]
                    else:
                        pool.view(torch.uint8)[p, :, :m] = x[:, s].float().to(torch.float8_e4m3fn).view(torch.uint8)
                        exp[p, :, :m] = (e[:, s] + 127).to(torch.uint8)
            pools.append(pool)
            exps.append(exp)
        self.cache = binding.PagedCache(pools[0], pools[1], k_exp=exps[0], v_exp=exps[1])


def _limit(n, NQ, i, causal):
    return max(0, n - (NQ - 1 - i)) if causal else n


def score_error(q, k, scale):
    """Bound on a base-e score's error: products of bf16 (or e4m3 and a scaled fp16 query, exact to 2^-40) are
    exact in fp32; d / 16 sums of 16 products and four roundings of the result, each at most 2^-23
    of the sum of magnitudes (tensor-core sums may truncate: twice half a step)."""
    size = torch.einsum("hd,hkd->hk", q.double().abs(), k.abs()).amax() * scale
    return float((q.shape[-1] / 16 + 4) * 2.0 ** -23 * size)


def attention(case, q, scale, causal):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits."""
    B, Hq, NQ, d = q.shape
    group = Hq // case.Hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, NQ), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(case.lengths):
        k, v = (x[b].repeat_interleave(group, 0) for x in (case.kc, case.vc))
        for i in range(NQ):
            m = _limit(n, NQ, i, causal)
            if m == 0:
                continue
            s = torch.einsum("hd,hkd->hk", q[b, :, i].double(), k[:, :m]) * scale
            p = torch.softmax(s, -1)
            out[b, :, i] = torch.einsum("hk,hkd->hd", p, v[:, :m])
            lse[b, :, i] = torch.logsumexp(s, -1)
            size = torch.einsum("hk,hkd->hd", p, v[:, :m].abs())
            e = score_error(q[b, :, i], k[:, :m], scale)
            # weights: the scores' error in numerator and sum, 2^-21 each for exp2 and the rescalings; two
            # bf16 terms keep 2^-16, one fp16 term 2^-11; fp32 sums over m / 16 products
            weight = 2 * e + 2.0 ** -20 + (2.0 ** -16 if case.kind == "bf16" else 2.0 ** -11) + (m / 16) * 2.0 ** -23
            tol[b, :, i] = out[b, :, i].abs() * 2.0 ** -8 + size * weight
            if case.kind != "bf16":
                # weights below fp16's normal numbers: half its smallest step, 2^-25 of the reference 2^m', and m'
                # may be the bound max s + max e over keys whose e differ by at most 4: it exceeds the largest
                # s_j + e_j by at most 4, so 2^-21 of the largest p_j 2^e_j for each of m codes of at most 448
                row = v[:, :m].abs().amax(-1)
                unit = torch.exp2(torch.ceil(torch.log2(row.clamp(min=2.0 ** -200) / 448)))
                tol[b, :, i] += m * 2.0 ** -21 * 448 * (p * unit).amax(-1, keepdim=True)
            tol_lse[b, :, i] = e + 2.0 ** -21 + lse[b, :, i].abs() * 2.0 ** -22
    return out, lse, tol, tol_lse


def divergence(case1, q1, case2, q2, scale, causal):
    """(kl, lse1, lse2, tolerance of kl, tolerance of the lse) in 64 bits."""
    B, Hq, NQ, d = q1.shape
    group = Hq // case1.Hkv
    kl = torch.zeros((B, Hq, NQ), dtype=torch.float64, device="cuda")
    lse = [torch.full_like(kl, -math.inf) for _ in range(2)]
    tol, tol_lse = torch.zeros_like(kl), torch.zeros_like(kl)
    for b, n in enumerate(case1.lengths):
        k1, k2 = case1.kc[b].repeat_interleave(group, 0), case2.kc[b].repeat_interleave(group, 0)
        for i in range(NQ):
            m = _limit(n, NQ, i, causal)
            if m == 0:
                continue
            a = torch.einsum("hd,hkd->hk", q1[b, :, i].double(), k1[:, :m]) * scale
            c = torch.einsum("hd,hkd->hk", q2[b, :, i].double(), k2[:, :m]) * scale
            pa, pc = torch.log_softmax(a, -1), torch.log_softmax(c, -1)
            kl[b, :, i] = (pa.exp() * (pa - pc)).sum(-1)
            lse[0][b, :, i], lse[1][b, :, i] = torch.logsumexp(a, -1), torch.logsumexp(c, -1)
            e = max(score_error(q1[b, :, i], k1[:, :m], scale), score_error(q2[b, :, i], k2[:, :m], scale))
            # dKL = sum p1 (r - KL) ds1 + sum (p2 - p1) ds2, |ds| <= e, r = log(p1 / p2); exp2 and the sums
            # of the weights: 2^-20 relative on terms of size |a - c|
            spread = (pa.exp() * (pa - pc).abs()).sum(-1) + kl[b, :, i]
            size = (pa.exp() * (a - c).abs()).sum(-1) + 1
            tol[b, :, i] = e * (spread + 2) + size * 2.0 ** -20
            tol_lse[b, :, i] = e + 2.0 ** -21 + torch.maximum(lse[0][b, :, i].abs(), lse[1][b, :, i].abs()) * 2.0 ** -22
    return kl, lse[0], lse[1], tol, tol_lse


def close(got, want, tol, what):
    got = got.double()
    same = (got == want) | ((got - want).abs() <= tol)
    if not bool(same.all()):
        bad = (~same).nonzero()[0].tolist()
        worst = ((got - want).abs() / tol.clamp(min=1e-300))[~same].max()
        raise AssertionError("%s: %d of %d off, first at %s: got %r, want %r, allowed %r; worst %.3g times" % (
            what, int((~same).sum()), same.numel(), bad, float(got[tuple(bad)]), float(want[tuple(bad)]),
            float(tol[tuple(bad)]), float(worst)))


def queries(B, Hq, NQ, d, seed, near=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 77)
    x = torch.randn((B, Hq, NQ, d), generator=g, device="cuda")
    if near is not None:
        x = near.float() + 0.5 * x
    return x.to(torch.bfloat16)
