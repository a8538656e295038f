"""Values near the largest bf16 number: attention over a few of them stays finite wherever the result is."""
import pytest
import torch

from attention_kl_divergence_02_b200 import binding

import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,NQ,n", [(4, 1, 120), (16, 1, 3000), (4, 10, 120), (16, 5, 3000)])
def test_large_values(kind, Hq, NQ, n):
    """Scores that rise by up to 8 octaves from key to key and one key that ends up far above the rest, so that the sum
    of weights times values is about the result."""
    d = 64
    c = ref.Case([n], 2, d, 16, kind, seed=70)
    g = torch.Generator(device="cuda")
    g.manual_seed(71)
    u = torch.where(torch.rand((2, d), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    rise = torch.tensor([0.0, 4.0, 8.0, 11.0], device="cuda").repeat(-(-n // 4))[:n] / 16      # times log2(e): 0 to 16 octaves
    rise[n - 40] = 2.0
    c.k[0] = (u[:, None] * rise[None, :, None]).to(torch.bfloat16)
    c.v[0] = torch.randn((2, n, d), generator=g, device="cuda").clamp(-4, 4).mul(2.0 ** 122).to(torch.bfloat16)
    c.fill()
    q = (u.repeat_interleave(Hq // 2, 0)[None, :, None] * torch.ones(1, Hq, NQ, 1, device="cuda")).to(torch.bfloat16)
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len, scale=0.25, causal=False)
    want, want_lse, tol, tol_lse = ref.attention(c, q, 0.25, False)
    ref.close(out, want, tol, "out")
    ref.close(lse, want_lse, tol_lse, "lse")
