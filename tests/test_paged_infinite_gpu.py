"""Infinite values that a row of paged attention sees: the row's columns are that infinity."""
import math

import pytest
import torch

from attention_kl_divergence_02_b200 import binding

import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,NQ,lengths", [
    (4, 1, [1, 2, 85, 16]), (4, 1, [5000]), (16, 1, [300, 1]), (4, 10, [77, 200]), (4, 16, [333]), (16, 5, [40, 999]),
])
def test_an_infinite_value_that_is_seen(Hq, NQ, lengths, d):
    """One token's values are +inf, -inf or ordinary by column; every row's weight of it is a normal number."""
    c = ref.Case(lengths, 2, d, 16, "bf16", seed=60)
    q = ref.queries(len(lengths), Hq, NQ, d, seed=61)
    want, want_lse, tol, tol_lse = ref.attention(c, q, d ** -0.5, False)
    for b, n in enumerate(lengths):
        j = n // 2
        page = int(c.table[b, j // 16])
        c.cache.v[page, :, j % 16, 0::3] = math.inf
        c.cache.v[page, :, j % 16, 1::3] = -math.inf
    out, lse = binding.paged_attn(q, c.cache, c.table, c.len, causal=False)
    assert bool((out[..., 0::3] == math.inf).all())
    assert bool((out[..., 1::3] == -math.inf).all())
    ref.close(out[..., 2::3], want[..., 2::3], tol[..., 2::3], "out")
    ref.close(lse, want_lse, tol_lse, "lse")


def test_both_infinities_in_a_column():
    c = ref.Case([50], 2, 64, 16, "bf16", seed=62)
    q = ref.queries(1, 4, 1, 64, seed=63)
    for j, x in ((3, math.inf), (40, -math.inf)):
        c.cache.v[int(c.table[0, j // 16]), :, j % 16, 7] = x
    out, _ = binding.paged_attn(q, c.cache, c.table, c.len)
    assert bool(torch.isnan(out[..., 7]).all()) and bool(torch.isfinite(out[..., :7]).all())
