"""A scale whose product with log2(e) is no fp32 number is refused on the host, like the other bad scales."""
import pytest

from attention_kl_divergence_02_b200 import binding, build

from test_paged_host import attn, cache, kl


@pytest.mark.parametrize("scale", [3e38, 2.4e38])
def test_a_scale_beyond_the_range(scale):
    build.build()
    assert attn(cache(), scale=scale) == binding.ERR_UNSUPPORTED
    assert kl(cache(), cache(k=1 << 21), scale=scale) == binding.ERR_UNSUPPORTED
