"""Paged calls from Python: both ways of a call (the extension and the plain path) refuse alike, and the device
status loses nothing."""
import pytest
import torch

from attention_kl_divergence_02_b200 import binding

import paged_ref as ref

pytestmark = pytest.mark.gpu


def status():
    return binding.streamkl_device_status()


def batch(kind="bf16"):
    c = ref.Case([40, 20], 2, 64, 16, kind, seed=120)
    q = ref.queries(2, 4, 1, 64, seed=121)
    return c, q, binding.paged_workspace(2, 4, 2, 1, 64)


@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("shape", ["pages", "Hkv", "page_size", "d"])
def test_caches_that_do_not_match_are_refused_alike(fast, shape, monkeypatch):
    c, q, ws = batch()
    if not fast:
        monkeypatch.setattr(binding, "_fast", None)
    pages, Hkv, page_size, d = c.cache.shape
    other = binding.PagedCache.empty(*{"pages": (pages + 1, Hkv, page_size, d), "Hkv": (pages, 1, page_size, d),
                                       "page_size": (pages, Hkv, 32, d), "d": (pages, Hkv, page_size, 128)}[shape])
    with pytest.raises(ValueError, match="both caches must agree"):
        binding.paged_kl(q, c.cache, q, other, c.table, c.len, workspace=ws)
    assert status() == binding.OK


def a_bad_page(c, q, ws):
    table = c.table.clone()
    table[0, 0] = c.pages
    binding.paged_attn(q, c.cache, table, c.len, workspace=ws)


def test_a_bad_page_does_not_reach_the_watchdog_s_self_test():
    """The self-test answers for its own waits; what a call before it recorded stays for the status call."""
    c, q, ws = batch()
    a_bad_page(c, q, ws)
    rc, _ = binding.streamkl_selftest_watchdog(0)
    assert rc == binding.OK
    assert status() == binding.ERR_PAGE and status() == binding.OK
    a_bad_page(c, q, ws)
    rc, _ = binding.streamkl_selftest_watchdog(1)       # waits that run out, and return
    assert rc == binding.ERR_TIMEOUT
    assert status() == binding.ERR_PAGE and status() == binding.OK
