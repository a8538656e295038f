"""Paged calls from Python: the extension is what runs, both ways of a call refuse alike, and the device status
loses nothing."""
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


def test_everyday_calls_run_in_the_extension(monkeypatch):
    """It is loaded, takes the everyday case of every call itself, and agrees with the plain path."""
    c, q, ws = batch()
    assert binding._fast is not None
    scale = 0.125
    done = binding._fast.attn(q, c.cache.address, c.cache.index, c.table, c.len, scale, True, ws)
    assert done is not NotImplemented and done[0] == binding.OK
    kl = binding._fast.kl(q, c.cache.address, q, c.cache.address, c.cache.index, c.table, c.len, scale, True, ws)
    assert kl is not NotImplemented and kl[0] == binding.OK
    new = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    zero, one = (torch.full((2,), x, dtype=torch.int32, device="cuda") for x in (0, 1))
    assert binding._fast.move(c.cache.address, c.cache.index, False, new, new.clone(), c.table, None, one) == binding.OK
    want = binding.paged_attn(q, c.cache, c.table, c.len, workspace=ws)
    monkeypatch.setattr(binding, "_fast", None)
    plain = binding.paged_attn(q, c.cache, c.table, c.len, workspace=ws)
    for a, b in zip((*done[1:], *want), (*plain, *plain)):
        assert torch.equal(a, b)
    for a, b in zip(kl[1], binding.paged_kl(q, c.cache, q, c.cache, c.table, c.len, workspace=ws)):
        assert torch.equal(a, b)
    assert status() == binding.OK


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


def test_a_captured_fork_and_join():
    """Captured behind a copy, beside a call on another stream, and behind both: every launch is a programmatic
    dependent of all that it has to wait for."""
    c, q, _ = batch()
    other = (q.float() * 2).to(torch.bfloat16)
    want = [binding.paged_attn(x, c.cache, c.table, c.len) for x in (q, other)]
    spaces = [binding.paged_workspace(2, 4, 2, 1, 64) for _ in range(2)]
    out = [(torch.empty_like(q), torch.empty((2, 4, 1), device="cuda")) for _ in range(2)]
    source, rows = q.clone(), torch.empty_like(q)
    side = torch.cuda.Stream()

    def step():
        rows.copy_(source)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            binding.paged_attn(rows, c.cache, c.table, c.len, out=out[1], workspace=spaces[1])
        binding.paged_attn(rows, c.cache, c.table, c.len, out=out[0], workspace=spaces[0])
        torch.cuda.current_stream().wait_stream(side)
        return binding.paged_attn(rows, c.cache, c.table, c.len)

    first = torch.cuda.Stream()
    first.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(first):
        step()
    torch.cuda.current_stream().wait_stream(first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.append(step())
    for x, w in ((q, want[0]), (other, want[1]), (q, want[0])):
        source.copy_(x)
        for o in out:
            o[0].zero_(), o[1].zero_()
        graph.replay()
        for o in out:
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    assert status() == binding.OK
