"""Paged-cache calls refuse bad arguments on the host, before any device work."""
import ctypes

import pytest
import torch

from attention_kl_divergence_02_b200 import binding, build

FAKE = 1 << 20     # 16-byte aligned, never dereferenced: every call below fails its checks first
INVALID, UNSUPPORTED = binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE, type=binding.CACHE_E4M3, pages=8, page_size=16, Hkv=2, d=64)
    f.update(kw)
    return binding.CacheStruct(*(f[n] for n, _ in binding.CacheStruct._fields_))


BAD_CACHES = [
    (dict(k=None), INVALID),
    (dict(v=None), INVALID),
    (dict(k_exp=None), INVALID),
    (dict(type=2), INVALID),
    (dict(pages=0), INVALID),
    (dict(page_size=0), INVALID),
    (dict(Hkv=-1), INVALID),
    (dict(d=0), INVALID),
    (dict(d=96), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=2048), UNSUPPORTED),
    (dict(k=FAKE + 8), UNSUPPORTED),
    (dict(v_exp=FAKE + 4), UNSUPPORTED),
]


def move(append, c, **kw):
    a = dict(table=FAKE, width=4, start=FAKE, count=FAKE, B=2, NT=3, k=FAKE, v=FAKE)
    a.update(kw)
    if append:
        return binding.streamkl_cache_append(c, a["k"], a["v"], a["table"], a["width"], a["start"], a["count"], a["B"],
                                             a["NT"], stream=0)
    return binding.streamkl_cache_gather(c, a["table"], a["width"], a["start"], a["count"], a["B"], a["NT"], a["k"],
                                         a["v"], stream=0)


def attn(c, **kw):
    a = dict(q=FAKE, table=FAKE, width=4, lengths=FAKE, B=2, Hq=4, NQ=1, scale=0.125, causal=1, out=FAKE, lse=FAKE,
             ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return binding.streamkl_paged_attn(c, a["q"], a["table"], a["width"], a["lengths"], a["B"], a["Hq"], a["NQ"],
                                       a["scale"], a["causal"], a["out"], a["lse"], a["ws"], a["bytes"], stream=0)


def kl(c1, c2, **kw):
    a = dict(q1=FAKE, q2=FAKE, table=FAKE, width=4, lengths=FAKE, B=2, Hq=4, NQ=1, scale=0.125, causal=1, kl=FAKE,
             lse1=FAKE, lse2=FAKE, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return binding.streamkl_paged_kl(c1, a["q1"], c2, a["q2"], a["table"], a["width"], a["lengths"], a["B"], a["Hq"],
                                     a["NQ"], a["scale"], a["causal"], a["kl"], a["lse1"], a["lse2"], a["ws"],
                                     a["bytes"], stream=0)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches(kw, want):
    assert move(True, cache(**kw)) == want
    assert move(False, cache(**kw)) == want
    assert attn(cache(**kw)) == want
    if not {"v", "v_exp"} & set(kw):        # the divergence reads keys only
        assert kl(cache(**kw), cache()) == want
        assert kl(cache(), cache(**kw)) == want


def test_no_cache():
    assert move(True, None) == INVALID and attn(None) == INVALID and kl(cache(), None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(table=None), INVALID),
    (dict(width=0), INVALID),
    (dict(B=0), INVALID),
    (dict(NT=0), INVALID),
    (dict(k=None), INVALID),
    (dict(v=FAKE + 2), UNSUPPORTED),
    (dict(width=(1 << 26) + 1), UNSUPPORTED),       # over 2^30 tokens
    (dict(B=1 << 20, NT=1 << 10), UNSUPPORTED),     # 2^31 rows
])
def test_bad_moves(kw, want):
    assert move(True, cache(), **kw) == want
    assert move(False, cache(), **kw) == want


COMMON = [
    (dict(table=None), INVALID),
    (dict(width=0), INVALID),
    (dict(lengths=None), INVALID),
    (dict(B=0), INVALID),
    (dict(NQ=0), INVALID),
    (dict(Hq=0), INVALID),
    (dict(Hq=3), UNSUPPORTED),
    (dict(scale=0.0), UNSUPPORTED),
    (dict(scale=float("inf")), UNSUPPORTED),
    (dict(scale=float("nan")), UNSUPPORTED),
    (dict(width=(1 << 26) + 1), UNSUPPORTED),
    (dict(B=1 << 20, NQ=1 << 10), UNSUPPORTED),
    (dict(B=1 << 16, width=1 << 20), UNSUPPORTED),  # 2^35 units of keys
    (dict(ws=None), INVALID),
    (dict(bytes=64), INVALID),
    (dict(ws=FAKE + 8), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(lse=None), INVALID), (dict(q=FAKE + 2), UNSUPPORTED),
    (dict(out=FAKE + 8), UNSUPPORTED), (dict(lse=FAKE + 2), UNSUPPORTED)])
def test_bad_attention(kw, want):
    assert attn(cache(), **kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(q2=None), INVALID), (dict(kl=None), INVALID), (dict(lse2=FAKE + 2), UNSUPPORTED)])
def test_bad_divergence(kw, want):
    assert kl(cache(), cache(k=2 * FAKE), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=2 * FAKE, pages=9), UNSUPPORTED), (dict(k=2 * FAKE, page_size=32), UNSUPPORTED),
    (dict(k=2 * FAKE, Hkv=1), UNSUPPORTED), (dict(k=2 * FAKE, d=128), UNSUPPORTED),
    (dict(type=binding.CACHE_BF16), INVALID),       # one pool of keys cannot be of two types
    (dict(k_exp=2 * FAKE), INVALID)])
def test_caches_that_do_not_match(kw, want):
    assert kl(cache(), cache(**kw)) == want


def test_workspace_bytes():
    n = 4 * binding.streamkl_num_sms() * 2
    assert binding.streamkl_paged_workspace_bytes(1, 8, 8, 1, 128) == 4096 + n * 8 * 132 * 4
    assert binding.streamkl_paged_workspace_bytes(64, 32, 8, 3, 64) == 4096 + n * 16 * 68 * 4
    assert binding.streamkl_paged_workspace_bytes(1, 32, 1, 9, 64) == 4096 + n * 32 * 68 * 4
    for bad in ((0, 8, 8, 1, 128), (1, 8, 3, 1, 128), (1, 8, 8, 0, 128), (1, 8, 8, 1, 96)):
        assert binding.streamkl_paged_workspace_bytes(*bad) == 0


def test_status_text():
    assert binding.ERR_PAGE == 5 and "page" in binding.status_string(5)


def test_python_calls_refuse_host_tensors():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.PagedCache(k)
    with pytest.raises(ValueError):
        binding.PagedCache(k.float())


def test_the_extension_leaves_everything_odd_to_python():
    """csrc/fastcall.cpp answers NotImplemented, without an exception, for whatever is not its everyday case."""
    binding._start()
    if binding._fast is None:
        pytest.skip("the extension is not built (no Python headers)")
    struct = cache(type=binding.CACHE_BF16)
    at = ctypes.addressof(struct)
    q = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16)
    table, n = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(4096)
    new = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16)
    for args in ((q, at, 0, table, n, 0.1, True, ws),              # tensors on the host
                 (q, at, 0, table, n, 0.1, True, None),
                 (None, at, 0, table, n, 0.1, True, ws),
                 (q, 0, 0, table, n, 0.1, True, ws),
                 (q, "x", 0, table, n, 0.1, True, ws),
                 (q, at, 0, 7, n, 0.1, True, ws),
                 (q, at, 0, table, n, "x", True, ws),
                 (q,)):
        assert binding._fast.attn(*args) is NotImplemented
    assert binding._fast.kl(q, at, q, at, 0, table, n, 0.1, True, ws) is NotImplemented
    assert binding._fast.kl(q, at, object(), at, 0, table, n, 0.1, True, ws) is NotImplemented
    for append in (True, False):
        assert binding._fast.move(at, 0, append, new, new, table, n, n) is NotImplemented
        assert binding._fast.move(at, 0, append, new, None, table, None, None) is NotImplemented


def test_a_missing_tensor_is_named():
    """None in the place of a tensor meets a ValueError, as in the dense calls."""
    class Cache:
        v, shape, index, device = object(), (4, 2, 16, 64), 0, "cuda:0"
    rows = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    for call in (lambda: binding.cache_append(Cache, None, rows, rows, rows, stream=0),
                 lambda: binding.cache_gather(Cache, None, rows, rows=1, stream=0),
                 lambda: binding._need("start", None, torch.int32, (1,), Cache),
                 lambda: binding._width(None, 1, Cache),
                 lambda: binding.paged_attn(None, Cache, rows, rows, stream=0),
                 lambda: binding.paged_kl(None, Cache, rows, Cache, rows, rows, stream=0)):
        with pytest.raises(ValueError, match="is required"):
            call()
