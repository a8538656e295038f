"""ctypes binding of libstreamkl (include/streamkl.h).

Argument marshalling only: torch tensors are turned into device pointers and the CUDA
stream handle, and every step of the computation runs in the library's kernels.  The
library is loaded on first use; if it is missing or fails to load this raises, there is
no other implementation to fall back to.

Low-level functions carry the C names and arguments (pointers may be ints or tensors).
``fwd``/``bwd`` are conveniences that allocate outputs with torch (device memory is
torch's job; the library allocates nothing).
"""
import ctypes
import math
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libstreamkl.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_CUDA = 3
ERR_TIMEOUT = 4
ERR_PAGE = 5
CACHE_BF16 = 0
CACHE_E4M3 = 1

EXPORTS = (
    "streamkl_fwd",
    "streamkl_fwd_sym",
    "streamkl_fwd_splitk",
    "streamkl_fwd_splits",
    "streamkl_fwd_splitk_workspace_bytes",
    "streamkl_bwd",
    "streamkl_bwd_workspace_bytes",
    "streamkl_bwd_noalloc",
    "streamkl_status_string",
    "streamkl_device_status",
    "streamkl_selftest_watchdog",
    "streamkl_last_cuda_error",
    "streamkl_version",
    "streamkl_probe_exp2",
    "streamkl_num_sms",
    "streamkl_probe_clock",
    "streamkl_eval_exp2",
    "streamkl_cache_append",
    "streamkl_cache_gather",
    "streamkl_paged_workspace_bytes",
    "streamkl_paged_attn",
    "streamkl_paged_kl",
)

_lib = None


class CacheStruct(ctypes.Structure):
    """streamkl_cache of the header."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p), ("type", ctypes.c_int), ("pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int)]


class StreamKLError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = "%s: %s" % (where, status_string(status))
        if status == ERR_CUDA:
            msg += " (%s)" % last_cuda_error()
        super().__init__(msg)


def load(path=None):
    """Load the shared library (once) and declare the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError("libstreamkl.so not built at %s (run python -m "
                          "attention_kl_divergence_02_b200.build)" % p)
    lib = ctypes.CDLL(p)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.streamkl_fwd.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, vp, vp, vp]
    lib.streamkl_fwd.restype = i
    lib.streamkl_fwd_sym.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, vp, vp, vp, vp]
    lib.streamkl_fwd_sym.restype = i
    lib.streamkl_fwd_splitk.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp, vp, vp, vp, sz, vp]
    lib.streamkl_fwd_splitk.restype = i
    lib.streamkl_fwd_splits.argtypes = [i, i, i, i]
    lib.streamkl_fwd_splits.restype = i
    lib.streamkl_fwd_splitk_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.streamkl_fwd_splitk_workspace_bytes.restype = sz
    lib.streamkl_bwd.argtypes = ([i, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i,
                                  vp, vp, vp, sz, vp])
    lib.streamkl_bwd.restype = i
    lib.streamkl_bwd_noalloc.argtypes = ([i, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i,
                                          vp, vp, vp])
    lib.streamkl_bwd_noalloc.restype = i
    lib.streamkl_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.streamkl_bwd_workspace_bytes.restype = sz
    lib.streamkl_status_string.argtypes = [i]
    lib.streamkl_status_string.restype = ctypes.c_char_p
    lib.streamkl_device_status.argtypes = [vp]
    lib.streamkl_device_status.restype = i
    lib.streamkl_selftest_watchdog.argtypes = [i, ctypes.POINTER(ctypes.c_longlong), vp]
    lib.streamkl_selftest_watchdog.restype = i
    lib.streamkl_last_cuda_error.argtypes = []
    lib.streamkl_last_cuda_error.restype = ctypes.c_char_p
    lib.streamkl_version.argtypes = []
    lib.streamkl_version.restype = i
    lib.streamkl_probe_exp2.argtypes = [i, i, ctypes.POINTER(ctypes.c_longlong), vp]
    lib.streamkl_probe_exp2.restype = i
    lib.streamkl_num_sms.argtypes = []
    lib.streamkl_num_sms.restype = i
    lib.streamkl_probe_clock.argtypes = [ctypes.c_longlong, ctypes.c_longlong, vp, i, vp]
    lib.streamkl_probe_clock.restype = i
    lib.streamkl_eval_exp2.argtypes = [i, vp, vp, ctypes.c_longlong, vp]
    lib.streamkl_eval_exp2.restype = i
    lib.streamkl_cache_append.argtypes = [vp, vp, vp, vp, i, vp, vp, i, i, vp]
    lib.streamkl_cache_append.restype = i
    lib.streamkl_cache_gather.argtypes = [vp, vp, i, vp, vp, i, i, vp, vp, vp]
    lib.streamkl_cache_gather.restype = i
    lib.streamkl_paged_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.streamkl_paged_workspace_bytes.restype = sz
    lib.streamkl_paged_attn.argtypes = [vp, vp, vp, i, vp, i, i, i, f, i, vp, vp, vp, sz, vp]
    lib.streamkl_paged_attn.restype = i
    lib.streamkl_paged_kl.argtypes = [vp, vp, vp, vp, vp, i, vp, i, i, i, f, i, vp, vp, vp, vp, sz, vp]
    lib.streamkl_paged_kl.restype = i
    if path is None:
        _lib = lib
    return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ C-named calls
def streamkl_fwd(q1, k1, q2, k2, B, Hq, Hkv, NQ, NK, d, scale, causal, kl, lse1, lse2, stream=None):
    return load().streamkl_fwd(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), B, Hq, Hkv, NQ, NK, d,
                               float(scale), int(bool(causal)), _ptr(kl), _ptr(lse1), _ptr(lse2),
                               _stream(stream))


def streamkl_fwd_sym(q1, k1, q2, k2, B, Hq, Hkv, NQ, NK, d, scale, causal, kl12, kl21, lse1, lse2,
                     stream=None):
    return load().streamkl_fwd_sym(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), B, Hq, Hkv, NQ, NK, d,
                                   float(scale), int(bool(causal)), _ptr(kl12), _ptr(kl21), _ptr(lse1),
                                   _ptr(lse2), _stream(stream))


def streamkl_fwd_splitk(q1, k1, q2, k2, B, Hq, Hkv, NQ, NK, d, scale, causal, splits, kl, lse1, lse2,
                        workspace, workspace_bytes, stream=None):
    return load().streamkl_fwd_splitk(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), B, Hq, Hkv, NQ, NK, d,
                                      float(scale), int(bool(causal)), int(splits), _ptr(kl),
                                      _ptr(lse1), _ptr(lse2), _ptr(workspace), int(workspace_bytes),
                                      _stream(stream))


def streamkl_fwd_splits(B, Hq, NQ, NK):
    return load().streamkl_fwd_splits(B, Hq, NQ, NK)


def streamkl_fwd_splitk_workspace_bytes(B, Hq, NQ, NK, splits):
    return load().streamkl_fwd_splitk_workspace_bytes(B, Hq, NQ, NK, splits)


def streamkl_bwd(mode, q1, k1, q2, k2, kl, lse1, lse2, dkl, B, Hq, Hkv, NQ, NK, d, scale, causal,
                 dq, dk, workspace, workspace_bytes, stream=None):
    return load().streamkl_bwd(int(mode), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), _ptr(kl),
                               _ptr(lse1), _ptr(lse2), _ptr(dkl), B, Hq, Hkv, NQ, NK, d,
                               float(scale), int(bool(causal)), _ptr(dq), _ptr(dk),
                               _ptr(workspace), int(workspace_bytes), _stream(stream))


# Built-in scratch of streamkl_bwd_noalloc (STREAMKL_NOALLOC_SCRATCH_BYTES in the header).
NOALLOC_SCRATCH_BYTES = 32 << 20


def streamkl_bwd_noalloc(mode, q1, k1, q2, k2, kl, lse1, lse2, dkl, B, Hq, Hkv, NQ, NK, d, scale,
                         causal, dq, dk, stream=None):
    """Backward without a workspace argument, for callers that may not allocate device
    memory: the library's fixed 32 MiB built-in buffer holds what streamkl_bwd keeps in its
    workspace (the dK accumulator, plus the dQ partial sums when keys are split into ranges),
    so sizes with streamkl_bwd_workspace_bytes(...) > 32 MiB return ERR_UNSUPPORTED.  Calls
    that can overlap on the GPU share that buffer and race."""
    return load().streamkl_bwd_noalloc(int(mode), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), _ptr(kl),
                                       _ptr(lse1), _ptr(lse2), _ptr(dkl), B, Hq, Hkv, NQ, NK, d,
                                       float(scale), int(bool(causal)), _ptr(dq), _ptr(dk),
                                       _stream(stream))


def streamkl_bwd_workspace_bytes(B, Hq, Hkv, NQ, NK, d):
    return load().streamkl_bwd_workspace_bytes(B, Hq, Hkv, NQ, NK, d)


def streamkl_device_status(stream=None):
    return load().streamkl_device_status(_stream(stream))


def streamkl_selftest_watchdog(starve, stream=None):
    """Runs the bounded-wait self-test; returns (status, [ns of wait 0, ns of wait 1])."""
    ns = (ctypes.c_longlong * 2)()
    rc = load().streamkl_selftest_watchdog(int(starve), ns, _stream(stream))
    return rc, [ns[0], ns[1]]


def streamkl_probe_exp2(kind, iters, stream=None):
    """Launches the exponential-throughput probe; returns (status, exponentials evaluated)."""
    n = ctypes.c_longlong(0)
    rc = load().streamkl_probe_exp2(int(kind), int(iters), ctypes.byref(n), _stream(stream))
    return rc, n.value


def streamkl_num_sms():
    return load().streamkl_num_sms()


def streamkl_probe_clock(duration_ns, interval_ns, samples, stream=None):
    """Launches the clock probe into `samples` (int64 device tensor of 2 + 2 * max_pairs
    elements); returns the status."""
    import torch
    if samples.dtype != torch.int64 or not samples.is_cuda or not samples.is_contiguous() \
            or samples.numel() < 6:
        raise ValueError("samples must be a contiguous int64 CUDA tensor of at least 6 elements")
    n = samples.numel()
    return load().streamkl_probe_clock(int(duration_ns), int(interval_ns), _ptr(samples),
                                       int((n - 2) // 2), _stream(stream))


def streamkl_eval_exp2(kind, x, stream=None):
    """2^x by the kernels' exponential path `kind` (0: exponential unit, 1: FMA-pipe
    polynomial) for a contiguous fp32 CUDA tensor; returns (status, y)."""
    import torch
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous fp32 CUDA tensor")
    y = torch.empty_like(x)
    rc = load().streamkl_eval_exp2(int(kind), _ptr(x), _ptr(y), x.numel(), _stream(stream))
    return rc, y


def _cache_ref(cache):
    """A pointer to the streamkl_cache of a PagedCache or CacheStruct (None stays NULL)."""
    if cache is None:
        return None
    return ctypes.byref(cache.struct if isinstance(cache, PagedCache) else cache)


def streamkl_cache_append(cache, k, v, table, width, start, count, B, NT, stream=None):
    return load().streamkl_cache_append(_cache_ref(cache), _ptr(k), _ptr(v), _ptr(table), width, _ptr(start),
                                        _ptr(count), B, NT, _stream(stream))


def streamkl_cache_gather(cache, table, width, start, count, B, NT, k, v, stream=None):
    return load().streamkl_cache_gather(_cache_ref(cache), _ptr(table), width, _ptr(start), _ptr(count), B, NT,
                                        _ptr(k), _ptr(v), _stream(stream))


def streamkl_paged_workspace_bytes(B, Hq, Hkv, NQ, d):
    return load().streamkl_paged_workspace_bytes(B, Hq, Hkv, NQ, d)


def streamkl_paged_attn(cache, q, table, width, lengths, B, Hq, NQ, scale, causal, out, lse, workspace,
                        workspace_bytes, stream=None):
    return load().streamkl_paged_attn(_cache_ref(cache), _ptr(q), _ptr(table), width, _ptr(lengths), B, Hq, NQ,
                                      float(scale), int(bool(causal)), _ptr(out), _ptr(lse), _ptr(workspace),
                                      int(workspace_bytes), _stream(stream))


def streamkl_paged_kl(cache1, q1, cache2, q2, table, width, lengths, B, Hq, NQ, scale, causal, kl, lse1, lse2,
                      workspace, workspace_bytes, stream=None):
    return load().streamkl_paged_kl(_cache_ref(cache1), _ptr(q1), _cache_ref(cache2), _ptr(q2), _ptr(table), width,
                                    _ptr(lengths), B, Hq, NQ, float(scale), int(bool(causal)), _ptr(kl),
                                    _ptr(lse1), _ptr(lse2), _ptr(workspace), int(workspace_bytes),
                                    _stream(stream))


def status_string(status):
    return load().streamkl_status_string(int(status)).decode()


def last_cuda_error():
    return load().streamkl_last_cuda_error().decode()


def version():
    return load().streamkl_version()


# ------------------------------------------------------------------ conveniences
def _dims(q1, k1):
    B, Hq, NQ, d = q1.shape
    _, Hkv, NK, _ = k1.shape
    return B, Hq, Hkv, NQ, NK, d


def _check_inputs(q1, k1, q2, k2):
    """Refuses inputs whose shapes or devices disagree: the library sizes every tensor map
    from q1's batch and head dimension and k1's key count, so a mismatch would make a kernel
    read past an allocation."""
    import torch
    for t in (q1, k1, q2, k2):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous bf16 CUDA tensors")
    if q1.dim() != 4 or k1.dim() != 4 or q1.shape != q2.shape or k1.shape != k2.shape:
        raise ValueError("q1/q2 must be [B,Hq,NQ,d], k1/k2 [B,Hkv,NK,d]")
    if q1.shape[0] != k1.shape[0] or q1.shape[3] != k1.shape[3]:
        raise ValueError("q and k must share batch size and head dim (q %s, k %s)"
                         % (tuple(q1.shape), tuple(k1.shape)))
    if k1.shape[1] < 1 or q1.shape[1] % k1.shape[1] != 0:
        raise ValueError("query heads (%d) must be a multiple of KV heads (%d)"
                         % (q1.shape[1], k1.shape[1]))
    if len({t.device for t in (q1, k1, q2, k2)}) != 1:
        raise ValueError("q1, k1, q2, k2 must be on one device")


def _check_tensor(name, t, shape, dtype, device):
    """Refuses a tensor the kernels would read or write out of bounds or misinterpret."""
    if t is None:
        raise ValueError("%s is required" % name)
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s (got %s %s on %s)"
                         % (name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device))


def _check_workspace(workspace, nbytes, device):
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    have = workspace.numel() * workspace.element_size()
    if have < nbytes:
        raise ValueError("workspace holds %d bytes, %d needed" % (have, nbytes))


def fwd(q1, k1, q2, k2, scale=None, causal=False, out=None, stream=None):
    """Returns (kl, lse1, lse2), fp32 [B,Hq,NQ].  Pass k2 = k1 (same tensor) for shared keys."""
    import torch
    _check_inputs(q1, k1, q2, k2)
    B, Hq, Hkv, NQ, NK, d = _dims(q1, k1)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = tuple(torch.empty((B, Hq, NQ), dtype=torch.float32, device=q1.device) for _ in range(3))
    for name, o in zip(("kl", "lse1", "lse2"), out):
        _check_tensor(name, o, (B, Hq, NQ), torch.float32, q1.device)
    rc = streamkl_fwd(q1, k1, q2, k2, B, Hq, Hkv, NQ, NK, d, scale, causal, *out, stream=stream)
    if rc != OK:
        raise StreamKLError(rc, "streamkl_fwd")
    return out


def fwd_sym(q1, k1, q2, k2, scale=None, causal=False, out=None, stream=None):
    """Returns (kl12, kl21, lse1, lse2), fp32 [B,Hq,NQ]: KL(P1||P2), KL(P2||P1) and both LSEs in
    one pass over the keys; kl12 + kl21 is the symmetric divergence."""
    import torch
    _check_inputs(q1, k1, q2, k2)
    B, Hq, Hkv, NQ, NK, d = _dims(q1, k1)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = tuple(torch.empty((B, Hq, NQ), dtype=torch.float32, device=q1.device) for _ in range(4))
    for name, o in zip(("kl12", "kl21", "lse1", "lse2"), out):
        _check_tensor(name, o, (B, Hq, NQ), torch.float32, q1.device)
    rc = streamkl_fwd_sym(q1, k1, q2, k2, B, Hq, Hkv, NQ, NK, d, scale, causal, *out, stream=stream)
    if rc != OK:
        raise StreamKLError(rc, "streamkl_fwd_sym")
    return out


def fwd_splitk(q1, k1, q2, k2, scale=None, causal=False, splits=0, out=None, workspace=None,
               stream=None):
    """Split-K forward (key ranges merged exactly); same outputs as fwd.  splits = 0 lets
    the library choose; `workspace` (fp32 tensor) is allocated here when not given."""
    import torch
    _check_inputs(q1, k1, q2, k2)
    B, Hq, Hkv, NQ, NK, d = _dims(q1, k1)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = tuple(torch.empty((B, Hq, NQ), dtype=torch.float32, device=q1.device) for _ in range(3))
    for name, o in zip(("kl", "lse1", "lse2"), out):
        _check_tensor(name, o, (B, Hq, NQ), torch.float32, q1.device)
    need = streamkl_fwd_splitk_workspace_bytes(B, Hq, NQ, NK, splits)
    if workspace is None and need > 0:
        workspace = torch.empty((need + 3) // 4, dtype=torch.float32, device=q1.device)
    if workspace is not None:
        _check_workspace(workspace, need, q1.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = streamkl_fwd_splitk(q1, k1, q2, k2, B, Hq, Hkv, NQ, NK, d, scale, causal, splits, *out,
                             workspace, wbytes, stream=stream)
    if rc != OK:
        raise StreamKLError(rc, "streamkl_fwd_splitk")
    return out


def bwd(mode, q1, k1, q2, k2, kl, lse1, lse2, dkl, scale=None, causal=False, out=None,
        workspace=None, stream=None):
    """Returns (dq, dk) of the free distribution: mode 1 -> (dQ2, dK2), mode 2 -> (dQ1, dK1)."""
    import torch
    _check_inputs(q1, k1, q2, k2)
    B, Hq, Hkv, NQ, NK, d = _dims(q1, k1)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    for name, v in zip(("kl", "lse1", "lse2", "dkl"), (kl, lse1, lse2, dkl)):
        _check_tensor(name, v, (B, Hq, NQ), torch.float32, q1.device)
    if out is None:
        out = (torch.empty_like(q1), torch.empty_like(k1))
    _check_tensor("dq", out[0], q1.shape, torch.bfloat16, q1.device)
    _check_tensor("dk", out[1], k1.shape, torch.bfloat16, q1.device)
    nbytes = streamkl_bwd_workspace_bytes(B, Hq, Hkv, NQ, NK, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16) // 4, dtype=torch.float32, device=q1.device)
    _check_workspace(workspace, nbytes, q1.device)
    rc = streamkl_bwd(mode, q1, k1, q2, k2, kl, lse1, lse2, dkl, B, Hq, Hkv, NQ, NK, d, scale,
                      causal, out[0], out[1], workspace, workspace.numel() * workspace.element_size(),
                      stream=stream)
    if rc != OK:
        raise StreamKLError(rc, "streamkl_bwd")
    return out


# ------------------------------------------------------------------ paged key-value cache
# torch, and the extension that does the everyday case of a call (csrc/fastcall.cpp; None where it was not
# built), from the first PagedCache on: these calls are made once per token, and an import statement, a tuple
# or a device object in each check adds up to the time of a kernel.
_torch = None
_fast = None


def _load_fastcall():
    """The extension that was built for this torch version; None where there is none that loads."""
    import importlib.util
    from . import build
    import torch
    path = build.fastcall_path(torch.__version__)
    if not os.path.exists(path):
        return None
    try:
        spec = importlib.util.spec_from_file_location(__package__ + "._fastcall", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError:
        return None
    return module


def _start():
    global _torch, _fast
    import torch
    _torch = torch
    _fastcall = _load_fastcall()
    if _fastcall is None:
        return
    lib = load()
    _fastcall.setup(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.streamkl_paged_attn, lib.streamkl_paged_kl, lib.streamkl_cache_append, lib.streamkl_cache_gather)))
    _fast = _fastcall


class PagedCache:
    """The pages of a key-value cache: k and v [pages, Hkv, page_size, d], bf16 or float8_e4m3fn; with
    e4m3, k_exp and v_exp uint8 [pages, Hkv, page_size] (a row's scale is 2^(byte - 127)).  v may be
    None for a cache that only paged_kl reads.  Holds the tensors and the C struct that points to
    them; page tables, lengths and positions are the caller's int32 tensors."""

    def __init__(self, k, v=None, k_exp=None, v_exp=None):
        import torch
        if _torch is None:
            _start()
        if k.dim() != 4 or k.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or not k.is_cuda:
            raise ValueError("k must be a bf16 or float8_e4m3fn CUDA tensor [pages, Hkv, page_size, d]")
        quantised = k.dtype == torch.float8_e4m3fn
        rows = tuple(k.shape[:3])
        _check_tensor("k", k, k.shape, k.dtype, k.device)
        if v is not None:
            _check_tensor("v", v, k.shape, k.dtype, k.device)
        if quantised:
            _check_tensor("k_exp", k_exp, rows, torch.uint8, k.device)
            if v is not None:
                _check_tensor("v_exp", v_exp, rows, torch.uint8, k.device)
        elif k_exp is not None or v_exp is not None:
            raise ValueError("a bf16 cache has no scales")
        pages, Hkv, page_size, d = k.shape
        if d not in (64, 128) or page_size not in (16, 32, 64, 128, 256, 512, 1024) or pages < 1 or Hkv < 1:
            raise ValueError("pages of 16 to 1024 rows (a power of two) and d = 64 or 128 are supported (got %s)"
                             % (tuple(k.shape),))
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.shape = (pages, Hkv, page_size, d)
        self.device = k.device
        self.index = k.get_device()
        self.struct = CacheStruct(_ptr(k), _ptr(v), _ptr(k_exp), _ptr(v_exp),
                                  CACHE_E4M3 if quantised else CACHE_BF16, pages, page_size, Hkv, d)
        self.ref = ctypes.byref(self.struct)
        self.address = ctypes.addressof(self.struct)

    @classmethod
    def empty(cls, pages, Hkv, page_size, d, quantised=False, values=True, device="cuda"):
        """A cache of zeros."""
        import torch
        dtype = torch.float8_e4m3fn if quantised else torch.bfloat16
        n = 2 if values else 1
        rows = [torch.zeros((pages, Hkv, page_size, d), dtype=torch.uint8 if quantised else dtype,
                            device=device).view(dtype) for _ in range(n)]
        exps = [torch.full((pages, Hkv, page_size), 127, dtype=torch.uint8, device=device) if quantised else None
                for _ in range(n)]
        return cls(rows[0], rows[1] if values else None, exps[0], exps[1] if values else None)


PAGED_COUNTER_BYTES = 4096     # STREAMKL_PAGED_COUNTER_BYTES of the header


def _new_workspace(nbytes, device):
    import torch
    workspace = torch.empty(nbytes // 4, dtype=torch.float32, device=device)
    workspace[:PAGED_COUNTER_BYTES // 4].zero_()
    return workspace


def paged_workspace(B, Hq, Hkv, NQ, d, device="cuda"):
    """A workspace for paged_attn and paged_kl of these sizes (or smaller ones), to be kept between calls: its
    first PAGED_COUNTER_BYTES are zero, and every call leaves them so."""
    import torch
    device = torch.device(device)
    with torch.cuda.device(device):
        nbytes = streamkl_paged_workspace_bytes(B, Hq, Hkv, NQ, d)
    if nbytes == 0:
        raise ValueError("unsupported sizes: B %d, Hq %d, Hkv %d, NQ %d, d %d" % (B, Hq, Hkv, NQ, d))
    return _new_workspace(nbytes, device)


def _enter(cache, stream):
    """(guard, stream handle) of a call on a cache's device: what the call allocates belongs to the stream
    it runs on, the caller's `stream` (an object or a handle) or the device's current one."""
    if stream is None:
        guard = None
        if cache.index != _torch._C._cuda_getDevice():
            guard = _torch.cuda.device(cache.device)
            guard.__enter__()
        return guard, _torch._C._cuda_getCurrentRawStream(cache.index)
    if isinstance(stream, int):
        stream = _torch.cuda.ExternalStream(stream, cache.device) if stream else _torch.cuda.default_stream(cache.device)
    if stream.device != cache.device:
        raise ValueError("the stream is on %s, the cache is on %s" % (stream.device, cache.device))
    guard = _torch.cuda.stream(stream)
    guard.__enter__()
    return guard, stream.cuda_stream


def _leave(guard):
    if guard is not None:
        guard.__exit__(None, None, None)


def _given(name, t):
    if t is None:
        raise ValueError("%s is required" % name)


def _need(name, t, dtype, shape, cache):
    """Refuses a tensor that the kernels would misread; `shape` is a tuple."""
    _given(name, t)
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == cache.index and t.is_contiguous()):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s (got %s %s on %s)"
                         % (name, dtype, shape, cache.device, t.dtype, tuple(t.shape), t.device))


def _width(table, B, cache):
    """Pages of a row of the table [B, width]."""
    _given("table", table)
    shape = table.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError("table must be int32 [B, width]")
    _need("table", table, _torch.int32, (B, shape[1]), cache)
    return shape[1]


def _rows_shape(cache, k, v):
    """Shape of dense rows [B, Hkv, rows, d] that fit the cache."""
    _given("k", k)
    shape = tuple(k.shape)
    if cache.v is None:
        raise ValueError("this cache has no values")
    if len(shape) != 4 or shape[1] != cache.shape[1] or shape[3] != cache.shape[3] or shape[0] < 1 or shape[2] < 1:
        raise ValueError("k and v must be [B, %d, rows, %d] (got %s)" % (cache.shape[1], cache.shape[3], shape))
    _need("k", k, _torch.bfloat16, shape, cache)
    _need("v", v, _torch.bfloat16, shape, cache)
    return shape


def cache_append(cache, k, v, table, start, count=None, stream=None):
    """Writes k, v (bf16 [B, Hkv, NT, d]) into the cache: row i < count[b] (NT without `count`) of
    sequence b at position start[b] + i.  table int32 [B, width], start and count int32 [B]."""
    if stream is None and _fast is not None and start is not None:
        rc = _fast.move(cache.address, cache.index, True, k, v, table, start, count)
        if rc is not NotImplemented:
            if rc != OK:
                raise StreamKLError(rc, "streamkl_cache_append")
            return
    B, _, NT, _ = _rows_shape(cache, k, v)
    width = _width(table, B, cache)
    _need("start", start, _torch.int32, (B,), cache)
    if count is not None:
        _need("count", count, _torch.int32, (B,), cache)
    guard, handle = _enter(cache, stream)
    try:
        rc = load().streamkl_cache_append(cache.ref, k.data_ptr(), v.data_ptr(), table.data_ptr(), width, start.data_ptr(),
                                          None if count is None else count.data_ptr(), B, NT, handle)
    finally:
        _leave(guard)
    if rc != OK:
        raise StreamKLError(rc, "streamkl_cache_append")


def cache_gather(cache, table, count, start=None, rows=None, out=None, stream=None):
    """Reads rows back into (k, v), bf16 [B, Hkv, rows, d]: row i < count[b] is the cached row at position
    start[b] + i (from 0 without `start`); rows behind the count are left as they were (zeros in
    tensors allocated here)."""
    if stream is None and out is not None and rows is None and _fast is not None and count is not None:
        rc = _fast.move(cache.address, cache.index, False, out[0], out[1], table, start, count)
        if rc is not NotImplemented:
            if rc != OK:
                raise StreamKLError(rc, "streamkl_cache_gather")
            return out
    _given("table", table)
    if out is None and (rows is None or rows < 1 or table.dim() != 2):
        raise ValueError("out, or rows of at least 1 and a table [B, width], are required")
    guard, handle = _enter(cache, stream)
    try:
        if out is None:
            out = tuple(_torch.zeros((table.shape[0], cache.shape[1], rows, cache.shape[3]), dtype=_torch.bfloat16,
                                     device=cache.device) for _ in range(2))
        k, v = out
        B, _, NT, _ = _rows_shape(cache, k, v)
        if rows is not None and rows != NT:
            raise ValueError("out has %d rows, not %d" % (NT, rows))
        width = _width(table, B, cache)
        _need("count", count, _torch.int32, (B,), cache)
        if start is not None:
            _need("start", start, _torch.int32, (B,), cache)
        rc = load().streamkl_cache_gather(cache.ref, table.data_ptr(), width, None if start is None else start.data_ptr(),
                                          count.data_ptr(), B, NT, k.data_ptr(), v.data_ptr(), handle)
    finally:
        _leave(guard)
    if rc != OK:
        raise StreamKLError(rc, "streamkl_cache_gather")
    return out


def _query_shape(name, q, cache):
    """Shape of queries [B, Hq, NQ, d] that fit the cache."""
    _given(name, q)
    shape = tuple(q.shape)
    if len(shape) != 4 or shape[3] != cache.shape[3] or min(shape) < 1 or shape[1] % cache.shape[1]:
        raise ValueError("%s must be [B, Hq, NQ, %d], Hq a multiple of %d (got %s)"
                         % (name, cache.shape[3], cache.shape[1], shape))
    _need(name, q, _torch.bfloat16, shape, cache)
    return shape


def _scratch(workspace, shape, cache):
    """The caller's workspace, checked, or a new one; (tensor, bytes).  The library checks its size."""
    if workspace is None:
        B, Hq, NQ, d = shape
        nbytes = streamkl_paged_workspace_bytes(B, Hq, cache.shape[1], NQ, d)
        return _new_workspace(nbytes, cache.device), nbytes
    if workspace.dtype is not _torch.float32 or workspace.get_device() != cache.index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous fp32 tensor on %s (see paged_workspace)" % (cache.device,))
    return workspace, workspace.numel() * 4


def paged_attn(q, cache, table, lengths, scale=None, causal=True, out=None, workspace=None, stream=None):
    """Attention of new tokens over the cache: (out bf16 [B, Hq, NQ, d], lse fp32 [B, Hq, NQ]).  lengths int32
    [B] count the new tokens; causal: they are the last NQ and see their own past only.  `workspace`
    (paged_workspace) is allocated here when not given."""
    if out is None and stream is None and _fast is not None:
        done = _fast.attn(q, cache.address, cache.index, table, lengths, cache.shape[3] ** -0.5 if scale is None else scale,
                          causal, workspace)
        if done is not NotImplemented:
            if done[0] != OK:
                raise StreamKLError(done[0], "streamkl_paged_attn")
            return done[1:]
    shape = _query_shape("q", q, cache)
    if cache.v is None:
        raise ValueError("this cache has no values")
    B, Hq, NQ, d = shape
    width = _width(table, B, cache)
    _need("lengths", lengths, _torch.int32, (B,), cache)
    guard, handle = _enter(cache, stream)
    try:
        workspace, nbytes = _scratch(workspace, shape, cache)
        if out is None:
            o, lse = out = _torch.empty_like(q), workspace.new_empty((B, Hq, NQ))
        else:
            o, lse = out
            _need("out", o, _torch.bfloat16, shape, cache)
            _need("lse", lse, _torch.float32, (B, Hq, NQ), cache)
        rc = load().streamkl_paged_attn(cache.ref, q.data_ptr(), table.data_ptr(), width, lengths.data_ptr(), B, Hq, NQ,
                                        d ** -0.5 if scale is None else scale, 1 if causal else 0, o.data_ptr(),
                                        lse.data_ptr(), workspace.data_ptr(), nbytes, handle)
    finally:
        _leave(guard)
    if rc != OK:
        raise StreamKLError(rc, "streamkl_paged_attn")
    return out


def paged_kl(q1, cache1, q2, cache2, table, lengths, scale=None, causal=True, out=None, workspace=None, stream=None):
    """KL(P1 || P2) of two attentions of the new tokens over paged key caches: (kl, lse1, lse2), fp32
    [B, Hq, NQ].  P1 from q1 and cache1's keys, P2 from q2 and cache2's; pass the same cache twice
    for shared keys.  Other arguments as paged_attn."""
    if out is None and stream is None and _fast is not None and cache1.index == cache2.index:
        done = _fast.kl(q1, cache1.address, q2, cache2.address, cache1.index, table, lengths,
                        cache1.shape[3] ** -0.5 if scale is None else scale, causal, workspace)
        if done is not NotImplemented:
            if done[0] != OK:
                raise StreamKLError(done[0], "streamkl_paged_kl")
            return done[1]
    shape = _query_shape("q1", q1, cache1)
    if cache1.shape != cache2.shape or cache1.index != cache2.index:
        raise ValueError("both caches must agree in shape and device (%s on %s, %s on %s)"
                         % (cache1.shape, cache1.device, cache2.shape, cache2.device))
    _need("q2", q2, _torch.bfloat16, shape, cache1)
    B, Hq, NQ, d = shape
    width = _width(table, B, cache1)
    _need("lengths", lengths, _torch.int32, (B,), cache1)
    guard, handle = _enter(cache1, stream)
    try:
        workspace, nbytes = _scratch(workspace, shape, cache1)
        if out is None:
            out = workspace.new_empty((3, B, Hq, NQ)).unbind(0)
        else:
            for name, o in zip(("kl", "lse1", "lse2"), out):
                _need(name, o, _torch.float32, (B, Hq, NQ), cache1)
        kl, lse1, lse2 = out
        rc = load().streamkl_paged_kl(cache1.ref, q1.data_ptr(), cache2.ref, q2.data_ptr(), table.data_ptr(), width,
                                      lengths.data_ptr(), B, Hq, NQ, d ** -0.5 if scale is None else scale,
                                      1 if causal else 0, kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(),
                                      workspace.data_ptr(), nbytes, handle)
    finally:
        _leave(guard)
    if rc != OK:
        raise StreamKLError(rc, "streamkl_paged_kl")
    return out
