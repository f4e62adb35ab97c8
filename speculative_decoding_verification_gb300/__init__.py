"""libspecverify Python binding: argument marshalling for the C ABI, nothing else.

Every function here forwards to the entry point of the same name in libspecverify.so (built
for sm_103a by ``build.build()``).  Tensors are torch CUDA tensors; torch supplies device
memory and the current stream, the computation runs in the library's kernels.  If the shared
library is absent, importing the binding still works but every call raises ImportError; no
other implementation stands in.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import threading

import torch

from . import _abi
from ._abi import (DBG, SV_BF16, SV_F32, SV_MAX_K, STATS_BYTES, STATS_FIELDS, SvError,  # noqa: F401
                   load, status_string)

__all__ = ["sv_verify", "sv_saguaro_sample", "sv_fanout", "sv_cache_keys", "sv_cache_lookup", "sv_topk_rows",
           "sv_mirror_reuse", "sv_rope_frequencies", "sv_rope", "sv_kv_append", "sv_kv_attend", "sv_kv_commit",
           "sv_kv_append8", "sv_kv_attend8", "sv_kv_commit8", "sv_kv_fork", "sv_kv_compact",
           "sv_selftest_timeout", "sv_selftest_exp2", "read_stats", "load", "status_string",
           "SvError", "Workspace"]


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream, dev):
    """The stream a call runs on: the caller's, which must belong to `dev`, or dev's current one.
    The library launches on this stream and plans for the current device, so the two agree."""
    if stream is None:
        s = torch.cuda.current_stream(dev)
    else:
        s = stream
        if s.device != dev:
            raise ValueError(f"the stream is on {s.device}, the call's arrays on {dev}")
    return ctypes.c_void_p(s.cuda_stream)


def _on(dev, fn, *args):
    """Call the library with `dev` current: it takes the device of its workspace plan, static
    scratch and SM count from the current device."""
    with torch.cuda.device(dev):
        return fn(*args)


def _call(dev, stream, fn, *args):
    """_on with the stream (_stream's rule) as the last argument, without the context manager where `dev` is current
    already: the short calls of a decoding step are bound by what the host does for them."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev.index)
    else:
        raw = _stream(stream, dev)
    if torch._C._cuda_getDevice() == dev.index:
        return fn(*args, raw)
    with torch.cuda.device(dev):
        return fn(*args, raw)


def _on_stream(fn):
    """Runs a call with its `stream` argument as the current stream: what the call allocates is that stream's memory, and the
    caller's tensors are marked as used there (and its results on the caller's stream), so that none of them is given out
    again while one of the two streams still works on it."""
    place = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        s = kw.get("stream") if len(args) <= place else args[place]
        if s is None:
            return fn(*args, **kw)
        outer = torch.cuda.current_stream(s.device)
        if s == outer:
            return fn(*args, **kw)
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(s)
        with torch.cuda.stream(s):
            out = fn(*args, **kw)
        for t in out if isinstance(out, tuple) else (out,):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(outer)
        return out
    return call


def _dtype_code(t):
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _rows(t, name):
    """(row pitch in elements, rows per sequence) of a [B, R, V] or [N, V] logit tensor."""
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: the vocabulary axis must be contiguous")
    if t.dim() == 3:
        if t.shape[1] > 1 and t.stride(0) != t.shape[1] * t.stride(1):
            raise ValueError(f"{name}: rows of a sequence must be consecutive rows of one pitch")
        pitch = t.stride(1) if t.shape[1] > 1 else t.stride(0)
        return pitch, t.shape[1]
    if t.dim() == 2:
        return t.stride(0), 1
    raise ValueError(f"{name}: expected [B, R, V] or [N, V]")


def _current_raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _capture_id(index, raw):
    """The capture that `raw`, the current stream of device `index`, belongs to; 0 for none."""
    if torch._C._cuda_getDevice() == index and not torch._C._cuda_isCurrentStreamCapturing():
        return 0
    return load().sv_stream_capture_id(raw)


class Workspace:
    """Device workspaces (torch memory) reused from call to call: one for each host thread, device and current stream, so
    that calls which may run at the same time never share one.

    A call that is captured into a CUDA graph gets a buffer of that capture alone, which is kept as long as the
    Workspace: the graph holds its address.  Capture with a Workspace of your own (workspace=), dropped with the graph,
    to have that memory back."""

    def __init__(self):
        self._local = threading.local()   # .bufs: (device, stream) -> buffer of that stream's memory
        self._captured = {}               # (device, stream, capture) -> buffers, the largest last

    def get(self, nbytes: int, device) -> torch.Tensor:
        index = device.index if type(device) is torch.device else torch.device(device).index
        if index is None:
            index = torch.cuda.current_device()
        raw = _current_raw_stream(index)
        capture = _capture_id(index, raw)
        if capture:
            bufs = self._captured.setdefault((index, raw, capture), [])
            if not bufs or bufs[-1].numel() < nbytes:
                bufs.append(torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device))
            return bufs[-1]
        try:
            bufs = self._local.bufs
        except AttributeError:
            bufs = self._local.bufs = {}
        buf = bufs.get((index, raw))
        if buf is None or buf.numel() < nbytes:
            # The old one goes back to the memory of its own stream, which runs what still uses it first.
            buf = bufs[index, raw] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        return buf


_default_ws = Workspace()


def new_stats(device) -> torch.Tensor:
    return torch.zeros(STATS_BYTES, dtype=torch.uint8, device=device)


def read_stats(t: torch.Tensor) -> dict:
    """Decode an sv_stats block (synchronises with the device)."""
    raw = t.detach().cpu()
    i32 = raw.view(torch.int32)
    i64 = raw.view(torch.int64)
    out = {"status": int(i32[0]), "error_index": int(i32[1])}
    for k, name in enumerate(STATS_FIELDS[2:]):
        out[name] = int(i64[1 + k])
    return out


def _cuda(t, name):
    """The CUDA device of a logit tensor: the device entry points read device memory only."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (host buffers go through sv_verify_host)")
    return t.device


def _arr(t, name, dtype, n, dev):
    """t as the library reads or writes it: a contiguous `dtype` tensor on `dev` holding at least
    n elements.  Anything else would be read with the wrong layout or past its end, so it is
    refused here, before any work is queued."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {n}")
    return t


def _opt(t, name, dtype, n, dev):
    return None if t is None else _arr(t, name, dtype, n, dev)


def _out(t, name, dtype, shape, dev):
    """An output array: allocated when the caller passes none, else checked like an input."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    n = 1
    for d in shape:
        n *= d
    return _arr(t, name, dtype, n, dev)


def _pair(first, second, names, K, dev):
    """Row pitch and rows of the first logit tensor and, when K > 0, of the second (same dtype and
    device); with K = 0 the second is not read and its pointer is null."""
    f_pitch, _ = _rows(first, names[0])
    if K == 0:
        return f_pitch, f_pitch, 1, ctypes.c_void_p(0)
    if _cuda(second, names[1]) != dev:
        raise ValueError(f"{names[0]} and {names[1]} must be on one device")
    if second.dtype != first.dtype:
        raise TypeError(f"{names[0]} and {names[1]} logits must share a dtype")
    s_pitch, s_rows = _rows(second, names[1])
    return f_pitch, s_pitch, s_rows, _ptr(second)


def _seq_inputs(draft_tokens, uniforms, temperature, top_p, top_k, B, K, dev):
    """The per-sequence inputs of the verify entry points, checked (draft tokens only when K > 0)."""
    if K > 0:
        _arr(draft_tokens, "draft_tokens", torch.int32, B * K, dev)
    _arr(uniforms, "uniforms", torch.float64, B * (K + 1), dev)
    _arr(temperature, "temperature", torch.float32, B, dev)
    _opt(top_p, "top_p", torch.float32, B, dev)
    _opt(top_k, "top_k", torch.int32, B, dev)


def _stats(stats, dev):
    return new_stats(dev) if stats is None else _arr(stats, "stats", torch.uint8, STATS_BYTES, dev)


@_on_stream
def sv_verify(target, draft, draft_tokens, uniforms, temperature, top_p=None, saguaro_F=0, saguaro_C=1.0,
              accept_len=None, out_tokens=None, debug=False, stats=None, workspace=None, stream=None, lazy=False,
              top_k=None):
    """sv_verify (or, with lazy=True, sv_verify_lazy: same outputs, rows after each sequence's
    first rejection left unread) on torch CUDA tensors.

    target [B, K+1, V] and draft [B, R>=K, V] (float32 or bfloat16, same dtype); draft_tokens
    int32 [B, K]; uniforms float64 [B, K+1]; temperature float32 [B]; top_p float32 [B] or None;
    top_k int32 [B] or None (top-k acts before top-p).
    Returns (accept_len int32 [B], out_tokens int32 [B, K+1], debug float64 [B, K+1, 8] or None,
    stats uint8 block).
    """
    lib = load()
    B, K1, V = target.shape
    K = K1 - 1
    dev = _cuda(target, "target")
    t_pitch, d_pitch, d_rows, d_ptr = _pair(target, draft, ("target", "draft"), K, dev)
    _seq_inputs(draft_tokens, uniforms, temperature, top_p, top_k, B, K, dev)
    accept_len = _out(accept_len, "accept_len", torch.int32, (B,), dev)
    out_tokens = _out(out_tokens, "out_tokens", torch.int32, (B, K + 1), dev)
    dbg = torch.empty((B, K + 1, _abi.SV_DEBUG_FIELDS), dtype=torch.float64, device=dev) if debug else None
    stats = _stats(stats, dev)
    ws_bytes = lib.sv_verify_workspace_size(B, K, V)
    ws = (workspace or _default_ws).get(ws_bytes, dev)
    fn = lib.sv_verify_lazy if lazy else lib.sv_verify
    code = _on(dev, fn, _ptr(target), t_pitch, d_ptr, d_pitch, d_rows, _dtype_code(target),
              _ptr(draft_tokens if K > 0 else None), _ptr(uniforms), B, K, V, _ptr(temperature),
              _ptr(top_p), _ptr(top_k), int(saguaro_F), float(saguaro_C), _ptr(accept_len),
              _ptr(out_tokens), _ptr(dbg), _ptr(stats), _ptr(ws), ws.numel(), _stream(stream, dev))
    _abi.check("sv_verify_lazy" if lazy else "sv_verify", code)
    return accept_len, out_tokens, dbg, stats


@_on_stream
def sv_verify_host(target, draft, draft_tokens, uniforms, temperature, top_p=None, saguaro_F=0, saguaro_C=1.0,
                   accept_len=None, out_tokens=None, stats=None, workspace=None, stream=None, top_k=None,
                   device=None):
    """sv_verify_host on host (CPU) tensors: the library copies the rows the verification reads
    (every target row; the draft rows of sequences with a nonzero temperature) and the small
    inputs to the device, verifies there, and copies the outputs back, all on `stream`.

    Pinned tensors (tensor.pin_memory()) make the copies asynchronous and full-speed.  target
    [B, K+1, V] and draft [B, R>=K, V] (float32 or bfloat16); draft_tokens int32 [B, K]; uniforms
    float64 [B, K+1]; temperature float32 [B]; top_p float32 [B] or None; top_k int32 [B] or
    None.  Returns (accept_len int32 [B], out_tokens int32 [B, K+1]) as CPU tensors, valid once
    the stream has synchronised, the stats block (device) and the bytes copied to the device."""
    lib = load()
    for name, t in (("target", target), ("draft", draft), ("draft_tokens", draft_tokens), ("uniforms", uniforms),
                    ("temperature", temperature), ("top_p", top_p), ("top_k", top_k)):
        if t is not None and t.is_cuda:
            raise TypeError(f"sv_verify_host: {name} must be a host tensor")
    dev = torch.device(device if device is not None else "cuda")
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    B, K1, V = target.shape
    K = K1 - 1
    t_pitch, _ = _rows(target, "target")
    if K > 0:
        if draft.dtype != target.dtype:
            raise TypeError("target and draft logits must share a dtype")
        d_pitch, d_rows = _rows(draft, "draft")
        d_ptr = _ptr(draft)
    else:
        d_pitch, d_rows, d_ptr = t_pitch, 1, ctypes.c_void_p(0)
    pin = target.is_pinned()
    if accept_len is None:
        accept_len = torch.empty(B, dtype=torch.int32, pin_memory=pin)
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, pin_memory=pin)
    host = torch.device("cpu")
    for name, t, dt, n in (("draft_tokens", draft_tokens if K > 0 else None, torch.int32, B * K),
                           ("uniforms", uniforms, torch.float64, B * (K + 1)),
                           ("temperature", temperature, torch.float32, B), ("top_p", top_p, torch.float32, B),
                           ("top_k", top_k, torch.int32, B), ("accept_len", accept_len, torch.int32, B),
                           ("out_tokens", out_tokens, torch.int32, B * (K + 1))):
        _opt(t, name, dt, n, host)
    stats = _stats(stats, dev)
    ws_bytes = lib.sv_verify_host_workspace_size(B, K, V, _dtype_code(target))
    ws = (workspace or _default_ws).get(ws_bytes, dev)
    moved = ctypes.c_size_t(0)
    code = _on(dev, lib.sv_verify_host, _ptr(target), t_pitch, d_ptr, d_pitch, d_rows, _dtype_code(target),
                              _ptr(draft_tokens if K > 0 else None), _ptr(uniforms), B, K, V, _ptr(temperature),
                              _ptr(top_p), _ptr(top_k), int(saguaro_F), float(saguaro_C), _ptr(accept_len),
                              _ptr(out_tokens), _ptr(stats), _ptr(ws), ws.numel(), ctypes.c_void_p(ctypes.addressof(moved)),
                              _stream(stream, dev))
    _abi.check("sv_verify_host", code)
    return accept_len, out_tokens, stats, moved.value


@_on_stream
def sv_verify_static(target, draft, draft_tokens, uniforms, temperature, top_p=None, saguaro_F=0, saguaro_C=1.0,
                     accept_len=None, out_tokens=None, debug=None, stats=None, stream=None, top_k=None):
    """sv_verify without a workspace, for callers that cannot allocate device memory (a server
    whose KV-cache pool holds all free HBM, a host program that owns every allocation).

    The library's own scratch array (SV_STATIC_SCRATCH_BYTES, 32 MiB per device) stands in for
    the workspace, so the C call allocates nothing.  Pass accept_len int32 [B], out_tokens int32
    [B, K+1], stats (new_stats) and, optionally, debug float64 [B, K+1, 8] to keep this wrapper
    from allocating them.  Calls that overlap on the GPU share the scratch and race; the first
    call on a device looks up the array's address and belongs before any stream capture.
    Returns (accept_len, out_tokens, debug, stats) like sv_verify.
    """
    lib = load()
    B, K1, V = target.shape
    K = K1 - 1
    dev = _cuda(target, "target")
    t_pitch, d_pitch, d_rows, d_ptr = _pair(target, draft, ("target", "draft"), K, dev)
    _seq_inputs(draft_tokens, uniforms, temperature, top_p, top_k, B, K, dev)
    accept_len = _out(accept_len, "accept_len", torch.int32, (B,), dev)
    out_tokens = _out(out_tokens, "out_tokens", torch.int32, (B, K + 1), dev)
    if debug is True:
        debug = torch.empty((B, K + 1, _abi.SV_DEBUG_FIELDS), dtype=torch.float64, device=dev)
    elif debug is False:
        debug = None
    _opt(debug, "debug", torch.float64, B * (K + 1) * _abi.SV_DEBUG_FIELDS, dev)
    stats = _stats(stats, dev)
    code = _on(dev, lib.sv_verify_static, _ptr(target), t_pitch, d_ptr, d_pitch, d_rows, _dtype_code(target),
                                _ptr(draft_tokens if K > 0 else None), _ptr(uniforms), B, K, V, _ptr(temperature),
                                _ptr(top_p), _ptr(top_k), int(saguaro_F), float(saguaro_C), _ptr(accept_len),
                                _ptr(out_tokens), _ptr(debug), _ptr(stats), _stream(stream, dev))
    if code == _abi.SV_ERR_WORKSPACE:
        raise ValueError(f"sv_verify_static: B={B}, K={K}, V={V} needs more scratch than the "
                         f"{_abi.SV_STATIC_SCRATCH_BYTES >> 20} MiB static array; use sv_verify with a workspace")
    _abi.check("sv_verify_static", code)
    return accept_len, out_tokens, debug, stats


@_on_stream
def sv_fuzzy_verify(verifier, drafter, draft_tokens, uniforms, temperature, tau=0.5, mode="divergence",
                    divergence=False, accept_len=None, out_tokens=None, stats=None, workspace=None, stream=None):
    """sv_fuzzy_verify: one stage of three-model speculative decoding on torch CUDA tensors.

    verifier [B, K+1, V] and drafter [B, R>=K, V] logits (same dtype); draft_tokens int32 [B, K];
    uniforms float64 [B, K+1]; temperature float32 [B]; mode "divergence" (accept while the
    Jensen-Shannon divergence <= tau) or "assisted".  Returns (accept_len, out_tokens,
    divergence float64 [B, K] or None, stats).
    """
    lib = load()
    B, K1, V = verifier.shape
    K = K1 - 1
    dev = _cuda(verifier, "verifier")
    v_pitch, d_pitch, d_rows, d_ptr = _pair(verifier, drafter, ("verifier", "drafter"), K, dev)
    _seq_inputs(draft_tokens, uniforms, temperature, None, None, B, K, dev)
    code_mode = {"divergence": _abi.SV_ACCEPT_DIVERGENCE, "assisted": _abi.SV_ACCEPT_ASSISTED}[mode]
    accept_len = _out(accept_len, "accept_len", torch.int32, (B,), dev)
    out_tokens = _out(out_tokens, "out_tokens", torch.int32, (B, K + 1), dev)
    div = torch.full((B, max(K, 1)), float("nan"), dtype=torch.float64, device=dev) if divergence else None
    stats = _stats(stats, dev)
    ws_bytes = lib.sv_fuzzy_verify_workspace_size(B, K, V)
    ws = (workspace or _default_ws).get(ws_bytes, dev)
    code = _on(dev, lib.sv_fuzzy_verify, _ptr(verifier), v_pitch, d_ptr, d_pitch, d_rows, _dtype_code(verifier),
                               _ptr(draft_tokens if K > 0 else None), _ptr(uniforms), B, K, V, _ptr(temperature),
                               float(tau), code_mode, _ptr(accept_len), _ptr(out_tokens), _ptr(div), _ptr(stats),
                               _ptr(ws), ws.numel(), _stream(stream, dev))
    _abi.check("sv_fuzzy_verify", code)
    return accept_len, out_tokens, (div[:, :K] if div is not None else None), stats


@_on_stream
def sv_tree_verify(target, draft, parents, tokens, uniforms, temperature, accept_len=None, out_tokens=None, path=True,
                   stats=None, workspace=None, stream=None):
    """sv_tree_verify on torch CUDA tensors: target and draft [B, N+1, V] (same dtype; row i follows
    node i), parents and tokens int32 [B, N], uniforms float64 [B, N+1], temperature float32 [B].
    Returns (accept_len int32 [B], out_tokens int32 [B, N+1], path int32 [B, N] or None, stats)."""
    lib = load()
    B, N1, V = target.shape
    N = N1 - 1
    dev = _cuda(target, "target")
    if _cuda(draft, "draft") != dev:
        raise ValueError("target and draft must be on one device")
    if draft.dtype != target.dtype or draft.shape[1] < N1:
        raise TypeError("draft must share the target's dtype and hold N+1 rows per sequence")
    t_pitch, _ = _rows(target, "target")
    d_pitch, _ = _rows(draft, "draft")
    if N > 0:
        _arr(parents, "parents", torch.int32, B * N, dev)
        _arr(tokens, "tokens", torch.int32, B * N, dev)
    _arr(uniforms, "uniforms", torch.float64, B * (N + 1), dev)
    _arr(temperature, "temperature", torch.float32, B, dev)
    accept_len = _out(accept_len, "accept_len", torch.int32, (B,), dev)
    out_tokens = _out(out_tokens, "out_tokens", torch.int32, (B, N + 1), dev)
    if path is True:
        path = torch.empty((B, max(N, 1)), dtype=torch.int32, device=dev)
    elif path is False:
        path = None
    _opt(path, "path", torch.int32, B * N, dev)
    stats = _stats(stats, dev)
    ws = (workspace or _default_ws).get(lib.sv_tree_verify_workspace_size(B, N, V), dev)
    code = _on(dev, lib.sv_tree_verify, _ptr(target), t_pitch, _ptr(draft), d_pitch, _dtype_code(target),
                              _ptr(parents if N > 0 else None), _ptr(tokens if N > 0 else None), _ptr(uniforms), B, N,
                              V, _ptr(temperature), _ptr(accept_len), _ptr(out_tokens), _ptr(path), _ptr(stats),
                              _ptr(ws), ws.numel(), _stream(stream, dev))
    _abi.check("sv_tree_verify", code)
    return accept_len, out_tokens, (path[:, :N] if path is not None else None), stats


@_on_stream
def sv_tree_reuse(parents, tokens, accept_len, out_tokens, reuse_node=None, stream=None):
    """sv_tree_reuse: per sequence the node where the committed prefix ends as a path of the
    drafted tree (parents / tokens int32 [B, N]), or -1."""
    lib = load()
    B, N = parents.shape
    K = out_tokens.shape[1] - 1
    dev = _cuda(parents, "parents")
    _arr(parents, "parents", torch.int32, B * N, dev)
    _arr(tokens, "tokens", torch.int32, B * N, dev)
    _arr(accept_len, "accept_len", torch.int32, B, dev)
    _arr(out_tokens, "out_tokens", torch.int32, B * (K + 1), dev)
    reuse_node = _out(reuse_node, "reuse_node", torch.int32, (B,), dev)
    code = _on(dev, lib.sv_tree_reuse, _ptr(parents), _ptr(tokens), N, _ptr(accept_len), _ptr(out_tokens), K, B,
                             _ptr(reuse_node), _stream(stream, dev))
    _abi.check("sv_tree_reuse", code)
    return reuse_node


@_on_stream
def sv_saguaro_sample(draft, uniforms, temperature, top_p=None, F=0, C=1.0, n_rows=None, tokens=None, debug=False,
                      stats=None, workspace=None, stream=None, top_k=None):
    """sv_saguaro_sample: one token per row j < n_rows of each sequence of draft [B, R, V].
    uniforms float64 [B, n_rows]; temperature float32 [B]; top_p float32 [B] or None; top_k
    int32 [B] or None; returns (tokens int32 [B, n_rows],
    debug float64 [B, n_rows, 4] or None, stats)."""
    lib = load()
    B, R, V = draft.shape
    n_rows = R if n_rows is None else n_rows
    dev = _cuda(draft, "draft")
    pitch, rows = _rows(draft, "draft")
    _arr(uniforms, "uniforms", torch.float64, B * n_rows, dev)
    _arr(temperature, "temperature", torch.float32, B, dev)
    _opt(top_p, "top_p", torch.float32, B, dev)
    _opt(top_k, "top_k", torch.int32, B, dev)
    tokens = _out(tokens, "tokens", torch.int32, (B, n_rows), dev)
    dbg = torch.empty((B, n_rows, 4), dtype=torch.float64, device=dev) if debug else None
    stats = _stats(stats, dev)
    ws_bytes = lib.sv_saguaro_sample_workspace_size(B, n_rows, V)
    ws = (workspace or _default_ws).get(ws_bytes, dev)
    code = _on(dev, lib.sv_saguaro_sample, _ptr(draft), pitch, rows, _dtype_code(draft), B, n_rows, V, _ptr(temperature),
                                 _ptr(top_p), _ptr(top_k), int(F), float(C), _ptr(uniforms), _ptr(tokens),
                                 _ptr(dbg), _ptr(stats),
                                 _ptr(ws), ws.numel(), _stream(stream, dev))
    _abi.check("sv_saguaro_sample", code)
    return tokens, dbg, stats


def sv_fanout(budget: float, a: float, r: float, K: int):
    """Host-only Theorem 12 fan-out: returns (F_real list[float], F_int list[int])."""
    lib = load()
    fr = (ctypes.c_double * (K + 1))()
    fi = (ctypes.c_int32 * (K + 1))()
    code = lib.sv_fanout(float(budget), float(a), float(r), int(K), ctypes.cast(fr, ctypes.c_void_p),
                         ctypes.cast(fi, ctypes.c_void_p))
    _abi.check("sv_fanout", code)
    return list(fr), list(fi)


def _host_i32(values):
    arr = (ctypes.c_int32 * len(values))(*[int(v) for v in values])
    return arr, ctypes.cast(arr, ctypes.c_void_p)


@_on_stream
def sv_cache_keys(draft, draft_tokens, F_int, keys=None, stats=None, workspace=None, stream=None):
    """sv_cache_keys: draft [B, R>=K+1, V]; draft_tokens int32 [B, K]; F_int host list of K+1 ints.
    Returns keys int32 [B, sum F_int]."""
    lib = load()
    B, R, V = draft.shape
    K = len(F_int) - 1
    dev = _cuda(draft, "draft")
    pitch, rows = _rows(draft, "draft")
    if K > 0:
        _arr(draft_tokens, "draft_tokens", torch.int32, B * K, dev)
    keys = _out(keys, "keys", torch.int32, (B, int(sum(F_int))), dev)
    stats = _stats(stats, dev)
    f_arr, f_ptr = _host_i32(F_int)
    ws_bytes = lib.sv_cache_keys_workspace_size(B, K, V)
    ws = (workspace or _default_ws).get(ws_bytes, dev)
    code = _on(dev, lib.sv_cache_keys, _ptr(draft), pitch, rows, _dtype_code(draft), _ptr(draft_tokens), f_ptr, B, K, V,
                             _ptr(keys), _ptr(stats), _ptr(ws), ws.numel(), _stream(stream, dev))
    _abi.check("sv_cache_keys", code)
    return keys, stats


@_on_stream
def sv_cache_lookup(accept_len, out_tokens, keys, F_int, hit=None, stream=None):
    lib = load()
    B = accept_len.shape[0]
    K = len(F_int) - 1
    dev = _cuda(accept_len, "accept_len")
    _arr(accept_len, "accept_len", torch.int32, B, dev)
    _arr(out_tokens, "out_tokens", torch.int32, B * (K + 1), dev)
    _arr(keys, "keys", torch.int32, B * int(sum(F_int)), dev)
    hit = _out(hit, "hit", torch.uint8, (B,), dev)
    f_arr, f_ptr = _host_i32(F_int)
    code = _on(dev, lib.sv_cache_lookup, _ptr(accept_len), _ptr(out_tokens), _ptr(keys), f_ptr, B, K, _ptr(hit),
                               _stream(stream, dev))
    _abi.check("sv_cache_lookup", code)
    return hit


@_on_stream
def sv_topk_rows(logits, kappa, temperature=None, ids=None, logprobs=None, stats=None, workspace=None, stream=None):
    """sv_topk_rows: logits [N, V]; returns (ids int32 [N, kappa], logprobs float64 [N, kappa], stats)."""
    lib = load()
    N, V = logits.shape
    dev = _cuda(logits, "logits")
    pitch, _ = _rows(logits, "logits")
    _opt(temperature, "temperature", torch.float32, N, dev)
    ids = _out(ids, "ids", torch.int32, (N, kappa), dev)
    logprobs = _out(logprobs, "logprobs", torch.float64, (N, kappa), dev)
    stats = _stats(stats, dev)
    ws_bytes = lib.sv_topk_rows_workspace_size(N, V)
    ws = (workspace or _default_ws).get(ws_bytes, dev)
    code = _on(dev, lib.sv_topk_rows, _ptr(logits), pitch, _dtype_code(logits), N, V, int(kappa), _ptr(temperature), _ptr(ids),
                            _ptr(logprobs), _ptr(stats), _ptr(ws), ws.numel(), _stream(stream, dev))
    _abi.check("sv_topk_rows", code)
    return ids, logprobs, stats


@_on_stream
def sv_mirror_reuse(branches, accept_len, out_tokens, reuse=None, stream=None):
    lib = load()
    B, kappa, gamma = branches.shape
    dev = _cuda(branches, "branches")
    _arr(branches, "branches", torch.int32, B * kappa * gamma, dev)
    _arr(accept_len, "accept_len", torch.int32, B, dev)
    _arr(out_tokens, "out_tokens", torch.int32, B * (gamma + 1), dev)
    reuse = _out(reuse, "reuse", torch.uint8, (B,), dev)
    code = _on(dev, lib.sv_mirror_reuse, _ptr(branches), _ptr(accept_len), _ptr(out_tokens), B, kappa, gamma, _ptr(reuse),
                               _stream(stream, dev))
    _abi.check("sv_mirror_reuse", code)
    return reuse


def _style(style):
    code = _abi.SV_ROPE_STYLES.get(style)
    if code is None:
        raise ValueError(f"style must be one of {sorted(_abi.SV_ROPE_STYLES)}, got {style!r}")
    return code


def _heads(t, name, like=None):
    """(row stride, head stride) in elements of a [rows, heads, dim] or [B, n, heads, dim] tensor whose
    rows lie one stride apart."""
    shape, st = t.shape, t.stride()
    if len(shape) == 4:
        if shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
            raise ValueError(f"{name}: rows of a sequence must be consecutive rows of one stride")
        row = st[1] if shape[1] > 1 else st[0]
    elif len(shape) == 3:
        row = st[0]
    else:
        raise ValueError(f"{name}: expected [rows, heads, dim] or [B, n, heads, dim]")
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    if like is not None:
        if t.get_device() != like.get_device():
            raise ValueError(f"{name} must be on {like.device}, got {t.device}")
        if t.dtype is not like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    return row, st[-2]


def _ints(t, name, dtype, n, dev):
    """_arr's checks for the small arrays of a block, cheapest first; its address."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == dev.index and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    return _arr(t, name, dtype, n, dev).data_ptr()


def sv_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                        low: float = 1.0, high: float = 32.0, original_len: int = 0):
    """Host-only: the frequencies of sv_rope (list of rotary_dim/2 floats) and their magnitude.  scaling: "none",
    "linear", "base", "turns" or "dims" (formulas in specverify.h)."""
    if scaling not in _abi.SV_ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_abi.SV_ROPE_SCALINGS)}, got {scaling!r}")
    lib = load()
    f = (ctypes.c_float * max(1, rotary_dim // 2))()
    mag = ctypes.c_float(0.0)
    code = lib.sv_rope_frequencies(int(rotary_dim), float(base), _abi.SV_ROPE_SCALINGS[scaling], float(factor), float(low),
                                   float(high), int(original_len), ctypes.addressof(f), ctypes.addressof(mag))
    _abi.check("sv_rope_frequencies", code)
    return list(f), mag.value


@_on_stream
def sv_rope(x, positions, inv_freq, style="half", magnitude=1.0, backward=False, out=None, stream=None):
    """sv_rope: rotary positions of x [rows, heads, dim] or [B, n, heads, dim] (float32 or bfloat16).

    positions int32 [rows]; inv_freq float32 [rotary_dim/2] on the device; style "half" or "interleaved".
    backward=True takes the gradient of the output to the input's.  out may be x.  Returns out."""
    lib = load()
    dev = _cuda(x, "x")
    shape, (row, head) = x.shape, _heads(x, "x")
    rows = shape[0] if len(shape) == 3 else shape[0] * shape[1]
    pos = _ints(positions, "positions", torch.int32, rows, dev)
    freq = _ints(inv_freq, "inv_freq", torch.float32, 1, dev)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=dev)
    o_row, o_head = _heads(out, "out", x)
    if out.shape != shape:
        raise ValueError(f"out must have shape {tuple(shape)}")
    code = _call(dev, stream, lib.sv_rope, x.data_ptr(), row, head, out.data_ptr(), o_row, o_head, _dtype_code(x), rows, shape[-2],
                 shape[-1], pos, freq, 2 * inv_freq.numel(), _style(style), magnitude, bool(backward))
    if code:
        _abi.check("sv_rope", code)
    return out


def _paged(k_cache, v_cache, dims):
    """(device, shape, strides) of paged tensors [pages, page_size, kv_heads, dim] (with a leading layer axis where dims is 5): one shape,
    dtype, device and set of strides for keys and values."""
    dev = _cuda(k_cache, "k_cache")
    shape, st = k_cache.shape, k_cache.stride()
    if len(shape) != dims:
        raise ValueError(f"k_cache: expected {dims} axes, [{'layers, ' if dims == 5 else ''}pages, page_size, kv_heads, dim]")
    if v_cache.shape != shape or v_cache.stride() != st:
        raise ValueError("k_cache and v_cache must share their shape and strides")
    if v_cache.dtype is not k_cache.dtype:
        raise TypeError("k_cache and v_cache must share a dtype")
    if v_cache.get_device() != dev.index:
        raise ValueError("k_cache and v_cache must be on one device")
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("k_cache: the last axis must be contiguous")
    return dev, shape, st


def _kv_cache(k_cache, v_cache, dims):
    """_paged's, and the packed sv_kv_cache."""
    dev, shape, st = _paged(k_cache, v_cache, dims)
    return dev, shape, st, _abi.KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), st[-4], st[-3], st[-2], shape[-4], shape[-3],
                                              shape[-2], shape[-1], _dtype_code(k_cache))


def _on_device(t, name, dev):
    if t.get_device() != dev.index:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _page_table(page_table, B, dev, name="page_table"):
    """(address, pitch, pages, B) of a page table, checked."""
    shape, st = page_table.shape, page_table.stride()
    if len(shape) != 2 or (B is not None and shape[0] != B) or page_table.dtype is not torch.int32 or \
            page_table.get_device() != dev.index or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be an int32 [{'B' if B is None else B}, pages] tensor on {dev} with contiguous rows")
    return page_table.data_ptr(), st[0], shape[1], shape[0]


def _kv_batch(dev, context_len, page_table, shape, row_start, parents, max_rows):
    """(B, rows, packed sv_kv_batch) of a call whose row tensors have `shape`."""
    table, pitch, pages, B = _page_table(page_table, None, dev)
    ctx = _ints(context_len, "context_len", torch.int32, B, dev)
    starts = par = 0
    if row_start is None:
        if len(shape) != 4 or shape[0] != B:
            raise ValueError(f"without row_start the block's tensors are [B, n, heads, dim] with B = {B}")
        n = shape[1]
        rows = B * n
        if parents is not None:
            if parents.dim() == 2 and parents.shape[1] != n - 1:   # would be read with the wrong row length
                raise ValueError(f"parents must be [B, n - 1] = [{B}, {n - 1}], got {list(parents.shape)}")
            par = _ints(parents, "parents", torch.int32, B * (n - 1), dev)
    else:
        if len(shape) != 3:
            raise ValueError("with row_start the block's tensors are [rows, heads, dim]")
        if parents is not None:
            raise ValueError("parents needs blocks of one size (no row_start)")
        starts = _ints(row_start, "row_start", torch.int32, B + 1, dev)
        rows = shape[0]
        n = rows if max_rows is None else int(max_rows)
    return B, rows, _abi.KV_BATCH.pack(ctx, table, starts, par, pitch, pages, B, max(n, 1), rows)


def _append(fn, dev, c_shape, cache, dtype, like, k, v, context_len, page_table, q, q_out, inv_freq, style, magnitude, parents, row_start,
            max_rows, stats, stream):
    """The body of sv_kv_append and sv_kv_append8; k, v and q are of the type of `like` and on its device."""
    shape, (k_row, k_head), (v_row, v_head) = k.shape, _heads(k, "k", like), _heads(v, "v", like)
    if v.shape != shape or shape[-2:] != c_shape[-2:]:
        raise ValueError("k and v must share a shape that ends in the cache's [kv_heads, dim]")
    _, rows, batch = _kv_batch(dev, context_len, page_table, shape, row_start, parents, max_rows)
    freq = rotary = 0
    if inv_freq is not None:
        freq, rotary = _ints(inv_freq, "inv_freq", torch.float32, 1, dev), 2 * inv_freq.numel()
    q_row = q_head = o_row = o_head = heads = q_ptr = o_ptr = 0
    if q is not None:
        q_shape, (q_row, q_head) = q.shape, _heads(q, "q", like)
        if q_shape[:-2] != shape[:-2] or q_shape[-1] != shape[-1]:
            raise ValueError("q must have the rows and head width of k")
        if q_out is None:
            q_out = torch.empty(q_shape, dtype=q.dtype, device=dev)
        o_row, o_head = _heads(q_out, "q_out", like)
        if q_out.shape != q_shape:
            raise ValueError(f"q_out must have shape {tuple(q_shape)}")
        heads, q_ptr, o_ptr = q_shape[-2], q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    st = _stats(stats, dev).data_ptr() if stats is not None else 0
    if rows == 0:
        return q_out
    code = _call(dev, stream, fn, cache, batch, *dtype, q_ptr, q_row, q_head, o_ptr, o_row, o_head, heads, k.data_ptr(), k_row,
                 k_head, v.data_ptr(), v_row, v_head, freq, rotary, _style(style), magnitude, st)
    if code:
        _abi.check(fn.__name__, code)
    return q_out


@_on_stream
def sv_kv_append(k, v, k_cache, v_cache, context_len, page_table, q=None, q_out=None, inv_freq=None, style="half",
                 magnitude=1.0, parents=None, row_start=None, max_rows=None, stats=None, stream=None):
    """sv_kv_append: write the block's keys and values to the paged cache, rotating keys and queries.

    k, v [B, n, kv_heads, dim], q [B, n, heads, dim] or None (views of one projection are fine); k_cache, v_cache
    [pages, page_size, kv_heads, dim]; context_len int32 [B]; page_table int32 [B, pages].  inv_freq float32
    [rotary_dim/2] or None (no rotation).  parents int32 [B, n-1]: the block is a tree (as sv_tree_verify's).
    row_start int32 [B+1]: ragged blocks, with k, v, q [rows, heads, dim] and at most max_rows rows a sequence.
    Returns the rotated queries (q_out, which may be q), or None without q.  Device-side errors are written to
    stats where one is passed (new_stats)."""
    lib = _abi.load_packed()
    dev, c_shape, _, cache = _kv_cache(k_cache, v_cache, 4)
    return _append(lib.sv_kv_append, dev, c_shape, cache, (), k_cache, k, v, context_len, page_table, q, q_out, inv_freq, style, magnitude,
                   parents, row_start, max_rows, stats, stream)


@functools.lru_cache(maxsize=1024)
def _attend_ws_bytes(rows, heads, dim, B, groups):
    return load().sv_kv_attend_workspace_size(rows, heads, dim, B, groups)


def _attend(fn, dev, c_shape, cache, dtype, like, q, context_len, page_table, scale, parents, row_start, max_rows, group_start, prefix_len, out,
            lse, stats, workspace, stream):
    """The body of sv_kv_attend and sv_kv_attend8; q and out are of the type of `like` and on its device."""
    shape, (q_row, q_head) = q.shape, _heads(q, "q", like)
    heads, dim = shape[-2], shape[-1]
    if dim != c_shape[-1]:
        raise ValueError("q must have the cache's head width")
    B, rows, batch = _kv_batch(dev, context_len, page_table, shape, row_start, parents, max_rows)
    groups = starts = lens = 0
    if (group_start is None) != (prefix_len is None):
        raise ValueError("group_start and prefix_len come together")
    if prefix_len is not None:
        groups = prefix_len.numel()
        lens = _ints(prefix_len, "prefix_len", torch.int32, 1, dev)
        starts = _ints(group_start, "group_start", torch.int32, groups + 1, dev)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=dev)
    o_row, o_head = _heads(out, "out", like)
    if out.shape != shape:
        raise ValueError(f"out must have shape {tuple(shape)}")
    if lse is True:
        lse = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    elif lse is False:
        lse = None
    else:
        _opt(lse, "lse", torch.float32, rows * heads, dev)
    st = _stats(stats, dev).data_ptr() if stats is not None else 0
    if rows == 0:
        return out, lse
    ws = (workspace or _default_ws).get(_attend_ws_bytes(rows, heads, dim, B, groups), dev)
    code = _call(dev, stream, fn, cache, batch, *dtype, q.data_ptr(), q_row, q_head, heads,
                 dim ** -0.5 if scale is None else scale, starts, lens, groups, out.data_ptr(), o_row, o_head,
                 lse.data_ptr() if lse is not None else 0, st, ws.data_ptr(), ws.numel())
    if code:
        _abi.check(fn.__name__, code)
    return out, lse


@_on_stream
def sv_kv_attend(q, k_cache, v_cache, context_len, page_table, scale=None, parents=None, row_start=None, max_rows=None,
                 group_start=None, prefix_len=None, out=None, lse=False, stats=None, workspace=None, stream=None):
    """sv_kv_attend: attention of the block's rows over the paged cache, their own tokens included.

    q [B, n, heads, dim] (or [rows, heads, dim] with row_start); the other arguments as sv_kv_append's.  scale defaults to
    dim ** -0.5.  group_start int32 [G+1] and prefix_len int32 [G]: the sequences of a group share their first
    prefix_len tokens, which are read once for all of them.  lse: True, or a float32 tensor of q's shape without
    the last axis.  out must not overlap q.  With row_start, max_rows picks the kernel: left out, all rows count as one
    block's, which is right and may be slower.  Returns (out, lse or None)."""
    lib = _abi.load_packed()
    dev, c_shape, _, cache = _kv_cache(k_cache, v_cache, 4)
    return _attend(lib.sv_kv_attend, dev, c_shape, cache, (), k_cache, q, context_len, page_table, scale, parents, row_start, max_rows,
                   group_start, prefix_len, out, lse, stats, workspace, stream)


def _commit(fn, dev, cache, layers, context_len, page_table, accept_len, path, context_out, stats, stream, row_start):
    """The body of sv_kv_commit and sv_kv_commit8; layers: their number and strides."""
    B, N = path.shape
    table, pitch, pages, _ = _page_table(page_table, B, dev)
    ctx = _ints(context_len, "context_len", torch.int32, B, dev)
    acc = _ints(accept_len, "accept_len", torch.int32, B, dev)
    nodes = _ints(path, "path", torch.int32, B * N, dev)
    if context_out is not None and context_out.data_ptr() == ctx:
        raise ValueError("context_out must not be context_len")
    context_out = _out(context_out, "context_out", torch.int32, (B,), dev)
    starts = 0 if row_start is None else _ints(row_start, "row_start", torch.int32, B + 1, dev)
    st = _stats(stats, dev).data_ptr() if stats is not None else 0
    batch = _abi.KV_BATCH.pack(ctx, table, starts, 0, pitch, pages, B, N + 1, B * (N + 1))
    code = _call(dev, stream, fn, cache, batch, *layers, acc, nodes if N else 0, context_out.data_ptr(), st)
    if code:
        _abi.check(fn.__name__, code)
    return context_out


@_on_stream
def sv_kv_commit(k_cache, v_cache, context_len, page_table, accept_len, path, context_out=None, stats=None, stream=None,
                 row_start=None):
    """sv_kv_commit: after sv_tree_verify, move the accepted path's keys and values to consecutive slots in every
    layer.  k_cache, v_cache [layers, pages, page_size, kv_heads, dim]; accept_len int32 [B] and path int32 [B, N]
    as sv_tree_verify gives them.  row_start int32 [B+1]: the blocks were ragged, as in sv_kv_append (at most N + 1 rows a
    sequence).  Returns context_out int32 [B]: context_len + 1 + accept_len, or context_len of an empty block."""
    lib = _abi.load_packed()
    dev, c_shape, strides, cache = _kv_cache(k_cache, v_cache, 5)
    return _commit(lib.sv_kv_commit, dev, cache, (c_shape[0], strides[0]), context_len, page_table, accept_len, path, context_out, stats, stream,
                   row_start)


def _cache8(k_cache, v_cache, k_scale, v_scale, dims):
    """(device, shape, strides, strides of the scales) of a cache held in 8 bits: codes [pages, page_size, kv_heads, dim], scales [pages,
    kv_heads] (with a leading layer axis each where dims is 5), one set of strides for keys and values."""
    dev, shape, st = _paged(k_cache, v_cache, dims)
    if k_cache.dtype is not torch.float8_e4m3fn:
        raise TypeError(f"k_cache and v_cache must be torch.float8_e4m3fn, got {k_cache.dtype}")
    return dev, shape, st, _scales(k_scale, v_scale, shape, dev)


def _scales(k_scale, v_scale, shape, dev):
    want, st = shape[:-3] + shape[-2:-1], k_scale.stride()
    if k_scale.dtype not in (torch.uint8, torch.float8_e8m0fnu) or v_scale.dtype is not k_scale.dtype:
        raise TypeError("k_scale and v_scale must both be torch.float8_e8m0fnu or torch.uint8 (biased exponents)")
    if k_scale.shape != want or v_scale.shape != want or v_scale.stride() != st:
        raise ValueError(f"k_scale and v_scale must have shape {tuple(want)} and one set of strides")
    if k_scale.get_device() != dev.index or v_scale.get_device() != dev.index:
        raise ValueError(f"k_scale and v_scale must be on {dev}")
    return st


def _pack8(k_cache, v_cache, k_scale, v_scale, shape, st, sst):
    return _abi.KV_CACHE8.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), st[-4], st[-3], st[-2], sst[-2],
                               sst[-1], shape[-4], shape[-3], shape[-2], shape[-1])


@_on_stream
def sv_kv_append8(k, v, k_cache, v_cache, k_scale, v_scale, context_len, page_table, q=None, q_out=None, inv_freq=None, style="half",
                  magnitude=1.0, parents=None, row_start=None, max_rows=None, stats=None, stream=None):
    """sv_kv_append8: sv_kv_append to a cache held in 8 bits.

    k_cache, v_cache float8_e4m3fn [pages, page_size, kv_heads, dim]; k_scale, v_scale float8_e8m0fnu (or uint8, the same
    bytes) [pages, kv_heads].  The other arguments are sv_kv_append's; k, v and q are float32 or bfloat16.  A page that the
    block writes belongs to one sequence alone: its scale may grow, and its earlier codes are then rounded to it."""
    lib = _abi.load_packed()
    dev, c_shape, st, sst = _cache8(k_cache, v_cache, k_scale, v_scale, 4)
    _on_device(k, "k", dev)
    return _append(lib.sv_kv_append8, dev, c_shape, _pack8(k_cache, v_cache, k_scale, v_scale, c_shape, st, sst), (_dtype_code(k),), k, k, v,
                   context_len, page_table, q, q_out, inv_freq, style, magnitude, parents, row_start, max_rows, stats, stream)


@_on_stream
def sv_kv_attend8(q, k_cache, v_cache, k_scale, v_scale, context_len, page_table, scale=None, parents=None, row_start=None, max_rows=None,
                  group_start=None, prefix_len=None, out=None, lse=False, stats=None, workspace=None, stream=None):
    """sv_kv_attend8: sv_kv_attend over a cache held in 8 bits (arrays as sv_kv_append8's; the other arguments as
    sv_kv_attend's; q and out are float32 or bfloat16).  Returns (out, lse or None)."""
    lib = _abi.load_packed()
    dev, c_shape, st, sst = _cache8(k_cache, v_cache, k_scale, v_scale, 4)
    _on_device(q, "q", dev)
    return _attend(lib.sv_kv_attend8, dev, c_shape, _pack8(k_cache, v_cache, k_scale, v_scale, c_shape, st, sst), (_dtype_code(q),), q, q,
                   context_len, page_table, scale, parents, row_start, max_rows, group_start, prefix_len, out, lse, stats, workspace, stream)


@_on_stream
def sv_kv_commit8(k_cache, v_cache, k_scale, v_scale, context_len, page_table, accept_len, path, context_out=None, stats=None, stream=None,
                  row_start=None):
    """sv_kv_commit8: sv_kv_commit in a cache held in 8 bits: k_cache, v_cache float8_e4m3fn [layers, pages, page_size, kv_heads, dim],
    k_scale, v_scale [layers, pages, kv_heads] as sv_kv_append8's.  Returns context_out."""
    lib = _abi.load_packed()
    dev, c_shape, st, sst = _cache8(k_cache, v_cache, k_scale, v_scale, 5)
    return _commit(lib.sv_kv_commit8, dev, _pack8(k_cache, v_cache, k_scale, v_scale, c_shape, st, sst), (c_shape[0], st[0], sst[0]),
                   context_len, page_table, accept_len, path, context_out, stats, stream, row_start)


def _kv_pool(k_cache, v_cache, k_scale, v_scale):
    """(device, pages, packed sv_kv_pool) of caches [layers, pages, page_size, kv_heads, dim] of any element type."""
    dev, shape, st = _paged(k_cache, v_cache, 5)
    es = k_cache.element_size()   # other one-byte caches (with one scale a tensor, say) have no scales of their pages
    scale_at, sst = (0, 0), (0, 0, 0)
    if (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale come together")
    if k_scale is not None:
        sst = _scales(k_scale, v_scale, shape, dev)
        scale_at = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_cache.dtype is torch.float8_e4m3fn:
        raise ValueError("a cache held in 8 bits has scales: pass k_scale and v_scale")
    return dev, shape[1], _abi.KV_POOL.pack(k_cache.data_ptr(), v_cache.data_ptr(), *scale_at, st[0] * es, st[1] * es, st[2] * es, st[3] * es,
                                            shape[4] * es, *sst, shape[0], shape[1], shape[2], shape[3])


def _table_out(table_out, shape, dev, name="table_out"):
    """table_out or a new one, (address, pitch) of its rows."""
    if table_out is None:
        table_out = torch.empty(shape, dtype=torch.int32, device=dev)
    at, pitch, pages, _ = _page_table(table_out, shape[0], dev, name)
    if pages != shape[1]:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return table_out, at, pitch


@functools.lru_cache(maxsize=1024)
def _fork_ws_bytes(pages, n):
    return load().sv_kv_fork_workspace_size(pages, n)


@functools.lru_cache(maxsize=1024)
def _compact_ws_bytes(pages):
    return load().sv_kv_compact_workspace_size(pages)


@_on_stream
def sv_kv_fork(k_cache, v_cache, page_refs, context_len, page_table, src, reserve=0, k_scale=None, v_scale=None, refs_out=None, table_out=None,
               context_out=None, stats=None, workspace=None, stream=None):
    """sv_kv_fork: a new batch whose sequence j continues sequence src[j] of the old one (-1: an empty sequence).

    k_cache, v_cache [layers, pages, page_size, kv_heads, dim] of any type (with k_scale, v_scale [layers, pages, kv_heads] where
    they are held in 8 bits, float8_e4m3fn); page_refs int32 [pages]: holders of each page, 0 free; context_len int32 [B]; page_table int32 [B,
    max_pages], -1 where an entry names no page; src int32 [N].  Full pages are shared, a partly filled one is copied for all but its
    first new sequence, entries up to slot context + reserve are given free pages.  With N 0 the whole batch ends.  refs_out may be page_refs.
    Returns (table_out [N, max_pages], context_out [N], refs_out [pages])."""
    lib = _abi.load_packed()
    dev, pages, pool = _kv_pool(k_cache, v_cache, k_scale, v_scale)
    table, pitch, width, B = _page_table(page_table, None, dev)
    ctx = _ints(context_len, "context_len", torch.int32, B, dev)
    refs = _ints(page_refs, "page_refs", torch.int32, pages, dev)
    N = src.numel()
    of = _ints(src, "src", torch.int32, N, dev)
    table_out, to, to_pitch = _table_out(table_out, (N, width), dev)
    context_out = ctx_out = _out(context_out, "context_out", torch.int32, (N,), dev)
    if N == 0:   # the whole batch ends: a new one of a single empty sequence, which nobody sees
        none = torch.full((width + 2,), -1, dtype=torch.int32, device=dev)
        N, of, to, to_pitch, ctx_out = 1, none.data_ptr(), none[1:].data_ptr(), width, none[width + 1:]
    refs_out = _out(refs_out, "refs_out", torch.int32, (pages,), dev)
    st = _stats(stats, dev).data_ptr() if stats is not None else 0
    ws = (workspace or _default_ws).get(_fork_ws_bytes(pages, N), dev)
    code = _call(dev, stream, lib.sv_kv_fork, pool, refs, ctx, table, pitch, width, B, of, N, int(reserve), refs_out.data_ptr(), to, to_pitch,
                 ctx_out.data_ptr(), st, ws.data_ptr(), ws.numel())
    if code:
        _abi.check("sv_kv_fork", code)
    return table_out, context_out, refs_out


@_on_stream
def sv_kv_compact(k_cache, v_cache, page_refs, page_table=None, k_scale=None, v_scale=None, refs_out=None, table_out=None, moved_to=None,
                  live=None, stats=None, workspace=None, stream=None):
    """sv_kv_compact: the pages that are held move to the pool's front, in every layer.

    Caches, scales and page_refs as sv_kv_fork's; page_table int32 [B, max_pages] or None; refs_out may be page_refs and table_out
    page_table.  moved_to int32 [pages] or None takes each page's new number (-1: it was free).
    Returns (table_out or None, refs_out, live int32 [1])."""
    lib = _abi.load_packed()
    dev, pages, pool = _kv_pool(k_cache, v_cache, k_scale, v_scale)
    table = pitch = width = B = to = to_pitch = 0
    if page_table is not None:
        table, pitch, width, B = _page_table(page_table, None, dev)
        table_out, to, to_pitch = _table_out(table_out, (B, width), dev)
    elif table_out is not None:
        raise ValueError("table_out without page_table")
    refs = _ints(page_refs, "page_refs", torch.int32, pages, dev)
    refs_out = _out(refs_out, "refs_out", torch.int32, (pages,), dev)
    moved = 0 if moved_to is None else _ints(moved_to, "moved_to", torch.int32, pages, dev)
    live = _out(live, "live", torch.int32, (1,), dev)
    st = _stats(stats, dev).data_ptr() if stats is not None else 0
    ws = (workspace or _default_ws).get(_compact_ws_bytes(pages), dev)
    code = _call(dev, stream, lib.sv_kv_compact, pool, refs, table, pitch, width, B, refs_out.data_ptr(), to, to_pitch, moved, live.data_ptr(),
                 st, ws.data_ptr(), ws.numel())
    if code:
        _abi.check("sv_kv_compact", code)
    return table_out, refs_out, live


@_on_stream
def sv_selftest_timeout(limit_cycles: int, stats=None, stream=None):
    lib = load()
    dev = torch.device("cuda", torch.cuda.current_device())
    if stats is None:
        stats = new_stats(dev)
    _abi.check("sv_selftest_timeout", lib.sv_selftest_timeout(int(limit_cycles), _ptr(stats), _stream(stream, dev)))
    return stats


@_on_stream
def sv_selftest_exp2(lo: float, hi: float, n: int, stream=None):
    lib = load()
    dev = torch.device("cuda", torch.cuda.current_device())
    out = torch.zeros(2, dtype=torch.float64, device=dev)
    _abi.check("sv_selftest_exp2", lib.sv_selftest_exp2(float(lo), float(hi), int(n), _ptr(out), _stream(stream, dev)))
    return out


@_on_stream
def sv_selftest_exp2_all(lo: float, hi: float, stream=None):
    """Largest relative errors (fast, float-float) of the library's exponentials over every
    float32 input in [lo, hi], and the number of inputs evaluated."""
    lib = load()
    dev = torch.device("cuda", torch.cuda.current_device())
    out = torch.zeros(3, dtype=torch.float64, device=dev)
    _abi.check("sv_selftest_exp2_all", lib.sv_selftest_exp2_all(float(lo), float(hi), _ptr(out), _stream(stream, dev)))
    torch.cuda.synchronize()
    r = out.cpu().tolist()
    return r[0], r[1], int(r[2])
