"""ctypes binding of libgdr (include/gdr.h): argument marshalling only.

Every function here checks tensor devices, dtypes, shapes and contiguity,
allocates outputs with torch (device memory is torch's job), and passes raw
pointers plus the current CUDA stream to the C ABI.  All arithmetic of the
method runs in the library's CUDA kernels; there is no fallback.  Importing this
module raises if libgdr.so has not been built.
"""

import contextlib
import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# GDR_LIBRARY=checks loads the debug build with device-side index checks
# (libgdr_checks.so, see build.py) instead of the product library.
LIB_PATH = os.path.join(_HERE, "libgdr_checks.so" if os.environ.get("GDR_LIBRARY") == "checks"
                        else "libgdr.so")

GDR_OK, GDR_ERR_INVALID_ARG, GDR_ERR_UNSUPPORTED, GDR_ERR_CUDA, GDR_ERR_TIMEOUT = range(5)
GDR_F32, GDR_BF16 = 0, 1
CHUNK = 64

EXPORTS = ["gdr_version", "gdr_last_error", "gdr_prefill_workspace_bytes", "gdn_prefill",
           "kda_prefill", "gdn_decode", "kda_decode", "gdr_workspace_status",
           "gdr_prefill_path", "gdn_prefill_noalloc", "gdr_noalloc_status", "gdr_check_status",
           "gdr_timing_start", "gdr_timing_stop",
           "gdn_verify", "kda_verify", "gdr_prefill_varlen_workspace_bytes",
           "gdn_prefill_varlen", "kda_prefill_varlen", "gdr_backward_workspace_bytes",
           "gdn_backward", "kda_backward", "gdn_prefill_ex", "kda_prefill_ex", "gdn_decode_ex",
           "kda_decode_ex", "gdn_verify_ex", "kda_verify_ex", "gdn_prefill_varlen_ex",
           "kda_prefill_varlen_ex", "gdr_lin_workspace_bytes", "lin_prefill", "lin_decode",
           "lin_backward", "gdr_attn_workspace_bytes", "attn_prefill", "attn_backward",
           "gdr_attn_decode_workspace_bytes", "attn_decode", "kv_append"]

# fused prologue flags of the *_ex entry points (prologue= keyword below)
PROLOGUE_L2NORM_QK = 1   # q, k raw: L2-normalised per (token, head) inside the kernels
PROLOGUE_GATE_LOGIT = 2  # alpha holds x: the gate is exp(-softplus(x))


class GdrError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"[gdr status {status}] {message}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m gated_delta_rule_79_b200.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, fp, i, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.gdr_version.restype = i
    lib.gdr_version.argtypes = []
    lib.gdr_last_error.restype = ctypes.c_char_p
    lib.gdr_last_error.argtypes = []
    lib.gdr_prefill_workspace_bytes.restype = sz
    lib.gdr_prefill_workspace_bytes.argtypes = [i, i, i, i, i, i]
    for name in ("gdn_prefill", "kda_prefill"):
        f = getattr(lib, name)
        f.restype = i
        f.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, i, i, i, i, i, i, i, i, vp, sz, vp]
    for name in ("gdn_decode", "kda_decode"):
        f = getattr(lib, name)
        f.restype = i
        f.argtypes = [vp, vp, vp, fp, fp, fp, vp, i, i, i, i, i, i, vp]
    for name in ("gdn_verify", "kda_verify"):
        f = getattr(lib, name)
        f.restype = i
        f.argtypes = [vp, vp, vp, fp, fp, fp, fp, vp, i, i, i, i, i, i, i, vp]
    lib.gdr_prefill_varlen_workspace_bytes.restype = sz
    lib.gdr_prefill_varlen_workspace_bytes.argtypes = [i, i, i, i, i, i]
    for name in ("gdn_prefill_varlen", "kda_prefill_varlen"):
        f = getattr(lib, name)
        f.restype = i
        f.argtypes = [vp, vp, vp, fp, fp, vp, vp, fp, vp, i, i, i, i, i, i, i, i, vp, sz, vp]
    for name in ("gdn_prefill", "kda_prefill", "gdn_decode", "kda_decode", "gdn_verify",
                 "kda_verify", "gdn_prefill_varlen", "kda_prefill_varlen"):
        f = getattr(lib, name + "_ex")
        f.restype = i
        f.argtypes = list(getattr(lib, name).argtypes) + [ctypes.c_uint]
    lib.gdr_backward_workspace_bytes.restype = sz
    lib.gdr_backward_workspace_bytes.argtypes = [i, i, i, i, i, i]
    for name in ("gdn_backward", "kda_backward"):
        f = getattr(lib, name)
        f.restype = i
        f.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, fp, fp, fp, fp, fp, fp,
                      i, i, i, i, i, i, i, vp, sz, vp]
    lib.gdn_prefill_noalloc.restype = i
    lib.gdn_prefill_noalloc.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, i, i, i, i, i, i, i, i, vp]
    lib.gdr_noalloc_status.restype = i
    lib.gdr_noalloc_status.argtypes = [vp]
    lib.gdr_check_status.restype = i
    lib.gdr_check_status.argtypes = [vp]
    lib.gdr_prefill_path.restype = i
    lib.gdr_prefill_path.argtypes = [i, i, i, i]
    lib.gdr_workspace_status.restype = i
    lib.gdr_workspace_status.argtypes = [vp, sz, vp]
    u = ctypes.c_float
    for name, args in (
            ("lin_prefill", [vp, vp, vp, fp, fp, vp, fp, i, i, i, i, i, i, vp, sz, vp]),
            ("lin_decode", [vp, vp, vp, fp, fp, vp, i, i, i, i, i, vp]),
            ("lin_backward", [vp, vp, vp, fp, fp, vp, fp, vp, vp, vp, fp, i, i, i, i, i, i, vp, sz,
                              vp]),
            ("attn_prefill", [vp, vp, vp, vp, vp, fp, i, i, i, i, i, i, i, i, u, i, vp, sz, vp]),
            ("attn_backward", [vp, vp, vp, vp, vp, fp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, u,
                               i, vp, sz, vp]),
            ("attn_decode", [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, u, i, vp,
                             sz, vp]),
            ("kv_append", [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, vp, sz, vp])):
        f = getattr(lib, name)
        f.restype = i
        f.argtypes = args
    for name, n in (("gdr_lin_workspace_bytes", 7), ("gdr_attn_workspace_bytes", 10),
                    ("gdr_attn_decode_workspace_bytes", 9)):
        f = getattr(lib, name)
        f.restype = sz
        f.argtypes = [i] * n
    lib.gdr_timing_start.restype = i
    lib.gdr_timing_start.argtypes = []
    lib.gdr_timing_stop.restype = i
    lib.gdr_timing_stop.argtypes = [ctypes.POINTER(ctypes.c_float), i, ctypes.POINTER(i)]
    return lib


lib = _load()


def _check(status):
    if status != GDR_OK:
        raise GdrError(status, lib.gdr_last_error().decode())


def _pick(name, prologue):
    """The plain entry point, or its fused-prologue variant with the flags appended."""
    if prologue:
        return getattr(lib, name + "_ex"), (int(prologue),)
    return getattr(lib, name), ()


def _code(dtype):
    if dtype == torch.float32:
        return GDR_F32
    if dtype == torch.bfloat16:
        return GDR_BF16
    raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, shape, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_ws_lock = threading.Lock()
_ws_cache = {}


def prefill_workspace(B, T, H, dk, dv, kda, device, stream=None):
    """Zero-initialised device workspace for a prefill call, cached per
    (device, stream) and grown on demand.  Returns (tensor, nbytes)."""
    need = lib.gdr_prefill_workspace_bytes(B, T, H, dk, dv, int(kda))
    if need == 0:
        raise GdrError(GDR_ERR_INVALID_ARG, "invalid prefill sizes")
    s = stream if stream is not None else torch.cuda.current_stream(device)
    key = (device, s.cuda_stream)
    with _ws_lock:
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < need:
            with torch.cuda.stream(s):
                buf = torch.zeros(max(need, 1 << 12), dtype=torch.uint8, device=device)
            _ws_cache[key] = buf
    return buf, buf.numel()


def _prefill(kda, q, k, v, alpha, beta, s0, out_dtype, o, s_final, chunk, stream, workspace,
             prologue=0):
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, d_k]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    dt = q.dtype
    _need(q, "q", (B, T, H, dk), dt, dev)
    _need(k, "k", (B, T, H, dk), dt, dev)
    _need(v, "v", (B, T, H, dv), dt, dev)
    _need(alpha, "alpha", (B, T, H, dk) if kda else (B, T, H), torch.float32, dev)
    _need(beta, "beta", (B, T, H), torch.float32, dev)
    if s0 is not None:
        _need(s0, "s0", (B, H, dv, dk), torch.float32, dev)
    out_dtype = out_dtype or dt
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=out_dtype, device=dev)
    _need(o, "o", (B, T, H, dv), out_dtype, dev)
    if s_final is None:
        s_final = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    elif s_final is not False:
        _need(s_final, "s_final", (B, H, dv, dk), torch.float32, dev)
    sf = None if s_final is False else s_final
    if workspace is None:
        ws, nws = prefill_workspace(B, T, H, dk, dv, kda, dev, stream)
    else:
        ws, nws = workspace, workspace.numel() * workspace.element_size()
    fn, extra = _pick("kda_prefill" if kda else "gdn_prefill", prologue)
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(s0), _ptr(o), _ptr(sf),
              B, T, H, dk, dv, _code(dt), _code(out_dtype), chunk, _ptr(ws), nws,
              _stream(dev, stream), *extra))
    return o, sf


def gdn_prefill(q, k, v, alpha, beta, s0=None, *, out_dtype=None, o=None, s_final=None,
                chunk=CHUNK, stream=None, workspace=None, prologue=0):
    """Gated DeltaNet chunked prefill (scalar gate alpha [B, T, H]).

    q, k [B, T, H, d_k] and v [B, T, H, d_v] in float32 or bfloat16; alpha, beta
    float32; s0 [B, H, d_v, d_k] float32 or None.  Returns (o, s_final); pass
    s_final=False to skip writing the final state, or s_final=s0 to carry in place.
    prologue: PROLOGUE_* flags (raw q, k normalised in the kernel; alpha given as the
    gate pre-activation x, alpha = exp(-softplus(x))).
    """
    return _prefill(False, q, k, v, alpha, beta, s0, out_dtype, o, s_final, chunk, stream,
                    workspace, prologue)


def kda_prefill(q, k, v, alpha, beta, s0=None, *, out_dtype=None, o=None, s_final=None,
                chunk=CHUNK, stream=None, workspace=None, prologue=0):
    """Kimi Delta Attention chunked prefill (per-channel gate alpha [B, T, H, d_k]);
    otherwise as ``gdn_prefill``."""
    return _prefill(True, q, k, v, alpha, beta, s0, out_dtype, o, s_final, chunk, stream,
                    workspace, prologue)


def _decode(kda, q, k, v, alpha, beta, state, out_dtype, o, stream, prologue=0):
    if q.dim() != 3:
        raise ValueError("q must be [N, H, d_k]")
    N, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    dt = q.dtype
    _need(q, "q", (N, H, dk), dt, dev)
    _need(k, "k", (N, H, dk), dt, dev)
    _need(v, "v", (N, H, dv), dt, dev)
    _need(alpha, "alpha", (N, H, dk) if kda else (N, H), torch.float32, dev)
    _need(beta, "beta", (N, H), torch.float32, dev)
    _need(state, "state", (N, H, dv, dk), torch.float32, dev)
    out_dtype = out_dtype or dt
    if o is None:
        o = torch.empty((N, H, dv), dtype=out_dtype, device=dev)
    _need(o, "o", (N, H, dv), out_dtype, dev)
    fn, extra = _pick("kda_decode" if kda else "gdn_decode", prologue)
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state), _ptr(o),
              N, H, dk, dv, _code(dt), _code(out_dtype), _stream(dev, stream), *extra))
    return o


def gdn_decode(q, k, v, alpha, beta, state, *, out_dtype=None, o=None, stream=None, prologue=0):
    """One Gated DeltaNet decode step for N sequences; ``state`` [N, H, d_v, d_k]
    float32 is updated in place.  Returns o [N, H, d_v]."""
    return _decode(False, q, k, v, alpha, beta, state, out_dtype, o, stream, prologue)


def kda_decode(q, k, v, alpha, beta, state, *, out_dtype=None, o=None, stream=None, prologue=0):
    """One Kimi Delta Attention decode step (alpha [N, H, d_k]); as ``gdn_decode``."""
    return _decode(True, q, k, v, alpha, beta, state, out_dtype, o, stream, prologue)


def _prefill_varlen(kda, q, k, v, alpha, beta, cu_seqlens, state, slots, out_dtype, o,
                    chunk, stream, workspace, prologue=0):
    if q.dim() != 3:
        raise ValueError("q must be [total, H, d_k] (sequences packed along the tokens)")
    total, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    dt = q.dtype
    _need(q, "q", (total, H, dk), dt, dev)
    _need(k, "k", (total, H, dk), dt, dev)
    _need(v, "v", (total, H, dv), dt, dev)
    _need(alpha, "alpha", (total, H, dk) if kda else (total, H), torch.float32, dev)
    _need(beta, "beta", (total, H), torch.float32, dev)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.device != dev:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor on the inputs' device")
    nseq = cu_seqlens.numel() - 1
    if nseq < 0:
        raise ValueError("cu_seqlens needs nseq + 1 entries")
    if state.dim() != 4 or state.shape[1:] != (H, dv, dk) or state.dtype != torch.float32:
        raise ValueError("state must be a float32 pool [nslots, H, d_v, d_k]")
    if not state.is_contiguous() or state.device != dev:
        raise ValueError("state must be contiguous on the inputs' device")
    if slots is not None and (slots.dtype != torch.int32 or slots.numel() != nseq
                              or slots.device != dev):
        raise ValueError("slots must be an int32 tensor of nseq entries on the inputs' device")
    if slots is None and state.shape[0] < nseq:
        raise ValueError("without slots the pool needs one slot per sequence")
    out_dtype = out_dtype or dt
    if o is None:
        o = torch.empty((total, H, dv), dtype=out_dtype, device=dev)
    _need(o, "o", (total, H, dv), out_dtype, dev)
    need = lib.gdr_prefill_varlen_workspace_bytes(nseq, total, H, dk, dv, int(kda))
    if workspace is None:
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        with torch.cuda.stream(s):
            workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
    fn, extra = _pick("kda_prefill_varlen" if kda else "gdn_prefill_varlen", prologue)
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(cu_seqlens), _ptr(slots),
              _ptr(state), _ptr(o), nseq, total, H, dk, dv, _code(dt), _code(out_dtype), chunk,
              _ptr(workspace), workspace.numel(), _stream(dev, stream), *extra))
    return o


def gdn_prefill_varlen(q, k, v, alpha, beta, cu_seqlens, state, *, slots=None, out_dtype=None,
                       o=None, chunk=CHUNK, stream=None, workspace=None, prologue=0):
    """Gated DeltaNet prefill of nseq sequences packed along the tokens: q, k
    [total, H, d_k], v [total, H, d_v] bf16; alpha, beta [total, H] float32; cu_seqlens
    int32 [nseq + 1] on the device; state a float32 pool [nslots, H, d_v, d_k] read
    from and written back to slot slots[i] (default i) in place.  Returns o."""
    return _prefill_varlen(False, q, k, v, alpha, beta, cu_seqlens, state, slots, out_dtype, o,
                           chunk, stream, workspace, prologue)


def kda_prefill_varlen(q, k, v, alpha, beta, cu_seqlens, state, *, slots=None, out_dtype=None,
                       o=None, chunk=CHUNK, stream=None, workspace=None, prologue=0):
    """Kimi Delta Attention (alpha [total, H, d_k]); as ``gdn_prefill_varlen``."""
    return _prefill_varlen(True, q, k, v, alpha, beta, cu_seqlens, state, slots, out_dtype, o,
                           chunk, stream, workspace, prologue)


VERIFY_MAX_TOKENS = 16


def _verify(kda, q, k, v, alpha, beta, state, snapshots, out_dtype, o, stream, prologue=0):
    if q.dim() != 4:
        raise ValueError("q must be [N, K, H, d_k]")
    N, K, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    dt = q.dtype
    _need(q, "q", (N, K, H, dk), dt, dev)
    _need(k, "k", (N, K, H, dk), dt, dev)
    _need(v, "v", (N, K, H, dv), dt, dev)
    _need(alpha, "alpha", (N, K, H, dk) if kda else (N, K, H), torch.float32, dev)
    _need(beta, "beta", (N, K, H), torch.float32, dev)
    _need(state, "state", (N, H, dv, dk), torch.float32, dev)
    if snapshots is True:
        snapshots = torch.empty((K, N, H, dv, dk), dtype=torch.float32, device=dev)
    elif snapshots is False:
        snapshots = None
    if snapshots is not None:
        _need(snapshots, "snapshots", (K, N, H, dv, dk), torch.float32, dev)
    out_dtype = out_dtype or dt
    if o is None:
        o = torch.empty((N, K, H, dv), dtype=out_dtype, device=dev)
    _need(o, "o", (N, K, H, dv), out_dtype, dev)
    fn, extra = _pick("kda_verify" if kda else "gdn_verify", prologue)
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state), _ptr(snapshots),
              _ptr(o), N, K, H, dk, dv, _code(dt), _code(out_dtype), _stream(dev, stream),
              *extra))
    return o, snapshots


def gdn_verify(q, k, v, alpha, beta, state, *, snapshots=True, out_dtype=None, o=None,
               stream=None, prologue=0):
    """Gated DeltaNet over K tokens per sequence from a carried state, keeping the
    state after every token.  q, k [N, K, H, d_k]; v [N, K, H, d_v]; alpha, beta
    [N, K, H]; state [N, H, d_v, d_k] float32.  snapshots=True allocates, or pass a
    [K, N, H, d_v, d_k] float32 tensor; snapshots[t] is the state after token t+1 and
    ``state`` is left as it was.  snapshots=False updates ``state`` in place to the
    state after the K tokens instead.  Returns (o [N, K, H, d_v], snapshots or None)."""
    return _verify(False, q, k, v, alpha, beta, state, snapshots, out_dtype, o, stream,
                   prologue)


def kda_verify(q, k, v, alpha, beta, state, *, snapshots=True, out_dtype=None, o=None,
               stream=None, prologue=0):
    """Kimi Delta Attention (alpha [N, K, H, d_k]); as ``gdn_verify``."""
    return _verify(True, q, k, v, alpha, beta, state, snapshots, out_dtype, o, stream,
                   prologue)


def _backward(kda, q, k, v, alpha, beta, s0, do, ds_final, workspace, stream):
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, d_k]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    dt = q.dtype
    _need(q, "q", (B, T, H, dk), dt, dev)
    _need(k, "k", (B, T, H, dk), dt, dev)
    _need(v, "v", (B, T, H, dv), dt, dev)
    _need(alpha, "alpha", (B, T, H, dk) if kda else (B, T, H), torch.float32, dev)
    _need(beta, "beta", (B, T, H), torch.float32, dev)
    if s0 is not None:
        _need(s0, "s0", (B, H, dv, dk), torch.float32, dev)
    _need(do, "do", (B, T, H, dv), None, dev)
    if ds_final is not None:
        _need(ds_final, "ds_final", (B, H, dv, dk), torch.float32, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    dq = torch.empty((B, T, H, dk), **f32)
    dk_ = torch.empty((B, T, H, dk), **f32)
    dv_ = torch.empty((B, T, H, dv), **f32)
    dalpha = torch.empty(alpha.shape, **f32)
    dbeta = torch.empty((B, T, H), **f32)
    ds0 = torch.empty((B, H, dv, dk), **f32)
    need = lib.gdr_backward_workspace_bytes(B, T, H, dk, dv, int(kda))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    nws = workspace.numel() * workspace.element_size()
    fn = lib.kda_backward if kda else lib.gdn_backward
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(s0), _ptr(do),
              _ptr(ds_final), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dalpha), _ptr(dbeta),
              _ptr(ds0), B, T, H, dk, dv, _code(dt), _code(do.dtype), _ptr(workspace), nws,
              _stream(dev, stream)))
    return dq, dk_, dv_, dalpha, dbeta, ds0


def gdn_backward(q, k, v, alpha, beta, s0, do, ds_final=None, *, workspace=None, stream=None):
    """Gradients (dq, dk, dv, dalpha [B,T,H], dbeta, ds0), all fp32, of
    L = sum <do, o> + <ds_final, S_T> for gdn_prefill(q, k, v, alpha, beta, s0)."""
    return _backward(False, q, k, v, alpha, beta, s0, do, ds_final, workspace, stream)


def kda_backward(q, k, v, alpha, beta, s0, do, ds_final=None, *, workspace=None, stream=None):
    """As gdn_backward with the per-channel gate: dalpha is [B, T, H, d_k]."""
    return _backward(True, q, k, v, alpha, beta, s0, do, ds_final, workspace, stream)


def backward_workspace_bytes(B, T, H, dk, dv, kda):
    return lib.gdr_backward_workspace_bytes(B, T, H, dk, dv, int(kda))


# ---- linear attention with one decay per head; sliding-window softmax attention -----------

# A decode step runs for a few microseconds, so these calls keep their own cost low: one test a
# tensor (the reason for a refusal is worked out by _need afterwards), plain integers for pointers.

def _on(device, stream):
    """Context in which a call on `stream` (None: the device's current one) allocates and
    launches: outputs and workspaces belong to that stream, the launch goes to that device."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if device.index != torch.cuda.current_device():
        return torch.cuda.device(device)
    return _HERE_ALREADY


_HERE_ALREADY = contextlib.nullcontext()

# workspace sizes by the sizes of a call
_lin_bytes = functools.lru_cache(maxsize=256)(lib.gdr_lin_workspace_bytes)
_attn_bytes = functools.lru_cache(maxsize=256)(lib.gdr_attn_workspace_bytes)
_decode_bytes = functools.lru_cache(maxsize=256)(lib.gdr_attn_decode_workspace_bytes)


def _raw(device, stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def _same(t, name, shape, dtype, device):
    """data_ptr of t after _need's checks."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype \
            and t.device == device and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, shape, dtype, device)
    return t.data_ptr()


def _maybe(t, name, shape, dtype, device):
    return None if t is None else _same(t, name, shape, dtype, device)


_kept = {}             # (device, stream): (workspace, its bytes, lock)


def mixer_workspace(device=None, stream=None):
    """The workspace of the linear- and softmax-attention calls on `stream` (None: the device's
    current one) that are given none.  Its status word is kept from call to call until
    workspace_status reads it, so that ``workspace_status(mixer_workspace())`` tells of a wait
    that gave up, or of a length or page outside a paged cache, in any of them.  (A call that is
    captured into a graph takes a workspace from the graph's own pool instead, which nothing
    reads: give such a call a zero-filled one to be told.)  It grows to what the largest call on
    the stream needs (..._workspace_bytes) and is kept; calls given one leave it alone."""
    dev = torch.device("cuda" if device is None else device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    with _on(dev, stream):
        return _keep(256, dev, _raw(dev, stream))[0]


def _keep(need, device, raw):
    """A kept workspace of at least `need` bytes, inside _on(device, stream)."""
    key = device.index, raw
    got = _kept.get(key)
    if got is None or got[1] < need:
        with _ws_lock:
            got = _kept.get(key)
            if got is None or got[1] < need:
                buf = torch.zeros(max(need, 1 << 12), dtype=torch.uint8, device=device)
                if got is not None:              # what is on record stays so
                    buf[:256].copy_(got[0][:256])
                got = _kept[key] = (buf, buf.numel(), threading.Lock())
    return got


def _scratch(workspace, need, device, what, raw):
    """The call's workspace, inside _on(device, stream): the caller's, or the one kept for this
    stream, or in a capture one from torch's allocator (so a captured graph owns what it uses).
    Returns (tensor, nbytes, what to hold while the call enqueues its kernels: those of two
    threads on one stream must not mix in one workspace)."""
    if need == 0:
        raise GdrError(GDR_ERR_INVALID_ARG, f"invalid {what} sizes")
    if workspace is None:
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(need, dtype=torch.uint8, device=device), need, _HERE_ALREADY
        return _keep(need, device, raw)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace, workspace.numel() * workspace.element_size(), _HERE_ALREADY


def _cuda(t, name, dim, form):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dim:
        raise ValueError(f"{name} must be {form}")
    if not t.is_cuda:
        raise ValueError("inputs must be CUDA tensors (there is no CPU path)")
    return t.device


def _out(t, name, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _same(t, name, shape, dtype, device)
    return t


def _out_like(t, name, like):
    """An output of the shape and type of `like`, one of the checked inputs."""
    if t is None:
        return torch.empty_like(like)
    _same(t, name, like.shape, like.dtype, like.device)
    return t


def lin_workspace_bytes(B, T, H, dk, dv, dtype, backward=False):
    """Bytes of device workspace for lin_prefill (or lin_backward) at these sizes."""
    return lib.gdr_lin_workspace_bytes(B, T, H, dk, dv, _code(dtype), int(backward))


def lin_prefill(q, k, v, decay, s0=None, *, o=None, s_final=None, stream=None, workspace=None):
    """Linear attention with one decay per head over T tokens:
    S_t = decay S_{t-1} + v_t k_t^T, o_t = S_t q_t.

    q, k [B, T, H, d_k] and v [B, T, H, d_v], all float32 or all bfloat16; decay [H] float32 in
    [0, 1]; s0 [B, H, d_v, d_k] float32 or None.  Returns (o, s_final), o in the inputs' type;
    pass s_final=False to skip the final state, or s_final=s0 to carry in place.  workspace:
    a zero-filled uint8 tensor of lin_workspace_bytes(...) to read with workspace_status
    (None: mixer_workspace()).
    """
    dev = _cuda(q, "q", 4, "[B, T, H, d_k]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    code = _code(dt)
    state = (B, H, dv, dk)
    ptrs = (_same(q, "q", (B, T, H, dk), dt, dev), _same(k, "k", (B, T, H, dk), dt, dev),
            _same(v, "v", (B, T, H, dv), dt, dev), _same(decay, "decay", (H,), torch.float32, dev),
            _maybe(s0, "s0", state, torch.float32, dev))
    with _on(dev, stream):
        o = _out_like(o, "o", v)
        sf = None if s_final is False else _out(s_final, "s_final", state, torch.float32, dev)
        raw = _raw(dev, stream)
        ws, nws, lock = _scratch(workspace, _lin_bytes(B, T, H, dk, dv, code, 0), dev,
                                 "lin_prefill", raw)
        with lock:
            _check(lib.lin_prefill(*ptrs, o.data_ptr(), None if sf is None else sf.data_ptr(),
                                   B, T, H, dk, dv, code, ws.data_ptr(), nws, raw))
    return o, sf


def lin_decode(q, k, v, decay, state, *, o=None, stream=None):
    """One token of linear attention for N sequences: q, k [N, H, d_k], v [N, H, d_v], decay
    [H]; ``state`` [N, H, d_v, d_k] float32 is updated in place.  Returns o [N, H, d_v]."""
    dev = _cuda(q, "q", 3, "[N, H, d_k]")
    N, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    code = _code(dt)
    ptrs = (_same(q, "q", (N, H, dk), dt, dev), _same(k, "k", (N, H, dk), dt, dev),
            _same(v, "v", (N, H, dv), dt, dev), _same(decay, "decay", (H,), torch.float32, dev),
            _same(state, "state", (N, H, dv, dk), torch.float32, dev))
    with _on(dev, stream):
        o = _out_like(o, "o", v)
        _check(lib.lin_decode(*ptrs, o.data_ptr(), N, H, dk, dv, code, _raw(dev, stream)))
    return o


def lin_backward(q, k, v, decay, s0, do, ds_final=None, *, workspace=None, stream=None):
    """Gradients (dq, dk, dv in the inputs' type, ds0 float32) of
    L = sum <do, o> + <ds_final, S_T> for lin_prefill(q, k, v, decay, s0).  The decay is a
    constant of the head and has none."""
    dev = _cuda(q, "q", 4, "[B, T, H, d_k]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    code = _code(dt)
    state = (B, H, dv, dk)
    ptrs = (_same(q, "q", (B, T, H, dk), dt, dev), _same(k, "k", (B, T, H, dk), dt, dev),
            _same(v, "v", (B, T, H, dv), dt, dev), _same(decay, "decay", (H,), torch.float32, dev),
            _maybe(s0, "s0", state, torch.float32, dev), _same(do, "do", (B, T, H, dv), dt, dev),
            _maybe(ds_final, "ds_final", state, torch.float32, dev))
    with _on(dev, stream):
        dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ds0 = torch.empty(state, dtype=torch.float32, device=dev)
        raw = _raw(dev, stream)
        ws, nws, lock = _scratch(workspace, _lin_bytes(B, T, H, dk, dv, code, 1), dev,
                                 "lin_backward", raw)
        with lock:
            _check(lib.lin_backward(*ptrs, dq.data_ptr(), dk_.data_ptr(), dv_.data_ptr(),
                                    ds0.data_ptr(), B, T, H, dk, dv, code, ws.data_ptr(), nws,
                                    raw))
    return dq, dk_, dv_, ds0


def attn_workspace_bytes(B, Tq, Tk, Hq, Hkv, d, dtype, backward=False, window=0, sinks=0):
    """Bytes of device workspace for attn_prefill (or attn_backward) at these sizes."""
    return lib.gdr_attn_workspace_bytes(B, Tq, Tk, Hq, Hkv, d, _int32(window, "window"),
                                        _int32(sinks, "sinks"), _code(dtype), int(backward))


def _int32(x, name):
    """A window or a number of sinks as the C int it becomes (None: 0)."""
    if x is None:
        return 0
    if x < 0 and name == "sinks":
        raise ValueError("sinks must not be negative")
    return min(max(int(x), 0), 0x7fffffff)


def _attn_shapes(q, k, v):
    dev = _cuda(q, "q", 4, "[B, Tq, Hq, d]")
    _cuda(k, "k", 4, "[B, Tk, Hkv, d]")
    B, Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[1], k.shape[2]
    ptrs = (_same(q, "q", (B, Tq, Hq, d), q.dtype, dev),
            _same(k, "k", (B, Tk, Hkv, d), q.dtype, dev),
            _same(v, "v", (B, Tk, Hkv, d), q.dtype, dev))
    return dev, ptrs, B, Tq, Tk, Hq, Hkv, d


def attn_prefill(q, k, v, *, window=0, sinks=0, scale=None, lengths=None, o=None, lse=None,
                 stream=None, workspace=None):
    """Causal softmax attention with an optional sliding window and sinks.

    q [B, Tq, Hq, d]; k, v [B, Tk, Hkv, d] (Hq a multiple of Hkv: query head h reads key head
    h // (Hq / Hkv)); all float32 or all bfloat16.  Query i sits at position p = Tk - Tq + i
    and sees key j when j <= p, j and p < lengths[b] (int32 [B]; None: Tk), and
    p - j < window (0 or None: no window) or j < sinks.  scale: None for d ** -0.5.
    Returns (o in q's type, lse [B, Hq, Tq] float32); a query that sees nothing has o = 0 and
    lse = -inf.  Pass lse=False to skip it.  workspace: a zero-filled uint8 tensor of
    attn_workspace_bytes(...) to read with workspace_status (None: mixer_workspace()).
    """
    dev, ptrs, B, Tq, Tk, Hq, Hkv, d = _attn_shapes(q, k, v)
    code = _code(q.dtype)
    lens = _maybe(lengths, "lengths", (B,), torch.int32, dev)
    w, n = _int32(window, "window"), _int32(sinks, "sinks")
    with _on(dev, stream):
        o = _out_like(o, "o", q)
        lse = None if lse is False else _out(lse, "lse", (B, Hq, Tq), torch.float32, dev)
        raw = _raw(dev, stream)
        ws, nws, lock = _scratch(workspace, _attn_bytes(B, Tq, Tk, Hq, Hkv, d, w, n, code, 0), dev,
                                 "attn_prefill", raw)
        with lock:
            _check(lib.attn_prefill(*ptrs, lens, o.data_ptr(),
                                    None if lse is None else lse.data_ptr(), B, Tq, Tk, Hq, Hkv, d,
                                    w, n, d ** -0.5 if scale is None else scale, code,
                                    ws.data_ptr(), nws, raw))
    return o, lse


def attn_backward(q, k, v, o, lse, do, *, window=0, sinks=0, scale=None, lengths=None,
                  stream=None, workspace=None):
    """Gradients (dq, dk, dv, in the inputs' type) of L = sum <do, o> for
    attn_prefill(q, k, v, ...), from its o and lse."""
    dev, ptrs, B, Tq, Tk, Hq, Hkv, d = _attn_shapes(q, k, v)
    code = _code(q.dtype)
    lens = _maybe(lengths, "lengths", (B,), torch.int32, dev)
    given = (_same(o, "o", (B, Tq, Hq, d), q.dtype, dev),
             _same(lse, "lse", (B, Hq, Tq), torch.float32, dev),
             _same(do, "do", (B, Tq, Hq, d), q.dtype, dev))
    w, n = _int32(window, "window"), _int32(sinks, "sinks")
    with _on(dev, stream):
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        raw = _raw(dev, stream)
        ws, nws, lock = _scratch(workspace, _attn_bytes(B, Tq, Tk, Hq, Hkv, d, w, n, code, 1), dev,
                                 "attn_backward", raw)
        with lock:
            _check(lib.attn_backward(*ptrs, lens, *given, dq.data_ptr(), dk.data_ptr(),
                                     dv.data_ptr(), B, Tq, Tk, Hq, Hkv, d, w, n,
                                     d ** -0.5 if scale is None else scale, code, ws.data_ptr(),
                                     nws, raw))
    return dq, dk, dv


def _paged(k_cache, v_cache, page_table, N, dt, dev):
    _cuda(k_cache, "k_cache", 4, "[npages, page, Hkv, d]")
    npages, page, Hkv, d = k_cache.shape
    _cuda(page_table, "page_table", 2, "[N, max_pages]")
    max_pages = page_table.shape[1]
    ptrs = (_same(k_cache, "k_cache", k_cache.shape, dt, dev),
            _same(v_cache, "v_cache", k_cache.shape, dt, dev),
            _same(page_table, "page_table", (N, max_pages), torch.int32, dev))
    return ptrs, npages, page, Hkv, d, max_pages


def attn_decode_workspace_bytes(N, Hq, Hkv, d, page, max_pages, dtype, window=0, sinks=0):
    """Bytes of device workspace for attn_decode at these sizes."""
    return lib.gdr_attn_decode_workspace_bytes(N, Hq, Hkv, d, page, max_pages,
                                               _int32(window, "window"), _int32(sinks, "sinks"),
                                               _code(dtype))


def attn_decode(q, k_cache, v_cache, page_table, lengths, *, k=None, v=None, window=0, sinks=0,
                scale=None, o=None, stream=None, workspace=None):
    """Attention of one new token for each of N sequences over a paged key-value cache.

    q [N, Hq, d]; k_cache, v_cache [npages, page, Hkv, d] (page a power of two); page_table
    [N, max_pages] int32: token t of sequence n lies in row t % page of page
    page_table[n, t // page]; lengths [N] int32, the new token counted.  With k, v [N, Hkv, d]
    the new token's key and value are stored at position lengths[n] - 1 by the same launch.
    window, sinks, scale as in attn_prefill.  Returns o [N, Hq, d]; 0 for an empty sequence.
    Lengths and table entries outside the cache are left out and recorded in the workspace's
    status word: read it with workspace_status, of the zero-filled workspace given, or of
    mixer_workspace() when there was none.
    """
    dev = _cuda(q, "q", 3, "[N, Hq, d]")
    N, Hq, d = q.shape
    dt = q.dtype
    code = _code(dt)
    qp = _same(q, "q", (N, Hq, d), dt, dev)
    ptrs, npages, page, Hkv, dc, max_pages = _paged(k_cache, v_cache, page_table, N, dt, dev)
    if dc != d:
        raise ValueError(f"the caches' head size {dc} is not q's {d}")
    lens = _same(lengths, "lengths", (N,), torch.int32, dev)
    if (k is None) != (v is None):
        raise ValueError("k and v are given together or not at all")
    kp, vp = _maybe(k, "k", (N, Hkv, d), dt, dev), _maybe(v, "v", (N, Hkv, d), dt, dev)
    w, s = _int32(window, "window"), _int32(sinks, "sinks")
    with _on(dev, stream):
        o = _out_like(o, "o", q)
        raw = _raw(dev, stream)
        need = _decode_bytes(N, Hq, Hkv, d, page, max_pages, w, s, code)
        ws, nws, lock = _scratch(workspace, need, dev, "attn_decode", raw)
        with lock:
            _check(lib.attn_decode(qp, kp, vp, *ptrs, lens, o.data_ptr(), N, Hq, Hkv, d, npages,
                                   page, max_pages, w, s, d ** -0.5 if scale is None else scale,
                                   code, ws.data_ptr(), nws, raw))
    return o


def kv_append(k, v, k_cache, v_cache, page_table, start, counts=None, *, stream=None,
              workspace=None):
    """Store K tokens of each of N sequences in a paged cache, in place: k, v [N, K, Hkv, d];
    token t < counts[n] (int32 [N]; None: K) goes to position start[n] + t (int32 [N]).
    Positions and pages outside the cache are skipped, and recorded in ``workspace`` (None:
    mixer_workspace())."""
    dev = _cuda(k, "k", 4, "[N, K, Hkv, d]")
    N, K, Hkv, d = k.shape
    dt = k.dtype
    code = _code(dt)
    kp, vp = _same(k, "k", (N, K, Hkv, d), dt, dev), _same(v, "v", (N, K, Hkv, d), dt, dev)
    ptrs, npages, page, hc, dc, max_pages = _paged(k_cache, v_cache, page_table, N, dt, dev)
    if (hc, dc) != (Hkv, d):
        raise ValueError(f"the caches hold heads {hc} x {dc}, k and v {Hkv} x {d}")
    sp = _same(start, "start", (N,), torch.int32, dev)
    cp = _maybe(counts, "counts", (N,), torch.int32, dev)
    with _on(dev, stream):
        raw = _raw(dev, stream)
        if workspace is None and torch.cuda.is_current_stream_capturing():
            ws, nws = None, 0
        else:
            w, nws, _ = _scratch(workspace, 256, dev, "kv_append", raw)
            ws = w.data_ptr()
        _check(lib.kv_append(kp, vp, *ptrs, sp, cp, N, K, Hkv, d, npages, page, max_pages, code,
                             ws, nws, raw))


def prefill_path(dk, dv, dtype, kda):
    """"tensor-core" or "cuda-core": which prefill kernel serves these parameters."""
    p = lib.gdr_prefill_path(dk, dv, _code(dtype), int(kda))
    if p < 0:
        raise GdrError(GDR_ERR_UNSUPPORTED, f"no prefill kernel for d_k={dk} d_v={dv}")
    return "tensor-core" if p == 1 else "cuda-core"


def check_status(stream=None):
    """Synchronise and read/clear the device-side index-check word of the checks build
    (libgdr_checks.so); raises GdrError(GDR_ERR_INVALID_ARG) if a check fired, and
    GdrError(GDR_ERR_UNSUPPORTED) in the product build, which has no checks."""
    dev = torch.device("cuda", torch.cuda.current_device())
    _check(lib.gdr_check_status(_stream(dev, stream)))


def noalloc_status(stream=None):
    """Synchronise and read/clear the sticky status of gdn_prefill_noalloc on the
    current device; raises GdrError(GDR_ERR_TIMEOUT) if a bounded device wait of a
    call since the last query gave up."""
    dev = torch.device("cuda", torch.cuda.current_device())
    _check(lib.gdr_noalloc_status(_stream(dev, stream)))


def workspace_status(workspace, stream=None):
    """Synchronise and read/clear the device status word of a workspace; raises
    GdrError(GDR_ERR_TIMEOUT) if a bounded device wait gave up, and
    GdrError(GDR_ERR_INVALID_ARG) if offsets, lengths or pages read on the device were wrong."""
    dev = workspace.device
    _check(lib.gdr_workspace_status(_ptr(workspace), workspace.numel(), _stream(dev, stream)))


def timing_start():
    """Start recording per-kernel CUDA events for every prefill call (measurement aid)."""
    lib.gdr_timing_start()


def timing_stop(max_kernels=8):
    """Stop recording; returns (mean ms of each kernel position of a call, calls)."""
    buf = (ctypes.c_float * max_kernels)()
    n = ctypes.c_int(0)
    k = lib.gdr_timing_stop(buf, max_kernels, ctypes.byref(n))
    if k < 0:
        raise GdrError(GDR_ERR_CUDA, "gdr_timing_stop: reading a CUDA event failed")
    return [float(buf[i]) for i in range(min(k, max_kernels))], int(n.value)
