"""ctypes binding over libkda.so.  Argument marshalling only: every step of
the layer runs in the library's kernels.  Torch supplies device memory and
the current stream; nothing here computes any part of the layer, and there
is no fallback when the library is missing -- the call raises.

The Python names match the C entry points (include/kda.h).
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkda.so")
PROBE_LIB_PATH = os.path.join(PKG, "libkda_probe.so")

KDA_BF16, KDA_F32, KDA_F16, KDA_E4M3 = 0, 1, 2, 3
STATUS = {
    0: "ok", 1: "invalid argument", 2: "unsupported shape or dtype",
    3: "pointer not 16-byte aligned", 4: "CUDA error", 5: "log_alpha outside [-5, 0]",
    6: "device wait timed out", 7: "workspace too small",
    8: "state-pass operand outside the fp16 range",
}

EXPORTS = ["kda_chunk_fwd", "kda_chunk_fwd_workspace_size", "kda_chunk_fwd_noalloc",
           "kda_chunk_fwd_segments", "kda_chunk_fwd_segments_workspace_size",
           "kda_chunk_fwd_checkpointed", "kda_chunk_fwd_launches", "kda_decode_verify",
           "kda_chunk_bwd", "kda_chunk_bwd_workspace_size",
           "kda_chunk_fwd_host", "kda_chunk_fwd_host_workspace_size",
           "kda_decode_commit",
           "kda_varlen_fwd",
           "kda_varlen_fwd_workspace_size", "kda_decode_step", "kda_cache_append",
           "kda_cache_attend", "kda_cache_attend_workspace_size", "kda_draft_accept",
           "kda_status_string",
           "kda_last_device_status", "kda_version"]


class KDAError(RuntimeError):
    def __init__(self, code, where):
        self.code = int(code)
        super().__init__(f"{where}: {STATUS.get(self.code, 'unknown')} (status {self.code})")


_lib = None
_probe = None

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong


def load(path: str = LIB_PATH):
    """Load libkda.so (raises if it was not built: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(
                f"libkda.so not found at {path}; build it with "
                "`python -m linear_attention_recurrence_fwd_gb300.build` (no CPU fallback exists)")
        lib = ctypes.CDLL(path)
        lib.kda_chunk_fwd.argtypes = [_vp] * 7 + [_i, _vp, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]
        lib.kda_chunk_fwd.restype = _i
        lib.kda_chunk_fwd_checkpointed.argtypes = ([_vp] * 7 + [_i, _vp, _i, _i, _i, _i, _i, _f] +
                                                   [_vp, _i, _vp, _sz, _vp])
        lib.kda_chunk_fwd_checkpointed.restype = _i
        lib.kda_chunk_fwd_host.argtypes = lib.kda_chunk_fwd.argtypes
        lib.kda_chunk_fwd_host.restype = _i
        lib.kda_chunk_fwd_host_workspace_size.argtypes = [_i] * 6
        lib.kda_chunk_fwd_host_workspace_size.restype = _sz
        lib.kda_chunk_bwd.argtypes = [_vp] * 14 + [_i, _i, _i, _i, _i, _f, _vp, _sz, _vp]
        lib.kda_chunk_bwd.restype = _i
        lib.kda_chunk_bwd_workspace_size.argtypes = [_i] * 5
        lib.kda_chunk_bwd_workspace_size.restype = _sz
        lib.kda_chunk_fwd_segments.argtypes = ([_vp] * 7 + [_i, _vp, _i, _i, _i, _i, _i, _f, _i] +
                                               [_vp, _sz, _vp])
        lib.kda_chunk_fwd_segments.restype = _i
        lib.kda_chunk_fwd_segments_workspace_size.argtypes = [_i] * 6
        lib.kda_chunk_fwd_segments_workspace_size.restype = _sz
        lib.kda_chunk_fwd_noalloc.argtypes = [_vp] * 7 + [_i, _vp, _i, _i, _i, _i, _i, _f, _vp]
        lib.kda_chunk_fwd_noalloc.restype = _i
        lib.kda_varlen_fwd.argtypes = [_vp] * 6 + [_i, _i, _i, _vp, _vp, _i, _vp, _i, _i, _i, _f,
                                                   _vp, _sz, _vp]
        lib.kda_varlen_fwd.restype = _i
        lib.kda_decode_step.argtypes = [_vp] * 7 + [_i, _i, _i, _i, _i, _f, _vp]
        lib.kda_decode_step.restype = _i
        lib.kda_decode_verify.argtypes = [_vp] * 7 + [_i, _i, _i, _i, _i, _i, _f, _vp]
        lib.kda_decode_verify.restype = _i
        lib.kda_decode_commit.argtypes = [_vp] * 7 + [_i, _i, _i, _i, _i, _vp]
        lib.kda_decode_commit.restype = _i
        lib.kda_chunk_fwd_workspace_size.argtypes = [_i] * 5
        lib.kda_chunk_fwd_workspace_size.restype = _sz
        lib.kda_varlen_fwd_workspace_size.argtypes = [_i] * 5
        lib.kda_varlen_fwd_workspace_size.restype = _sz
        lib.kda_chunk_fwd_launches.argtypes = [_i, _i, _i]
        lib.kda_chunk_fwd_launches.restype = _i
        lib.kda_cache_append.argtypes = [_vp] * 5 + [_i] + [_ll] * 4 + [_vp, _i, _i, _vp, _vp, _i, _i, _i, _vp]
        lib.kda_cache_append.restype = _i
        lib.kda_cache_attend.argtypes = [_vp, _vp, _i, _ll, _vp, _vp, _vp, _i, _i, _f, _i, _i, _vp, _sz, _vp]
        lib.kda_cache_attend.restype = _i
        lib.kda_cache_attend_workspace_size.argtypes = [_i] * 6
        lib.kda_cache_attend_workspace_size.restype = _sz
        lib.kda_draft_accept.argtypes = [_vp, _vp, _vp, _i] + [_ll] * 4 + [_vp] * 4 + [_i] * 3 + [_vp]
        lib.kda_draft_accept.restype = _i
        lib.kda_status_string.argtypes = [_i]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_last_device_status.argtypes = [_vp]
        lib.kda_last_device_status.restype = _i
        lib.kda_version.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def load_probe(path: str = PROBE_LIB_PATH):
    """Test-only layout probes (libkda_probe.so)."""
    global _probe
    if _probe is None:
        if not os.path.exists(path):
            raise RuntimeError(f"libkda_probe.so not found at {path}")
        lib = ctypes.CDLL(path)
        lib.kda_probe_umma.argtypes = [_vp, _vp, _vp] + [_i] * 14 + [_vp, _vp]
        lib.kda_probe_umma.restype = _i
        lib.kda_probe_tma.argtypes = [_vp, _vp] + [_i] * 5 + [_vp, _vp]
        lib.kda_probe_tma.restype = _i
        lib.kda_probe_umma_ta.argtypes = [_vp, _vp, _vp] + [_i] * 15 + [_vp, _vp]
        lib.kda_probe_umma_ta.restype = _i
        lib.kda_probe_wait_timeout.argtypes = [_i, _vp, _vp]
        lib.kda_probe_wait_timeout.restype = _i
        lib.kda_probe_attend_loaders.argtypes = [_vp, _i, _vp, _i, _vp] + [_i] * 4 + [_vp, _vp, _vp]
        lib.kda_probe_attend_loaders.restype = _i
        _probe = lib
    return _probe


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(code, where):
    if code != 0:
        raise KDAError(code, where)


def _dtype_code(dt):
    if dt == torch.bfloat16:
        return KDA_BF16
    if dt == torch.float32:
        return KDA_F32
    raise ValueError(f"unsupported output dtype {dt}")


def _need(t, dtype, name):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


def _need_host(t, dtype, name):
    if t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous host {dtype} tensor")


def kda_chunk_fwd(q, k, v, log_alpha, beta, initial_state=None, scale=1.0,
                  out_dtype=torch.float32, output_final_state=True, out=None,
                  final_state=None, stream=None):
    """Chunked prefill.  q,k,log_alpha [B,T,H,dk] bf16; v [B,T,H,dv] bf16;
    beta [B,T,H] bf16; initial_state [B,H,dk,dv] fp32 or None.
    Returns (out [B,T,H,dv], final_state [B,H,dk,dv] fp32 or None)."""
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_alpha, "log_alpha"), (beta, "beta")):
        _need(t, torch.bfloat16, n)
    if initial_state is not None:
        _need(initial_state, torch.float32, "initial_state")
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=out_dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ws_bytes = lib.kda_chunk_fwd_workspace_size(B, T, H, dk, dv)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device) if ws_bytes else None
    _check(lib.kda_chunk_fwd(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(initial_state),
                             _p(out), _dtype_code(out.dtype), _p(final_state), B, T, H, dk, dv,
                             float(scale), _p(ws), ws_bytes, _stream(stream)), "kda_chunk_fwd")
    return out, final_state


def kda_chunk_fwd_segments(q, k, v, log_alpha, beta, initial_state=None, scale=1.0,
                           n_segments=2, out_dtype=torch.float32, out=None, final_state=None,
                           stream=None):
    """kda_chunk_fwd with each sequence cut into n_segments segments walked in
    parallel and joined by a scan of their (transition, zero-start state)
    pairs.  Returns (out, final_state)."""
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_alpha, "log_alpha"), (beta, "beta")):
        _need(t, torch.bfloat16, n)
    if initial_state is not None:
        _need(initial_state, torch.float32, "initial_state")
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=out_dtype, device=q.device)
    if final_state is None:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ws_bytes = lib.kda_chunk_fwd_segments_workspace_size(B, T, H, dk, dv, int(n_segments))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device) if ws_bytes else None
    _check(lib.kda_chunk_fwd_segments(
        _p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(initial_state), _p(out),
        _dtype_code(out.dtype), _p(final_state), B, T, H, dk, dv, float(scale), int(n_segments),
        _p(ws), ws_bytes, _stream(stream)), "kda_chunk_fwd_segments")
    return out, final_state


def kda_chunk_fwd_checkpointed(q, k, v, log_alpha, beta, initial_state=None, scale=1.0,
                               checkpoint_every=512, out_dtype=torch.float32, out=None,
                               final_state=None, checkpoints=None, stream=None):
    """kda_chunk_fwd plus the state after every `checkpoint_every` tokens.
    Returns (out, final_state, checkpoints [B, T // checkpoint_every, H, dk, dv])."""
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_alpha, "log_alpha"), (beta, "beta")):
        _need(t, torch.bfloat16, n)
    if initial_state is not None:
        _need(initial_state, torch.float32, "initial_state")
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=out_dtype, device=q.device)
    if final_state is None:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    n_ckpt = T // checkpoint_every if checkpoint_every > 0 else 0
    if checkpoints is None:
        checkpoints = torch.empty((B, n_ckpt, H, dk, dv), dtype=torch.float32, device=q.device)
    ws_bytes = lib.kda_chunk_fwd_workspace_size(B, T, H, dk, dv)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device) if ws_bytes else None
    _check(lib.kda_chunk_fwd_checkpointed(
        _p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(initial_state), _p(out),
        _dtype_code(out.dtype), _p(final_state), B, T, H, dk, dv, float(scale),
        _p(checkpoints) if n_ckpt else None, int(checkpoint_every), _p(ws), ws_bytes,
        _stream(stream)), "kda_chunk_fwd_checkpointed")
    return out, final_state, checkpoints


def kda_chunk_fwd_host_workspace(B, T, H, dk=128, dv=128, out_dtype=torch.float32, device=None):
    """A device workspace for kda_chunk_fwd_host of this shape."""
    lib = load()
    n = lib.kda_chunk_fwd_host_workspace_size(B, T, H, dk, dv, _dtype_code(out_dtype))
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or torch.device("cuda"))


def kda_chunk_fwd_host(q, k, v, log_alpha, beta, initial_state=None, scale=1.0,
                       out_dtype=torch.float32, out=None, final_state=None, workspace=None,
                       stream=None):
    """kda_chunk_fwd with every tensor in host memory (CPU tensors, ideally
    pinned): the library copies each round's inputs in and its outputs back
    while other rounds compute.  Returns (out, final_state) on the host."""
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_alpha, "log_alpha"), (beta, "beta")):
        _need_host(t, torch.bfloat16, n)
    if initial_state is not None:
        _need_host(initial_state, torch.float32, "initial_state")
    pin = q.is_pinned()
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=out_dtype, pin_memory=pin)
    if final_state is None:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, pin_memory=pin)
    if workspace is None:
        workspace = kda_chunk_fwd_host_workspace(B, T, H, dk, dv, out.dtype)
    _check(lib.kda_chunk_fwd_host(
        _p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(initial_state), _p(out),
        _dtype_code(out.dtype), _p(final_state), B, T, H, dk, dv, float(scale), _p(workspace),
        workspace.numel(), _stream(stream)), "kda_chunk_fwd_host")
    return out, final_state


def kda_chunk_bwd(q, k, v, log_alpha, beta, d_out, initial_state=None, d_final_state=None,
                  scale=1.0, want_initial_state_grad=True, stream=None):
    """Gradients of <d_out, out> + <d_final_state, final_state> for the layer
    kda_chunk_fwd computes.  Returns a dict of fp32 tensors: q, k, v,
    log_alpha ([B, T, H, d]), beta ([B, T, H]) and initial_state
    ([B, H, dk, dv], or None when not asked for)."""
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_alpha, "log_alpha"), (beta, "beta")):
        _need(t, torch.bfloat16, n)
    _need(d_out, torch.float32, "d_out")
    for t, n in ((initial_state, "initial_state"), (d_final_state, "d_final_state")):
        if t is not None:
            _need(t, torch.float32, n)
    dev = q.device
    g = {name: torch.empty((B, T, H, d), dtype=torch.float32, device=dev)
         for name, d in (("q", dk), ("k", dk), ("v", dv), ("log_alpha", dk))}
    g["beta"] = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    g["initial_state"] = (torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
                          if want_initial_state_grad else None)
    ws_bytes = lib.kda_chunk_bwd_workspace_size(B, T, H, dk, dv)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    _check(lib.kda_chunk_bwd(
        _p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(initial_state), _p(d_out),
        _p(d_final_state), _p(g["q"]), _p(g["k"]), _p(g["v"]), _p(g["log_alpha"]), _p(g["beta"]),
        _p(g["initial_state"]), B, T, H, dk, dv, float(scale), _p(ws), ws_bytes,
        _stream(stream)), "kda_chunk_bwd")
    return g


def kda_chunk_fwd_noalloc(q, k, v, log_alpha, beta, initial_state=None, scale=1.0,
                          out_dtype=torch.float32, output_final_state=True, out=None,
                          final_state=None, stream=None):
    """kda_chunk_fwd without a workspace: the library's fixed device scratch is
    used instead (B * ceil(T/64) * H <= 1008).  Outputs are allocated here
    only when not passed in; pass `out` / `final_state` to allocate nothing."""
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_alpha, "log_alpha"), (beta, "beta")):
        _need(t, torch.bfloat16, n)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=out_dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _check(lib.kda_chunk_fwd_noalloc(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta),
                                     _p(initial_state), _p(out), _dtype_code(out.dtype),
                                     _p(final_state), B, T, H, dk, dv, float(scale),
                                     _stream(stream)), "kda_chunk_fwd_noalloc")
    return out, final_state


def kda_varlen_fwd(q, k, v, log_alpha, beta, cu_seqlens, max_seqlen, initial_state=None,
                   scale=1.0, out_dtype=torch.float32, output_final_state=True, out=None,
                   final_state=None, stream=None):
    """Packed prefill.  Tensors [T_total,H,*] (or [1,T_total,H,*]);
    cu_seqlens int32 [N+1] on the device.  Returns (out, final_state [N,H,dk,dv])."""
    lib = load()
    squeeze = q.dim() == 4
    if squeeze:
        q, k, v, log_alpha, beta = q[0], k[0], v[0], log_alpha[0], beta[0]
    T_total, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    if out is None:
        out = torch.empty((T_total, H, dv), dtype=out_dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    ws_bytes = lib.kda_varlen_fwd_workspace_size(N, T_total, H, dk, dv)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device) if ws_bytes else None
    _check(lib.kda_varlen_fwd(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(cu_seqlens), N,
                              T_total, int(max_seqlen), _p(initial_state), _p(out),
                              _dtype_code(out.dtype), _p(final_state), H, dk, dv, float(scale),
                              _p(ws), ws_bytes, _stream(stream)), "kda_varlen_fwd")
    return (out[None] if squeeze else out), final_state


def kda_decode_step(q, k, v, log_alpha, beta, state, scale=1.0, out=None,
                    out_dtype=torch.float32, stream=None):
    """One token per sequence; `state` [N,H,dk,dv] fp32 is updated in place.
    q,k,log_alpha [N,H,dk], v [N,H,dv], beta [N,H] (bf16).  Returns out [N,H,dv]."""
    lib = load()
    N, H, dk = q.shape
    dv = v.shape[-1]
    _need(state, torch.float32, "state")
    if out is None:
        out = torch.empty((N, H, dv), dtype=out_dtype, device=q.device)
    _check(lib.kda_decode_step(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(state), _p(out),
                               _dtype_code(out.dtype), N, H, dk, dv, float(scale),
                               _stream(stream)), "kda_decode_step")
    return out


def kda_decode_verify(q, k, v, log_alpha, beta, state, scale=1.0, out_dtype=torch.float32,
                      out=None, stream=None):
    """Outputs of K drafted tokens per sequence from `state` (only read).
    q, k, log_alpha, v [N,K,H,d] bf16; beta [N,K,H]; state [N,H,d,d] fp32.
    Returns out [N,K,H,d]."""
    lib = load()
    N, K, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_alpha, "log_alpha"), (beta, "beta")):
        _need(t, torch.bfloat16, n)
    _need(state, torch.float32, "state")
    if out is None:
        out = torch.empty((N, K, H, dv), dtype=out_dtype, device=q.device)
    _check(lib.kda_decode_verify(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(state),
                                 _p(out), _dtype_code(out.dtype), N, K, H, dk, dv, float(scale),
                                 _stream(stream)), "kda_decode_verify")
    return out


def kda_decode_commit(q, k, v, log_alpha, beta, state, accepted, stream=None):
    """Advance `state` in place by the first accepted[n] draft tokens of each
    sequence (accepted: int32 [N] on the device)."""
    lib = load()
    N, K, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_alpha, "log_alpha"), (beta, "beta")):
        _need(t, torch.bfloat16, n)
    _need(state, torch.float32, "state")
    _need(accepted, torch.int32, "accepted")
    _check(lib.kda_decode_commit(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(state),
                                 _p(accepted), N, K, H, dk, dv, _stream(stream)),
           "kda_decode_commit")
    return state


class _CacheStruct(ctypes.Structure):
    """kda_paged_cache_t (include/kda.h)."""
    _fields_ = ([(n, _vp) for n in ("k", "v", "block_table", "lens")] +
                [(n, _ll) for n in ("page_stride", "token_stride", "head_stride", "table_stride")] +
                [("k_scale", _f), ("v_scale", _f)] +
                [(n, _i) for n in ("dtype", "n_seq", "num_pages", "page_size", "table_width", "H_kv", "d")])


_CODES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32, torch.float16: KDA_F16,
          torch.float8_e4m3fn: KDA_E4M3}


class PagedCache:
    """The pages of one attention layer and which sequence holds them.

    k_pages, v_pages: [num_pages, page_size, H_kv, d] bf16, fp16 or
    float8_e4m3fn, of equal strides, channels contiguous (for pages laid out
    head by head, pass a transposed view); block_table: int32 [N, width];
    lens: int32 [N], the tokens held before a call's new ones.  The tensors
    stay the caller's: pages, table and lens are read by every call as they
    are then, and lens is advanced by the caller (`cache.lens.add_(counts)`).
    k_scale, v_scale: what a stored 1.0 stands for.  All six may be assigned
    later; an assignment is checked like the constructor's arguments and holds
    for the calls after it (a graph keeps the tensors of its capture).
    """

    def __init__(self, k_pages, v_pages, block_table, lens, k_scale=1.0, v_scale=1.0):
        self._struct = _CacheStruct()
        self._ref = ctypes.addressof(self._struct)
        self._set(k_pages, v_pages, block_table, lens, float(k_scale), float(v_scale))

    def _set(self, k_pages, v_pages, block_table, lens, k_scale, v_scale):
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if not t.is_cuda or t.dim() != 4 or t.dtype not in _CODES or t.dtype == torch.float32:
                raise ValueError(f"{name} must be a CUDA tensor [num_pages, page_size, H_kv, d] of "
                                 "bfloat16, float16 or float8_e4m3fn")
        if (k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride() or
                k_pages.dtype != v_pages.dtype):
            raise ValueError("k_pages and v_pages must agree in shape, strides and dtype")
        if k_pages.stride(3) != 1:
            raise ValueError("the channels of a page must be contiguous")
        if not block_table.is_cuda or block_table.dtype != torch.int32 or block_table.dim() != 2 or (
                block_table.shape[1] > 1 and block_table.stride(1) != 1):
            raise ValueError("block_table must be a CUDA int32 tensor [N, width] with contiguous rows")
        _need(lens, torch.int32, "lens")
        if lens.shape != (block_table.shape[0],):
            raise ValueError("lens must have one entry for each row of block_table")
        if not k_pages.device == v_pages.device == block_table.device == lens.device:
            raise ValueError("k_pages, v_pages, block_table and lens must be on one device")
        self._held = k_pages, v_pages, block_table, lens, k_scale, v_scale
        pages, page_size, heads, d = k_pages.shape
        self.n_seq, self.heads, self.d, self.page_size = lens.numel(), heads, d, page_size
        self.capacity = block_table.shape[1] * page_size  # tokens a row of the table holds
        self.device, self.device_index = k_pages.device, k_pages.get_device()
        # the calls hold the address of this struct: it is filled anew, not replaced
        self._struct.__init__(
            k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), lens.data_ptr(),
            k_pages.stride(0), k_pages.stride(1), k_pages.stride(2), block_table.stride(0),
            k_scale, v_scale, _CODES[k_pages.dtype], self.n_seq, pages, page_size,
            block_table.shape[1], heads, d)

    def _field(i, convert=lambda x: x):
        def assign(self, value):
            self._set(*self._held[:i], convert(value), *self._held[i + 1:])
        return property(lambda self: self._held[i], assign)

    k_pages, v_pages, block_table, lens = _field(0), _field(1), _field(2), _field(3)
    k_scale, v_scale = _field(4, float), _field(5, float)
    del _field


# The calls below take a few microseconds on the GPU for a single token, so what
# they do on the host is kept short: one look at a tensor's shape and strides,
# raw pointers, no context manager where the current stream is used.

def _token_stride(x, heads, d, name, dev):
    """The elements between the tokens of x ([T, heads, d] or [N, K, heads, d],
    heads packed, sequences of equal length one after the other) on GPU dev."""
    shape = x.shape
    if x.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    if x.is_contiguous() and shape[-1] == d and shape[-2] == heads:
        return heads * d
    s = x.stride()
    if shape[-1] != d or shape[-2] != heads or s[-1] != 1 or (s[-2] != d and heads > 1):
        raise ValueError(f"{name} must be a CUDA tensor of {heads} heads of {d} channels, packed within a token")
    if len(shape) == 3 or shape[1] == 1:
        return s[0]
    if shape[0] > 1 and s[0] != shape[1] * s[1]:
        raise ValueError(f"the tokens of {name} must be evenly spaced")
    return s[1]


def _int32_ptr(t, n, name, dev):
    """The address of a contiguous int32 tensor of n entries on GPU dev; None for None."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype != torch.int32 or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on cuda:{dev}")
    return t.data_ptr()


def _stream_of(stream, dev):
    """The raw handle of `stream`, or of the current one, on GPU dev, which must be the current one."""
    if dev != torch.cuda.current_device() or (stream is not None and stream.device_index != dev):
        raise ValueError(f"the tensors are on cuda:{dev}, which is not the current device or the stream's")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to `stream`, or to the current one."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


@functools.lru_cache(maxsize=1024)
def _attend_workspace(device, N, K, H_q, H_kv, d, max_len):
    """Bytes of kda_cache_attend's workspace for these sizes on the current device."""
    return load().kda_cache_attend_workspace_size(N, K, H_q, H_kv, d, max_len)


def kda_cache_append(k, v, cache, q=None, inv_freq=None, interleaved=False, cu_seqlens=None,
                     counts=None, q_out=None, stream=None):
    """New tokens' keys and values into their pages, keys (and queries, if
    given) rotated by position * inv_freq on the way.  k, v [N,K,H_kv,d], or
    packed [T,H_kv,d] with cu_seqlens int32 [N+1]; q the same with H_q heads;
    inv_freq fp64 [rot_dim/2] or None (no rotation); counts int32 [N]: how many
    of the K tokens are real.  Returns the rotated queries (q_out), or None."""
    lib = _lib or load()
    shape, dtype = k.shape, k.dtype
    code = _CODES.get(dtype)
    if code is None or v.dtype != dtype or (q is not None and q.dtype != dtype):
        raise ValueError("k, v and q must have one dtype, bfloat16 or float16")
    H, d, N = cache.heads, cache.d, cache.n_seq
    if len(shape) != (4 if cu_seqlens is None else 3) or v.shape != shape:
        raise ValueError("k and v must be [N, K, H_kv, d], or [T, H_kv, d] with cu_seqlens")
    if cu_seqlens is None:
        K = shape[1]
        T = N * K
        if shape[0] != N:
            raise ValueError(f"k has {shape[0]} sequences, the cache {N}")
    else:
        K, T = 0, shape[0]
    rot, freqs = 0, None
    dev = cache.device_index
    if inv_freq is not None:
        _need(inv_freq, torch.float64, "inv_freq")
        if inv_freq.get_device() != dev:
            raise ValueError(f"inv_freq must be on cuda:{dev}")
        rot = 2 * inv_freq.numel()
        freqs = inv_freq.data_ptr() if rot else None
    qp = qo = None
    qs = qos = Hq = 0
    if q is not None:
        q_shape = q.shape
        if q_shape[:-2] != shape[:-2]:
            raise ValueError("q and k must have the same tokens")
        Hq = q_shape[-2]
        qs = _token_stride(q, Hq, d, "q", dev)
        if q_out is None:
            q_out = _empty(q_shape, dtype, q.device, stream)
            qos = Hq * d
        elif q_out.shape != q_shape or q_out.dtype != dtype:
            raise ValueError("q_out must have q's shape and dtype")
        else:
            qos = _token_stride(q_out, Hq, d, "q_out", dev)
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    code = lib.kda_cache_append(
        cache._ref, k.data_ptr(), v.data_ptr(), qp, qo, code, _token_stride(k, H, d, "k", dev),
        _token_stride(v, H, d, "v", dev), qs, qos, freqs, rot, interleaved,
        _int32_ptr(cu_seqlens, N + 1, "cu_seqlens", dev), _int32_ptr(counts, N, "counts", dev), K, T, Hq,
        _stream_of(stream, dev))
    if code:
        raise KDAError(code, "kda_cache_append")
    return q_out


def kda_cache_attend(q, cache, scale=None, window=0, counts=None, max_len=0, out=None,
                     return_lse=False, stream=None):
    """Attention of each sequence's K newest tokens, already appended, over its
    pages: token i at position lens[n] + i sees every position up to its own,
    or the `window` newest of them.  q [N,K,H_q,d] bf16 or fp16; scale defaults
    to 1/sqrt(d); max_len: an upper bound on lens + K (0: what the table
    holds).  Returns out [N,K,H_q,d], and with return_lse also the fp32 log of
    the sum of exponentials [N,K,H_q]."""
    lib = _lib or load()
    shape, dtype = q.shape, q.dtype
    code = _CODES.get(dtype)
    if len(shape) != 4 or shape[0] != cache.n_seq or code is None:
        raise ValueError(f"q must be [{cache.n_seq}, K, H_q, {cache.d}] in bfloat16 or float16")
    N, K, Hq, d = shape
    index, dev = cache.device_index, cache.device
    qs = _token_stride(q, Hq, cache.d, "q", index)
    if out is not None and (out.shape != shape or out.dtype != dtype or out.get_device() != index or
                            not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous tensor on cuda:{index} with q's shape and dtype")
    # no length passes 2^30; ctypes would cut larger numbers to their lower 32 bits
    window, max_len = max(-1, min(window, 0x7fffffff)), max(-1, min(max_len, 0x7fffffff))
    real, raw_stream = _int32_ptr(counts, N, "counts", index), _stream_of(stream, index)
    need = _attend_workspace(index, N, K, Hq, cache.heads, d, max_len or cache.capacity)
    lse = ws = None
    if out is None:
        out = _empty(shape, dtype, dev, stream)
    if return_lse:
        lse = _empty((N, K, Hq), torch.float32, dev, stream)
    if need:
        ws = _empty(need, torch.uint8, dev, stream)
    code = lib.kda_cache_attend(
        cache._ref, q.data_ptr(), code, qs, out.data_ptr(), None if lse is None else lse.data_ptr(),
        real, K, Hq, d ** -0.5 if scale is None else scale, window, max_len,
        None if ws is None else ws.data_ptr(), need, raw_stream)
    if code:
        raise KDAError(code, "kda_cache_attend")
    return (out, lse) if return_lse else out


def kda_draft_accept(draft_tokens, draft_probs, target_probs, uniform, draft_lens=None, counts=None,
                     tokens=None, stream=None):
    """How many of each sequence's K drafted tokens are kept, and the token
    drawn after them.  draft_tokens int32 [N,K]; draft_probs [N,K,V] (or None:
    drafts that are no random draw) and target_probs [N,K+1,V] in one dtype
    (fp32, bf16 or fp16); uniform fp32 [N,K+1] in [0, 1); draft_lens int32 [N]
    (negative: an idle sequence).  Returns (counts int32 [N], the tokens gained
    by each sequence, and tokens int32 [N,K+1], -1 beyond them)."""
    lib = _lib or load()
    N, K1, V = target_probs.shape
    K = K1 - 1
    dtype = target_probs.dtype
    code = _CODES.get(dtype)
    ts = target_probs.stride()
    if code is None or not target_probs.is_cuda or (ts[2] != 1 and V > 1):
        raise ValueError("target_probs must be a CUDA tensor of float32, bfloat16 or float16 with contiguous rows")
    dev = target_probs.device
    index = dev.index
    _need(draft_tokens, torch.int32, "draft_tokens")
    _need(uniform, torch.float32, "uniform")
    if draft_tokens.get_device() != index or uniform.get_device() != index:
        raise ValueError(f"draft_tokens and uniform must be on cuda:{index}, as target_probs")
    if K < 0 or draft_tokens.shape != (N, K) or uniform.shape != (N, K1):
        raise ValueError("draft_tokens must be [N, K] and uniform [N, K + 1] for target_probs [N, K + 1, V]")
    dp, ds = None, (0, 0)
    if draft_probs is not None:
        ds = draft_probs.stride()
        if (draft_probs.dtype != dtype or draft_probs.get_device() != index or draft_probs.shape != (N, K, V) or
                (ds[2] != 1 and V > 1)):
            raise ValueError(f"draft_probs must be a tensor {(N, K, V)} on cuda:{index}, of target_probs' dtype with "
                             "contiguous rows")
        dp = draft_probs.data_ptr()
    if tokens is not None:
        _need(tokens, torch.int32, "tokens")
        if tokens.shape != (N, K1) or tokens.get_device() != index:
            raise ValueError(f"tokens must be {(N, K1)} on cuda:{index}")
    if counts is None:
        counts = _empty(N, torch.int32, dev, stream)
    if tokens is None:
        tokens = _empty((N, K1), torch.int32, dev, stream)
    code = lib.kda_draft_accept(
        draft_tokens.data_ptr(), dp, target_probs.data_ptr(), code, ds[0], ds[1], ts[0], ts[1],
        uniform.data_ptr(), _int32_ptr(draft_lens, N, "draft_lens", index), _int32_ptr(counts, N, "counts", index),
        tokens.data_ptr(), N, K, V, _stream_of(stream, index))
    if code:
        raise KDAError(code, "kda_draft_accept")
    return counts, tokens


def kda_chunk_fwd_launches(B, T, H):
    """Kernel launches one kda_chunk_fwd call of this shape makes on the current device."""
    return int(load().kda_chunk_fwd_launches(int(B), int(T), int(H)))


def kda_last_device_status(stream=None) -> int:
    return int(load().kda_last_device_status(_stream(stream)))


def kda_status_string(code: int) -> str:
    return load().kda_status_string(int(code)).decode()


def kda_version() -> str:
    return load().kda_version().decode()
