"""GB300-native Gated DeltaNet (gated delta rule) sequence mixer.

Thin ctypes binding over the C ABI in ``include/gdn.h``: it checks tensor
shapes, dtypes and devices, reads sizes off the tensors, and passes raw device
pointers and the current CUDA stream.  Every step of the computation runs in
the library's CUDA kernels; there is no CPU or PyTorch fallback, and calls
raise when the compiled library is missing.

    out, S_final = prefill(q, k, v, alpha, beta, S0=None, cu_seqlens=None)
    out, S_final = prefill(..., workspace=ws)  # caller-owned scratch, nothing allocated
    out = decode_step(q, k, v, alpha, beta, S)          # S updated in place
    grads = prefill_backward(q, k, v, alpha, beta, dout, S0, dS_final)   # training
    x = prepare(qkv, conv_w, a_raw, b_raw, A_log, dt_bias, heads)   # -> q, k, v, alpha, beta
    y = output_norm_gate(out, g, w)                     # Eq. 20 read-out
    y = decode_layer_step(qkv, conv_w, a_raw, b_raw, A_log, dt_bias, conv_state, S, g, w)
    q, scale, s = residual_norm_fp8(x, w, residual)      # the layer around the mixer:
    out = linear_fp8(q, scale, wq, w_scale)              # 8-bit projections,
    h = gated_ffn(x, w_gate, w_up)                       # gated feed-forward
    out, lse = attention_prefill(q, k, v, cu_seqlens, cu_seqlens_k)   # a hybrid's attention layers
    cache = kv_cache(layers, pages, kv_heads, rows, max_pages)        # and their paged cache:
    start = cache_reserve(cache, counts); cache_append(cache, k, v, start, layer=i)
    out = attention_decode_step(q, cache, layer=i)
    k, v = cache_gather(cache, cu_seqlens_k, tokens, layer=i)         # (prompts that go on)

Recurrence (Appendix A.3, Eq. 16-19 of "Long-Context Aware Upcycling"):
S_t = alpha_t S_{t-1}(I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
o_t = S_t q_t / sqrt(dk), with the state stored as [dv, dk].
"""
from __future__ import annotations

import ctypes
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libgdn_gb300.so"
_lib = None
_direct = None   # csrc/binding.cpp's module, once the library is loaded

GDN_F32, GDN_BF16, GDN_E4M3 = 0, 1, 2
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "alignment",
           4: "CUDA error", 5: "device timeout", 6: "malformed cu_seqlens",
           8: "no page of the attention cache left", 9: "outside the attention cache"}


class GDNError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed with status {code} ({_STATUS.get(code, 'unknown')})")
        self.code = code


def lib_path() -> str:
    return os.path.join(_HERE, LIB_NAME)


def load():
    """Load the compiled library (raises if it has not been built)."""
    global _lib, _direct
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{LIB_NAME} is not built; run __graft_entry__.build() "
                           f"(or python -m hybrid_linear_attention_deltanet_gb300._build)")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.gdn_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32,
                                vp]
    lib.gdn_prefill.restype = ctypes.c_int
    lib.gdn_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
    lib.gdn_decode_step.restype = ctypes.c_int
    lib.gdn_get_device_status.argtypes = [vp]
    lib.gdn_get_device_status.restype = ctypes.c_int
    lib.gdn_version.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_kernel_launches.restype = ctypes.c_uint64
    lib.gdn_prefill_path.argtypes = [ctypes.c_int32]
    lib.gdn_prefill_path.restype = ctypes.c_char_p
    lib.gdn_prefill_scan.argtypes = [vp] * 9 + [i32, i64, i32, i32, i32, i32, i32, vp]
    lib.gdn_prefill_scan.restype = ctypes.c_int
    lib.gdn_prefill_backward.argtypes = [vp] * 15 + [i32, i64, i32, i32, i32, i32, vp]
    lib.gdn_prefill_backward.restype = ctypes.c_int
    lib.gdn_prepare.argtypes = [vp] * 14 + [i32, i64, i32, i32, i32, i32, vp]
    lib.gdn_prepare.restype = ctypes.c_int
    lib.gdn_prepare_decode_step.argtypes = [vp] * 12 + [i32, i32, i32, i32, i32, vp]
    lib.gdn_prepare_decode_step.restype = ctypes.c_int
    lib.gdn_output_norm_gate.argtypes = [vp, vp, vp, ctypes.c_float, i32, vp, i64, i32, i32, i32,
                                         vp]
    lib.gdn_decode_layer_step.argtypes = [vp] * 10 + [ctypes.c_float, i32, vp, i32, i32, i32,
                                                      i32, i32, vp]
    lib.gdn_decode_layer_step.restype = ctypes.c_int
    lib.gdn_output_norm_gate.restype = ctypes.c_int
    sz = ctypes.c_size_t
    lib.gdn_prefill_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32, i32]
    lib.gdn_prefill_workspace_size.restype = sz
    lib.gdn_prefill_ws.argtypes = [vp] * 9 + [i32, i64, i32, i32, i32, i32, vp, sz, vp]
    lib.gdn_prefill_ws.restype = ctypes.c_int
    lib.gdn_prefill_scan_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32, i32, i32]
    lib.gdn_prefill_scan_workspace_size.restype = sz
    lib.gdn_prefill_scan_ws.argtypes = [vp] * 9 + [i32, i64, i32, i32, i32, i32, i32, vp, sz,
                                                    vp]
    lib.gdn_prefill_scan_ws.restype = ctypes.c_int
    lib.gdn_prefill_backward_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32, i32]
    lib.gdn_prefill_backward_workspace_size.restype = sz
    lib.gdn_prefill_backward_ws.argtypes = [vp] * 15 + [i32, i64, i32, i32, i32, i32, vp, sz, vp]
    lib.gdn_prefill_backward_ws.restype = ctypes.c_int
    lib.gdn_prefill_layer.argtypes = [vp] * 12 + [ctypes.c_float, i32, vp, vp, i32, i64, i32,
                                                  i32, i32, i32, vp]
    lib.gdn_prefill_layer.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.gdn_residual_norm.argtypes = [vp, vp, vp, f32, vp, vp, i64, i32, i32, vp]
    lib.gdn_residual_norm.restype = ctypes.c_int
    lib.gdn_residual_norm_fp8.argtypes = [vp, vp, vp, f32, vp, vp, vp, i64, i32, i32, vp]
    lib.gdn_residual_norm_fp8.restype = ctypes.c_int
    lib.gdn_residual_norm_backward.argtypes = [vp] * 4 + [f32, vp, vp, i64, i32, i32, vp]
    lib.gdn_residual_norm_backward.restype = ctypes.c_int
    lib.gdn_residual_norm_backward_workspace_size.argtypes = [i64, i32, i32]
    lib.gdn_residual_norm_backward_workspace_size.restype = sz
    lib.gdn_residual_norm_backward_ws.argtypes = [vp] * 4 + [f32, vp, vp, i64, i32, i32, vp, sz,
                                                             vp]
    lib.gdn_residual_norm_backward_ws.restype = ctypes.c_int
    lib.gdn_quantize_fp8.argtypes = [vp, vp, vp, i64, i32, i32, i32, vp]
    lib.gdn_quantize_fp8.restype = ctypes.c_int
    lib.gdn_linear_fp8.argtypes = [vp] * 5 + [i64, i32, i32, i32, vp]
    lib.gdn_linear_fp8.restype = ctypes.c_int
    lib.gdn_gated_ffn.argtypes = [vp, vp, vp, i32, vp, i64, i32, i32, i32, vp]
    lib.gdn_gated_ffn.restype = ctypes.c_int
    lib.gdn_gated_ffn_backward.argtypes = [vp] * 4 + [i32, vp, vp, vp, i64, i32, i32, i32, vp]
    lib.gdn_gated_ffn_backward.restype = ctypes.c_int
    lib.gdn_gated_ffn_backward_workspace_size.argtypes = [i64, i32, i32, i32]
    lib.gdn_gated_ffn_backward_workspace_size.restype = sz
    lib.gdn_gated_ffn_backward_ws.argtypes = [vp] * 4 + [i32, vp, vp, vp, i64, i32, i32, i32, vp,
                                                         sz, vp]
    lib.gdn_gated_ffn_backward_ws.restype = ctypes.c_int
    lib.gdn_attention_prefill.argtypes = [vp] * 5 + [f32, vp, vp, i32, i64, i64, i32, i32, i32,
                                                     i64, i64, i64, vp]
    lib.gdn_attention_prefill.restype = ctypes.c_int
    lib.gdn_attention_prefill_backward.argtypes = [vp] * 8 + [f32, vp, vp, vp, i32, i64, i64, i32,
                                                              i32, i32, i64, i64, i64, vp]
    lib.gdn_attention_prefill_backward.restype = ctypes.c_int
    lib.gdn_attention_prefill_backward_workspace_size.argtypes = [i32, i64, i64, i32, i32, i32,
                                                                  i32]
    lib.gdn_attention_prefill_backward_workspace_size.restype = sz
    lib.gdn_attention_prefill_backward_ws.argtypes = [vp] * 8 + [f32, vp, vp, vp, i32, i64, i64,
                                                                 i32, i32, i32, i64, i64, i64, vp,
                                                                 sz, vp]
    lib.gdn_attention_prefill_backward_ws.restype = ctypes.c_int
    lib.gdn_attention_decode_step.argtypes = [vp, vp, i32, i32, f32, vp, vp]
    lib.gdn_attention_decode_step.restype = ctypes.c_int
    lib.gdn_attention_decode_step_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.gdn_attention_decode_step_workspace_size.restype = sz
    lib.gdn_attention_decode_step_ws.argtypes = [vp, vp, i32, i32, f32, vp, vp, sz, vp]
    lib.gdn_attention_decode_step_ws.restype = ctypes.c_int
    lib.gdn_cache_reserve.argtypes = [vp] * 4
    lib.gdn_cache_reserve.restype = ctypes.c_int
    lib.gdn_cache_append.argtypes = [vp, i32, vp, vp, vp, vp, i64, i64, i64, vp]
    lib.gdn_cache_append.restype = ctypes.c_int
    lib.gdn_cache_gather.argtypes = [vp, i32, vp, i64, vp, vp, vp]
    lib.gdn_cache_gather.restype = ctypes.c_int
    lib.gdn_cache_free.argtypes = [vp, vp, i32, vp]
    lib.gdn_cache_free.restype = ctypes.c_int
    lib.gdn_cache_fork.argtypes = [vp, vp, vp, i32, vp]
    lib.gdn_cache_fork.restype = ctypes.c_int
    lib.gdn_cache_compact.argtypes = [vp, vp, vp]
    lib.gdn_cache_compact.restype = ctypes.c_int
    lib.gdn_release_scratch.restype = ctypes.c_int
    lib.gdn_testing_scratch_reserved.argtypes = [vp]
    lib.gdn_testing_scratch_reserved.restype = ctypes.c_int
    try:
        from . import _layer_calls
        _layer_calls.bind(path)
        _direct = _layer_calls
    except ImportError as e:   # built without Python's headers, or for another PyTorch
        _direct = _Declines()
        warnings.warn("the layer operators' direct calls are not available, each call takes "
                      f"10 to 20 us longer on the host: {e}", RuntimeWarning, stacklevel=2)
    _lib = lib
    return lib


class _Declines:
    """In the place of _layer_calls: every call takes the general path."""

    def __getattr__(self, name):
        return lambda *args: None


def _direct_calls():
    if _lib is None:
        load()
    return _direct


def _ws_args(workspace, index):
    """(pointer, bytes) of a caller workspace: a uint8 tensor on CUDA device `index`."""
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 \
            or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous torch.uint8 tensor")
    if workspace.get_device() != index:
        raise ValueError(f"workspace is on {workspace.device}, expected cuda:{index}")
    return ctypes.c_void_p(workspace.data_ptr()), workspace.numel()


def prefill_workspace_size(batch, seqlen, heads, dk=256, dv=256, io_dtype=torch.bfloat16,
                           varlen=False) -> int:
    """Bytes of device workspace ``prefill(..., workspace=...)`` needs
    (``gdn_prefill_workspace_size``)."""
    n = load().gdn_prefill_workspace_size(batch, seqlen, heads, dk, dv, _io_code(io_dtype),
                                          int(bool(varlen)))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported prefill arguments")
    return int(n)


def prefill_scan_workspace_size(batch, seqlen, heads, dk=256, dv=256, io_dtype=torch.bfloat16,
                                varlen=False, segments=8) -> int:
    n = load().gdn_prefill_scan_workspace_size(batch, seqlen, heads, dk, dv, _io_code(io_dtype),
                                               int(bool(varlen)), int(segments))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported prefill_scan arguments")
    return int(n)


def prefill_backward_workspace_size(batch, seqlen, heads, dk=256, dv=256,
                                    io_dtype=torch.bfloat16, varlen=False) -> int:
    n = load().gdn_prefill_backward_workspace_size(batch, seqlen, heads, dk, dv,
                                                   _io_code(io_dtype), int(bool(varlen)))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported prefill_backward arguments")
    return int(n)


def release_scratch() -> None:
    """Hand the library's scratch pool on the current device back to the system
    (``gdn_release_scratch``; synchronises the device)."""
    rc = load().gdn_release_scratch()
    if rc != 0:
        raise GDNError("gdn_release_scratch", rc)


def scratch_reserved() -> int:
    """Bytes the library's scratch pool holds mapped on the current device."""
    v = ctypes.c_uint64(0)
    rc = load().gdn_testing_scratch_reserved(ctypes.byref(v))
    if rc != 0:
        raise GDNError("gdn_testing_scratch_reserved", rc)
    return int(v.value)


def version() -> str:
    return load().gdn_version().decode()


def kernel_launches() -> int:
    """Cumulative count of the library's kernel launches in this process."""
    return int(load().gdn_kernel_launches())


def prefill_path(io_dtype=torch.bfloat16) -> str:
    """Kernel path gdn_prefill takes for this I/O dtype."""
    return load().gdn_prefill_path(_io_code(io_dtype)).decode()


def _stream_handle(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _io_code(dtype):
    if dtype == torch.bfloat16:
        return GDN_BF16
    if dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {dtype}")


def _check(t, name, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def prefill(q, k, v, alpha, beta, S0=None, cu_seqlens=None, out=None, S_final=None,
            return_final: bool = True, stream=None, workspace=None):
    """Chunkwise prefill (``gdn_prefill``).

    Dense: q, k [B, T, H, dk]; v [B, T, H, dv]; alpha, beta [B, T, H] fp32.
    Varlen: the same with B = 1 (or no batch axis) and ``cu_seqlens`` int32
    [N + 1] on the device.  S0 / S_final: [N, H, dv, dk] fp32.
    ``workspace``: a uint8 CUDA tensor of at least
    :func:`prefill_workspace_size` bytes (``gdn_prefill_ws``: the call then
    allocates nothing); None takes scratch from the library's pool.
    Returns (out, S_final); S_final is None when ``return_final`` is False.
    """
    return _prefill_call(q, k, v, alpha, beta, S0, cu_seqlens, out, S_final, return_final,
                         stream, workspace, None)


def prefill_scan(q, k, v, alpha, beta, S0=None, cu_seqlens=None, segments=8, out=None,
                 S_final=None, return_final: bool = True, stream=None, workspace=None):
    """``gdn_prefill_scan``: :func:`prefill` with every sequence cut into
    ``segments`` pieces of whole chunks, run as a scan over the segments
    (dense or packed, bf16 or fp32).  Returns (out, S_final)."""
    if int(segments) < 1:
        raise ValueError("segments must be >= 1")
    return _prefill_call(q, k, v, alpha, beta, S0, cu_seqlens, out, S_final, return_final,
                         stream, workspace, int(segments))


def _prefill_call(q, k, v, alpha, beta, S0, cu_seqlens, out, S_final, return_final, stream,
                  workspace, segments):
    lib = load()
    dev = q.device
    io = q.dtype
    _io_code(io)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(t, name, io, dev)
    _check(alpha, "alpha", torch.float32, dev)
    _check(beta, "beta", torch.float32, dev)
    if q.dim() not in (3, 4) or k.shape != q.shape:
        raise ValueError("q and k must be [B, T, H, dk] (or [T, H, dk]) and equal in shape")
    H, dk, dv = q.shape[-2], q.shape[-1], v.shape[-1]
    if v.shape[:-1] != q.shape[:-1] or alpha.shape != q.shape[:-1] or beta.shape != q.shape[:-1]:
        raise ValueError("v, alpha, beta must match q's leading [.., T, H] axes")
    if cu_seqlens is None:
        B, T = (q.shape[0], q.shape[1]) if q.dim() == 4 else (1, q.shape[0])
        N, seqlen = B, T
    else:
        _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if q.dim() == 4 and q.shape[0] != 1:
            raise ValueError("varlen input must have batch axis 1")
        N = cu_seqlens.numel() - 1
        seqlen = q.shape[-3]
    if S0 is not None:
        _check(S0, "S0", torch.float32, dev)
        if tuple(S0.shape) != (N, H, dv, dk):
            raise ValueError(f"S0 must be [{N}, {H}, {dv}, {dk}]")
    if out is None:
        out = torch.empty_like(v)
    else:
        _check(out, "out", io, dev)
    if S_final is None and return_final:
        S_final = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    elif S_final is not None:
        _check(S_final, "S_final", torch.float32, dev)
    with torch.cuda.device(dev):
        args = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
                _ptr(out), _ptr(S_final), N, seqlen, H, dk, dv, _io_code(io))
        if segments is not None:
            args = args + (segments,)
        name = "gdn_prefill" if segments is None else "gdn_prefill_scan"
        if workspace is None:
            rc = getattr(lib, name)(*args, _stream_handle(stream))
        else:
            name += "_ws"
            rc = getattr(lib, name)(*args, *_ws_args(workspace, q.get_device()), _stream_handle(stream))
    if rc != 0:
        raise GDNError(name, rc)
    return out, S_final


def prefill_backward(q, k, v, alpha, beta, dout, S0=None, dS_final=None, cu_seqlens=None,
                     want_dS0: bool = True, stream=None, workspace=None):
    """Gradients of the prefill (``gdn_prefill_backward``) for
    L = <dout, out> + <dS_final, S_final>: returns dict dq, dk, dv (dtype of
    q), dalpha, dbeta (fp32) and dS0 ([N, H, dv, dk] fp32, or None when
    ``want_dS0`` is False).  Arguments as in :func:`prefill`; dout like out."""
    lib = load()
    dev, io = q.device, q.dtype
    _io_code(io)
    for name, t in (("q", q), ("k", k), ("v", v), ("dout", dout)):
        _check(t, name, io, dev)
    _check(alpha, "alpha", torch.float32, dev)
    _check(beta, "beta", torch.float32, dev)
    if q.dim() not in (3, 4) or k.shape != q.shape or dout.shape != v.shape:
        raise ValueError("q, k must be [B, T, H, dk] (or [T, H, dk]); dout shaped like v")
    H, dk, dv = q.shape[-2], q.shape[-1], v.shape[-1]
    if v.shape[:-1] != q.shape[:-1] or alpha.shape != q.shape[:-1] or beta.shape != q.shape[:-1]:
        raise ValueError("v, alpha, beta must match q's leading [.., T, H] axes")
    if cu_seqlens is None:
        B, T = (q.shape[0], q.shape[1]) if q.dim() == 4 else (1, q.shape[0])
        N, seqlen = B, T
    else:
        _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if q.dim() == 4 and q.shape[0] != 1:
            raise ValueError("varlen input must have batch axis 1")
        N, seqlen = cu_seqlens.numel() - 1, q.shape[-3]
    for name, t in (("S0", S0), ("dS_final", dS_final)):
        if t is not None:
            _check(t, name, torch.float32, dev)
            if tuple(t.shape) != (N, H, dv, dk):
                raise ValueError(f"{name} must be [{N}, {H}, {dv}, {dk}]")
    g = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
             dalpha=torch.empty_like(alpha), dbeta=torch.empty_like(beta),
             dS0=torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev) if want_dS0 else None)
    with torch.cuda.device(dev):
        args = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
                _ptr(dout), _ptr(dS_final), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
                _ptr(g["dalpha"]), _ptr(g["dbeta"]), _ptr(g["dS0"]), N, seqlen, H, dk, dv,
                _io_code(io))
        if workspace is None:
            rc = lib.gdn_prefill_backward(*args, _stream_handle(stream))
        else:
            rc = lib.gdn_prefill_backward_ws(*args, *_ws_args(workspace, q.get_device()),
                                             _stream_handle(stream))
    if rc != 0:
        raise GDNError("gdn_prefill_backward", rc)
    return g


def decode_step(q, k, v, alpha, beta, S, out=None, stream=None):
    """One token per sequence (``gdn_decode_step``): q, k [N, H, dk];
    v [N, H, dv]; alpha, beta [N, H]; S [N, H, dv, dk] fp32 updated in place.
    Returns out [N, H, dv] in the dtype of v."""
    lib = load()
    dev = q.device
    io = q.dtype
    _io_code(io)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(t, name, io, dev)
    _check(alpha, "alpha", torch.float32, dev)
    _check(beta, "beta", torch.float32, dev)
    _check(S, "S", torch.float32, dev)
    N, H, dk = q.shape
    dv = v.shape[-1]
    if tuple(S.shape) != (N, H, dv, dk) or alpha.shape != (N, H) or beta.shape != (N, H):
        raise ValueError("shape mismatch in decode_step arguments")
    if out is None:
        out = torch.empty_like(v)
    else:
        _check(out, "out", io, dev)
    with torch.cuda.device(dev):
        rc = lib.gdn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S),
                                 _ptr(out), N, H, dk, dv, _io_code(io), _stream_handle(stream))
    if rc != 0:
        raise GDNError("gdn_decode_step", rc)
    return out


GATE_ACT = {"silu": 0, "sigmoid": 1}


def prepare(qkv, conv_w, a_raw, b_raw, A_log, dt_bias, heads, dk=256, dv=256, cu_seqlens=None,
            conv_state_in=None, conv_state_out=None, stream=None):
    """Pre-recurrence steps (``gdn_prepare``): short conv + SiLU on the packed
    q|k|v projection, q/k L2 normalisation, decay and write strength.

    qkv [B, T, C] or [T, C] (C = H*(2*dk + dv)); conv_w [C, 4] fp32;
    a_raw, b_raw [B, T, H] / [T, H] fp32; A_log, dt_bias [H] fp32;
    conv_state_in / conv_state_out [N, 3, C] in qkv's dtype (or None).
    Returns dict q, k [.., H, dk], v [.., H, dv], alpha, beta [.., H] ready
    for :func:`prefill`.
    """
    lib = load()
    dev, io = qkv.device, qkv.dtype
    _io_code(io)
    H = heads
    C = H * (2 * dk + dv)
    _check(qkv, "qkv", io, dev)
    if qkv.shape[-1] != C or qkv.dim() not in (2, 3):
        raise ValueError(f"qkv must be [B, T, {C}] or [T, {C}]")
    lead = tuple(qkv.shape[:-1])
    for name, t in (("a_raw", a_raw), ("b_raw", b_raw)):
        _check(t, name, torch.float32, dev)
        if tuple(t.shape) != lead + (H,):
            raise ValueError(f"{name} must be {list(lead + (H,))}")
    _check(conv_w, "conv_w", torch.float32, dev)
    if tuple(conv_w.shape) != (C, 4):
        raise ValueError(f"conv_w must be [{C}, 4]")
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias)):
        _check(t, name, torch.float32, dev)
        if tuple(t.shape) != (H,):
            raise ValueError(f"{name} must be [{H}]")
    if cu_seqlens is None:
        B, T = (qkv.shape[0], qkv.shape[1]) if qkv.dim() == 3 else (1, qkv.shape[0])
        N, seqlen = B, T
    else:
        _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if qkv.dim() == 3 and qkv.shape[0] != 1:
            raise ValueError("varlen input must have batch axis 1")
        N, seqlen = cu_seqlens.numel() - 1, qkv.shape[-2]
    for name, t in (("conv_state_in", conv_state_in), ("conv_state_out", conv_state_out)):
        if t is not None:
            _check(t, name, io, dev)
            if tuple(t.shape) != (N, 3, C):
                raise ValueError(f"{name} must be [{N}, 3, {C}]")
    out = dict(q=torch.empty(lead + (H, dk), dtype=io, device=dev),
               k=torch.empty(lead + (H, dk), dtype=io, device=dev),
               v=torch.empty(lead + (H, dv), dtype=io, device=dev),
               alpha=torch.empty(lead + (H,), dtype=torch.float32, device=dev),
               beta=torch.empty(lead + (H,), dtype=torch.float32, device=dev))
    with torch.cuda.device(dev):
        rc = lib.gdn_prepare(_ptr(qkv), _ptr(conv_w), _ptr(a_raw), _ptr(b_raw), _ptr(A_log),
                             _ptr(dt_bias), _ptr(cu_seqlens), _ptr(conv_state_in),
                             _ptr(conv_state_out), _ptr(out["q"]), _ptr(out["k"]),
                             _ptr(out["v"]), _ptr(out["alpha"]), _ptr(out["beta"]), N, seqlen,
                             H, dk, dv, _io_code(io), _stream_handle(stream))
    if rc != 0:
        raise GDNError("gdn_prepare", rc)
    return out


def prepare_decode_step(qkv, conv_w, a_raw, b_raw, A_log, dt_bias, conv_state, heads, dk=256,
                        dv=256, out=None, stream=None):
    """``gdn_prepare_decode_step``: one token per sequence, qkv [N, C],
    a_raw / b_raw [N, H], conv_state [N, 3, C] updated in place.  Returns
    dict q, k [N, H, dk], v [N, H, dv], alpha, beta [N, H] (or fills ``out``)."""
    lib = load()
    dev, io = qkv.device, qkv.dtype
    _io_code(io)
    H = heads
    C = H * (2 * dk + dv)
    _check(qkv, "qkv", io, dev)
    if qkv.dim() != 2 or qkv.shape[1] != C:
        raise ValueError(f"qkv must be [N, {C}]")
    N = qkv.shape[0]
    _check(conv_state, "conv_state", io, dev)
    _check(conv_w, "conv_w", torch.float32, dev)
    for name, t in (("a_raw", a_raw), ("b_raw", b_raw)):
        _check(t, name, torch.float32, dev)
    if (tuple(conv_state.shape) != (N, 3, C) or tuple(conv_w.shape) != (C, 4)
            or tuple(a_raw.shape) != (N, H) or tuple(b_raw.shape) != (N, H)):
        raise ValueError("shape mismatch in prepare_decode_step arguments")
    if out is None:
        out = dict(q=torch.empty((N, H, dk), dtype=io, device=dev),
                   k=torch.empty((N, H, dk), dtype=io, device=dev),
                   v=torch.empty((N, H, dv), dtype=io, device=dev),
                   alpha=torch.empty((N, H), dtype=torch.float32, device=dev),
                   beta=torch.empty((N, H), dtype=torch.float32, device=dev))
    with torch.cuda.device(dev):
        rc = lib.gdn_prepare_decode_step(
            _ptr(qkv), _ptr(conv_w), _ptr(a_raw), _ptr(b_raw), _ptr(A_log), _ptr(dt_bias),
            _ptr(conv_state), _ptr(out["q"]), _ptr(out["k"]), _ptr(out["v"]), _ptr(out["alpha"]),
            _ptr(out["beta"]), N, H, dk, dv, _io_code(io), _stream_handle(stream))
    if rc != 0:
        raise GDNError("gdn_prepare_decode_step", rc)
    return out


def output_norm_gate(o, g, w, eps=1e-5, act="silu", y=None, stream=None):
    """Eq. 20 read-out (``gdn_output_norm_gate``): o / rms(o) * w * act(g)
    per (token, head) over dv.  o, g [.., H, dv] (same dtype); w [dv] fp32.
    ``y`` defaults to a new tensor; pass ``y=o`` to normalise in place."""
    lib = load()
    dev, io = o.device, o.dtype
    _io_code(io)
    _check(o, "o", io, dev)
    _check(g, "g", io, dev)
    _check(w, "w", torch.float32, dev)
    if g.shape != o.shape or o.dim() < 2 or tuple(w.shape) != (o.shape[-1],):
        raise ValueError("o and g must share [.., H, dv]; w must be [dv]")
    H, dv = o.shape[-2], o.shape[-1]
    tokens = o.numel() // (H * dv)
    if y is None:
        y = torch.empty_like(o)
    else:
        _check(y, "y", io, dev)
    with torch.cuda.device(dev):
        rc = lib.gdn_output_norm_gate(_ptr(o), _ptr(g), _ptr(w), float(eps), GATE_ACT[act], _ptr(y),
                                      tokens, H, dv, _io_code(io), _stream_handle(stream))
    if rc != 0:
        raise GDNError("gdn_output_norm_gate", rc)
    return y


def decode_layer_step(qkv, conv_w, a_raw, b_raw, A_log, dt_bias, conv_state, S, gate, norm_w,
                      eps=1e-5, act="silu", y=None, stream=None):
    """One fused decode step of the mixer core (``gdn_decode_layer_step``):
    conv + SiLU + L2 norm + gates, the state update, and Eq. 20's gated
    RMSNorm.  qkv [N, C]; conv_state [N, 3, C] and S [N, H, dv, dk] updated in
    place; gate [N, H, dv]; norm_w [dv].  Returns y [N, H, dv]."""
    lib = load()
    dev, io = qkv.device, qkv.dtype
    _io_code(io)
    N, H, dv, dk = S.shape
    C = H * (2 * dk + dv)
    _check(qkv, "qkv", io, dev)
    _check(conv_state, "conv_state", io, dev)
    _check(gate, "gate", io, dev)
    _check(S, "S", torch.float32, dev)
    for name, t in (("conv_w", conv_w), ("a_raw", a_raw), ("b_raw", b_raw), ("A_log", A_log),
                    ("dt_bias", dt_bias), ("norm_w", norm_w)):
        _check(t, name, torch.float32, dev)
    if (tuple(qkv.shape) != (N, C) or tuple(conv_state.shape) != (N, 3, C)
            or tuple(conv_w.shape) != (C, 4) or tuple(a_raw.shape) != (N, H)
            or tuple(b_raw.shape) != (N, H) or tuple(gate.shape) != (N, H, dv)
            or tuple(norm_w.shape) != (dv,)):
        raise ValueError("shape mismatch in decode_layer_step arguments")
    if y is None:
        y = torch.empty_like(gate)
    else:
        _check(y, "y", io, dev)
    with torch.cuda.device(dev):
        rc = lib.gdn_decode_layer_step(
            _ptr(qkv), _ptr(conv_w), _ptr(a_raw), _ptr(b_raw), _ptr(A_log), _ptr(dt_bias),
            _ptr(conv_state), _ptr(S), _ptr(gate), _ptr(norm_w), float(eps), GATE_ACT[act],
            _ptr(y), N, H, dk, dv, _io_code(io), _stream_handle(stream))
    if rc != 0:
        raise GDNError("gdn_decode_layer_step", rc)
    return y


def prefill_layer(qkv, conv_w, a_raw, b_raw, A_log, dt_bias, gate, norm_w, heads, S0=None,
                  cu_seqlens=None, conv_state_in=None, conv_state_out=None, eps=1e-5, act="silu",
                  y=None, S_final=None, return_final=True, stream=None):
    """The mixer core over whole sequences in one call (``gdn_prefill_layer``):
    what :func:`prepare`, :func:`prefill` and :func:`output_norm_gate` compute,
    as the pre-recurrence pass and then the tensor-core prefill with the gated
    RMSNorm applied inside it (for sequences in the segmented form, the
    pre-recurrence steps inside the prefill's tile loads too); bf16, dk = dv =
    256.  qkv [B, T, C] or [T, C]
    (packed with ``cu_seqlens``); a_raw, b_raw [.., H]; gate [.., H, dv];
    S0 / S_final [N, H, dv, dk]; conv states [N, 3, C].  Returns (y, S_final)."""
    lib = load()
    dev, io = qkv.device, qkv.dtype
    if io != torch.bfloat16:
        raise TypeError("prefill_layer takes bf16 projections")
    H, dk, dv = heads, 256, 256
    C = H * (2 * dk + dv)
    _check(qkv, "qkv", io, dev)
    if qkv.shape[-1] != C or qkv.dim() not in (2, 3):
        raise ValueError(f"qkv must be [B, T, {C}] or [T, {C}]")
    lead = tuple(qkv.shape[:-1])
    for name, t in (("a_raw", a_raw), ("b_raw", b_raw)):
        _check(t, name, torch.float32, dev)
        if tuple(t.shape) != lead + (H,):
            raise ValueError(f"{name} must be {list(lead + (H,))}")
    for name, t, shape in (("conv_w", conv_w, (C, 4)), ("A_log", A_log, (H,)),
                           ("dt_bias", dt_bias, (H,)), ("norm_w", norm_w, (dv,))):
        _check(t, name, torch.float32, dev)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {list(shape)}")
    _check(gate, "gate", io, dev)
    if tuple(gate.shape) != lead + (H, dv):
        raise ValueError(f"gate must be {list(lead + (H, dv))}")
    if cu_seqlens is None:
        B, T = (qkv.shape[0], qkv.shape[1]) if qkv.dim() == 3 else (1, qkv.shape[0])
        N, seqlen = B, T
    else:
        _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if qkv.dim() == 3 and qkv.shape[0] != 1:
            raise ValueError("varlen input must have batch axis 1")
        N, seqlen = cu_seqlens.numel() - 1, qkv.shape[-2]
    for name, t in (("conv_state_in", conv_state_in), ("conv_state_out", conv_state_out)):
        if t is not None:
            _check(t, name, io, dev)
            if tuple(t.shape) != (N, 3, C):
                raise ValueError(f"{name} must be [{N}, 3, {C}]")
    if S0 is not None:
        _check(S0, "S0", torch.float32, dev)
        if tuple(S0.shape) != (N, H, dv, dk):
            raise ValueError(f"S0 must be [{N}, {H}, {dv}, {dk}]")
    if y is None:
        y = torch.empty_like(gate)
    else:
        _check(y, "y", io, dev)
    if S_final is None and return_final:
        S_final = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    elif S_final is not None:
        _check(S_final, "S_final", torch.float32, dev)
    with torch.cuda.device(dev):
        rc = lib.gdn_prefill_layer(
            _ptr(qkv), _ptr(conv_w), _ptr(a_raw), _ptr(b_raw), _ptr(A_log), _ptr(dt_bias),
            _ptr(conv_state_in), _ptr(conv_state_out), _ptr(S0), _ptr(cu_seqlens), _ptr(gate),
            _ptr(norm_w), float(eps), GATE_ACT[act], _ptr(y), _ptr(S_final), N, seqlen, H, dk,
            dv, GDN_BF16, _stream_handle(stream))
    if rc != 0:
        raise GDNError("gdn_prefill_layer", rc)
    return y, S_final


# ---------------------------------------------------------------------------
# The layer around the mixer: residual norm, 8-bit projections, feed-forward.
# A decoding step makes these calls for single tokens, where the host's time
# counts.  The ordinary call (new outputs, the current device and stream) goes
# through _layer_calls (csrc/binding.cpp), which returns None, having done
# nothing, where anything is out of the ordinary; the code here then checks,
# allocates and calls the library itself, and raises what is to be raised.
FP8 = torch.float8_e4m3fn
FP8_BLOCK = 128
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _blocks(n):
    return -(-n // FP8_BLOCK)


def _need(t, name, dtype, index):
    """t must be a contiguous tensor of this type on this device."""
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.get_device() == index
            and t.is_contiguous()):
        return
    _check(t, name, dtype, torch.device("cuda", index) if index >= 0 else torch.device("cpu"))


def _out(t, name, shape, dtype, index):
    """The caller's output tensor, checked."""
    _need(t, name, dtype, index)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return t


def _call(name, index, stream, *args):
    """lib.name(*args, stream) with device `index` current."""
    fn = getattr(load(), name)
    if index < 0:
        raise ValueError(f"{name} takes CUDA tensors")
    if index == torch.cuda.current_device():
        if stream is not None:
            handle = stream.cuda_stream
        elif _raw_stream is not None:
            handle = _raw_stream(index)
        else:
            handle = torch.cuda.current_stream().cuda_stream
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _stream_handle(stream))
    if rc != 0:
        raise GDNError(name, rc)


def _i32(**sizes):
    """Refuses what ctypes would cut to 32 bits in silence."""
    for name, n in sizes.items():
        if not -2 ** 31 <= n < 2 ** 31:
            raise ValueError(f"{name} {n} is out of range")


def _ws(workspace, index):
    """(address, bytes) of a caller workspace as integers."""
    p, n = _ws_args(workspace, index)
    return p.value, n


def _norm_inputs(x, w, residual, s):
    """(device index, dim, address of residual or None, the sum's tensor)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    index, io, shape = x.get_device(), x.dtype, x.shape
    if not shape:
        raise ValueError("x must be [.., dim]")
    _need(x, "x", io, index)
    _need(w, "w", torch.float32, index)
    if w.dim() != 1 or w.shape[0] != shape[-1]:
        raise ValueError(f"w must be [{shape[-1]}]")
    if residual is None:
        if s is not None:
            raise ValueError("s goes with a residual (without one the sum is x)")
        return index, shape, None, None
    _need(residual, "residual", io, index)
    if residual.shape != shape:
        raise ValueError("residual must be shaped like x")
    return index, shape, residual.data_ptr(), (torch.empty_like(x) if s is None else
                                               _out(s, "s", shape, io, index))


def residual_norm(x, w, residual=None, eps=1e-5, s=None, y=None, stream=None):
    """Residual addition and root-mean-square norm (``gdn_residual_norm``):
    s = x + residual (rounded to their dtype), y = s / sqrt(mean(s^2) + eps) * w
    over the last axis.  x, residual [.., dim] bf16 or fp32; w [dim] fp32.
    Returns (y, s); s is x itself without a residual.  ``s=residual`` updates
    the residual stream in place."""
    if s is None and y is None and stream is None:
        done = _direct_calls().residual_norm(x, w, residual, eps)
        if done is not None:
            return done
    code = _io_code(x.dtype)
    index, shape, r, total = _norm_inputs(x, w, residual, s)
    y = torch.empty_like(x) if y is None else _out(y, "y", shape, x.dtype, index)
    dim = shape[-1]
    _call("gdn_residual_norm", index, stream, x.data_ptr(), r, w.data_ptr(), eps,
          None if total is None else total.data_ptr(), y.data_ptr(), x.numel() // max(dim, 1), dim,
          code)
    return y, x if total is None else total


def residual_norm_fp8(x, w, residual=None, eps=1e-5, s=None, q=None, scale=None, stream=None):
    """:func:`residual_norm` with y in 8 bits (``gdn_residual_norm_fp8``).
    Returns (q, scale, s): q [.., dim] float8_e4m3fn and scale
    [.., ceil(dim / 128)] fp32, y ~ q * scale per 128 columns, as
    :func:`linear_fp8` reads them."""
    if s is None and q is None and scale is None and stream is None:
        done = _direct_calls().residual_norm_fp8(x, w, residual, eps)
        if done is not None:
            return done
    code = _io_code(x.dtype)
    index, shape, r, total = _norm_inputs(x, w, residual, s)
    dim = shape[-1]
    q = torch.empty_like(x, dtype=FP8) if q is None else _out(q, "q", shape, FP8, index)
    sc_shape = (*shape[:-1], -(-dim // FP8_BLOCK))
    scale = (torch.empty(sc_shape, dtype=torch.float32, device=x.device) if scale is None else
             _out(scale, "scale", sc_shape, torch.float32, index))
    _call("gdn_residual_norm_fp8", index, stream, x.data_ptr(), r, w.data_ptr(), eps,
          None if total is None else total.data_ptr(), q.data_ptr(), scale.data_ptr(),
          x.numel() // max(dim, 1), dim, code)
    return q, scale, x if total is None else total


def residual_norm_backward_workspace_size(tokens, dim, io_dtype=torch.bfloat16) -> int:
    n = load().gdn_residual_norm_backward_workspace_size(tokens, dim, _io_code(io_dtype))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported residual_norm_backward arguments")
    return int(n)


def residual_norm_backward(dy, s, w, ds=None, eps=1e-5, stream=None, workspace=None):
    """Gradients of :func:`residual_norm` (``gdn_residual_norm_backward``): dy
    [.., dim] of y, ds of s from its other uses (or None), s as the forward
    call returned it.  Returns dict dx (the gradient of x and of residual
    alike, dtype of s) and dw [dim] fp32."""
    if stream is None and workspace is None:
        done = _direct_calls().residual_norm_backward(dy, s, w, ds, eps)
        if done is not None:
            return dict(dx=done[0], dw=done[1])
    code = _io_code(s.dtype)
    index, shape, _, _ = _norm_inputs(s, w, None, None)
    _need(dy, "dy", s.dtype, index)
    if dy.shape != shape:
        raise ValueError("dy must be shaped like s")
    if ds is not None:
        _need(ds, "ds", s.dtype, index)
        if ds.shape != shape:
            raise ValueError("ds must be shaped like s")
    g = dict(dx=torch.empty_like(s), dw=torch.empty_like(w))
    dim = shape[-1]
    args = (dy.data_ptr(), s.data_ptr(), w.data_ptr(), None if ds is None else ds.data_ptr(), eps,
            g["dx"].data_ptr(), g["dw"].data_ptr(), s.numel() // max(dim, 1), dim, code)
    if workspace is None:
        _call("gdn_residual_norm_backward", index, stream, *args)
    else:
        _call("gdn_residual_norm_backward_ws", index, stream, *args, *_ws(workspace, index))
    return g


def quantize_fp8(x, block_rows=1, q=None, scale=None, stream=None):
    """x [.., cols] (bf16 or fp32) as e4m3 values with block scales
    (``gdn_quantize_fp8``): 1 x 128 blocks for activations, with
    ``block_rows=128`` 128 x 128 blocks for a weight [n, k].  Returns
    (q, scale)."""
    if q is None and scale is None and stream is None:
        done = _direct_calls().quantize_fp8(x, block_rows)
        if done is not None:
            return done
    code = _io_code(x.dtype)
    index, shape = x.get_device(), x.shape
    _need(x, "x", x.dtype, index)
    if not shape or (block_rows != 1 and len(shape) != 2):
        raise ValueError("x must be [.., cols] (a weight [n, k] with block_rows=128)")
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    cols = shape[-1]
    rows = x.numel() // max(cols, 1)
    sc_shape = (*(shape[:-1] if block_rows == 1 else (_blocks(rows),)), _blocks(cols))
    q = torch.empty_like(x, dtype=FP8) if q is None else _out(q, "q", shape, FP8, index)
    scale = (torch.empty(sc_shape, dtype=torch.float32, device=x.device) if scale is None else
             _out(scale, "scale", sc_shape, torch.float32, index))
    _call("gdn_quantize_fp8", index, stream, x.data_ptr(), q.data_ptr(), scale.data_ptr(), rows,
          cols, block_rows, code)
    return q, scale


def linear_fp8(x, x_scale, w, w_scale, out_dtype=torch.bfloat16, out=None, stream=None):
    """out = x w^T of 8-bit operands with block scales (``gdn_linear_fp8``):
    x [.., k] float8_e4m3fn with x_scale [.., ceil(k / 128)], w [n, k] with
    w_scale [ceil(n / 128), ceil(k / 128)] (as :func:`residual_norm_fp8` and
    :func:`quantize_fp8` give them).  Returns out [.., n] in ``out_dtype``
    (bf16 or fp32)."""
    code = _io_code(out_dtype)
    if out is None and stream is None:
        done = _direct_calls().linear_fp8(x, x_scale, w, w_scale, code)
        if done is not None:
            return done
    index = x.get_device()
    _need(x, "x", FP8, index)
    _need(w, "w", FP8, index)
    _need(x_scale, "x_scale", torch.float32, index)
    _need(w_scale, "w_scale", torch.float32, index)
    shape = x.shape
    if not shape or w.dim() != 2 or w.shape[1] != shape[-1]:
        raise ValueError("x must be [.., k] and w [n, k]")
    n, k = w.shape
    blocks, lead = -(-k // FP8_BLOCK), shape[:-1]
    if x_scale.shape != (*lead, blocks):
        raise ValueError(f"x_scale must be {[*lead, blocks]}")
    if w_scale.shape != (-(-n // FP8_BLOCK), blocks):
        raise ValueError(f"w_scale must be [{_blocks(n)}, {blocks}]")
    if out is None:
        out = torch.empty((*lead, n), dtype=out_dtype, device=x.device)
    else:
        _out(out, "out", (*lead, n), out_dtype, index)
    _call("gdn_linear_fp8", index, stream, x.data_ptr(), x_scale.data_ptr(), w.data_ptr(),
          w_scale.data_ptr(), out.data_ptr(), x.numel() // max(k, 1), k, n, code)
    return out


def _ffn_inputs(x, w_gate, w_up, act):
    """(device index, shape of x, hidden)."""
    io = torch.bfloat16
    if x.dtype != io:
        raise TypeError("the gated feed-forward takes bf16 tensors")
    if act not in GATE_ACT:
        raise ValueError(f"act must be one of {sorted(GATE_ACT)}")
    index, shape, w_shape = x.get_device(), x.shape, w_gate.shape
    _need(x, "x", io, index)
    _need(w_gate, "w_gate", io, index)
    _need(w_up, "w_up", io, index)
    if not shape or len(w_shape) != 2 or w_shape[1] != shape[-1] or w_up.shape != w_shape:
        raise ValueError("x must be [.., dim], w_gate and w_up [hidden, dim]")
    return index, shape, w_shape[0]


def gated_ffn(x, w_gate, w_up, act="silu", h=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T) in one kernel (``gdn_gated_ffn``):
    x [.., dim], w_gate and w_up [hidden, dim], all bf16.  Returns h
    [.., hidden]."""
    if h is None and stream is None:
        done = _direct_calls().gated_ffn(x, w_gate, w_up, GATE_ACT.get(act))
        if done is not None:
            return done
    index, shape, hidden = _ffn_inputs(x, w_gate, w_up, act)
    dim, h_shape = shape[-1], (*shape[:-1], hidden)
    if h is None:
        h = torch.empty(h_shape, dtype=torch.bfloat16, device=x.device)
    else:
        _out(h, "h", h_shape, torch.bfloat16, index)
    _call("gdn_gated_ffn", index, stream, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
          GATE_ACT[act], h.data_ptr(), x.numel() // max(dim, 1), dim, hidden, GDN_BF16)
    return h


def gated_ffn_backward_workspace_size(tokens, dim, hidden, io_dtype=torch.bfloat16) -> int:
    n = load().gdn_gated_ffn_backward_workspace_size(tokens, dim, hidden, _io_code(io_dtype))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported gated_ffn_backward arguments")
    return int(n)


def gated_ffn_backward(x, w_gate, w_up, dh, act="silu", stream=None, workspace=None):
    """Gradients of :func:`gated_ffn` from its inputs and dh [.., hidden]
    (``gdn_gated_ffn_backward``).  Returns dict dx, dw_gate, dw_up (bf16)."""
    if stream is None and workspace is None:
        done = _direct_calls().gated_ffn_backward(x, w_gate, w_up, dh, GATE_ACT.get(act))
        if done is not None:
            return dict(dx=done[0], dw_gate=done[1], dw_up=done[2])
    index, shape, hidden = _ffn_inputs(x, w_gate, w_up, act)
    _need(dh, "dh", torch.bfloat16, index)
    if dh.shape != (*shape[:-1], hidden):
        raise ValueError(f"dh must be {[*shape[:-1], hidden]}")
    g = dict(dx=torch.empty_like(x), dw_gate=torch.empty_like(w_gate),
             dw_up=torch.empty_like(w_up))
    dim = shape[-1]
    args = (x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), dh.data_ptr(), GATE_ACT[act],
            g["dx"].data_ptr(), g["dw_gate"].data_ptr(), g["dw_up"].data_ptr(),
            x.numel() // max(dim, 1), dim, hidden, GDN_BF16)
    if workspace is None:
        _call("gdn_gated_ffn_backward", index, stream, *args)
    else:
        _call("gdn_gated_ffn_backward_ws", index, stream, *args, *_ws(workspace, index))
    return g


# ---------------------------------------------------------------------------
# (Calls go through _layer_calls first, as above.)
# The attention layers that a hybrid keeps among its Gated DeltaNet layers, and
# the paged cache that they share.
def _token_rows(t, name, index):
    """(heads, d, elements from one token to the next) of bf16 t [.., T, heads, d],
    whose tokens may be rows of a wider tensor (a slice of a packed projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bf16")
    if t.get_device() != index:
        raise ValueError(f"{name} is on another device")
    if t.dim() not in (3, 4):
        raise ValueError(f"{name} must be [B, T, heads, d] or [T, heads, d]")
    heads, d = t.shape[-2:]
    step = heads * d
    if t.numel() == 0:
        return heads, d, step
    batch, tokens = (t.shape[0] if t.dim() == 4 else 1), t.shape[-3]
    if tokens > 1:
        step = t.stride(-3)
    elif batch > 1:
        step = t.stride(0)
    if ((d > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != d) or step < heads * d
            or (batch > 1 and tokens > 1 and t.stride(0) != tokens * step)):
        raise ValueError(f"{name}'s heads must be contiguous and its tokens evenly spaced")
    return heads, d, step


def _attention_inputs(q, k, v, cu_seqlens, cu_seqlens_k, scale):
    """(device index, the C ABI's sizes and strides, cu pointers, scale)."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    index = q.get_device()
    H, d, qs = _token_rows(q, "q", index)
    kv, dk, ks = _token_rows(k, "k", index)
    kv2, dv, vs = _token_rows(v, "v", index)
    if dk != d or dv != d or kv2 != kv or k.shape != v.shape or q.dim() != k.dim():
        raise ValueError("q [.., T, q_heads, d], k and v [.., T_k, kv_heads, d]")
    if cu_seqlens is None and cu_seqlens_k is None:
        N = q.shape[0] if q.dim() == 4 else 1
        if q.dim() == 4 and k.shape[0] != N:
            raise ValueError("q and k have different batch sizes")
        cu_q = cu_k = None
    else:
        if cu_seqlens is None:
            raise ValueError("cu_seqlens_k goes with cu_seqlens")
        if cu_seqlens_k is None:
            if q.shape[:-2] != k.shape[:-2]:
                raise ValueError("cu_seqlens_k is needed where k has other tokens than q")
            cu_seqlens_k = cu_seqlens
        for name, t in (("cu_seqlens", cu_seqlens), ("cu_seqlens_k", cu_seqlens_k)):
            _need(t, name, torch.int32, index)
            if t.dim() != 1 or t.shape[0] < 2 or t.shape != cu_seqlens.shape:
                raise ValueError("cu_seqlens and cu_seqlens_k must be [N + 1]")
        if q.dim() == 4 and (q.shape[0] != 1 or k.shape[0] != 1):
            raise ValueError("varlen input must have batch axis 1")
        N, cu_q, cu_k = cu_seqlens.shape[0] - 1, cu_seqlens.data_ptr(), cu_seqlens_k.data_ptr()
    scale = d ** -0.5 if scale is None else float(scale)
    return index, (N, q.shape[-3], k.shape[-3], H, kv, d, qs, ks, vs), (cu_q, cu_k), scale


def attention_prefill(q, k, v, cu_seqlens=None, cu_seqlens_k=None, scale=None, out=None, lse=None,
                      stream=None):
    """Causal attention with grouped heads over whole sequences
    (``gdn_attention_prefill``): q [B, T, q_heads, d] or packed [T, q_heads, d],
    k and v [.., T_k, kv_heads, d], bf16; d 64 or 128.  ``cu_seqlens`` [N + 1]
    packs the queries, ``cu_seqlens_k`` the keys (the same when None).  A
    sequence's mask ends at both last tokens, so longer keys are a stored
    context.  q, k and v may be slices of a packed projection (heads
    contiguous, tokens evenly spaced).  Returns (out like q, contiguous; lse
    [.., T, q_heads] fp32); a row that sees no key has out 0 and lse -inf."""
    if out is None and lse is None and stream is None:
        done = _direct_calls().attention_prefill(q, k, v, cu_seqlens, cu_seqlens_k, scale)
        if done is not None:
            return done
    index, sizes, cu, scale = _attention_inputs(q, k, v, cu_seqlens, cu_seqlens_k, scale)
    out = (torch.empty(q.shape, dtype=q.dtype, device=q.device) if out is None else
           _out(out, "out", q.shape, q.dtype, index))
    lse = (torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if lse is None else
           _out(lse, "lse", q.shape[:-1], torch.float32, index))
    _call("gdn_attention_prefill", index, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), *cu,
          scale, out.data_ptr(), lse.data_ptr(), *sizes)
    return out, lse


def attention_prefill_backward_workspace_size(batch, seqlen, q_heads, kv_heads, d, varlen=False,
                                              seqlen_k=None) -> int:
    """Bytes of ``attention_prefill_backward``'s workspace on the current device for batch
    sequences of seqlen queries (varlen: seqlen in all) and seqlen_k keys (as many when
    None).  It serves calls with fewer of each, too."""
    _i32(batch=batch, q_heads=q_heads, kv_heads=kv_heads, d=d)
    n = load().gdn_attention_prefill_backward_workspace_size(
        batch, seqlen, seqlen if seqlen_k is None else seqlen_k, int(bool(varlen)), q_heads,
        kv_heads, d)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported attention_prefill_backward arguments")
    return int(n)


def attention_prefill_backward(q, k, v, out, lse, dout, cu_seqlens=None, cu_seqlens_k=None,
                               scale=None, stream=None, workspace=None):
    """Gradients of :func:`attention_prefill` from its inputs, its results and
    dout (``gdn_attention_prefill_backward``).  Returns dict dq, dk, dv (bf16,
    contiguous)."""
    if stream is None and workspace is None:
        done = _direct_calls().attention_prefill_backward(q, k, v, cu_seqlens, cu_seqlens_k, scale,
                                                          out, lse, dout)
        if done is not None:
            return dict(dq=done[0], dk=done[1], dv=done[2])
    index, sizes, cu, scale = _attention_inputs(q, k, v, cu_seqlens, cu_seqlens_k, scale)
    for name, t in (("out", out), ("dout", dout)):
        _out(t, name, q.shape, torch.bfloat16, index)
    _out(lse, "lse", q.shape[:-1], torch.float32, index)
    g = {n: torch.empty(t.shape, dtype=t.dtype, device=t.device)
         for n, t in (("dq", q), ("dk", k), ("dv", v))}
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
            dout.data_ptr(), *cu, scale, g["dq"].data_ptr(), g["dk"].data_ptr(),
            g["dv"].data_ptr(), *sizes)
    if workspace is None:
        _call("gdn_attention_prefill_backward", index, stream, *args)
    else:
        _call("gdn_attention_prefill_backward_ws", index, stream, *args, *_ws(workspace, index))
    return g


class _CacheStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "table", "lengths",
                                               "refs")] + \
               [(n, ctypes.c_int32) for n in ("layers", "pages", "kv_heads", "page", "d", "rows",
                                              "max_pages", "dtype")]


class KVCache:
    """A paged cache of keys and values (``gdn_kv_cache``) over the caller's
    tensors: k and v [layers, pages, kv_heads, page, d] bf16, or float8_e4m3fn
    with k_scale and v_scale [layers, pages, kv_heads, page] fp32; table
    [rows, max_pages], lengths [rows] and refs [pages] int32.  The tensors are
    its attributes and do not change; their contents are the cache.  (A new,
    empty one: :func:`kv_cache`.)"""

    __slots__ = ("k", "v", "k_scale", "v_scale", "table", "lengths", "refs", "index", "struct",
                 "address")

    def __init__(self, k, v, table, lengths, refs, k_scale=None, v_scale=None):
        if not isinstance(k, torch.Tensor) or k.dim() != 5:
            raise ValueError("k must be [layers, pages, kv_heads, page, d]")
        if k.dtype not in (torch.bfloat16, FP8):
            raise TypeError("a cache holds bf16 or float8_e4m3fn")
        layers, pages, kv_heads, page, d = k.shape
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table must be [rows, max_pages]")
        rows, max_pages = table.shape
        index, eight = k.get_device(), k.dtype == FP8
        if (k_scale is not None) != eight or (v_scale is not None) != eight:
            raise ValueError("k_scale and v_scale go with an 8-bit cache")
        _i32(layers=layers, pages=pages, kv_heads=kv_heads, page=page, d=d, rows=rows,
             max_pages=max_pages)
        shapes = dict(k=k.shape, v=k.shape, table=(rows, max_pages), lengths=(rows,),
                      refs=(pages,), k_scale=k.shape[:-1], v_scale=k.shape[:-1])
        given = dict(k=k, v=v, table=table, lengths=lengths, refs=refs, k_scale=k_scale,
                     v_scale=v_scale)
        c = _CacheStruct(layers=layers, pages=pages, kv_heads=kv_heads, page=page, d=d, rows=rows,
                         max_pages=max_pages, dtype=GDN_E4M3 if eight else GDN_BF16)
        for name, t in given.items():
            if t is not None:
                io = (k.dtype if name in ("k", "v") else
                      torch.float32 if name.endswith("scale") else torch.int32)
                _out(t, name, shapes[name], io, index)
                setattr(c, name, t.data_ptr())
            object.__setattr__(self, name, t)
        object.__setattr__(self, "index", index)
        object.__setattr__(self, "struct", c)
        object.__setattr__(self, "address", ctypes.addressof(c))

    def __setattr__(self, name, value):
        raise AttributeError("a KVCache's tensors are fixed")


def kv_cache(layers, pages, kv_heads, rows, max_pages, page=64, d=128, dtype=torch.bfloat16,
             device="cuda") -> KVCache:
    """A new, empty paged cache for ``rows`` sequences of up to ``max_pages``
    pages of ``page`` tokens each, out of a pool of ``pages``, shared by
    ``layers`` layers; dtype bf16 or float8_e4m3fn."""
    new = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device=device)  # noqa: E731
    if dtype not in (torch.bfloat16, FP8):
        raise TypeError("a cache holds bf16 or float8_e4m3fn")
    shape = (layers, pages, kv_heads, page, d)
    pool = lambda: (new(*shape, t=torch.uint8).view(FP8) if dtype == FP8 else  # noqa: E731
                    new(*shape, t=dtype))
    scale = lambda: new(*shape[:-1], t=torch.float32) if dtype == FP8 else None  # noqa: E731
    return KVCache(pool(), pool(), new(rows, max_pages).fill_(-1), new(rows), new(pages), scale(),
                   scale())


def _cache(cache):
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    return cache.index, cache.address


def _row_numbers(t, name, index):
    _need(t, name, torch.int32, index)
    if t.dim() != 1:
        raise ValueError(f"{name} must be a vector of row numbers")
    return t.shape[0]


def cache_reserve(cache, counts, start=None, stream=None):
    """Places for counts [rows] new tokens of every row (``gdn_cache_reserve``):
    takes pages, advances the lengths, and returns start [rows] int32, each
    row's first new position (-1 where the pool or the row's table had no
    room; :func:`device_status` then says so)."""
    index, at = _cache(cache)
    if start is None and stream is None:
        done = _direct_calls().cache_reserve(at, index, counts)
        if done is not None:
            return done
    _out(counts, "counts", cache.lengths.shape, torch.int32, index)
    start = (torch.empty_like(counts) if start is None else
             _out(start, "start", counts.shape, torch.int32, index))
    _call("gdn_cache_reserve", index, stream, at, counts.data_ptr(), start.data_ptr())
    return start


def cache_append(cache, k, v, start, cu_seqlens=None, layer=0, stream=None):
    """Writes one layer's new keys and values [tokens, kv_heads, d] (bf16; rows
    of a wider tensor allowed) to the places that :func:`cache_reserve` gave
    (``gdn_cache_append``): one token a row, or row r's tokens
    cu_seqlens[r] .. cu_seqlens[r + 1]."""
    index, at = _cache(cache)
    if stream is None and _direct_calls().cache_append(at, index, k, v, start, cu_seqlens, layer):
        return
    heads, d, ks = _token_rows(k, "k", index)
    _, _, vs = _token_rows(v, "v", index)
    if k.dim() != 3 or k.shape != v.shape or (heads, d) != (cache.k.shape[2], cache.k.shape[4]):
        raise ValueError(f"k and v must be [tokens, {cache.k.shape[2]}, {cache.k.shape[4]}]")
    rows = cache.lengths.shape[0]
    _out(start, "start", (rows,), torch.int32, index)
    if cu_seqlens is not None:
        _out(cu_seqlens, "cu_seqlens", (rows + 1,), torch.int32, index)
    elif k.shape[0] != rows:
        raise ValueError(f"k and v must have a token for each of the {rows} rows (or cu_seqlens)")
    _i32(layer=layer)
    _call("gdn_cache_append", index, stream, at, layer, k.data_ptr(), v.data_ptr(),
          start.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(), k.shape[0], ks, vs)


def cache_gather(cache, cu_seqlens, tokens, layer=0, stream=None):
    """One layer's stored keys and values as :func:`attention_prefill` reads them
    (``gdn_cache_gather``): row r's first cu_seqlens[r+1] - cu_seqlens[r]
    tokens, packed; tokens = cu_seqlens[-1], which stays on the device.
    Returns (k, v) [tokens, kv_heads, d] bf16; zeros for tokens that the row
    does not hold (its reservation failed; :func:`device_status` then says so)."""
    index, at = _cache(cache)
    if stream is None:
        done = _direct_calls().cache_gather(at, index, cu_seqlens, tokens, layer)
        if done is not None:
            return done
    _out(cu_seqlens, "cu_seqlens", (cache.lengths.shape[0] + 1,), torch.int32, index)
    k, v = (torch.empty((tokens, cache.k.shape[2], cache.k.shape[4]), dtype=torch.bfloat16,
                        device=cache.k.device) for _ in range(2))
    _i32(layer=layer)
    _call("gdn_cache_gather", index, stream, at, layer, cu_seqlens.data_ptr(), tokens, k.data_ptr(),
          v.data_ptr())
    return k, v


def cache_free(cache, rows, stream=None):
    """Empties the named rows (int32) and gives their pages back
    (``gdn_cache_free``)."""
    index, at = _cache(cache)
    if stream is None and _direct_calls().cache_free(at, index, rows):
        return
    n = _row_numbers(rows, "rows", index)
    _call("gdn_cache_free", index, stream, at, rows.data_ptr(), n)


def cache_fork(cache, src, dst, stream=None):
    """The empty rows dst [n] (int32) become copies of rows src [n]
    (``gdn_cache_fork``): full pages are shared, a last page that is not full is
    copied, in all layers."""
    index, at = _cache(cache)
    if stream is None and _direct_calls().cache_fork(at, index, src, dst):
        return
    n = _row_numbers(src, "src", index)
    if _row_numbers(dst, "dst", index) != n:
        raise ValueError("src and dst must name as many rows")
    _call("gdn_cache_fork", index, stream, at, src.data_ptr(), dst.data_ptr(), n)


def cache_compact(cache, into, stream=None):
    """Moves a cache's rows to ``into``, their pages in order at the front of its
    pool (``gdn_cache_compact``), which may be larger or smaller; ``cache``
    stays as it is.  Returns ``into``."""
    index, at = _cache(cache)
    other, to = _cache(into)
    if stream is None and _direct_calls().cache_compact(at, index, to, other):
        return into
    if other != index:
        raise ValueError("the two caches are on different devices")
    _call("gdn_cache_compact", index, stream, at, to)
    return into


def attention_decode_step_workspace_size(rows, q_heads, kv_heads, d) -> int:
    _i32(rows=rows, q_heads=q_heads, kv_heads=kv_heads, d=d)
    n = load().gdn_attention_decode_step_workspace_size(rows, q_heads, kv_heads, d)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported attention_decode_step arguments")
    return int(n)


def attention_decode_step(q, cache, layer=0, scale=None, out=None, stream=None, workspace=None):
    """Attention of one new token of every row over the row's cached keys and
    values of one layer (``gdn_attention_decode_step``): q [rows, q_heads, d]
    bf16.  Returns out like q; 0 for an empty row."""
    index, at = _cache(cache)
    if out is None and stream is None and workspace is None:
        done = _direct_calls().attention_decode_step(at, index, q, layer, scale)
        if done is not None:
            return done
    _need(q, "q", torch.bfloat16, index)
    rows, d = cache.lengths.shape[0], cache.k.shape[4]
    if q.dim() != 3 or q.shape[0] != rows or q.shape[2] != d:
        raise ValueError(f"q must be [{rows}, q_heads, {d}]")
    _i32(layer=layer)
    out = torch.empty_like(q) if out is None else _out(out, "out", q.shape, q.dtype, index)
    args = (q.data_ptr(), at, layer, q.shape[1], d ** -0.5 if scale is None else float(scale),
            out.data_ptr())
    if workspace is None:
        _call("gdn_attention_decode_step", index, stream, *args)
    else:
        _call("gdn_attention_decode_step_ws", index, stream, *args, *_ws(workspace, index))
    return out


def device_status(stream=None) -> int:
    """Synchronise the stream; return and clear the device status word."""
    return int(load().gdn_get_device_status(_stream_handle(stream)))
