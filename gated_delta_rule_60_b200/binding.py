"""Thin ctypes binding of libkda (include/kda.h).

Argument marshalling only: every function here checks tensor placement,
dtype, shape and contiguity, passes raw device pointers and the current CUDA
stream to the C ABI, and turns a non-OK status into an exception.  All of the
operator's arithmetic runs in libkda's CUDA kernels; there is no fallback of
any kind, and importing a function from here on a machine without the built
library raises immediately.

The Python names are the C names.  As in the C ABI, the tensors of a call
must live on the current CUDA device (select it with torch.cuda.set_device or
a torch.cuda.device context); stream=None means that device's current stream.
"""
import ctypes
import functools
import os
from typing import Optional, Tuple, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")

KDA_OK = 0
KDA_ERR_INVALID_ARGUMENT = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_WORKSPACE = 3
KDA_ERR_CUDA = 4
KDA_ERR_TIMEOUT = 5
KDA_ERR_BAD_SEQLENS = 6

KDA_BF16 = 0
KDA_FP32 = 1

_DTYPES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_FP32}

_lib = None


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, kda_status_string(status),
                                                 status))


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libkda.so (built in-tree by gated_delta_rule_60_b200/build.py)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            "libkda.so is not built at %s; run `python -m "
            "gated_delta_rule_60_b200.build` (nvcc, sm_100a)" % path)
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.kda_chunk_fwd_workspace_size.restype = sz
    lib.kda_chunk_fwd_workspace_size.argtypes = [i32, i64, i32, i32, i32, ctypes.c_int]
    lib.kda_chunk_fwd.restype = ctypes.c_int
    lib.kda_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32,
                                  i32, ctypes.c_int, vp, vp, vp, sz, vp]
    lib.kda_chunk_fwd_gated.restype = ctypes.c_int
    lib.kda_chunk_fwd_gated.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32,
                                        i32, ctypes.c_int, vp, vp, vp, vp, sz, vp]
    lib.kda_chunk_fwd_noalloc.restype = ctypes.c_int
    lib.kda_chunk_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32,
                                          i32, ctypes.c_int, vp, vp, vp]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32,
                                    i32, ctypes.c_int, vp]
    lib.kda_stream_status.restype = ctypes.c_int
    lib.kda_stream_status.argtypes = [vp]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_version.restype = i32
    lib.kda_version.argtypes = []
    lib.kda_selftest_wait_timeout.restype = ctypes.c_int
    lib.kda_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
    lib.kda_chunk_bwd_workspace_size.restype = sz
    lib.kda_chunk_bwd_workspace_size.argtypes = [i32, i64, i32, i32, i32, ctypes.c_int]
    lib.kda_chunk_bwd.restype = ctypes.c_int
    lib.kda_chunk_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32,
                                  ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.kda_chunk_fwd_softplus.restype = ctypes.c_int
    lib.kda_chunk_fwd_softplus.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32,
                                           i32, ctypes.c_int, vp, vp, vp]
    lib.kda_decode_step_softplus.restype = ctypes.c_int
    lib.kda_decode_step_softplus.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32,
                                             i32, ctypes.c_int, vp]
    lib.kda_prologue.restype = ctypes.c_int
    lib.kda_prologue.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32,
                                 ctypes.c_int, vp, vp, vp, vp, vp]
    lib.kda_debug_stall_prefill.restype = ctypes.c_int
    lib.kda_debug_stall_prefill.argtypes = [i32, ctypes.c_uint64]
    lib.kda_debug_range_prefill.restype = ctypes.c_int
    lib.kda_debug_range_prefill.argtypes = [i32]
    lib.kda_debug_range_read.restype = ctypes.c_int
    lib.kda_debug_range_read.argtypes = [ctypes.POINTER(ctypes.c_float), sz]
    lib.kda_linear_chunk_fwd_workspace_size.restype = sz
    lib.kda_linear_chunk_fwd_workspace_size.argtypes = [i32, i64, i32, i32, ctypes.c_int]
    lib.kda_linear_chunk_fwd.restype = ctypes.c_int
    lib.kda_linear_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32,
                                         ctypes.c_int, i32, ctypes.c_float, vp, vp, vp, sz, vp]
    lib.kda_linear_decode_step.restype = ctypes.c_int
    lib.kda_linear_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                           ctypes.c_int, i32, ctypes.c_float, vp]
    lib.kda_linear_chunk_bwd_workspace_size.restype = sz
    lib.kda_linear_chunk_bwd_workspace_size.argtypes = [i32, i64, i32, i32, i32, ctypes.c_int]
    lib.kda_linear_chunk_bwd.restype = ctypes.c_int
    lib.kda_linear_chunk_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32,
                                         ctypes.c_int, i32, ctypes.c_float, vp, vp, vp, vp, vp, vp,
                                         vp, vp, sz, vp]
    lib.kda_rotary.restype = ctypes.c_int
    lib.kda_rotary.argtypes = [vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, ctypes.c_int, i32,
                               i32, ctypes.c_float, i64, i64, vp, vp, i64, i64, vp]
    lib.kda_rotary_frequencies.restype = ctypes.c_int
    lib.kda_rotary_frequencies.argtypes = [i32, ctypes.c_double, ctypes.c_int, ctypes.c_double,
                                           ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                           ctypes.POINTER(ctypes.c_float),
                                           ctypes.POINTER(ctypes.c_float)]
    lib.kda_layernorm_fwd.restype = ctypes.c_int
    lib.kda_layernorm_fwd.argtypes = [vp, vp, vp, i64, i32, i32, ctypes.c_int, ctypes.c_float, vp,
                                      vp, vp, vp]
    lib.kda_layernorm_bwd_workspace_size.restype = sz
    lib.kda_layernorm_bwd_workspace_size.argtypes = [i64, i32, i32, ctypes.c_int]
    lib.kda_layernorm_bwd.restype = ctypes.c_int
    lib.kda_layernorm_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, ctypes.c_int, vp, vp, vp,
                                      vp, sz, vp]
    _lib = lib
    return lib


def kda_status_string(status: int) -> str:
    return load_library().kda_status_string(int(status)).decode()


def kda_version() -> int:
    return int(load_library().kda_version())


def kda_chunk_fwd_workspace_size(N: int, T_tot: int, H: int, dk: int, dv: int,
                                 dtype: torch.dtype) -> int:
    return int(load_library().kda_chunk_fwd_workspace_size(
        int(N), int(T_tot), int(H), int(dk), int(dv), _DTYPES[dtype]))


def kda_chunk_bwd_workspace_size(N: int, T_tot: int, H: int, dk: int, dv: int,
                                 dtype: torch.dtype) -> int:
    return int(load_library().kda_chunk_bwd_workspace_size(
        int(N), int(T_tot), int(H), int(dk), int(dv), _DTYPES[dtype]))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t: torch.Tensor, name: str, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError("%s must be on %s, got %s" % (name, device or "cuda", t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape),
                                                            tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def kda_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  g: torch.Tensor, beta: torch.Tensor,
                  h0: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, *,
                  num_seqs: Optional[int] = None,
                  o: Optional[torch.Tensor] = None,
                  hT: Optional[torch.Tensor] = None,
                  output_final_state: bool = True,
                  workspace: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked KDA prefill.  Returns (o [T_tot,H,dv], hT [N,H,dk,dv] or None).

    q, k, g [T_tot, H, dk]; v [T_tot, H, dv]; beta [T_tot, H] share one dtype
    (bf16 or fp32); h0 fp32 [N, H, dk, dv] or None; cu_seqlens int32 [N+1] on
    the device, or None with num_seqs equal-length sequences (default 1).
    """
    lib = load_library()
    dev = q.device
    T_tot, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DTYPES:
        raise TypeError("unsupported dtype %s" % dt)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
        N = cu_seqlens.numel() - 1
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    for t, name, shp in ((q, "q", (T_tot, H, dk)), (k, "k", (T_tot, H, dk)),
                         (g, "g", (T_tot, H, dk)), (v, "v", (T_tot, H, dv)),
                         (beta, "beta", (T_tot, H))):
        _check(t, name, dt, shp, dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty(T_tot, H, dv, dtype=dt, device=dev)
    _check(o, "o", dt, (T_tot, H, dv), dev)
    if hT is None and output_final_state:
        hT = torch.empty(N, H, dk, dv, dtype=torch.float32, device=dev)
    if hT is not None:
        _check(hT, "hT", torch.float32, (N, H, dk, dv), dev)
    ws_need = kda_chunk_fwd_workspace_size(N, T_tot, H, dk, dv, dt)
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                           _ptr(h0), _ptr(cu_seqlens), N, T_tot, H, dk, dv,
                           _DTYPES[dt], _ptr(o), _ptr(hT), _ptr(workspace),
                           ws_bytes, _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd")
    return o, hT


def kda_chunk_fwd_gated(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        g: torch.Tensor, beta: torch.Tensor, z: torch.Tensor,
                        h0: Optional[torch.Tensor] = None,
                        cu_seqlens: Optional[torch.Tensor] = None, *,
                        num_seqs: Optional[int] = None,
                        o: Optional[torch.Tensor] = None,
                        hT: Optional[torch.Tensor] = None,
                        output_final_state: bool = True,
                        workspace: Optional[torch.Tensor] = None,
                        stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """kda_chunk_fwd with the output gate fused into the output store:
    o = (S^T q) * sigmoid(z), z [T_tot, H, dv] in the inputs' dtype."""
    lib = load_library()
    dev = q.device
    T_tot, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DTYPES:
        raise TypeError("unsupported dtype %s" % dt)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
        N = cu_seqlens.numel() - 1
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    for t, name, shp in ((q, "q", (T_tot, H, dk)), (k, "k", (T_tot, H, dk)),
                         (g, "g", (T_tot, H, dk)), (v, "v", (T_tot, H, dv)),
                         (beta, "beta", (T_tot, H)), (z, "z", (T_tot, H, dv))):
        _check(t, name, dt, shp, dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty(T_tot, H, dv, dtype=dt, device=dev)
    _check(o, "o", dt, (T_tot, H, dv), dev)
    if hT is None and output_final_state:
        hT = torch.empty(N, H, dk, dv, dtype=torch.float32, device=dev)
    if hT is not None:
        _check(hT, "hT", torch.float32, (N, H, dk, dv), dev)
    ws_need = kda_chunk_fwd_workspace_size(N, T_tot, H, dk, dv, dt)
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.kda_chunk_fwd_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                 _ptr(h0), _ptr(cu_seqlens), N, T_tot, H, dk, dv,
                                 _DTYPES[dt], _ptr(z), _ptr(o), _ptr(hT), _ptr(workspace),
                                 ws_bytes, _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_gated")
    return o, hT


def kda_chunk_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          g: torch.Tensor, beta: torch.Tensor,
                          h0: Optional[torch.Tensor] = None,
                          cu_seqlens: Optional[torch.Tensor] = None, *,
                          o: torch.Tensor, hT: Optional[torch.Tensor] = None,
                          num_seqs: Optional[int] = None,
                          stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """kda_chunk_fwd for callers that cannot allocate device memory: o (and
    hT, if wanted) must be given; the long-sequence scratch comes from the
    library's static device array, so nothing here allocates."""
    lib = load_library()
    dev = q.device
    T_tot, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DTYPES:
        raise TypeError("unsupported dtype %s" % dt)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
        N = cu_seqlens.numel() - 1
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    for t, name, shp in ((q, "q", (T_tot, H, dk)), (k, "k", (T_tot, H, dk)),
                         (g, "g", (T_tot, H, dk)), (v, "v", (T_tot, H, dv)),
                         (beta, "beta", (T_tot, H)), (o, "o", (T_tot, H, dv))):
        _check(t, name, dt, shp, dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, dk, dv), dev)
    if hT is not None:
        _check(hT, "hT", torch.float32, (N, H, dk, dv), dev)
    st = lib.kda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                   _ptr(h0), _ptr(cu_seqlens), N, T_tot, H, dk, dv,
                                   _DTYPES[dt], _ptr(o), _ptr(hT), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_noalloc")
    return o, hT


def kda_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    g: torch.Tensor, beta: torch.Tensor, S: torch.Tensor, *,
                    o: Optional[torch.Tensor] = None,
                    stream=None, _softplus: bool = False) -> torch.Tensor:
    """One KDA decode step; S [B,H,dk,dv] fp32 is updated in place.
    Returns o [B, H, dv] (dtype of q)."""
    lib = load_library()
    dev = q.device
    B, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DTYPES:
        raise TypeError("unsupported dtype %s" % dt)
    for t, name, shp in ((q, "q", (B, H, dk)), (k, "k", (B, H, dk)),
                         (g, "g", (B, H, dk)), (v, "v", (B, H, dv)),
                         (beta, "beta", (B, H))):
        _check(t, name, dt, shp, dev)
    _check(S, "S", torch.float32, (B, H, dk, dv), dev)
    if o is None:
        o = torch.empty(B, H, dv, dtype=dt, device=dev)
    _check(o, "o", dt, (B, H, dv), dev)
    fn = lib.kda_decode_step_softplus if _softplus else lib.kda_decode_step
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(o), B, H, dk, dv,
            _DTYPES[dt], _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_step" + ("_softplus" if _softplus else ""))
    return o


def kda_decode_step_softplus(q, k, v, g, beta, S, *, o=None, stream=None) -> torch.Tensor:
    """kda_decode_step with the unbounded gate log a = -softplus(g)."""
    return kda_decode_step(q, k, v, g, beta, S, o=o, stream=stream, _softplus=True)


def kda_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                  beta: torch.Tensor, dO: torch.Tensor, h0: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, dhT: Optional[torch.Tensor] = None,
                  *, num_seqs: Optional[int] = None, stream=None) -> dict:
    """Gradient of the prefill for L = <dO, O> + <dhT, hT>: returns a dict of
    dq, dk, dg [T_tot, H, dk], dv [T_tot, H, dv], dbeta [T_tot, H] (dtype of
    q) and dh0 [N, H, dk, dv] fp32."""
    lib = load_library()
    dev = q.device
    T_tot, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DTYPES:
        raise TypeError("unsupported dtype %s" % dt)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
        N = cu_seqlens.numel() - 1
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    for t, name, shp in ((q, "q", (T_tot, H, dk)), (k, "k", (T_tot, H, dk)),
                         (g, "g", (T_tot, H, dk)), (v, "v", (T_tot, H, dv)),
                         (beta, "beta", (T_tot, H)), (dO, "dO", (T_tot, H, dv))):
        _check(t, name, dt, shp, dev)
    for t, name in ((h0, "h0"), (dhT, "dhT")):
        if t is not None:
            _check(t, name, torch.float32, (N, H, dk, dv), dev)
    out = {"dq": torch.empty(T_tot, H, dk, dtype=dt, device=dev),
           "dk": torch.empty(T_tot, H, dk, dtype=dt, device=dev),
           "dv": torch.empty(T_tot, H, dv, dtype=dt, device=dev),
           "dg": torch.empty(T_tot, H, dk, dtype=dt, device=dev),
           "dbeta": torch.empty(T_tot, H, dtype=dt, device=dev),
           "dh0": torch.empty(N, H, dk, dv, dtype=torch.float32, device=dev)}
    ws_n = int(lib.kda_chunk_bwd_workspace_size(N, T_tot, H, dk, dv, _DTYPES[dt]))
    ws = torch.empty(max(ws_n, 256), dtype=torch.uint8, device=dev)
    st = lib.kda_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                           _ptr(cu_seqlens), N, T_tot, H, dk, dv, _DTYPES[dt], _ptr(dO),
                           _ptr(dhT), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                           _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(ws),
                           ws.numel(), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_bwd")
    return out


def kda_chunk_fwd_softplus(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                           g: torch.Tensor, beta: torch.Tensor,
                           h0: Optional[torch.Tensor] = None,
                           cu_seqlens: Optional[torch.Tensor] = None, *,
                           num_seqs: Optional[int] = None,
                           o: Optional[torch.Tensor] = None,
                           hT: Optional[torch.Tensor] = None,
                           output_final_state: bool = True,
                           stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked prefill with the unbounded gate log a = -softplus(g) (fp32
    CUDA-core path, any supported head size, bf16 or fp32 inputs)."""
    lib = load_library()
    dev = q.device
    T_tot, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in _DTYPES:
        raise TypeError("unsupported dtype %s" % dt)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
        N = cu_seqlens.numel() - 1
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    for t, name, shp in ((q, "q", (T_tot, H, dk)), (k, "k", (T_tot, H, dk)),
                         (g, "g", (T_tot, H, dk)), (v, "v", (T_tot, H, dv)),
                         (beta, "beta", (T_tot, H))):
        _check(t, name, dt, shp, dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, dk, dv), dev)
    if o is None:
        o = torch.empty(T_tot, H, dv, dtype=dt, device=dev)
    _check(o, "o", dt, (T_tot, H, dv), dev)
    if hT is None and output_final_state:
        hT = torch.empty(N, H, dk, dv, dtype=torch.float32, device=dev)
    if hT is not None:
        _check(hT, "hT", torch.float32, (N, H, dk, dv), dev)
    st = lib.kda_chunk_fwd_softplus(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                    _ptr(h0), _ptr(cu_seqlens), N, T_tot, H, dk, dv,
                                    _DTYPES[dt], _ptr(o), _ptr(hT), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_softplus")
    return o, hT


def kda_selftest_wait_timeout(limit_cycles: int, stream=None) -> None:
    """Let one bounded wait run out on the GPU (no fault): afterwards
    kda_stream_status() reports KDA_ERR_TIMEOUT."""
    st = load_library().kda_selftest_wait_timeout(int(limit_cycles), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_selftest_wait_timeout")


def kda_prologue(xq: torch.Tensor, xk: torch.Tensor, xv: torch.Tensor,
                 wq: torch.Tensor, wk: torch.Tensor, wv: torch.Tensor,
                 beta_raw: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, *,
                 num_seqs: Optional[int] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Short-conv prologue: (q, k, v, beta) for kda_chunk_fwd from the raw
    projections xq, xk, xv [T_tot, H, d], taps w* [H, d, 4] fp32 and
    beta_raw [T_tot, H] (see include/kda.h)."""
    lib = load_library()
    dev = xq.device
    T_tot, H, d = xq.shape
    dt = xq.dtype
    if dt not in _DTYPES:
        raise TypeError("unsupported dtype %s" % dt)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
        N = cu_seqlens.numel() - 1
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    for t, name in ((xq, "xq"), (xk, "xk"), (xv, "xv")):
        _check(t, name, dt, (T_tot, H, d), dev)
    for t, name in ((wq, "wq"), (wk, "wk"), (wv, "wv")):
        _check(t, name, torch.float32, (H, d, 4), dev)
    _check(beta_raw, "beta_raw", dt, (T_tot, H), dev)
    q, k, v = (torch.empty(T_tot, H, d, dtype=dt, device=dev) for _ in range(3))
    beta = torch.empty(T_tot, H, dtype=dt, device=dev)
    st = lib.kda_prologue(_ptr(xq), _ptr(xk), _ptr(xv), _ptr(wq), _ptr(wk), _ptr(wv),
                          _ptr(beta_raw), _ptr(cu_seqlens), N, T_tot, H, d, _DTYPES[dt],
                          _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _stream_handle(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_prologue")
    return q, k, v, beta


def kda_debug_stall_prefill(step: int, limit_cycles: int) -> None:
    """Make the next tensor-core kda_chunk_fwd call stall its scan at state
    step `step` on a wait that nothing completes, bounded by limit_cycles
    (no fault: the kernel reports KDA_ERR_TIMEOUT, drains and returns)."""
    st = load_library().kda_debug_stall_prefill(int(step), int(limit_cycles))
    if st != KDA_OK:
        raise KdaError(st, "kda_debug_stall_prefill")


RANGE_ROWS = ("Kr", "Qr", "Kh", "Z")
RANGE_COLS = ("max_abs", "min_nonzero_abs", "subnormal", "zero", "nonfinite", "count")


def kda_debug_range_prefill(step: int) -> None:
    """Make CTA 0 of the next tensor-core kda_chunk_fwd call record the
    magnitudes of its scaled operands (Kr, Qr, Kh in bf16) and of Z = Kh^T T
    (fp32, before the delta rescale) at state step `step`."""
    st = load_library().kda_debug_range_prefill(int(step))
    if st != KDA_OK:
        raise KdaError(st, "kda_debug_range_prefill")


def kda_debug_range_read() -> dict:
    """The record of kda_debug_range_prefill: {row: {column: value}}."""
    buf = (ctypes.c_float * (len(RANGE_ROWS) * len(RANGE_COLS)))()
    st = load_library().kda_debug_range_read(buf, len(buf))
    if st != KDA_OK:
        raise KdaError(st, "kda_debug_range_read")
    n = len(RANGE_COLS)
    return {r: {c: float(buf[i * n + j]) for j, c in enumerate(RANGE_COLS)}
            for i, r in enumerate(RANGE_ROWS)}


# The calls below serve single tokens too, where a call's own time counts: they
# hand plain integers to ctypes and ask torch for the raw stream and device.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _index(t: torch.Tensor, name: str) -> int:
    """The device index of t, which has to be the current CUDA device (the
    launch goes there whatever the tensors say)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    idx = t.get_device()
    if idx < 0:
        raise ValueError("%s must be on cuda, got %s" % (name, t.device))
    if idx != _current_device():
        raise ValueError("%s is on %s, which is not the current device" % (name, t.device))
    return idx


def _at(t, name: str, dtype, shape, idx: int) -> int:
    """The address of a dense tensor of this type, shape and device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and \
            t.get_device() == idx and t.is_contiguous():
        return t.data_ptr()
    _check(t, name, dtype, shape, torch.device("cuda", idx))
    return t.data_ptr()


def _maybe(t, name: str, dtype, shape, idx: int):
    return None if t is None else _at(t, name, dtype, shape, idx)


def _stream_at(stream, idx: int) -> int:
    if stream is None:
        return _raw_stream(idx)
    if stream.device.index != idx:
        raise ValueError("stream is on %s, the tensors on cuda:%d" % (stream.device, idx))
    return stream.cuda_stream


def _empty(stream, idx: int, shape, dtype) -> torch.Tensor:
    """Memory for a call on `stream`: torch's memory belongs to a stream, so what a
    call on another one writes has to come from that stream's."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=idx)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=idx)


def _workspace(need: int, given: Optional[torch.Tensor], stream, idx: int):
    """(address, bytes, tensor) of a call's scratch: the caller's, or a new one."""
    if given is None:
        if not need:
            return None, 0, None
        given = _empty(stream, idx, need, torch.uint8)
        return given.data_ptr(), need, given
    if given.get_device() != idx or not given.is_contiguous():
        raise ValueError("workspace must be contiguous on cuda:%d" % idx)
    return given.data_ptr(), given.numel() * given.element_size(), given


def _seqs(cu_seqlens, num_seqs, idx: int):
    """(address of cu_seqlens or None, number of sequences)"""
    if cu_seqlens is None:
        return None, 1 if num_seqs is None else int(num_seqs)
    n = cu_seqlens.numel() if isinstance(cu_seqlens, torch.Tensor) else 0
    return _at(cu_seqlens, "cu_seqlens", torch.int32, (n,), idx), n - 1


def _linear_sizes(q, v, g):
    """(device, T, Hk, H, d, dtype, its code, address of g, g_per_token)"""
    idx = _index(q, "q")
    if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("q, k and v must have three dimensions")
    T, Hk, d = q.shape
    H = v.shape[1]
    code = _DTYPES.get(q.dtype)
    if code is None:
        raise TypeError("unsupported dtype %s" % q.dtype)
    if not isinstance(g, torch.Tensor):
        raise TypeError("g must be a torch.Tensor")
    per_token = g.dim() == 2
    return idx, T, Hk, H, d, q.dtype, code, _at(g, "g", torch.float32, (T, H) if per_token else (H,), idx), \
        int(per_token)


@functools.lru_cache(maxsize=1024)
def _size(name: str, *sizes) -> int:
    """A workspace query: a pure function of the sizes."""
    return int(getattr(load_library(), name)(*sizes))


def kda_linear_chunk_fwd_workspace_size(N: int, T_tot: int, H: int, d: int,
                                        dtype: torch.dtype) -> int:
    return int(load_library().kda_linear_chunk_fwd_workspace_size(int(N), int(T_tot), int(H),
                                                                  int(d), _DTYPES[dtype]))


def kda_linear_chunk_bwd_workspace_size(N: int, T_tot: int, Hk: int, H: int, d: int,
                                        dtype: torch.dtype) -> int:
    return int(load_library().kda_linear_chunk_bwd_workspace_size(
        int(N), int(T_tot), int(Hk), int(H), int(d), _DTYPES[dtype]))


def kda_linear_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                         h0: Optional[torch.Tensor] = None,
                         cu_seqlens: Optional[torch.Tensor] = None, *,
                         num_seqs: Optional[int] = None, scale: float = 1.0,
                         o: Optional[torch.Tensor] = None, hT: Optional[torch.Tensor] = None,
                         output_final_state: bool = True,
                         workspace: Optional[torch.Tensor] = None,
                         stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a decay for each head over packed sequences:
    S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.  Returns
    (o [T, H, d], hT [N, H, d, d] fp32 or None).

    q, k [T, Hk, d] and v [T, H, d] share one dtype (bf16 or fp32), H a
    multiple of Hk; g fp32 log-decays, [T, H] or one constant a head [H]; h0
    fp32 [N, H, d, d] or None; hT may be h0; cu_seqlens int32 [N + 1], or None
    with num_seqs sequences of equal length.
    """
    lib = load_library()
    idx, T, Hk, H, d, dt, code, pg, per_token = _linear_sizes(q, v, g)
    cu, N = _seqs(cu_seqlens, num_seqs, idx)
    pq, pk = _at(q, "q", dt, (T, Hk, d), idx), _at(k, "k", dt, (T, Hk, d), idx)
    pv = _at(v, "v", dt, (T, H, d), idx)
    state = (N, H, d, d)
    ph = _maybe(h0, "h0", torch.float32, state, idx)
    handle = _stream_at(stream, idx)
    if o is None:
        o = _empty(stream, idx, (T, H, d), dt)
    if hT is None and output_final_state and N >= 0:
        hT = _empty(stream, idx, state, torch.float32)
    ws, ws_bytes, _keep = _workspace(_size("kda_linear_chunk_fwd_workspace_size", N, T, H, d, code),
                                     workspace, stream, idx)
    st = lib.kda_linear_chunk_fwd(pq, pk, pv, pg, ph, cu, N, T, Hk, H, d, code, per_token, scale,
                                  _at(o, "o", dt, (T, H, d), idx),
                                  _maybe(hT, "hT", torch.float32, state, idx), ws, ws_bytes, handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_linear_chunk_fwd")
    return o, hT


def kda_linear_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                           S: torch.Tensor, *, scale: float = 1.0,
                           o: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of the linear attention for each sequence; S [B, H, d, d]
    fp32 is updated in place.  q, k [B, Hk, d], v [B, H, d], g fp32 [B, H] or
    [H].  Returns o [B, H, d]."""
    lib = load_library()
    idx, B, Hk, H, d, dt, code, pg, per_token = _linear_sizes(q, v, g)
    pq, pk = _at(q, "q", dt, (B, Hk, d), idx), _at(k, "k", dt, (B, Hk, d), idx)
    pv, pS = _at(v, "v", dt, (B, H, d), idx), _at(S, "S", torch.float32, (B, H, d, d), idx)
    handle = _stream_at(stream, idx)
    if o is None:
        o = _empty(stream, idx, (B, H, d), dt)
    st = lib.kda_linear_decode_step(pq, pk, pv, pg, pS, _at(o, "o", dt, (B, H, d), idx), B, Hk, H, d,
                                    code, per_token, scale, handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_linear_decode_step")
    return o


def kda_linear_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                         dO: torch.Tensor, h0: Optional[torch.Tensor] = None,
                         cu_seqlens: Optional[torch.Tensor] = None,
                         dhT: Optional[torch.Tensor] = None, *, num_seqs: Optional[int] = None,
                         scale: float = 1.0, workspace: Optional[torch.Tensor] = None,
                         stream=None) -> dict:
    """Gradient of kda_linear_chunk_fwd for L = <dO, o> + <dhT, hT>: a dict of
    dq, dk [T, Hk, d], dv [T, H, d] (dtype of q), dg fp32 of g's shape and
    dh0 [N, H, d, d] fp32."""
    lib = load_library()
    idx, T, Hk, H, d, dt, code, pg, per_token = _linear_sizes(q, v, g)
    cu, N = _seqs(cu_seqlens, num_seqs, idx)
    pq, pk = _at(q, "q", dt, (T, Hk, d), idx), _at(k, "k", dt, (T, Hk, d), idx)
    pv, pd = _at(v, "v", dt, (T, H, d), idx), _at(dO, "dO", dt, (T, H, d), idx)
    state = (max(N, 0), H, d, d)
    ph, pT = _maybe(h0, "h0", torch.float32, state, idx), _maybe(dhT, "dhT", torch.float32, state, idx)
    handle = _stream_at(stream, idx)
    out = {"dq": _empty(stream, idx, (T, Hk, d), dt), "dk": _empty(stream, idx, (T, Hk, d), dt),
           "dv": _empty(stream, idx, (T, H, d), dt),
           "dg": _empty(stream, idx, g.shape, torch.float32),
           "dh0": _empty(stream, idx, state, torch.float32)}
    ws, ws_bytes, _keep = _workspace(
        _size("kda_linear_chunk_bwd_workspace_size", N, T, Hk, H, d, code), workspace, stream, idx)
    p = {n: t.data_ptr() for n, t in out.items()}
    st = lib.kda_linear_chunk_bwd(pq, pk, pv, pg, ph, cu, N, T, Hk, H, d, code, per_token, scale, pd, pT,
                                  p["dq"], p["dk"], p["dv"], p["dg"], p["dh0"], ws, ws_bytes, handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_linear_chunk_bwd")
    return out


KDA_ROPE_NONE = 0
KDA_ROPE_LINEAR = 1
KDA_ROPE_BASE = 2
KDA_ROPE_PARTS = 3


def kda_rotary_frequencies(rot: int, base: float = 10000.0, scaling: int = KDA_ROPE_NONE,
                           factor: float = 1.0, original_length: float = 0.0,
                           beta_fast: float = 32.0, beta_slow: float = 1.0, *,
                           device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq fp32 [rot / 2], scale) for kda_rotary; see include/kda.h for
    the ways of scaling.  inv_freq is on `device` (default: the current CUDA
    device)."""
    rot = int(rot)
    buf = (ctypes.c_float * max(1, rot // 2))()
    scale = ctypes.c_float()
    st = load_library().kda_rotary_frequencies(rot, float(base), int(scaling), float(factor),
                                               float(original_length), float(beta_fast),
                                               float(beta_slow), buf, ctypes.byref(scale))
    if st != KDA_OK:
        raise KdaError(st, "kda_rotary_frequencies")
    inv = torch.tensor(list(buf), dtype=torch.float32)
    return inv.to("cuda" if device is None else device), float(scale.value)


def _token_rows(t: torch.Tensor, name: str, dt, T: int, d: int, idx: int):
    """(address, heads, elements between tokens) of a [T, heads, d] tensor
    whose token rows are dense (the tokens themselves may be apart: a slice of
    a projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.get_device() != idx:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, idx, t.device))
    if t.dtype is not dt:
        raise TypeError("%s must be %s, got %s" % (name, dt, t.dtype))
    shape = t.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != d:
        raise ValueError("%s must have shape (%d, heads, %d), got %s" % (name, T, d, tuple(shape)))
    heads = shape[1]
    if t.is_contiguous():
        return t.data_ptr(), heads, heads * d
    s = t.stride()
    if (d > 1 and s[2] != 1) or (heads > 1 and s[1] != d) or (T > 1 and s[0] < heads * d):
        raise ValueError("%s must have dense heads, got strides %s" % (name, s))
    return t.data_ptr(), heads, s[0] if T > 1 else heads * d


def kda_rotary(q: torch.Tensor, k: Optional[torch.Tensor], inv_freq: Optional[torch.Tensor],
               positions: Optional[torch.Tensor] = None,
               cu_seqlens: Optional[torch.Tensor] = None, *, num_seqs: Optional[int] = None,
               interleaved: bool = False, inverse: bool = False, scale: float = 1.0,
               q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotary positions of q [T, Hq, d] and k [T, Hk, d] (or None) over the
    first 2 * len(inv_freq) channels of each head.  Returns (q_out, k_out);
    in place with q_out=q, k_out=k.

    Tokens may be apart (a slice of a fused projection); heads are dense.
    positions int32 [T], or None: a token's index in its sequence by
    cu_seqlens / num_seqs.  inverse turns back, which is also the gradient.
    """
    lib = load_library()
    idx = _index(q, "q")
    if q.dim() != 3:
        raise ValueError("q must have three dimensions")
    T, Hq, d = q.shape
    dt = q.dtype
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError("unsupported dtype %s" % dt)
    pq, _, sq = _token_rows(q, "q", dt, T, d, idx)
    rot, pf = 0, None
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        pf = _at(inv_freq, "inv_freq", torch.float32, (rot // 2,), idx)
    pp = _maybe(positions, "positions", torch.int32, (T,), idx)
    cu, N = _seqs(cu_seqlens, num_seqs, idx)
    handle = _stream_at(stream, idx)
    if q_out is None:
        q_out = _empty(stream, idx, (T, Hq, d), dt)
    pqo, heads, sqo = _token_rows(q_out, "q_out", dt, T, d, idx)
    if heads != Hq:
        raise ValueError("q_out must have shape %s" % ((T, Hq, d),))
    pk = pko = None
    Hk = sk = sko = 0
    if k is not None:
        pk, Hk, sk = _token_rows(k, "k", dt, T, d, idx)
        if k_out is None:
            k_out = _empty(stream, idx, (T, Hk, d), dt)
        pko, heads, sko = _token_rows(k_out, "k_out", dt, T, d, idx)
        if heads != Hk:
            raise ValueError("k_out must have shape %s" % ((T, Hk, d),))
    elif k_out is not None:
        raise ValueError("k_out without k")
    st = lib.kda_rotary(pq, pk, pf, pp, cu, N, T, Hq, Hk, d, rot, code, int(bool(interleaved)),
                        int(bool(inverse)), scale, sq, sk, pqo, pko, sqo, sko, handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_rotary")
    return q_out, k_out


def _norm_sizes(x, weight):
    """(device, T, G, D, dtype, its code): weight [D] norms the last axis,
    [G, D] the last axis of x [..., G, D] with a row for each of G."""
    idx = _index(x, "x")
    shape = x.shape
    if len(shape) < 1:
        raise ValueError("x must have a last axis")
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError("unsupported dtype %s" % x.dtype)
    D = shape[-1]
    G = 1
    if weight is not None and weight.dim() == 2:
        G = weight.shape[0]
        if len(shape) < 2 or shape[-2] != G:
            raise ValueError("a weight of shape %s needs x of shape (..., %d, %d)" % (
                tuple(weight.shape), G, D))
    if D == 0 or G == 0:
        raise ValueError("x must have a last axis")
    return idx, x.numel() // (G * D), G, D, x.dtype, code


def kda_layernorm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                      bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
                      y: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Layer norm over the last axis of x: (y, mean, rstd), mean and rstd fp32
    of x's shape without that axis.  weight, bias fp32 [D], or [G, D] with a
    row for each of the G in x [..., G, D] (heads); y may be x."""
    lib = load_library()
    by = weight if weight is not None else bias
    idx, T, G, D, dt, code = _norm_sizes(x, by)
    shape = x.shape
    px = _at(x, "x", dt, shape, idx)
    of = None if by is None else (D,) if by.dim() != 2 else (G, D)
    pw, pb = _maybe(weight, "weight", torch.float32, of, idx), _maybe(bias, "bias", torch.float32, of, idx)
    handle = _stream_at(stream, idx)
    if y is None:
        y = _empty(stream, idx, shape, dt)
    mean = _empty(stream, idx, shape[:-1], torch.float32)
    rstd = _empty(stream, idx, shape[:-1], torch.float32)
    st = lib.kda_layernorm_fwd(px, pw, pb, T, G, D, code, eps, _at(y, "y", dt, shape, idx),
                               mean.data_ptr(), rstd.data_ptr(), handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_layernorm_fwd")
    return y, mean, rstd


def kda_layernorm_bwd_workspace_size(T: int, G: int, D: int, dtype: torch.dtype) -> int:
    return int(load_library().kda_layernorm_bwd_workspace_size(int(T), int(G), int(D),
                                                               _DTYPES[dtype]))


def kda_layernorm_bwd(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                      weight: Optional[torch.Tensor] = None, *,
                      bias: Union[bool, torch.Tensor, None] = False,
                      dx: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradient of kda_layernorm_fwd: a dict of dx (dtype of x), dweight (with
    a weight) and dbias (with a bias), fp32 of the weight's shape.  bias: the
    forward's, whose shape alone counts, or True for one of the weight's shape
    (without a weight: [D])."""
    lib = load_library()
    given = isinstance(bias, torch.Tensor)
    idx, T, G, D, dt, code = _norm_sizes(x, weight if weight is not None or not given else bias)
    shape = x.shape
    px, pdy = _at(x, "x", dt, shape, idx), _at(dy, "dy", dt, shape, idx)
    pm = _at(mean, "mean", torch.float32, shape[:-1], idx)
    pr = _at(rstd, "rstd", torch.float32, shape[:-1], idx)
    by = weight if weight is not None else bias if given else None
    of = (G, D) if by is not None and by.dim() == 2 else (D,)
    pw = _maybe(weight, "weight", torch.float32, of, idx)
    if given:
        _at(bias, "bias", torch.float32, of, idx)
    bias = given or bool(bias)
    handle = _stream_at(stream, idx)
    if dx is None:
        dx = _empty(stream, idx, shape, dt)
    out = {"dx": dx}
    pdw = pdb = None
    if weight is not None:
        out["dweight"] = _empty(stream, idx, of, torch.float32)
        pdw = out["dweight"].data_ptr()
    if bias:
        out["dbias"] = _empty(stream, idx, of, torch.float32)
        pdb = out["dbias"].data_ptr()
    need = _size("kda_layernorm_bwd_workspace_size", T, G, D, code) if pdw or pdb else 0
    ws, ws_bytes, _keep = _workspace(need, workspace, stream, idx)
    st = lib.kda_layernorm_bwd(pdy, px, pm, pr, pw, T, G, D, code, _at(dx, "dx", dt, shape, idx), pdw, pdb,
                               ws, ws_bytes, handle)
    if st != KDA_OK:
        raise KdaError(st, "kda_layernorm_bwd")
    return out


def kda_stream_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(load_library().kda_stream_status(_stream_handle(stream)))
