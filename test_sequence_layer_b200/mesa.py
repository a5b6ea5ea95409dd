"""ctypes binding of libmesa_b200.so (argument marshalling only).

Every step of the layer runs in the library's CUDA kernels; this module only
turns torch tensors into the pointers, sizes and stream the C ABI takes
(include/mesa.h) and turns status codes into exceptions. There is no
fallback: if the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libmesa_b200.so")
_lib = None

MESA_F32, MESA_BF16 = 0, 1
_STATUS = {0: "MESA_OK", 1: "MESA_ERR_INVALID_ARG", 2: "MESA_ERR_UNSUPPORTED", 3: "MESA_ERR_WORKSPACE",
           4: "MESA_ERR_CUDA", 5: "MESA_ERR_DEVICE_TIMEOUT"}


class MesaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_STATUS.get(status, status)}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing; build it with `python -m test_sequence_layer_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    fwd = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, P, P, P, P, P, P, P, Z, P]
    lib.mesa_forward.argtypes = fwd
    lib.mesa_forward.restype = I
    lib.mesa_forward_host.argtypes = fwd
    lib.mesa_forward_warm.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, P, P, P, P, P, P, P, P, P, Z, P]
    lib.mesa_forward_warm.restype = I
    lib.mesa_forward_host.restype = I
    lib.mesa_forward_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.mesa_forward_workspace_size.restype = Z
    lib.mesa_forward_host_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.mesa_forward_host_workspace_size.restype = Z
    lib.mesa_step.argtypes = [P, P, P, P, P, P, I, I, I, I, P, P, I, F, P, P, P]
    lib.mesa_step.restype = I
    lib.mesa_step_warm.argtypes = [P, P, P, P, P, P, I, I, I, I, P, P, P, I, F, P, P, P]
    lib.mesa_step_warm.restype = I
    lib.mesa_get_error.argtypes = [P]
    lib.mesa_get_error.restype = I
    lib.mesa_status_string.argtypes = [I]
    lib.mesa_status_string.restype = ctypes.c_char_p
    lib.mesa_version.argtypes = []
    lib.mesa_version.restype = I
    lib.mesa_timing_enable.argtypes = [I]
    lib.mesa_timing_enable.restype = I
    lib.mesa_timing_read.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(I),
                                     ctypes.POINTER(ctypes.c_double), I]
    lib.mesa_timing_read.restype = I
    lib.mesa_preprocess.argtypes = [P, P, P, P, I, I, I, I, I, I, P, P, P]
    lib.mesa_preprocess.restype = I
    lib.mesa_forward_preprocessed.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P, P, P, P,
                                              P, P, P, Z, P]
    lib.mesa_forward_preprocessed.restype = I
    lib.mesa_forward_preprocessed_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.mesa_forward_preprocessed_workspace_size.restype = Z
    lib.mesa_chunk_state_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.mesa_chunk_state_workspace_size.restype = Z
    lib.mesa_chunk_state.argtypes = [P, P, P, P, I, I, I, I, I, I, I, P, P, P, P, P, P, Z, P]
    lib.mesa_chunk_state.restype = I
    lib.mesa_state_prefix.argtypes = [P, P, P, I, I, I, I, I, I, P, P, P]
    lib.mesa_state_prefix.restype = I
    lib.mesa_backward_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.mesa_backward_workspace_size.restype = Z
    lib.mesa_backward.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, P, P, P, P, P, P, P, P, Z, P]
    lib.mesa_backward.restype = I
    lib.mesa_lru_saved_size.argtypes = [I, I, I]
    lib.mesa_lru_saved_size.restype = Z
    lib.mesa_lru_forward.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P, P]
    lib.mesa_lru_forward.restype = I
    lib.mesa_lru_backward_workspace_size.argtypes = [I, I, I, I, I]
    lib.mesa_lru_backward_workspace_size.restype = Z
    lib.mesa_lru_backward.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P, P, P, P, P, P, P, Z, P]
    lib.mesa_lru_backward.restype = I
    lib.mesa_lru_step.argtypes = [P, P, P, P, I, I, I, P, P, P, P]
    lib.mesa_lru_step.restype = I
    lib.mesa_swa_forward.argtypes = [P, P, P, I, I, I, I, I, I, I, I, F, I, P, P, P]
    lib.mesa_swa_forward.restype = I
    lib.mesa_swa_backward_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
    lib.mesa_swa_backward_workspace_size.restype = Z
    lib.mesa_swa_backward.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, P, P, P, P, Z, P]
    lib.mesa_swa_backward.restype = I
    lib.mesa_swa_step_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.mesa_swa_step_workspace_size.restype = Z
    lib.mesa_swa_step.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, Z, P]
    lib.mesa_swa_step.restype = I
    lib.mesa_swa_cache_fill.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, P]
    lib.mesa_swa_cache_fill.restype = I
    _lib = lib
    return lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MESA_F32
    if t.dtype == torch.bfloat16:
        return MESA_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, where: str):
    if rc != 0:
        raise MesaError(rc, where)


def workspace_size(B, H, T, dk, dv, chunk, dtype=torch.bfloat16) -> int:
    code = MESA_BF16 if dtype == torch.bfloat16 else MESA_F32
    return int(_load().mesa_forward_workspace_size(B, H, T, dk, dv, chunk, code))


def host_workspace_size(B, H, T, dk, dv, chunk, dtype=torch.bfloat16) -> int:
    code = MESA_BF16 if dtype == torch.bfloat16 else MESA_F32
    return int(_load().mesa_forward_host_workspace_size(B, H, T, dk, dv, chunk, code))


def forward(q, k, v, gamma, beta, lam, *, chunk=64, cg_steps=15, tol=0.0, out=None,
            return_iters=False, iters=None, H_in=None, G_in=None, return_state=False, workspace=None,
            stream=None):
    """Chunkwise-parallel Mesa forward on CUDA tensors.

    q, k: [B,H,T,dk]; v: [B,H,T,dv] (float32 or bfloat16, same dtype);
    gamma, beta: [B,H,T] float32; lam: [H,dk] float32.
    Returns out [B,H,T,dv] float32, plus iters [B,H,T] int32 if return_iters
    (written into `iters` when given), plus (H_out, G_out) if return_state.
    """
    lib = _load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    code = _dtype_code(q)
    dev = q.device
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=torch.float32, device=dev)
    if return_iters and iters is None:
        iters = torch.empty((B, H, T), dtype=torch.int32, device=dev)
    H_out = torch.empty((B, H, dk, dk), dtype=torch.float32, device=dev) if return_state else None
    G_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev) if return_state else None
    need = int(lib.mesa_forward_workspace_size(B, H, T, dk, dv, chunk, code))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.mesa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta), _ptr(lam),
                          B, H, T, dk, dv, chunk, code, int(cg_steps), float(tol),
                          _ptr(out), _ptr(iters), _ptr(H_in), _ptr(G_in), _ptr(H_out), _ptr(G_out),
                          _ptr(workspace), ws_bytes, _stream(stream, dev))
    _check(rc, "mesa_forward")
    res = (out,)
    if return_iters:
        res += (iters,)
    if return_state:
        res += (H_out, G_out)
    return res[0] if len(res) == 1 else res


def forward_warm(q, k, v, gamma, beta, lam, x0, *, chunk=64, cg_steps=15, tol=0.0, out=None, x_out=None,
                 return_iters=False, iters=None, H_in=None, G_in=None, return_state=False, workspace=None,
                 stream=None):
    """forward() with every token's CG started from x0 [B,H,T,dk] float32
    (None: from zero). Returns (out, x) where x [B,H,T,dk] float32 holds the
    solutions (written into `x_out` when given; x_out may be x0 itself), plus
    iters if return_iters, plus (H_out, G_out) if return_state."""
    lib = _load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    code = _dtype_code(q)
    dev = q.device
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=torch.float32, device=dev)
    if x_out is None:
        x_out = torch.empty((B, H, T, dk), dtype=torch.float32, device=dev)
    if return_iters and iters is None:
        iters = torch.empty((B, H, T), dtype=torch.int32, device=dev)
    H_out = torch.empty((B, H, dk, dk), dtype=torch.float32, device=dev) if return_state else None
    G_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev) if return_state else None
    need = int(lib.mesa_forward_workspace_size(B, H, T, dk, dv, chunk, code))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.mesa_forward_warm(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta), _ptr(lam),
                               B, H, T, dk, dv, chunk, code, int(cg_steps), float(tol), _ptr(x0), _ptr(x_out),
                               _ptr(out), _ptr(iters), _ptr(H_in), _ptr(G_in), _ptr(H_out), _ptr(G_out),
                               _ptr(workspace), ws_bytes, _stream(stream, dev))
    _check(rc, "mesa_forward_warm")
    res = (out, x_out)
    if return_iters:
        res += (iters,)
    if return_state:
        res += (H_out, G_out)
    return res


def backward(q, k, v, gamma, beta, lam, dout, *, chunk=64, cg_steps=15, tol=0.0, workspace=None, stream=None):
    """Gradients of L given dout = dL/do for the inputs of forward() with zero
    initial states (implicit differentiation, adjoint CG under the same rule).

    dout: [B,H,T,dv] float32. Returns (dq, dk, dv, dgamma, dbeta, dlambda),
    all float32 with the shapes of q, k, v, gamma, beta, lam.
    """
    lib = _load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    code = _dtype_code(q)
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    dq = torch.empty((B, H, T, dk), **f32)
    dk_ = torch.empty((B, H, T, dk), **f32)
    dv_ = torch.empty((B, H, T, dv), **f32)
    dgamma = torch.empty((B, H, T), **f32)
    dbeta = torch.empty((B, H, T), **f32)
    dlam = torch.empty((H, dk), **f32)
    need = int(lib.mesa_backward_workspace_size(B, H, T, dk, dv, chunk, code))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.mesa_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta), _ptr(lam),
                           B, H, T, dk, dv, chunk, code, int(cg_steps), float(tol), _ptr(dout),
                           _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dgamma), _ptr(dbeta), _ptr(dlam),
                           _ptr(workspace), ws_bytes, _stream(stream, dev))
    _check(rc, "mesa_backward")
    return dq, dk_, dv_, dgamma, dbeta, dlam


def chunk_state(k, v, gamma, beta, *, chunk=64, H_in=None, G_in=None, workspace=None, stream=None):
    """The scan of forward() without the solve: (H_out, G_out, decay) with the
    states after the T tokens (from H_in, G_in or zero) and decay [B,H] =
    prod_t gamma_t. The summary a slice of a sequence-sharded forward exchanges."""
    lib = _load()
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    code = _dtype_code(k)
    dev = k.device
    H_out = torch.empty((B, H, dk, dk), dtype=torch.float32, device=dev)
    G_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    decay = torch.empty((B, H), dtype=torch.float32, device=dev)
    need = int(lib.mesa_chunk_state_workspace_size(B, H, T, dk, dv, chunk, code))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.mesa_chunk_state(_ptr(k), _ptr(v), _ptr(gamma), _ptr(beta), B, H, T, dk, dv, chunk, code,
                              _ptr(H_in), _ptr(G_in), _ptr(H_out), _ptr(G_out), _ptr(decay),
                              _ptr(workspace), ws_bytes, _stream(stream, dev))
    _check(rc, "mesa_chunk_state")
    return H_out, G_out, decay


def state_prefix(H_slices, G_slices, decay_slices, r, *, stream=None):
    """State entering slice r from the stacked summaries [n, B, H, ...] of the
    slices before it (in sequence order). Returns (H_in, G_in)."""
    lib = _load()
    n, B, H, dk, _ = H_slices.shape
    dv = G_slices.shape[3]
    dev = H_slices.device
    H_in = torch.empty((B, H, dk, dk), dtype=torch.float32, device=dev)
    G_in = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    rc = lib.mesa_state_prefix(_ptr(H_slices), _ptr(G_slices), _ptr(decay_slices), n, int(r), B, H, dk, dv,
                               _ptr(H_in), _ptr(G_in), _stream(stream, dev))
    _check(rc, "mesa_state_prefix")
    return H_in, G_in


def forward_host(q, k, v, gamma, beta, lam, *, chunk=64, cg_steps=15, tol=0.0, out=None,
                 iters=None, H_in=None, G_in=None, H_out=None, G_out=None, workspace=None,
                 device=None, stream=None):
    """Forward with HOST (CPU, ideally pinned) tensors; the library copies them to the
    device, runs the forward and copies results back before returning."""
    lib = _load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    code = _dtype_code(q)
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=torch.float32)
    need = int(lib.mesa_forward_host_workspace_size(B, H, T, dk, dv, chunk, code))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib.mesa_forward_host(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta), _ptr(lam),
                               B, H, T, dk, dv, chunk, code, int(cg_steps), float(tol),
                               _ptr(out), _ptr(iters), _ptr(H_in), _ptr(G_in), _ptr(H_out), _ptr(G_out),
                               _ptr(workspace), ws_bytes, _stream(stream, device))
    _check(rc, "mesa_forward_host")
    return out


def preprocess(q_raw, k_raw, conv_q, conv_k, *, q_out=None, k_out=None, stream=None):
    """mesa_preprocess: causal depthwise convolution over time (conv [H,W,d],
    w = lag), then per-token L2 normalisation, for q and k. q_raw, k_raw:
    [B,H,T,d] float32 or bfloat16 CUDA tensors. Returns (q, k) in the same
    dtype, ready for forward()."""
    lib = _load()
    B, H, T, d = q_raw.shape
    W = conv_q.shape[1]
    assert k_raw.shape == q_raw.shape and k_raw.dtype == q_raw.dtype
    assert conv_q.shape == (H, W, d) and conv_k.shape == (H, W, d)
    assert conv_q.dtype == torch.float32 and conv_k.dtype == torch.float32
    for t in (q_raw, k_raw, conv_q, conv_k):
        assert t.is_cuda and t.is_contiguous()
    q_out = torch.empty_like(q_raw) if q_out is None else q_out
    k_out = torch.empty_like(k_raw) if k_out is None else k_out
    rc = lib.mesa_preprocess(_ptr(q_raw), _ptr(k_raw), _ptr(conv_q), _ptr(conv_k), B, H, T, d, W,
                             _dtype_code(q_raw), _ptr(q_out), _ptr(k_out), _stream(stream, q_raw.device))
    _check(rc, "mesa_preprocess")
    return q_out, k_out


def forward_preprocessed(q_raw, k_raw, v, gamma, beta, lam, conv_q, conv_k, *, chunk=64, cg_steps=15, tol=0.0,
                         out=None, return_iters=False, iters=None, H_in=None, G_in=None, return_state=False,
                         workspace=None, stream=None):
    """forward() of preprocess(q_raw, k_raw, conv_q, conv_k) in one call
    (mesa_forward_preprocessed): on the tensor-core shape the scan and the
    solve convolve and normalise the raw rows as they stage them. Same
    returns as forward()."""
    lib = _load()
    B, H, T, dk = q_raw.shape
    dv = v.shape[-1]
    W = conv_q.shape[1]
    assert conv_q.shape == (H, W, dk) and conv_k.shape == (H, W, dk)
    code = _dtype_code(q_raw)
    dev = q_raw.device
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=torch.float32, device=dev)
    if return_iters and iters is None:
        iters = torch.empty((B, H, T), dtype=torch.int32, device=dev)
    H_out = torch.empty((B, H, dk, dk), dtype=torch.float32, device=dev) if return_state else None
    G_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev) if return_state else None
    need = int(lib.mesa_forward_preprocessed_workspace_size(B, H, T, dk, dv, chunk, code))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.mesa_forward_preprocessed(_ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(gamma), _ptr(beta), _ptr(lam),
                                       _ptr(conv_q), _ptr(conv_k), W, B, H, T, dk, dv, chunk, code, int(cg_steps),
                                       float(tol), _ptr(out), _ptr(iters), _ptr(H_in), _ptr(G_in), _ptr(H_out),
                                       _ptr(G_out), _ptr(workspace), ws_bytes, _stream(stream, dev))
    _check(rc, "mesa_forward_preprocessed")
    res = (out,)
    if return_iters:
        res += (iters,)
    if return_state:
        res += (H_out, G_out)
    return res[0] if len(res) == 1 else res


def step(q, k, v, gamma, beta, lam, Hstate, Gstate, *, cg_steps=15, tol=0.0, out=None,
         iters=None, x_state=None, stream=None):
    """One decode step; Hstate [B,H,dk,dk] and Gstate [B,H,dv,dk] (float32) are
    updated in place. q, k: [B,H,dk]; v: [B,H,dv]; gamma, beta: [B,H].
    x_state [B,H,dk] float32 (optional, in/out): the CG starts from it and it
    receives the solution (mesa_step_warm)."""
    lib = _load()
    B, H, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
    rc = lib.mesa_step_warm(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta), _ptr(lam), B, H, dk, dv,
                            _ptr(Hstate), _ptr(Gstate), _ptr(x_state), int(cg_steps), float(tol), _ptr(out),
                            _ptr(iters), _stream(stream, q.device))
    _check(rc, "mesa_step_warm")
    return out


def get_error(stream=None) -> int:
    """Synchronises the stream and reads/clears the device error word (0 = none)."""
    lib = _load()
    s = ctypes.c_void_p(None) if stream is None else ctypes.c_void_p(stream.cuda_stream)
    return int(lib.mesa_get_error(s))


def timing_enable(on: bool = True):
    """Bracket every library kernel launch with CUDA events on its stream."""
    _load().mesa_timing_enable(1 if on else 0)


def timing_read() -> dict:
    """{kernel kind: (launches, total device ms)} since the last read (synchronises)."""
    lib = _load()
    n = 32
    names = (ctypes.c_char_p * n)()
    launches = (ctypes.c_int * n)()
    ms = (ctypes.c_double * n)()
    k = lib.mesa_timing_read(names, launches, ms, n)
    if k < 0:
        raise MesaError(4, "mesa_timing_read")
    return {names[i].decode(): (int(launches[i]), float(ms[i])) for i in range(k)}


def forward_noalloc(q, k, v, gamma, beta, lam, *, chunk=64, cg_steps=15, tol=0.0, out=None, iters=None,
                    H_in=None, G_in=None, H_out=None, G_out=None, stream=None):
    """mesa_forward_noalloc: the forward for callers that cannot allocate device
    memory; its scratch is a fixed library-owned device array (sizes beyond it
    raise MesaError MESA_ERR_WORKSPACE)."""
    lib = _load()
    if not getattr(lib, "_noalloc_typed", False):
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.mesa_forward_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, P, P, P, P, P, P, P]
        lib.mesa_forward_noalloc.restype = I
        lib._noalloc_typed = True
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=torch.float32, device=q.device)
    rc = lib.mesa_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(gamma), _ptr(beta), _ptr(lam), B, H, T, dk, dv,
                                  chunk, _dtype_code(q), int(cg_steps), float(tol), _ptr(out), _ptr(iters),
                                  _ptr(H_in), _ptr(G_in), _ptr(H_out), _ptr(G_out), _stream(stream, q.device))
    _check(rc, "mesa_forward_noalloc")
    return out


# ---- the other mixers of a hybrid stack (include/mesa_mixers.h) ----

def _arg(name, t, shape, dtype, index):
    """Checks that the library may take t by its pointer: shape, type, CUDA device, contiguous."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return
    except (AttributeError, RuntimeError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device.type != "cuda" or t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{max(index, 0)}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _first(name, t, dims):
    """Device index of the argument that fixes type, sizes and device of a call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.float32:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.get_device()


class _On:
    """Runs a call on the tensors' device; what it allocates belongs to its
    stream. `raw` is that stream's handle. Where the caller names a stream the
    tensors are marked as used on it: memory that the caller drops while the
    call is still to run is not handed out again before it has."""

    __slots__ = ("contexts", "raw")

    def __init__(self, index, stream, *tensors):
        self.contexts = ()
        if torch.cuda.current_device() != index:
            self.contexts = (torch.cuda.device(index),)
        if stream is None:
            self.raw = torch._C._cuda_getCurrentRawStream(index)
        else:
            if stream.device_index != index:
                raise ValueError(f"stream belongs to cuda:{stream.device_index}, the tensors to cuda:{index}")
            self.contexts += (torch.cuda.stream(stream),)
            self.raw = stream.cuda_stream
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()
        return self.raw

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _p(t):
    return None if t is None else t.data_ptr()


def _workspace(given, need, device, index):
    if given is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    if given.get_device() != index or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on cuda:{index}")
    return given


def _lru_inputs(x, gate_a, gate_x, lam, dims):
    index = _first("x", x, dims)
    shape, dtype = x.shape, x.dtype
    if shape[0] < 1 or shape[-1] < 1:
        raise ValueError(f"x needs at least one sequence and one channel, got {tuple(shape)}")
    _arg("gate_a", gate_a, shape, dtype, index)
    _arg("gate_x", gate_x, shape, dtype, index)
    _arg("lam", lam, shape[-1:], torch.float32, index)
    return index


def lru_forward(x, gate_a, gate_x, lam, *, h0=None, y=None, return_state=False, return_saved=False, stream=None):
    """Gated linear recurrence over a sequence (mesa_lru_forward):
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_x_t) x_t with
    log a_t = -8 softplus(lam) sigmoid(gate_a_t).

    x, gate_a, gate_x: [B,T,D] float32 or bfloat16; lam: [D] float32;
    h0: [B,D] float32 or None (zero). Returns y [B,T,D] in x's type, plus the
    final state [B,D] float32 if return_state, plus the states lru_backward
    takes ([B, ceil(T/64), D] float32) if return_saved.
    """
    lib = _load()
    index = _lru_inputs(x, gate_a, gate_x, lam, 3)
    (B, T, D), dev = x.shape, x.device
    if h0 is not None:
        _arg("h0", h0, (B, D), torch.float32, index)
    if y is not None:
        _arg("y", y, x.shape, x.dtype, index)
    with _On(index, stream, x, gate_a, gate_x, lam, h0, y) as raw:
        y = torch.empty_like(x) if y is None else y
        h_T = torch.empty((B, D), dtype=torch.float32, device=dev) if return_state else None
        saved = torch.empty((B, -(-T // 64), D), dtype=torch.float32, device=dev) if return_saved else None
        _check(lib.mesa_lru_forward(_p(x), _p(gate_a), _p(gate_x), _p(lam), B, T, D, _dtype_code(x), _p(h0),
                                    _p(y), _p(h_T), _p(saved), raw), "mesa_lru_forward")
    res = (y,) + ((h_T,) if return_state else ()) + ((saved,) if return_saved else ())
    return res[0] if len(res) == 1 else res


def lru_backward(x, gate_a, gate_x, lam, dy, *, h0=None, saved=None, dh_T=None, workspace=None, stream=None):
    """Gradients of lru_forward (mesa_lru_backward) given dy = dL/dy [B,T,D]
    and dh_T = dL/dh_T [B,D] float32 (None: zero). `saved` is what lru_forward
    returned for these inputs; without it the states are recomputed from h0.
    Returns (dx, dgate_a, dgate_x, dlam, dh0): the first three in x's type,
    dlam [D] and dh0 [B,D] float32."""
    lib = _load()
    index = _lru_inputs(x, gate_a, gate_x, lam, 3)
    (B, T, D), dev, code = x.shape, x.device, _dtype_code(x)
    _arg("dy", dy, x.shape, x.dtype, index)
    if h0 is not None:
        _arg("h0", h0, (B, D), torch.float32, index)
    if saved is not None:
        _arg("saved", saved, (B, -(-T // 64), D), torch.float32, index)
    if dh_T is not None:
        _arg("dh_T", dh_T, (B, D), torch.float32, index)
    with _On(index, stream, x, gate_a, gate_x, lam, dy, h0, saved, dh_T, workspace) as raw:
        dx, dga, dgx = (torch.empty_like(x) for _ in range(3))
        dlam = torch.empty(D, dtype=torch.float32, device=dev)
        dh0 = torch.empty((B, D), dtype=torch.float32, device=dev)
        need = int(lib.mesa_lru_backward_workspace_size(B, T, D, code, saved is not None))
        workspace = _workspace(workspace, need, dev, index)
        _check(lib.mesa_lru_backward(_p(x), _p(gate_a), _p(gate_x), _p(lam), B, T, D, code, _p(h0),
                                     _p(saved), _p(dy), _p(dh_T), _p(dx), _p(dga), _p(dgx), _p(dlam),
                                     _p(dh0), _p(workspace), workspace.numel() * workspace.element_size(),
                                     raw), "mesa_lru_backward")
    return dx, dga, dgx, dlam, dh0


def lru_step(x, gate_a, gate_x, lam, h, *, h_out=None, y=None, stream=None):
    """One decoded token of the recurrence (mesa_lru_step): x, gate_a, gate_x
    [B,D]; the state h [B,D] float32 is updated in place, or left as it is and
    the new one written to h_out. Returns y [B,D] in x's type."""
    lib = _load()
    index = _lru_inputs(x, gate_a, gate_x, lam, 2)
    (B, D), dev = x.shape, x.device
    _arg("h", h, (B, D), torch.float32, index)
    if h_out is not None:
        _arg("h_out", h_out, (B, D), torch.float32, index)
    if y is not None:
        _arg("y", y, x.shape, x.dtype, index)
    with _On(index, stream, x, gate_a, gate_x, lam, h, h_out, y) as raw:
        y = torch.empty_like(x) if y is None else y
        _check(lib.mesa_lru_step(_p(x), _p(gate_a), _p(gate_x), _p(lam), B, D, _dtype_code(x), _p(h),
                                 _p(h if h_out is None else h_out), _p(y), raw), "mesa_lru_step")
    return y


def _swa_inputs(q, k, v, dims):
    """Checks q [B,Hq,(T,)d] against k, v [B,Hkv,(S,)d]."""
    index = _first("q", q, dims)
    if not isinstance(k, torch.Tensor) or k.dim() != dims:
        raise ValueError(f"k must be a tensor of {dims} dimensions")
    if k.shape[0] != q.shape[0] or k.shape[-1] != q.shape[-1]:
        raise ValueError(f"k {tuple(k.shape)} does not go with q {tuple(q.shape)}")
    _arg("k", k, k.shape, q.dtype, index)
    _arg("v", v, k.shape, q.dtype, index)
    return index


def _size(name, v):
    """A size the C ABI takes as a 32-bit integer; its range is checked there."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} = {v} does not fit 32 bits")
    return v


def _scale(scale, d):
    return float(d) ** -0.5 if scale is None else float(scale)


def swa_forward(q, k, v, *, window, sinks=0, scale=None, out=None, return_lse=False, stream=None):
    """Causal sliding-window attention with sinks (mesa_swa_forward).

    q: [B,Hq,T,d]; k, v: [B,Hkv,S,d] (float32 or bfloat16, one type), Hq a
    multiple of Hkv, S >= T: the queries are the last T positions. Position p
    sees key j if j <= p and (p - j < window or j < sinks); d in {16,32,64,128},
    sinks <= 128. scale defaults to 1/sqrt(d). Returns out [B,Hq,T,d] in q's
    type, plus lse [B,Hq,T] float32 if return_lse.
    """
    lib = _load()
    index = _swa_inputs(q, k, v, 4)
    (B, Hq, T, d), (_, Hkv, S, _), dev = q.shape, k.shape, q.device
    if out is not None:
        _arg("out", out, q.shape, q.dtype, index)
    with _On(index, stream, q, k, v, out) as raw:
        out = torch.empty_like(q) if out is None else out
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=dev) if return_lse else None
        _check(lib.mesa_swa_forward(_p(q), _p(k), _p(v), B, Hq, Hkv, T, S, d, _size("window", window), _size("sinks", sinks),
                                    _scale(scale, d), _dtype_code(q), _p(out), _p(lse), raw),
               "mesa_swa_forward")
    return (out, lse) if return_lse else out


def swa_backward(q, k, v, out, lse, dout, *, window, sinks=0, scale=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv), in the inputs' type, of swa_forward for the
    same arguments, from its out and lse and dout = dL/dout (mesa_swa_backward)."""
    lib = _load()
    index = _swa_inputs(q, k, v, 4)
    (B, Hq, T, d), (_, Hkv, S, _), dev, code = q.shape, k.shape, q.device, _dtype_code(q)
    _arg("out", out, q.shape, q.dtype, index)
    _arg("lse", lse, (B, Hq, T), torch.float32, index)
    _arg("dout", dout, q.shape, q.dtype, index)
    with _On(index, stream, q, k, v, out, lse, dout, workspace) as raw:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        need = int(lib.mesa_swa_backward_workspace_size(B, Hq, Hkv, T, S, d, _size("sinks", sinks), code))
        workspace = _workspace(workspace, need, dev, index)
        _check(lib.mesa_swa_backward(_p(q), _p(k), _p(v), _p(out), _p(lse), _p(dout), B, Hq, Hkv, T, S, d,
                                     _size("window", window), _size("sinks", sinks), _scale(scale, d), code, _p(dq), _p(dk), _p(dv),
                                     _p(workspace), workspace.numel() * workspace.element_size(),
                                     raw), "mesa_swa_backward")
    return dq, dk, dv


def _caches(k_cache, v_cache, B, Hkv, slots, d, dtype, index):
    _arg("k_cache", k_cache, (B, Hkv, slots, d), dtype, index)
    _arg("v_cache", v_cache, (B, Hkv, slots, d), dtype, index)


def swa_step(q, k, v, k_cache, v_cache, pos, *, window, sinks=0, scale=None, out=None, workspace=None, stream=None):
    """One decoded token over rolling caches (mesa_swa_step): q [B,Hq,d],
    k, v [B,Hkv,d], k_cache, v_cache [B,Hkv,sinks+window,d] updated in place,
    pos [B] int32 on the device: the token's position, negative for an idle
    row (its caches untouched, its output zero). Returns out [B,Hq,d]."""
    lib = _load()
    index = _swa_inputs(q, k, v, 3)
    (B, Hq, d), Hkv, dev, code = q.shape, k.shape[1], q.device, _dtype_code(q)
    window, sinks = _size("window", window), _size("sinks", sinks)
    _caches(k_cache, v_cache, B, Hkv, sinks + window, d, q.dtype, index)
    _arg("pos", pos, (B,), torch.int32, index)
    if out is not None:
        _arg("out", out, q.shape, q.dtype, index)
    with _On(index, stream, q, k, v, k_cache, v_cache, pos, out, workspace) as raw:
        out = torch.empty_like(q) if out is None else out
        need = lib.mesa_swa_step_workspace_size(B, Hq, Hkv, d, window, sinks, code)
        if need or workspace is not None:
            workspace = _workspace(workspace, need, dev, index)
        _check(lib.mesa_swa_step(_p(q), _p(k), _p(v), _p(k_cache), _p(v_cache), _p(pos), B, Hq, Hkv, d, window, sinks,
                                 _scale(scale, d), code, _p(out), _p(workspace),
                                 0 if workspace is None else workspace.numel() * workspace.element_size(), raw),
               "mesa_swa_step")
    return out


def swa_cache_fill(k, v, k_cache, v_cache, *, window, sinks=0, start=0, lens=None, stream=None):
    """Puts the tokens k, v [B,Hkv,S,d] at positions start, start + 1, ...
    into rolling caches (mesa_swa_cache_fill), as S swa_step calls would.
    lens: int32 [B] on the device, the tokens of each sequence (None: S)."""
    lib = _load()
    index = _first("k", k, 4)
    (B, Hkv, S, d), dev = k.shape, k.device
    _arg("v", v, k.shape, k.dtype, index)
    _caches(k_cache, v_cache, B, Hkv, _size("sinks", sinks) + _size("window", window), d, k.dtype, index)
    if lens is not None:
        _arg("lens", lens, (B,), torch.int32, index)
    with _On(index, stream, k, v, k_cache, v_cache, lens) as raw:
        _check(lib.mesa_swa_cache_fill(_p(k), _p(v), _p(k_cache), _p(v_cache), _p(lens), B, Hkv, S, d,
                                       _size("window", window), _size("sinks", sinks), _size("start", start), _dtype_code(k), raw),
               "mesa_swa_cache_fill")
