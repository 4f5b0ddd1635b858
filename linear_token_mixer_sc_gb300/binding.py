"""Python binding of the C ABI in ``include/ida.h`` (``_lib/libida.so``).

Argument marshalling only: every step of the mixer runs in the library's CUDA
kernels.  Torch supplies device memory and the stream.  There is no fallback:
if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import threading
from pathlib import Path

import torch

LIB_PATH = Path(__file__).resolve().parent / "_lib" / "libida.so"

IDA_OK, IDA_ERR_ARG, IDA_ERR_UNSUPPORTED, IDA_ERR_CUDA, IDA_ERR_DEVICE = range(5)
IDA_F32, IDA_BF16 = 0, 1
IDA_READOUT_ETA = 1
IDA_FEAT_L2 = 2
IDA_PATH_SEQUENTIAL = 256

EXPORTED = ("ida_state_floats", "ida_forward", "ida_forward_ws", "ida_forward_from", "ida_forward_workspace_bytes",
            "ida_forward_noalloc", "ida_decode_step", "ida_device_error", "ida_status_str",
            "ida_last_error", "ida_selftest_bounded_wait", "ida_backward", "ida_backward_workspace_bytes",
            "ida_forward_ideal", "ida_rope", "ida_forward_host", "ida_forward_host_staging_bytes",
            "ida_ssm_conv", "ida_ssm_conv_backward", "ida_ssm_conv_backward_workspace_bytes", "ida_ssm_scan",
            "ida_ssm_scan_workspace_bytes", "ida_ssm_scan_backward", "ida_ssm_scan_backward_workspace_bytes",
            "ida_ssm_step", "ida_rmsnorm", "ida_rmsnorm_backward", "ida_rmsnorm_backward_workspace_bytes",
            "ida_ffn", "ida_ffn_workspace_bytes", "ida_ffn_backward", "ida_ffn_backward_workspace_bytes",
            "ida_quant_e4m3", "ida_gemm_e4m3", "ida_glu_e4m3")

_lock = threading.Lock()
_lib = None
_vp, _fp, _i = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int


class IdaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def load() -> ctypes.CDLL:
    """Load ``libida.so``; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not LIB_PATH.exists():
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with linear_token_mixer_sc_gb300.build.build()")
            L = ctypes.CDLL(str(LIB_PATH))
            L.ida_state_floats.restype = ctypes.c_size_t
            L.ida_state_floats.argtypes = [_i, _i, _i, _i]
            L.ida_forward.restype = _i
            L.ida_forward.argtypes = [_vp, _vp, _vp, _fp, _fp, _fp, _fp, _fp, _vp, _fp,
                                      _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp]
            L.ida_forward_ws.restype = _i
            L.ida_forward_ws.argtypes = [_vp, _vp, _vp, _fp, _fp, _fp, _fp, _fp, _vp, _fp,
                                         _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp, ctypes.c_size_t, _vp]
            L.ida_forward_from.restype = _i
            L.ida_forward_from.argtypes = [_vp, _vp, _vp, _fp, _fp, _fp, _fp, _fp, _fp, _vp, _fp,
                                           _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp, ctypes.c_size_t, _vp]
            L.ida_forward_workspace_bytes.restype = ctypes.c_size_t
            L.ida_forward_workspace_bytes.argtypes = [_i] * 9
            L.ida_forward_host.restype = _i
            L.ida_forward_host.argtypes = [_vp, _vp, _vp, _fp, _fp, _fp, _fp, _fp, _fp, _vp, _fp,
                                           _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp, ctypes.c_size_t, _vp]
            L.ida_forward_host_staging_bytes.restype = ctypes.c_size_t
            L.ida_forward_host_staging_bytes.argtypes = [_i] * 9
            L.ida_forward_noalloc.restype = _i
            L.ida_forward_noalloc.argtypes = [_vp, _vp, _vp, _fp, _fp, _fp, _fp, _fp, _vp, _fp,
                                              _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp]
            L.ida_decode_step.restype = _i
            L.ida_decode_step.argtypes = [_vp, _vp, _vp, _fp, _fp, _fp, _fp, _fp, _fp, _vp,
                                          _i, _i, _i, _i, _i, _i, _i, _i, _vp]
            L.ida_backward.restype = _i
            L.ida_backward.argtypes = [_vp, _vp, _vp, _fp, _fp, _fp, _fp, _fp, _vp, _vp, _vp, _vp,
                                       _fp, _fp, _fp, _fp, _fp,
                                       _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp, ctypes.c_size_t, _vp]
            L.ida_backward_workspace_bytes.restype = ctypes.c_size_t
            L.ida_backward_workspace_bytes.argtypes = [_i] * 9
            L.ida_forward_ideal.restype = _i
            L.ida_forward_ideal.argtypes = [_vp, _vp, _vp, _fp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _vp]
            L.ida_rope.restype = _i
            L.ida_rope.argtypes = [_vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _i, _vp]
            ll, sz = ctypes.c_longlong, ctypes.c_size_t
            for name, args in (
                    ("ida_ssm_conv", [_vp] * 6 + [_i] * 3 + [ll] + [_i] * 2 + [_vp]),
                    ("ida_ssm_conv_backward", [_vp] * 7 + [_i] * 3 + [ll] * 2 + [_i] * 2 + [_vp, sz, _vp]),
                    ("ida_ssm_scan", [_vp] * 10 + [_i] * 6 + [ll] * 4 + [_i, _vp, sz, _vp]),
                    ("ida_ssm_scan_backward", [_vp] * 15 + [_i] * 6 + [ll] * 8 + [_i, _vp, sz, _vp]),
                    ("ida_ssm_step", [_vp] * 10 + [_i] * 5 + [ll] * 2 + [_i] * 2 + [_vp]),
                    ("ida_rmsnorm", [_vp] * 7 + [_i] * 3 + [ctypes.c_float, _i, _vp]),
                    ("ida_rmsnorm_backward", [_vp] * 6 + [_i] * 2 + [ctypes.c_float, _i, _vp, sz, _vp]),
                    ("ida_ffn", [_vp] * 6 + [_i] * 3 + [ll, _i, _vp, sz, _vp]),
                    ("ida_ffn_backward", [_vp] * 10 + [_i] * 3 + [ll, _i, _vp, sz, _vp]),
                    ("ida_quant_e4m3", [_vp] * 3 + [_i] * 3 + [ll, _i, _vp]),
                    ("ida_gemm_e4m3", [_vp] * 5 + [_i] * 4 + [_vp]),
                    ("ida_glu_e4m3", [_vp] * 8 + [_i] * 3 + [_vp])):
                getattr(L, name).restype = _i
                getattr(L, name).argtypes = args
            for name, n in (("ida_ssm_conv_backward_workspace_bytes", 4), ("ida_ssm_scan_workspace_bytes", 7),
                            ("ida_ssm_scan_backward_workspace_bytes", 7), ("ida_rmsnorm_backward_workspace_bytes", 2),
                            ("ida_ffn_workspace_bytes", 5), ("ida_ffn_backward_workspace_bytes", 4)):
                getattr(L, name).restype = sz
                getattr(L, name).argtypes = [_i] * n
            L.ida_selftest_bounded_wait.restype = _i
            L.ida_selftest_bounded_wait.argtypes = [ctypes.c_longlong, _vp]
            L.ida_device_error.restype = _i
            L.ida_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint)]
            L.ida_status_str.restype = ctypes.c_char_p
            L.ida_status_str.argtypes = [_i]
            L.ida_last_error.restype = ctypes.c_char_p
            L.ida_last_error.argtypes = []
            _lib = L
    return _lib


def _check(status: int, what: str) -> None:
    if status != IDA_OK:
        L = load()
        raise IdaError(status, f"{what}: {L.ida_status_str(status).decode()} "
                               f"({L.ida_last_error().decode()})")


def ida_state_floats(d: int, R: int, M: int, W: int) -> int:
    return int(load().ida_state_floats(d, R, M, W))


def ida_status_str(status: int) -> str:
    return load().ida_status_str(status).decode()


def ida_last_error() -> str:
    return load().ida_last_error().decode()


def ida_device_error() -> int:
    code = ctypes.c_uint(0)
    load().ida_device_error(ctypes.byref(code))
    return int(code.value)


def _p(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return IDA_F32
    if t.dtype == torch.bfloat16:
        return IDA_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _params(p: dict):
    out = []
    for key in ("conv_w", "norm_w", "bias", "lambda", "Bvec"):
        t = p[key]
        if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()):
            raise ValueError(f"parameter {key} must be a contiguous float32 CUDA tensor")
        out.append(t)
    return out


def ida_forward_workspace_bytes(B: int, H: int, N: int, d: int, R: int, M: int, dtype: int,
                                W: int, flags: int = 0) -> int:
    return int(load().ida_forward_workspace_bytes(B, H, N, d, R, M, dtype, W, flags))


def ida_forward_host_staging_bytes(B: int, H: int, N: int, d: int, R: int, M: int, dtype: int,
                                   W: int, flags: int = 0) -> int:
    return int(load().ida_forward_host_staging_bytes(B, H, N, d, R, M, dtype, W, flags))


def ida_forward_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, params: dict,
                     out: torch.Tensor | None = None, final_state: torch.Tensor | bool | None = None,
                     state_in: torch.Tensor | None = None, flags: int = 0,
                     staging: torch.Tensor | None = None, stream=None):
    """Prefill from host memory (``ida_forward_host``).  q, k [B,N,H,R], v [B,N,H,d]
    contiguous CPU tensors (fp32/bf16; pinned memory lets the copies overlap the
    kernels).  ``params`` as for ``ida_forward`` (CUDA).  ``out``: CPU tensor to fill,
    or None to allocate a pinned one.  ``final_state``: CPU float32 [B,H,S] tensor,
    True to allocate a pinned one, or None.  ``state_in``: CPU float32 [B,H,S] or None.
    ``staging``: CUDA tensor of at least ``ida_forward_host_staging_bytes`` bytes, or
    None to allocate one.  Asynchronous on ``stream``: synchronise it before reading
    ``out`` / ``final_state``.  Returns (out, final_state).
    """
    for t in (q, k, v):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CPU tensors")
    dt = _dtype_code(q)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share a dtype")
    B, N, H, R = q.shape
    d = v.shape[3]
    cw, nw, bs, lam, bv = _params(params)
    M, W = lam.shape[1], cw.shape[3]
    if tuple(k.shape) != (B, N, H, R) or tuple(v.shape[:3]) != (B, N, H):
        raise ValueError("shape mismatch between q, k and v")
    if out is None:
        out = torch.empty((B, N, H, d), dtype=q.dtype).pin_memory()
    if out.is_cuda or not out.is_contiguous() or out.dtype != q.dtype or out.numel() != B * N * H * d:
        raise ValueError("out must be a contiguous CPU tensor of q's dtype with B*N*H*d elements")
    S = ida_state_floats(d, R, M, W)
    if final_state is True:
        final_state = torch.empty((B, H, S), dtype=torch.float32).pin_memory()
    elif final_state is False:
        final_state = None
    for name, t in (("final_state", final_state), ("state_in", state_in)):
        if t is not None and (t.is_cuda or not t.is_contiguous() or t.dtype != torch.float32
                              or t.numel() < B * H * S):
            raise ValueError(f"{name} must be a contiguous float32 CPU tensor with B*H*ida_state_floats elements")
    if staging is None:
        nbytes = ida_forward_host_staging_bytes(B, H, N, d, R, M, dt, W, flags)
        staging = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=cw.device)
    if not staging.is_cuda:
        raise ValueError("staging must be a CUDA tensor")
    st = load().ida_forward_host(_p(q), _p(k), _p(v), _p(cw), _p(nw), _p(bs), _p(lam), _p(bv), _p(state_in),
                                 _p(out), _p(final_state), B, H, N, d, R, M, dt, W, int(flags), _p(staging),
                                 staging.numel() * staging.element_size(), _stream_handle(stream))
    _check(st, "ida_forward_host")
    return out, final_state


def ida_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, params: dict,
                out: torch.Tensor | None = None, final_state: torch.Tensor | bool | None = None,
                flags: int = 0, stream=None, workspace: torch.Tensor | None = None,
                state_in: torch.Tensor | None = None):
    """Prefill.  q, k [B,N,H,R], v [B,N,H,d] CUDA tensors (fp32/bf16, contiguous).

    ``params``: dict of float32 CUDA tensors conv_w [2,H,R,W], norm_w/bias
    [H,R+d], lambda/Bvec [H,M,2].  ``final_state``: a [B,H,S] float32 tensor to
    fill, True to allocate one, or None.  ``workspace``: optional CUDA tensor
    (any dtype) handed to ``ida_forward_ws``.  ``state_in``: optional [B,H,S]
    float32 CUDA tensor, the state before position 0 (``ida_forward_from``).
    Returns (out, final_state).
    """
    for t in (q, k, v):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("q, k, v must be contiguous CUDA tensors")
    dt = _dtype_code(q)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share a dtype")
    B, N, H, R = q.shape
    d = v.shape[3]
    cw, nw, bs, lam, bv = _params(params)
    M, W = lam.shape[1], cw.shape[3]
    if tuple(k.shape) != (B, N, H, R) or tuple(v.shape[:3]) != (B, N, H):
        raise ValueError("shape mismatch between q, k and v")
    if out is None:
        out = torch.empty((B, N, H, d), dtype=q.dtype, device=q.device)
    S = ida_state_floats(d, R, M, W)
    if final_state is True:
        final_state = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    elif final_state is False:
        final_state = None
    if final_state is not None and (final_state.dtype != torch.float32 or final_state.numel() < B * H * S):
        raise ValueError("final_state must be float32 with B*H*ida_state_floats elements")
    if state_in is not None:
        if not (state_in.is_cuda and state_in.is_contiguous() and state_in.dtype == torch.float32
                and state_in.numel() >= B * H * S):
            raise ValueError("state_in must be a contiguous float32 CUDA tensor with B*H*ida_state_floats elements")
        wp, nbytes = None, 0
        if workspace is not None:
            if not workspace.is_cuda:
                raise ValueError("workspace must be a CUDA tensor")
            wp, nbytes = workspace, workspace.numel() * workspace.element_size()
        st = load().ida_forward_from(_p(q), _p(k), _p(v), _p(cw), _p(nw), _p(bs), _p(lam), _p(bv),
                                     _p(state_in), _p(out), _p(final_state), B, H, N, d, R, M, dt, W,
                                     int(flags), _p(wp), nbytes, _stream_handle(stream))
        _check(st, "ida_forward_from")
    elif workspace is None:
        st = load().ida_forward(_p(q), _p(k), _p(v), _p(cw), _p(nw), _p(bs), _p(lam), _p(bv), _p(out),
                                _p(final_state), B, H, N, d, R, M, dt, W, int(flags),
                                _stream_handle(stream))
        _check(st, "ida_forward")
    else:
        if not workspace.is_cuda:
            raise ValueError("workspace must be a CUDA tensor")
        nbytes = workspace.numel() * workspace.element_size()
        st = load().ida_forward_ws(_p(q), _p(k), _p(v), _p(cw), _p(nw), _p(bs), _p(lam), _p(bv),
                                   _p(out), _p(final_state), B, H, N, d, R, M, dt, W, int(flags),
                                   _p(workspace), nbytes, _stream_handle(stream))
        _check(st, "ida_forward_ws")
    return out, final_state


def ida_forward_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, params: dict,
                        out: torch.Tensor, final_state: torch.Tensor | None = None, flags: int = 0,
                        stream=None):
    """Prefill through ``ida_forward_noalloc``: for callers that may not allocate device
    memory, so ``out`` (and ``final_state``, if wanted) must be passed in; the scratch is
    the library's static device array.  Marshalling only, like ``ida_forward``."""
    for t in (q, k, v, out):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("q, k, v and out must be contiguous CUDA tensors")
    dt = _dtype_code(q)
    B, N, H, R = q.shape
    d = v.shape[3]
    cw, nw, bs, lam, bv = _params(params)
    M, W = lam.shape[1], cw.shape[3]
    st = load().ida_forward_noalloc(_p(q), _p(k), _p(v), _p(cw), _p(nw), _p(bs), _p(lam), _p(bv),
                                    _p(out), _p(final_state), B, H, N, d, R, M, dt, W, int(flags),
                                    _stream_handle(stream))
    _check(st, "ida_forward_noalloc")
    return out, final_state


def forward_workspace(q: torch.Tensor, v: torch.Tensor, params: dict, flags: int = 0):
    """A device workspace sized by ``ida_forward_workspace_bytes`` (None when none applies)."""
    B, N, H, R = q.shape
    d = v.shape[3]
    M, W = params["lambda"].shape[1], params["conv_w"].shape[3]
    n = ida_forward_workspace_bytes(B, H, N, d, R, M, _dtype_code(q), W, flags)
    return None if n == 0 else torch.empty(n, dtype=torch.uint8, device=q.device)


def ida_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, params: dict,
                    state: torch.Tensor, out: torch.Tensor | None = None, flags: int = 0,
                    stream=None) -> torch.Tensor:
    """One decode step.  q, k [B,H,R], v [B,H,d]; ``state`` [B,H,S] float32 updated in place."""
    for t in (q, k, v, state):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("q, k, v and state must be contiguous CUDA tensors")
    dt = _dtype_code(q)
    B, H, R = q.shape
    d = v.shape[2]
    cw, nw, bs, lam, bv = _params(params)
    M, W = lam.shape[1], cw.shape[3]
    if state.dtype != torch.float32 or state.numel() < B * H * ida_state_floats(d, R, M, W):
        raise ValueError("state must be float32 with B*H*ida_state_floats elements")
    if out is None:
        out = torch.empty((B, H, d), dtype=q.dtype, device=q.device)
    st = load().ida_decode_step(_p(q), _p(k), _p(v), _p(cw), _p(nw), _p(bs), _p(lam), _p(bv),
                                _p(state), _p(out), B, H, d, R, M, dt, W, int(flags),
                                _stream_handle(stream))
    _check(st, "ida_decode_step")
    return out


def ida_backward_workspace_bytes(B: int, H: int, N: int, d: int, R: int, M: int, dtype: int,
                                 W: int, flags: int = 0) -> int:
    return int(load().ida_backward_workspace_bytes(B, H, N, d, R, M, dtype, W, flags))


def ida_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, params: dict, dout: torch.Tensor,
                 flags: int = 0, workspace: torch.Tensor | None = None, stream=None,
                 grads: dict | None = None) -> dict:
    """Gradients of the prefill.  q, k [B,N,H,R], v and dout [B,N,H,d] CUDA tensors of one
    dtype.  Returns dict q, k, v (input dtype) and conv_w, norm_w, bias, lambda, Bvec
    (float32, the parameters' shapes), written into ``grads`` when given.  ``workspace``: a
    CUDA tensor of at least ``ida_backward_workspace_bytes`` bytes (allocated here when None)."""
    for t in (q, k, v, dout):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("q, k, v and dout must be contiguous CUDA tensors")
    dt = _dtype_code(q)
    if k.dtype != q.dtype or v.dtype != q.dtype or dout.dtype != q.dtype:
        raise TypeError("q, k, v and dout must share a dtype")
    B, N, H, R = q.shape
    d = v.shape[3]
    cw, nw, bs, lam, bv = _params(params)
    M, W = lam.shape[1], cw.shape[3]
    if tuple(dout.shape) != (B, N, H, d):
        raise ValueError("dout must have the shape of out")
    nbytes = ida_backward_workspace_bytes(B, H, N, d, R, M, dt, W, flags)
    if workspace is None and nbytes > 0:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    g = grads if grads is not None else {
        "q": torch.empty_like(q), "k": torch.empty_like(k), "v": torch.empty_like(v),
        "conv_w": torch.empty_like(cw), "norm_w": torch.empty_like(nw), "bias": torch.empty_like(bs),
        "lambda": torch.empty_like(lam), "Bvec": torch.empty_like(bv)}
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().ida_backward(_p(q), _p(k), _p(v), _p(cw), _p(nw), _p(bs), _p(lam), _p(bv), _p(dout),
                             _p(g["q"]), _p(g["k"]), _p(g["v"]), _p(g["conv_w"]), _p(g["norm_w"]),
                             _p(g["bias"]), _p(g["lambda"]), _p(g["Bvec"]), B, H, N, d, R, M, dt, W,
                             int(flags), _p(workspace), wbytes, _stream_handle(stream))
    _check(st, "ida_backward")
    return g


def ida_forward_ideal(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, omega: torch.Tensor, params: dict,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The ideal layer on random Fourier features.  q, k [B,N,H,R_in], v [B,N,H,d] CUDA
    tensors of one dtype; omega [H,D,R_in] float32 CUDA; ``params`` as for ida_forward (only
    lambda and Bvec are read).  Returns out [B,N,H,d]."""
    for t in (q, k, v, omega):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("q, k, v and omega must be contiguous CUDA tensors")
    dt = _dtype_code(q)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share a dtype")
    if omega.dtype != torch.float32:
        raise TypeError("omega must be float32")
    B, N, H, Rin = q.shape
    d = v.shape[3]
    D = omega.shape[1]
    lam, bv = params["lambda"], params["Bvec"]
    M = lam.shape[1]
    if out is None:
        out = torch.empty((B, N, H, d), dtype=q.dtype, device=q.device)
    st = load().ida_forward_ideal(_p(q), _p(k), _p(v), _p(omega), _p(lam), _p(bv), _p(out), B, H, N, d, Rin, D, M,
                                  dt, _stream_handle(stream))
    _check(st, "ida_forward_ideal")
    return out


def ida_rope(q: torch.Tensor, k: torch.Tensor | None = None, pos0: int = 0, base: float = 10000.0,
             stream=None) -> None:
    """Rotary position embeddings on q (and k) [B,N,H,R] CUDA tensors, in place: channel
    pairs (2i, 2i+1) of the row at position pos0 + t rotate by (pos0 + t) * base^(-2i/R)."""
    for t in (q, k):
        if t is not None and not (t.is_cuda and t.is_contiguous()):
            raise ValueError("q and k must be contiguous CUDA tensors")
    if k is not None and (k.shape != q.shape or k.dtype != q.dtype):
        raise ValueError("k must match q in shape and dtype")
    B, N, H, R = q.shape
    st = load().ida_rope(_p(q), _p(k), B, N, H, R, int(pos0), float(base), _dtype_code(q), _stream_handle(stream))
    _check(st, "ida_rope")


# ---- the selective mixer and the residual pre-norm --------------------------------------------

def _placed(fn):
    """Give ``fn`` a keyword ``stream`` (a torch.cuda.Stream; None: the current one), and run it with its
    first tensor's device and that stream current, so that what it allocates belongs to the stream its
    kernels run on."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if first is None:
            raise TypeError(f"{fn.__name__}() needs {name}")
        dev = first.get_device()
        if dev < 0:
            raise ValueError(f"{fn.__name__}: expected CUDA tensors")
        if stream is not None:
            if stream.device_index != dev:
                raise ValueError(f"{fn.__name__}: the stream is on another device than the tensors")
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
        if dev != _current_device():
            with torch.cuda.device(dev):
                return fn(*args, **kw)
        return fn(*args, **kw)
    return call


# What torch.cuda.current_device() and current_stream().cuda_stream return, without building a
# Stream object: the calls below are a few microseconds long.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _fits(*sizes: int) -> None:
    """Sizes that the C ABI's ints hold (ctypes would cut off the others' high bits)."""
    if max(sizes) > 0x7FFFFFFF or min(sizes) < -0x80000000:
        raise ValueError(f"a size is above 2^31 - 1: {sizes}")


def _misfit(name: str, t: torch.Tensor, shape, dtype):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous and on the inputs' CUDA device")


def _dense(name: str, t: torch.Tensor, shape, dtype, dev: int) -> int:
    """The address of a contiguous tensor of this shape, dtype and device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        _misfit(name, t, shape, dtype)
    return t.data_ptr()


def _rows(name: str, t: torch.Tensor, shape, dtype, dev: int, lead: int):
    """(address, row stride) of a tensor whose last dimensions are dense rows and whose ``lead``
    first ones (1 or 2) count rows at one stride."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _misfit(name, t, shape, dtype)
    strides, row = t.stride(), 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] > 1 and strides[i] != row and t.numel():
            raise ValueError(f"the rows of {name} must be dense")
        row *= shape[i]
    n = shape[lead - 1]
    if lead == 2 and n > 1 and t.numel():
        ld = strides[1]
        if shape[0] > 1 and strides[0] != n * ld:
            raise ValueError(f"the rows of {name} must lie at one stride")
        return t.data_ptr(), ld
    if shape[0] > 1 and t.numel():
        return t.data_ptr(), strides[0]
    return t.data_ptr(), (row + 7) // 8 * 8  # a single row has no stride


def _work_buffer(given: torch.Tensor | None, nbytes: int, dev: int):
    """(tensor kept alive, address, bytes) of the given workspace or of a new one."""
    if given is None:
        if not nbytes:
            return None, None, 0
        given = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    elif given.get_device() != dev or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' CUDA device")
    return given, given.data_ptr(), given.numel() * given.element_size()


def ida_ssm_conv_backward_workspace_bytes(B: int, N: int, C: int, W: int) -> int:
    _fits(B, N, C, W)
    return int(load().ida_ssm_conv_backward_workspace_bytes(B, N, C, W))


def ida_ssm_scan_workspace_bytes(B: int, H: int, N: int, d: int, G: int, M: int, dtype: int) -> int:
    _fits(B, H, N, d, G, M, dtype)
    return int(load().ida_ssm_scan_workspace_bytes(B, H, N, d, G, M, dtype))


def ida_ssm_scan_backward_workspace_bytes(B: int, H: int, N: int, d: int, G: int, M: int, dtype: int) -> int:
    _fits(B, H, N, d, G, M, dtype)
    return int(load().ida_ssm_scan_backward_workspace_bytes(B, H, N, d, G, M, dtype))


def ida_rmsnorm_backward_workspace_bytes(rows: int, D: int) -> int:
    _fits(rows, D)
    return int(load().ida_rmsnorm_backward_workspace_bytes(rows, D))


@_placed
def ida_ssm_conv(x: torch.Tensor, conv_w: torch.Tensor, conv_b: torch.Tensor, state_in: torch.Tensor | None = None,
                 final_state: torch.Tensor | bool | None = None, out: torch.Tensor | None = None):
    """Short causal convolution and SiLU of the selective mixer.  x [B,N,C] (a slice of wider rows
    is taken as it is), conv_w [C,W] and conv_b [C] float32; ``state_in`` [B,W-1,C] float32 or None
    (zero); ``final_state``: a tensor to fill, True to allocate one, or None.
    Returns (out [B,N,C], final_state)."""
    dt, dev = _dtype_code(x), x.get_device()
    B, N, C = x.shape
    W = conv_w.shape[1]
    _fits(B, N, C, W)
    xp, ldx = _rows("x", x, x.shape, x.dtype, dev, 2)
    if out is None:
        out = torch.empty((B, N, C), dtype=x.dtype, device=x.device)
    if final_state is True:
        final_state = torch.empty((B, W - 1, C), dtype=torch.float32, device=x.device)
    elif final_state is False:
        final_state = None
    S, f32 = (B, W - 1, C), torch.float32
    st = load().ida_ssm_conv(xp, _dense("conv_w", conv_w, (C, W), f32, dev), _dense("conv_b", conv_b, (C,), f32, dev),
                             None if state_in is None else _dense("state_in", state_in, S, f32, dev),
                             _dense("out", out, x.shape, x.dtype, dev),
                             None if final_state is None else _dense("final_state", final_state, S, f32, dev),
                             B, N, C, ldx, dt, W, _raw_stream(dev))
    _check(st, "ida_ssm_conv")
    return out, final_state


@_placed
def ida_ssm_conv_backward(x: torch.Tensor, dout: torch.Tensor, conv_w: torch.Tensor, conv_b: torch.Tensor,
                          dx: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> dict:
    """Gradients of ``ida_ssm_conv`` from a zero state: dict x (written into ``dx`` when given, which
    may be a slice of wider rows), conv_w, conv_b.  dout [B,N,C] dense.  ``workspace``: a tensor of at
    least ``ida_ssm_conv_backward_workspace_bytes`` bytes (allocated here when None)."""
    dt, dev = _dtype_code(x), x.get_device()
    B, N, C = x.shape
    W = conv_w.shape[1]
    _fits(B, N, C, W)
    f32 = torch.float32
    xp, ldx = _rows("x", x, x.shape, x.dtype, dev, 2)
    wp, bp = _dense("conv_w", conv_w, (C, W), f32, dev), _dense("conv_b", conv_b, (C,), f32, dev)
    dp = _dense("dout", dout, x.shape, x.dtype, dev)
    if dx is None:
        dx = torch.empty((B, N, C), dtype=x.dtype, device=x.device)
    dxp, lddx = _rows("dx", dx, x.shape, x.dtype, dev, 2)
    dw, db = (torch.empty(t.shape, dtype=f32, device=x.device) for t in (conv_w, conv_b))
    L = load()
    ws, wsp, n = _work_buffer(workspace, L.ida_ssm_conv_backward_workspace_bytes(B, N, C, W), dev)
    st = L.ida_ssm_conv_backward(xp, dp, wp, bp, dxp, dw.data_ptr(), db.data_ptr(), B, N, C, ldx, lddx, dt, W, wsp, n,
                                 _raw_stream(dev))
    _check(st, "ida_ssm_conv_backward")
    return {"x": dx, "conv_w": dw, "conv_b": db}


def _scan_inputs(x, b, c, dt, params):
    """Addresses, strides and sizes of the scan's inputs."""
    dev, f32 = x.get_device(), torch.float32
    B, N, H, d = x.shape
    G, M = b.shape[2:]
    _fits(B, N, H, d, G, M)
    xp, ldx = _rows("x", x, x.shape, x.dtype, dev, 2)
    bp, ldb = _rows("b", b, (B, N, G, M), x.dtype, dev, 2)
    cp, ldc = _rows("c", c, (B, N, G, M), x.dtype, dev, 2)
    tp, ldt = _rows("dt", dt, (B, N, H), x.dtype, dev, 2)
    ptrs = [xp, bp, cp, tp] + [_dense(k, params[k], (H,), f32, dev) for k in ("a_log", "dt_bias", "D")]
    return dev, ptrs, (B, H, N, d, G, M), (ldx, ldb, ldc, ldt)


@_placed
def ida_ssm_scan(x: torch.Tensor, b: torch.Tensor, c: torch.Tensor, dt: torch.Tensor, params: dict,
                 state_in: torch.Tensor | None = None, final_state: torch.Tensor | bool | None = None,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Selective scan over a prompt.  x [B,N,H,d], b and c [B,N,G,M], dt [B,N,H] of one dtype, each a
    slice of wider rows if need be; ``params``: dict of float32 [H] tensors a_log, dt_bias, D.
    ``state_in`` [B,H,M,d] float32 or None (zero); ``final_state``: a tensor to fill, True to
    allocate one, or None.  ``workspace``: a tensor of ``ida_ssm_scan_workspace_bytes`` bytes
    (allocated here when None).  Returns (y [B,N,H,d], final_state)."""
    code = _dtype_code(x)
    dev, ptrs, sizes, strides = _scan_inputs(x, b, c, dt, params)
    B, H, N, d, G, M = sizes
    if out is None:
        out = torch.empty((B, N, H, d), dtype=x.dtype, device=x.device)
    if final_state is True:
        final_state = torch.empty((B, H, M, d), dtype=torch.float32, device=x.device)
    elif final_state is False:
        final_state = None
    S, f32 = (B, H, M, d), torch.float32
    sip = None if state_in is None else _dense("state_in", state_in, S, f32, dev)
    fsp = None if final_state is None else _dense("final_state", final_state, S, f32, dev)
    L = load()
    ws, wsp, n = _work_buffer(workspace, L.ida_ssm_scan_workspace_bytes(B, H, N, d, G, M, code)
                              if workspace is None else 0, dev)
    st = L.ida_ssm_scan(*ptrs, sip, _dense("out", out, x.shape, x.dtype, dev), fsp, *sizes, *strides, code, wsp, n,
                        _raw_stream(dev))
    _check(st, "ida_ssm_scan")
    return out, final_state


@_placed
def ida_ssm_scan_backward(x: torch.Tensor, b: torch.Tensor, c: torch.Tensor, dt: torch.Tensor, params: dict,
                          dy: torch.Tensor, workspace: torch.Tensor | None = None) -> dict:
    """Gradients of ``ida_ssm_scan`` from a zero state, given dy [B,N,H,d]: dict x, b, c, dt (input
    dtype; x, b and c are slices of the dense rows ``xbc`` [B,N,H d + 2 G M], what
    ``ida_ssm_conv_backward`` takes as dout) and a_log, dt_bias, D (float32 [H]).  ``workspace``: a
    tensor of at least ``ida_ssm_scan_backward_workspace_bytes`` bytes (allocated here when None)."""
    code = _dtype_code(x)
    dev, ptrs, sizes, strides = _scan_inputs(x, b, c, dt, params)
    B, H, N, d, G, M = sizes
    dyp = _dense("dy", dy, x.shape, x.dtype, dev)
    C = H * d + 2 * G * M
    xbc = torch.empty((B, N, C), dtype=x.dtype, device=x.device)
    ddt = torch.empty((B, N, H), dtype=x.dtype, device=x.device)
    par = torch.empty((3, H), dtype=torch.float32, device=x.device)
    L = load()
    ws, wsp, n = _work_buffer(workspace, L.ida_ssm_scan_backward_workspace_bytes(B, H, N, d, G, M, code)
                              if workspace is None else 0, dev)
    e, p, pp = xbc.element_size(), xbc.data_ptr(), par.data_ptr()
    st = L.ida_ssm_scan_backward(*ptrs, dyp, p, p + H * d * e, p + (H * d + G * M) * e, ddt.data_ptr(),
                                 pp, pp + 4 * H, pp + 8 * H, *sizes, *strides, C, C, C, H, code, wsp, n, _raw_stream(dev))
    _check(st, "ida_ssm_scan_backward")
    da_log, ddt_bias, dD = par.unbind()
    bc = (B, N, G, M), (N * C, C, M, 1)
    return {"x": xbc.as_strided((B, N, H, d), (N * C, C, d, 1)), "b": xbc.as_strided(*bc, H * d),
            "c": xbc.as_strided(*bc, H * d + G * M), "xbc": xbc, "dt": ddt, "a_log": da_log, "dt_bias": ddt_bias, "D": dD}


@_placed
def ida_ssm_step(xbc: torch.Tensor, dt: torch.Tensor, params: dict, conv_state: torch.Tensor, state: torch.Tensor,
                 groups: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """One position of the selective mixer, convolution included.  xbc [B, H d + 2 G M] raw rows and
    dt [B,H] of one dtype, each a slice of wider rows if need be; ``params``: dict of float32 tensors
    conv_w [C,W], conv_b [C], a_log, dt_bias, D [H]; ``conv_state`` [B,W-1,C] and ``state`` [B,H,M,d]
    float32, updated in place; ``groups``: G.  Returns y [B,H,d]."""
    code, dev, f32 = _dtype_code(xbc), xbc.get_device(), torch.float32
    B, C = xbc.shape
    _, H, M, d = state.shape
    conv_w = params["conv_w"]
    W = conv_w.shape[1]
    _fits(B, H, M, d, W, groups)
    if C != H * d + 2 * groups * M:
        raise ValueError("xbc must have H d + 2 G M channels")
    xp, ldx = _rows("xbc", xbc, (B, C), xbc.dtype, dev, 1)
    tp, ldt = _rows("dt", dt, (B, H), xbc.dtype, dev, 1)
    if out is None:
        out = torch.empty((B, H, d), dtype=xbc.dtype, device=xbc.device)
    st = load().ida_ssm_step(xp, tp, _dense("conv_w", conv_w, (C, W), f32, dev),
                             _dense("conv_b", params["conv_b"], (C,), f32, dev),
                             *[_dense(k, params[k], (H,), f32, dev) for k in ("a_log", "dt_bias", "D")],
                             _dense("conv_state", conv_state, (B, W - 1, C), f32, dev),
                             _dense("state", state, (B, H, M, d), f32, dev),
                             _dense("out", out, (B, H, d), xbc.dtype, dev), B, H, d, groups, M, ldx, ldt, code, W,
                             _raw_stream(dev))
    _check(st, "ida_ssm_step")
    return out


@_placed
def ida_rmsnorm(x: torch.Tensor, w: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                group: int = 0, res_out: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """Root-mean-square norm of r = x + residual, rows of D channels (any leading dimensions, dense);
    w [D] float32.  Returns (out, r, q, scale): r is the new residual stream (written into
    ``res_out`` when given, which may be x or residual; x itself without a residual).  With
    ``group`` = 0 out is r / rms * w in x's dtype and q, scale are None.  With 32, 64, 128 or D
    channels per scale, q is the result divided by scale [..., D / group] in float8_e4m3fn and out
    is None unless passed in."""
    dt, dev = _dtype_code(x), x.get_device()
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    _fits(rows, D, group)
    xp, wp = _dense("x", x, x.shape, x.dtype, dev), _dense("w", w, (D,), torch.float32, dev)
    rp = None if residual is None else _dense("residual", residual, x.shape, x.dtype, dev)
    if residual is not None and res_out is None:
        res_out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    q = scale = None
    if group:
        if group < 0 or D % group:
            raise ValueError("group must divide the channels")
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        scale = torch.empty((*x.shape[:-1], D // group), dtype=torch.float32, device=x.device)
    elif out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    st = load().ida_rmsnorm(xp, rp, wp, None if res_out is None else _dense("res_out", res_out, x.shape, x.dtype, dev),
                            None if out is None else _dense("out", out, x.shape, x.dtype, dev),
                            None if q is None else q.data_ptr(), None if scale is None else scale.data_ptr(),
                            rows, D, group, eps, dt, _raw_stream(dev))
    _check(st, "ida_rmsnorm")
    return out, x if res_out is None else res_out, q, scale


@_placed
def ida_rmsnorm_backward(r: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, dres: torch.Tensor | None = None,
                         eps: float = 1e-6, dx: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None) -> dict:
    """Gradients of ``ida_rmsnorm``'s out, given the r it returned, dy and what reaches r from elsewhere
    (``dres`` or None): dict x (the gradient of x and of residual alike; into ``dx`` when given) and w."""
    dt, dev = _dtype_code(r), r.get_device()
    D = r.shape[-1]
    rows = r.numel() // D if D else 0
    _fits(rows, D)
    rp, wp = _dense("r", r, r.shape, r.dtype, dev), _dense("w", w, (D,), torch.float32, dev)
    gp = _dense("dy", dy, r.shape, r.dtype, dev)
    sp = None if dres is None else _dense("dres", dres, r.shape, r.dtype, dev)
    if dx is None:
        dx = torch.empty(r.shape, dtype=r.dtype, device=r.device)
    dw = torch.empty(w.shape, dtype=w.dtype, device=w.device)
    L = load()
    ws, wsp, n = _work_buffer(workspace, L.ida_rmsnorm_backward_workspace_bytes(rows, D) if workspace is None else 0, dev)
    st = L.ida_rmsnorm_backward(rp, wp, gp, sp, _dense("dx", dx, r.shape, r.dtype, dev), dw.data_ptr(), rows, D, eps,
                                dt, wsp, n, _raw_stream(dev))
    _check(st, "ida_rmsnorm_backward")
    return {"x": dx, "w": dw}


# ---- the feed-forward block and products in 8 bits --------------------------------------------

@functools.lru_cache(maxsize=256)  # host arithmetic on the sizes alone
def ida_ffn_workspace_bytes(rows: int, D: int, F: int, dtype: int, keep: bool = False) -> int:
    _fits(rows, D, F, dtype)
    return int(load().ida_ffn_workspace_bytes(rows, D, F, dtype, int(keep)))


@functools.lru_cache(maxsize=256)
def ida_ffn_backward_workspace_bytes(rows: int, D: int, F: int, dtype: int) -> int:
    _fits(rows, D, F, dtype)
    return int(load().ida_ffn_backward_workspace_bytes(rows, D, F, dtype))


_INT = 0x7FFFFFFF


def _leading(name: str, t: torch.Tensor, dev: int):
    """(address, row stride, rows) of a tensor of rows: any leading dimensions where it is dense, one or
    two at one stride where it is a slice of wider rows."""
    n = t.shape[-1]
    rows = t.numel() // n if n else 0
    if t.is_contiguous():
        return t.data_ptr(), n, rows
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be contiguous, or rows in one or two dimensions at one stride")
    return (*_rows(name, t, t.shape, t.dtype, dev, t.dim() - 1), rows)


def _ffn_inputs(x, w_gate, w_up, w_down):
    """Device, addresses, row stride and sizes of the block's inputs."""
    dev = x.get_device()
    F, D = w_gate.shape
    xp, ldx, rows = _leading("x", x, dev)
    if x.shape[-1] != D:
        raise ValueError(f"x must have rows of {D} channels, got {x.shape[-1]}")
    if rows > _INT or D > _INT or F > _INT:
        _fits(rows, D, F)
    ptrs = [xp, _dense("w_gate", w_gate, (F, D), x.dtype, dev), _dense("w_up", w_up, (F, D), x.dtype, dev),
            _dense("w_down", w_down, (D, F), x.dtype, dev)]
    return dev, ptrs, ldx, (rows, D, F)


@_placed
def ida_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
            acts: torch.Tensor | bool | None = None, out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None):
    """Gated feed-forward block, out = (silu(x w_gate^T) * (x w_up^T)) w_down^T, tensors of one dtype.
    x: rows of D channels (any leading dimensions, or a slice of wider rows), w_gate and w_up [F,D],
    w_down [D,F].  ``acts``: a [3,...,F] tensor to fill with both factors and their product (what
    ``ida_ffn_backward`` takes), True to allocate one, or None.  ``workspace``: a tensor of at least
    ``ida_ffn_workspace_bytes`` bytes (allocated here when None).  Returns (out [...,D], acts)."""
    code = _dtype_code(x)
    dev, ptrs, ldx, sizes = _ffn_inputs(x, w_gate, w_up, w_down)
    rows, D, F = sizes
    # (what is allocated here needs none of the checks)
    op = ap = None
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        op = _dense("out", out, x.shape, x.dtype, dev)
    if acts is True:
        acts = torch.empty((3, *x.shape[:-1], F), dtype=x.dtype, device=x.device)
        ap = acts.data_ptr()
    elif acts is None or acts is False:
        acts = None
    else:
        ap = _dense("acts", acts, (3, *x.shape[:-1], F), x.dtype, dev)
    ws, wsp, n = _work_buffer(workspace, ida_ffn_workspace_bytes(rows, D, F, code, acts is not None) if workspace is None else 0, dev)
    st = (_lib or load()).ida_ffn(*ptrs, op or out.data_ptr(), ap, *sizes, ldx, code, wsp, n, _raw_stream(dev))
    _check(st, "ida_ffn")
    return out, acts


@_placed
def ida_ffn_backward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                     acts: torch.Tensor, dout: torch.Tensor, grads: dict | None = None,
                     workspace: torch.Tensor | None = None) -> dict:
    """Gradients of ``ida_ffn``'s out, given its inputs, the ``acts`` it returned and dout [...,D]: dict x,
    w_gate, w_up, w_down in their tensors' shapes and dtype, written into ``grads`` when given.
    ``workspace``: a tensor of at least ``ida_ffn_backward_workspace_bytes`` bytes (allocated here when
    None)."""
    code = _dtype_code(x)
    dev, ptrs, ldx, sizes = _ffn_inputs(x, w_gate, w_up, w_down)
    rows, D, F = sizes
    ap = _dense("acts", acts, (3, *x.shape[:-1], F), x.dtype, dev)
    dp = _dense("dout", dout, x.shape, x.dtype, dev)
    like = (("x", x), ("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down))
    if grads is None:
        g = {k: torch.empty(t.shape, dtype=x.dtype, device=x.device) for k, t in like}
        gp = [t.data_ptr() for t in g.values()]
    else:
        g = grads
        gp = [_dense(f"grads[{k!r}]", g[k], t.shape, x.dtype, dev) for k, t in like]
    ws, wsp, n = _work_buffer(workspace, ida_ffn_backward_workspace_bytes(rows, D, F, code)
                              if workspace is None else 0, dev)
    st = (_lib or load()).ida_ffn_backward(*ptrs, ap, dp, *gp, *sizes, ldx, code, wsp, n, _raw_stream(dev))
    _check(st, "ida_ffn_backward")
    return g


_E4M3 = torch.float8_e4m3fn


@_placed
def ida_quant_e4m3(x: torch.Tensor, rows: int = 1, q: torch.Tensor | None = None,
                   scale: torch.Tensor | None = None):
    """x, rows of K channels (any leading dimensions, or a slice of wider rows; float32 or bfloat16), in e4m3
    with a float32 scale for 128 channels of each row (``rows`` = 1, for activations) or of each 128 rows
    (``rows`` = 128, x [N,K], for weights).  Returns (q, scale): q [...,K] in float8_e4m3fn, scale
    [...,ceil(K/128)] or [ceil(N/128),ceil(K/128)]; x is q times its scale."""
    code, dev = _dtype_code(x), x.get_device()
    K = x.shape[-1]
    if rows == 128 and x.dim() != 2:
        raise ValueError("blocks of 128 rows are of a tensor [N, K]")
    xp, ldx, n = _leading("x", x, dev)
    _fits(n, K, rows)
    lead = x.shape[:-1] if rows == 1 else ((n + 127) // 128,)
    shape = (*lead, (K + 127) // 128)
    qp = sp = None
    if q is None:
        q = torch.empty(x.shape, dtype=_E4M3, device=x.device)
    else:
        qp = _dense("q", q, x.shape, _E4M3, dev)
    if scale is None:
        scale = torch.empty(shape, dtype=torch.float32, device=x.device)
    else:
        sp = _dense("scale", scale, shape, torch.float32, dev)
    st = (_lib or load()).ida_quant_e4m3(xp, qp or q.data_ptr(), sp or scale.data_ptr(), n, K, rows, ldx, code,
                                         _raw_stream(dev))
    _check(st, "ida_quant_e4m3")
    return q, scale


@_placed
def ida_gemm_e4m3(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                  dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """(a times its scales) (b times its scales)^T: a [...,K] with a_scale [...,ceil(K/128)], as
    ``ida_rmsnorm`` (group 128), ``ida_glu_e4m3`` and ``ida_quant_e4m3`` make them, b [N,K] with b_scale
    [ceil(N/128),ceil(K/128)] of ``ida_quant_e4m3`` with 128 rows; contiguous, q's in float8_e4m3fn.
    Returns out [...,N] in ``dtype`` (bfloat16 or float32; that of ``out`` when given)."""
    dev = a.get_device()
    K, lead = a.shape[-1], a.shape[:-1]
    N, kb = b.shape[0], (K + 127) // 128
    rows = a.numel() // K if K else 0
    if rows > _INT or K > _INT or N > _INT:
        _fits(rows, K, N)
    f32 = torch.float32
    ptrs = (_dense("a", a, a.shape, _E4M3, dev), _dense("a_scale", a_scale, (*lead, kb), f32, dev),
            _dense("b", b, (N, K), _E4M3, dev), _dense("b_scale", b_scale, ((N + 127) // 128, kb), f32, dev))
    op = None
    if out is None:
        out = torch.empty((*lead, N), dtype=dtype, device=a.device)
    else:
        op = _dense("out", out, (*lead, N), out.dtype, dev)
    code = _dtype_code(out)
    st = (_lib or load()).ida_gemm_e4m3(*ptrs, op or out.data_ptr(), rows, K, N, code, _raw_stream(dev))
    _check(st, "ida_gemm_e4m3")
    return out


@_placed
def ida_glu_e4m3(a: torch.Tensor, a_scale: torch.Tensor, w_gate: torch.Tensor, gate_scale: torch.Tensor,
                 w_up: torch.Tensor, up_scale: torch.Tensor, q: torch.Tensor | None = None,
                 scale: torch.Tensor | None = None):
    """First half of the feed-forward block in 8 bits: silu(a w_gate^T) * (a w_up^T) of operands as
    ``ida_gemm_e4m3`` takes them (a [...,D], w_gate and w_up [F,D]), quantised with a scale for 128
    channels of each row.  Returns (q [...,F] in float8_e4m3fn, scale [...,ceil(F/128)])."""
    dev = a.get_device()
    D, lead = a.shape[-1], a.shape[:-1]
    F, kb = w_gate.shape[0], (D + 127) // 128
    rows = a.numel() // D if D else 0
    if rows > _INT or D > _INT or F > _INT:
        _fits(rows, D, F)
    blocks = (F + 127) // 128
    f32 = torch.float32
    ptrs = (_dense("a", a, a.shape, _E4M3, dev), _dense("a_scale", a_scale, (*lead, kb), f32, dev),
            _dense("w_gate", w_gate, (F, D), _E4M3, dev), _dense("gate_scale", gate_scale, (blocks, kb), f32, dev),
            _dense("w_up", w_up, (F, D), _E4M3, dev), _dense("up_scale", up_scale, (blocks, kb), f32, dev))
    qp = sp = None
    if q is None:
        q = torch.empty((*lead, F), dtype=_E4M3, device=a.device)
    else:
        qp = _dense("q", q, (*lead, F), _E4M3, dev)
    if scale is None:
        scale = torch.empty((*lead, blocks), dtype=f32, device=a.device)
    else:
        sp = _dense("scale", scale, (*lead, blocks), f32, dev)
    st = (_lib or load()).ida_glu_e4m3(*ptrs, qp or q.data_ptr(), sp or scale.data_ptr(), rows, D, F, _raw_stream(dev))
    _check(st, "ida_glu_e4m3")
    return q, scale


def ida_selftest_bounded_wait(limit_cycles: int, stream=None) -> None:
    """Launch the library's bounded-wait self-test (a wait that runs out on purpose)."""
    _check(load().ida_selftest_bounded_wait(int(limit_cycles), _stream_handle(stream)),
           "ida_selftest_bounded_wait")


def params_to_device(p: dict, device="cuda") -> dict:
    """float32 parameter arrays (e.g. from ``inputs.make_params``) as CUDA tensors."""
    keys = ("conv_w", "norm_w", "bias", "lambda", "Bvec")
    return {k: torch.as_tensor(p[k], dtype=torch.float32).contiguous().to(device) for k in keys}
