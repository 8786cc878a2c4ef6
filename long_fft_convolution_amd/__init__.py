"""MI355X (gfx950) exact long causal FFT convolution -- Python binding.

Thin ctypes layer over the C ABI of ``libfftconv.so`` (include/fftconv.h):
every function has the C function's name and only marshals arguments.
torch tensors supply device memory and the current HIP stream; every step of
the convolution runs in the library's HIP kernels.  There is no CPU fallback:
if the library is not built, importing the functions raises.

    y[b,h,t] = v[b,h,t] * sum_{s<=min(t,L-1)} k[h,s] * u[b,h,t-s] * w[b,h,t-s]

(FlashFFTConv summary page: exact FFT convolution, gated, with partial and
frequency-sparse filters.)
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

import numpy as np
import torch  # loads torch's HIP runtime first, so the library shares it

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfftconv.so")

FFTCONV_F32, FFTCONV_F16, FFTCONV_BF16 = 0, 1, 2
_DTYPE_CODE = {torch.float32: FFTCONV_F32, torch.float16: FFTCONV_F16, torch.bfloat16: FFTCONV_BF16}
STATUS = {0: "FFTCONV_OK", 1: "FFTCONV_ERR_INVALID_ARGUMENT", 2: "FFTCONV_ERR_UNSUPPORTED",
          3: "FFTCONV_ERR_WORKSPACE", 4: "FFTCONV_ERR_FILTER_MISMATCH", 5: "FFTCONV_ERR_HIP"}

_lib = None


class FFTConvError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status
        self.detail = detail


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m long_fft_convolution_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    lib.fftconv_filter_bytes.argtypes = [i64, i64, ctypes.c_int]
    lib.fftconv_filter_bytes.restype = sz
    lib.fftconv_workspace_bytes.argtypes = [i64, i64, i64, ctypes.c_int]
    lib.fftconv_workspace_bytes.restype = sz
    lib.fftconv_mask_blocks.argtypes = [i64]
    lib.fftconv_mask_blocks.restype = i64
    lib.fftconv_prepare_filter.argtypes = [vp, i64, i64, i64, ctypes.c_int, vp, sz, vp, sz, vp]
    lib.fftconv_prepare_filter.restype = ctypes.c_int
    lib.fftconv_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, ctypes.c_int, vp, sz, vp]
    lib.fftconv_fwd.restype = ctypes.c_int
    lib.fftconv_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, ctypes.c_int, vp]
    lib.fftconv_fwd_noalloc.restype = ctypes.c_int
    lib.fftconv_fwd_noalloc_scratch_bytes.argtypes = []
    lib.fftconv_fwd_noalloc_scratch_bytes.restype = sz
    lib.fftconv_fwd_taps_workspace_bytes.argtypes = [i64, i64, i64, ctypes.c_int]
    lib.fftconv_fwd_taps_workspace_bytes.restype = sz
    lib.fftconv_fwd_taps.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, ctypes.c_int, vp, sz, vp]
    lib.fftconv_fwd_taps.restype = ctypes.c_int
    lib.fftconv_bwd_workspace_bytes.argtypes = [i64, i64, i64, ctypes.c_int]
    lib.fftconv_bwd_workspace_bytes.restype = sz
    lib.fftconv_bwd.argtypes = [vp] * 9 + [i64, i64, i64, i64, vp, ctypes.c_int, vp, sz, vp]
    lib.fftconv_bwd.restype = ctypes.c_int
    lib.fftconv_init.argtypes = []
    lib.fftconv_init.restype = ctypes.c_int
    lib.fftconv_status_string.argtypes = [ctypes.c_int]
    lib.fftconv_status_string.restype = ctypes.c_char_p
    lib.fftconv_last_error.argtypes = []
    lib.fftconv_last_error.restype = ctypes.c_char_p
    lib.fftconv_export_filter_rfft.argtypes = [vp, i64, i64, ctypes.c_int,
                                               ctypes.POINTER(ctypes.c_double), vp]
    lib.fftconv_export_filter_rfft.restype = ctypes.c_int
    lib.fftconv_short_filter_bytes.argtypes = [i64, ctypes.c_int]
    lib.fftconv_short_filter_bytes.restype = sz
    lib.fftconv_prepare_short_filter.argtypes = [vp, i64, i64, ctypes.c_int, vp, sz, vp]
    lib.fftconv_prepare_short_filter.restype = ctypes.c_int
    lib.fftconv_fwd_short.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, vp]
    lib.fftconv_fwd_short.restype = ctypes.c_int
    lib.fftconv_bwd_short.argtypes = [vp] * 9 + [i64, i64, i64, i64, ctypes.c_int, vp]
    lib.fftconv_bwd_short.restype = ctypes.c_int
    lib.fftconv_eqlinear_weight_bytes.argtypes = [i64, i64, i64, ctypes.c_int]
    lib.fftconv_eqlinear_weight_bytes.restype = sz
    lib.fftconv_eqlinear_prepare.argtypes = [vp, i64, i64, i64, ctypes.c_int, vp, sz, vp]
    lib.fftconv_eqlinear_prepare.restype = ctypes.c_int
    lib.fftconv_eqlinear_fwd.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, vp]
    lib.fftconv_eqlinear_fwd.restype = ctypes.c_int
    ints = [i64] * 6
    lib.fftconv_decay_fwd_workspace_bytes.argtypes = [i64] * 5 + [ctypes.c_int]
    lib.fftconv_decay_fwd_workspace_bytes.restype = sz
    lib.fftconv_decay_fwd.argtypes = [vp] * 9 + [i64, vp] + ints + [ctypes.c_float, ctypes.c_int, vp, sz, vp]
    lib.fftconv_decay_fwd.restype = ctypes.c_int
    lib.fftconv_decay_step.argtypes = [vp] * 8 + [i64] * 6 + [ctypes.c_float, ctypes.c_int, vp]
    lib.fftconv_decay_step.restype = ctypes.c_int
    lib.fftconv_decay_bwd_workspace_bytes.argtypes = ints + [ctypes.c_int]
    lib.fftconv_decay_bwd_workspace_bytes.restype = sz
    lib.fftconv_decay_bwd.argtypes = [vp] * 13 + ints + [ctypes.c_float, ctypes.c_int, vp, sz, vp]
    lib.fftconv_decay_bwd.restype = ctypes.c_int
    lib.fftconv_linear_fwd_workspace_bytes.argtypes = [i64] * 3 + [ctypes.c_int]
    lib.fftconv_linear_fwd_workspace_bytes.restype = sz
    lib.fftconv_linear_fwd.argtypes = [vp] * 7 + [i64] * 3 + [ctypes.c_int, ctypes.c_int, vp, sz, vp]
    lib.fftconv_linear_fwd.restype = ctypes.c_int
    lib.fftconv_linear_bwd_workspace_bytes.argtypes = [i64] * 3 + [ctypes.c_int]
    lib.fftconv_linear_bwd_workspace_bytes.restype = sz
    lib.fftconv_linear_bwd.argtypes = [vp] * 8 + [i64] * 3 + [ctypes.c_int, ctypes.c_int, vp, sz, vp]
    lib.fftconv_linear_bwd.restype = ctypes.c_int
    lib.fftconv_delta_fwd_workspace_bytes.argtypes = ints + [ctypes.c_int]
    lib.fftconv_delta_fwd_workspace_bytes.restype = sz
    lib.fftconv_delta_fwd.argtypes = [vp] * 10 + [i64, vp] + ints + [ctypes.c_float, ctypes.c_int, vp, sz, vp]
    lib.fftconv_delta_fwd.restype = ctypes.c_int
    lib.fftconv_delta_step.argtypes = [vp] * 9 + [i64] * 6 + [ctypes.c_float, ctypes.c_int, vp]
    lib.fftconv_delta_step.restype = ctypes.c_int
    lib.fftconv_delta_bwd_workspace_bytes.argtypes = ints + [ctypes.c_int]
    lib.fftconv_delta_bwd_workspace_bytes.restype = sz
    lib.fftconv_delta_bwd.argtypes = [vp] * 16 + ints + [ctypes.c_float, ctypes.c_int, vp, sz, vp]
    lib.fftconv_delta_bwd.restype = ctypes.c_int
    lib.fftconv_norm_fwd.argtypes = [vp] * 7 + [i64] * 3 + [ctypes.c_float, ctypes.c_int, vp]
    lib.fftconv_norm_fwd.restype = ctypes.c_int
    lib.fftconv_norm_bwd_workspace_bytes.argtypes = [i64, i64]
    lib.fftconv_norm_bwd_workspace_bytes.restype = sz
    lib.fftconv_norm_bwd.argtypes = [vp] * 7 + [i64] * 3 + [ctypes.c_float, ctypes.c_int, vp, sz, vp]
    lib.fftconv_norm_bwd.restype = ctypes.c_int
    _lib = lib
    return lib


def lib():
    """The loaded ctypes library (raises ImportError when not built)."""
    return _load()


def _check(status: int):
    if status != 0:
        raise FFTConvError(status, _load().fftconv_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _raw_stream(stream, device):
    """The stream's handle as an integer, without making a Stream object for the current one."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _at(t):
    """A tensor's address for a pointer argument."""
    return None if t is None else t.data_ptr()


def _dev_tensor(t, name):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def dtype_code(dtype: torch.dtype) -> int:
    return _DTYPE_CODE[dtype]


def fftconv_filter_bytes(H: int, N: int, dtype) -> int:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return int(_load().fftconv_filter_bytes(H, N, code))


def fftconv_workspace_bytes(B: int, H: int, N: int, dtype) -> int:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return int(_load().fftconv_workspace_bytes(B, H, N, code))


def fftconv_mask_blocks(N: int) -> int:
    return int(_load().fftconv_mask_blocks(N))


def fftconv_init(device=None) -> None:
    """Build the library's constant tables on `device` (default: the current one); synchronous."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check(_load().fftconv_init())


def fftconv_status_string(status: int) -> str:
    return _load().fftconv_status_string(status).decode()


def fftconv_last_error() -> str:
    return _load().fftconv_last_error().decode()


def fftconv_prepare_filter(k: torch.Tensor, N: int, K_f: torch.Tensor,
                           workspace: torch.Tensor | None = None, stream=None) -> None:
    """K_f <- prepared spectrum of the (H, L) filter k for sequence length N."""
    _dev_tensor(k, "k")
    _dev_tensor(K_f, "K_f")
    _dev_tensor(workspace, "workspace")
    H, L = k.shape
    _check(_load().fftconv_prepare_filter(
        _ptr(k), H, L, N, dtype_code(k.dtype), _ptr(K_f), K_f.numel() * K_f.element_size(),
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream, k.device)))


def fftconv_fwd(u: torch.Tensor, K_f: torch.Tensor, w: torch.Tensor | None,
                v: torch.Tensor | None, out: torch.Tensor, L_filter: int,
                sparsity_mask: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> None:
    """out <- v * causal_conv(u * w, k) through the prepared filter K_f."""
    for name, t in (("u", u), ("K_f", K_f), ("w", w), ("v", v), ("out", out),
                    ("sparsity_mask", sparsity_mask), ("workspace", workspace)):
        _dev_tensor(t, name)
    B, H, N = u.shape
    _check(_load().fftconv_fwd(
        _ptr(u), _ptr(K_f), _ptr(w), _ptr(v), _ptr(out), B, H, N, L_filter, _ptr(sparsity_mask),
        dtype_code(u.dtype), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream, u.device)))


def fftconv_fwd_noalloc(u: torch.Tensor, K_f: torch.Tensor, w: torch.Tensor | None,
                        v: torch.Tensor | None, out: torch.Tensor, L_filter: int,
                        sparsity_mask: torch.Tensor | None = None, stream=None) -> None:
    """fftconv_fwd with the library's static scratch instead of a workspace (after fftconv_init)."""
    for name, t in (("u", u), ("K_f", K_f), ("w", w), ("v", v), ("out", out),
                    ("sparsity_mask", sparsity_mask)):
        _dev_tensor(t, name)
    B, H, N = u.shape
    _check(_load().fftconv_fwd_noalloc(
        _ptr(u), _ptr(K_f), _ptr(w), _ptr(v), _ptr(out), B, H, N, L_filter, _ptr(sparsity_mask),
        dtype_code(u.dtype), _stream(stream, u.device)))


def fftconv_fwd_noalloc_scratch_bytes() -> int:
    return int(_load().fftconv_fwd_noalloc_scratch_bytes())


def fftconv_fwd_taps_workspace_bytes(B: int, H: int, N: int, dtype) -> int:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return int(_load().fftconv_fwd_taps_workspace_bytes(B, H, N, code))


def fftconv_fwd_taps(u: torch.Tensor, k: torch.Tensor, w: torch.Tensor | None,
                     v: torch.Tensor | None, out: torch.Tensor, workspace: torch.Tensor,
                     sparsity_mask: torch.Tensor | None = None, stream=None) -> None:
    """out <- v * causal_conv(u * w, k) from the (H, L) taps k, transformed within the call."""
    for name, t in (("u", u), ("k", k), ("w", w), ("v", v), ("out", out),
                    ("sparsity_mask", sparsity_mask), ("workspace", workspace)):
        _dev_tensor(t, name)
    B, H, N = u.shape
    _check(_load().fftconv_fwd_taps(
        _ptr(u), _ptr(k), _ptr(w), _ptr(v), _ptr(out), B, H, N, k.shape[1], _ptr(sparsity_mask),
        dtype_code(u.dtype), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream, u.device)))


def fftconv_bwd_workspace_bytes(B: int, H: int, N: int, dtype) -> int:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return int(_load().fftconv_bwd_workspace_bytes(B, H, N, code))


def fftconv_bwd(dy: torch.Tensor, u: torch.Tensor, K_f: torch.Tensor, w: torch.Tensor | None,
                v: torch.Tensor | None, du: torch.Tensor | None, dk: torch.Tensor | None,
                dw: torch.Tensor | None, dv: torch.Tensor | None, L_filter: int,
                sparsity_mask: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                stream=None) -> None:
    """Gradients of sum(dy * fftconv_fwd(u, K_f, w, v)) into du, dk, dw, dv (None = skip)."""
    for name, t in (("dy", dy), ("u", u), ("K_f", K_f), ("w", w), ("v", v), ("du", du), ("dk", dk),
                    ("dw", dw), ("dv", dv), ("sparsity_mask", sparsity_mask), ("workspace", workspace)):
        _dev_tensor(t, name)
    B, H, N = u.shape
    _check(_load().fftconv_bwd(
        _ptr(dy), _ptr(u), _ptr(K_f), _ptr(w), _ptr(v), _ptr(du), _ptr(dk), _ptr(dw), _ptr(dv),
        B, H, N, L_filter, _ptr(sparsity_mask), dtype_code(u.dtype), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream, u.device)))


def fftconv_export_filter_rfft(K_f: torch.Tensor, H: int, N: int, dtype, stream=None) -> np.ndarray:
    """Synchronous: natural-order rfft bins (H, N+1) complex128 decoded from K_f."""
    _dev_tensor(K_f, "K_f")
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    outbuf = np.empty((H, N + 1, 2), dtype=np.float64)
    _check(_load().fftconv_export_filter_rfft(
        _ptr(K_f), H, N, code, outbuf.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
        _stream(stream, K_f.device)))
    return outbuf[..., 0] + 1j * outbuf[..., 1]


# ---------------------------------------------------------------- plumbing
def fftconv_short_filter_bytes(H: int, dtype) -> int:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return int(_load().fftconv_short_filter_bytes(H, code))


def fftconv_prepare_short_filter(k: torch.Tensor, K_s: torch.Tensor, stream=None) -> None:
    """K_s <- spectrum of the (H, L) filter k, L <= 1024, for the chunked short-filter path."""
    _dev_tensor(k, "k")
    _dev_tensor(K_s, "K_s")
    H, L = k.shape
    _check(_load().fftconv_prepare_short_filter(
        _ptr(k), H, L, dtype_code(k.dtype), _ptr(K_s), K_s.numel() * K_s.element_size(),
        _stream(stream, k.device)))


def fftconv_fwd_short(u: torch.Tensor, K_s: torch.Tensor, w: torch.Tensor | None, v: torch.Tensor | None,
                      out: torch.Tensor, L_filter: int, stream=None) -> None:
    """out <- v * causal_conv(u * w, k) through the short-filter spectrum K_s (N a multiple of 1024)."""
    for name, t in (("u", u), ("K_s", K_s), ("w", w), ("v", v), ("out", out)):
        _dev_tensor(t, name)
    B, H, N = u.shape
    _check(_load().fftconv_fwd_short(
        _ptr(u), _ptr(K_s), _ptr(w), _ptr(v), _ptr(out), B, H, N, L_filter, dtype_code(u.dtype),
        _stream(stream, u.device)))


def fftconv_bwd_short(dy: torch.Tensor, u: torch.Tensor, K_s: torch.Tensor, w: torch.Tensor | None,
                      v: torch.Tensor | None, du: torch.Tensor | None, dk: torch.Tensor | None,
                      dw: torch.Tensor | None, dv: torch.Tensor | None, L_filter: int, stream=None) -> None:
    """Gradients of sum(dy * fftconv_fwd_short(u, K_s, w, v)) into du, dk, dw, dv (None = skip)."""
    for name, t in (("dy", dy), ("u", u), ("K_s", K_s), ("w", w), ("v", v), ("du", du), ("dk", dk),
                    ("dw", dw), ("dv", dv)):
        _dev_tensor(t, name)
    B, H, N = u.shape
    _check(_load().fftconv_bwd_short(
        _ptr(dy), _ptr(u), _ptr(K_s), _ptr(w), _ptr(v), _ptr(du), _ptr(dk), _ptr(dw), _ptr(dv),
        B, H, N, L_filter, dtype_code(u.dtype), _stream(stream, u.device)))


def causal_conv_short(u, k, w=None, v=None, stream=None):
    """Prepare a short filter k (L <= 1024) and run one chunked forward call."""
    H, L = k.shape
    K_s = torch.empty(fftconv_short_filter_bytes(H, u.dtype), dtype=torch.uint8, device=u.device)
    fftconv_prepare_short_filter(k, K_s, stream)
    out = torch.empty_like(u)
    fftconv_fwd_short(u, K_s, w, v, out, L, stream)
    return out


def causal_conv_short_bwd(u, k, dy, w=None, v=None, stream=None):
    """Prepare a short filter k and run one backward call; returns (du, dk, dw, dv)."""
    H, L = k.shape
    K_s = torch.empty(fftconv_short_filter_bytes(H, u.dtype), dtype=torch.uint8, device=u.device)
    fftconv_prepare_short_filter(k, K_s, stream)
    du = torch.empty_like(u)
    dk = torch.empty((H, L), dtype=u.dtype, device=u.device)
    dw = torch.empty_like(u) if w is not None else None
    dv = torch.empty_like(u) if v is not None else None
    fftconv_bwd_short(dy, u, K_s, w, v, du, dk, dw, dv, L, stream)
    return du, dk, dw, dv


def fftconv_eqlinear_weight_bytes(T: int, C_out: int, C_in: int, dtype) -> int:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return int(_load().fftconv_eqlinear_weight_bytes(T, C_out, C_in, code))


def fftconv_eqlinear_prepare(W: torch.Tensor, W_f: torch.Tensor, stream=None) -> None:
    """W_f <- the group-axis real DFT of W (T, C_out, C_in)."""
    _dev_tensor(W, "W")
    _dev_tensor(W_f, "W_f")
    T, C_out, C_in = W.shape
    _check(_load().fftconv_eqlinear_prepare(
        _ptr(W), T, C_out, C_in, dtype_code(W.dtype), _ptr(W_f), W_f.numel() * W_f.element_size(),
        _stream(stream, W.device)))


def fftconv_eqlinear_fwd(x: torch.Tensor, W_f: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    """y (N, T, C_out) <- group circular convolution of x (N, T, C_in) with the prepared W_f."""
    for name, t in (("x", x), ("W_f", W_f), ("y", y)):
        _dev_tensor(t, name)
    N, T, C_in = x.shape
    C_out = y.shape[2]
    _check(_load().fftconv_eqlinear_fwd(
        _ptr(x), _ptr(W_f), _ptr(y), N, T, C_in, C_out, dtype_code(x.dtype), _stream(stream, x.device)))


def eqlinear(x, W, stream=None):
    """Prepare W and run the group convolution once (allocations by torch)."""
    T, C_out, C_in = W.shape
    W_f = torch.empty(fftconv_eqlinear_weight_bytes(T, C_out, C_in, W.dtype), dtype=torch.uint8, device=x.device)
    fftconv_eqlinear_prepare(W, W_f, stream)
    y = torch.empty((x.shape[0], T, C_out), dtype=x.dtype, device=x.device)
    fftconv_eqlinear_fwd(x, W_f, y, stream)
    return y


# ---------------------------------------------------------------- decay attention
def _dtype_of(dtype) -> int:
    return dtype if isinstance(dtype, int) else dtype_code(dtype)


def _rows_tensor(t, name, like, shape):
    """Checks a tensor argument whose rows must be contiguous (other strides are free)."""
    # the common case in few steps: this is on the path of a single token
    if t.dtype is like.dtype and t.shape == shape and t.device == like.device and t.is_cuda and \
            (t.is_contiguous() or t.stride(-1) == 1):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}")
    if t.dtype != like.dtype:
        raise ValueError(f"{name} must have dtype {like.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def _plain_tensor(t, name, dtype, shape, device):
    if t is None:
        return
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")


_strides_of = {n: ctypes.c_int64 * n for n in (5, 6, 8, 12, 21)}


def _strides(tensors, packed):
    """(batch, token, head) of each tensor, None where all are dense (an absent gradient counts as dense)."""
    if all(t is None or t.is_contiguous() for t in tensors):
        return None
    flat = []
    for t in tensors:
        if t is None:
            flat += (0, 0, 0)
        elif packed:
            flat += (0, t.stride(0), t.stride(1))
        else:
            flat += t.stride()[:3]
    return _strides_of[len(flat)](*flat)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _decay_shapes(q, k, v, log_decay, cu_seqlens):
    qs, ks, vs = q.shape, k.shape, v.shape
    dims = 4 if cu_seqlens is None else 3
    if len(qs) != dims or len(ks) != dims or len(vs) != dims:
        raise ValueError(f"q, k and v must have {dims} dimensions, not {len(qs)}, {len(ks)} and {len(vs)}")
    H, Hk, Dk, Dv = qs[-2], ks[-2], qs[-1], vs[-1]
    _rows_tensor(q, "q", q, qs)
    _rows_tensor(k, "k", q, (*qs[:-2], Hk, Dk))
    _rows_tensor(v, "v", q, (*qs[:-2], Hk, Dv))
    _plain_tensor(log_decay, "log_decay", torch.float32, (H,), q.device)
    if cu_seqlens is None:
        return qs[0], qs[1], H, Hk, Dk, Dv
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold B + 1 values")
    _plain_tensor(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, q.device)
    return cu_seqlens.numel() - 1, qs[0], H, Hk, Dk, Dv


def fftconv_decay_fwd_workspace_bytes(B: int, T: int, H: int, Dk: int, Dv: int, dtype) -> int:
    return int(_load().fftconv_decay_fwd_workspace_bytes(B, T, H, Dk, Dv, _dtype_of(dtype)))


def fftconv_decay_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, out: torch.Tensor,
                      scale: float, state_in: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
                      state_slots: torch.Tensor | None = None, cu_seqlens: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> None:
    """out <- decay attention of q, k, v: (B, N, heads, width), or packed (T, heads, width) with cu_seqlens.

    state_in / state_out: fp32 (B, H, Dk, Dv), or pools of such matrices with state_slots (B) int32.
    """
    B, N, H, Hk, Dk, Dv = _decay_shapes(q, k, v, log_decay, cu_seqlens)
    _rows_tensor(out, "out", q, (*q.shape[:-1], Dv))
    n_slots, device = 0, q.device
    if state_slots is not None:
        _plain_tensor(state_slots, "state_slots", torch.int32, (B,), device)
        pool = state_in if state_in is not None else state_out
        n_slots = pool.shape[0] if pool is not None else 0
    states = (B if state_slots is None else n_slots, H, Dk, Dv)
    _plain_tensor(state_in, "state_in", torch.float32, states, device)
    _plain_tensor(state_out, "state_out", torch.float32, states, device)
    _dev_tensor(workspace, "workspace")
    _check((_lib or _load()).fftconv_decay_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), out.data_ptr(),
        _strides((q, k, v, out), cu_seqlens is not None), _at(state_in), _at(state_out), _at(state_slots), n_slots,
        _at(cu_seqlens), B, N, H, Hk, Dk, Dv, scale, _DTYPE_CODE[q.dtype], _at(workspace), _nbytes(workspace),
        _raw_stream(stream, device)))


def fftconv_decay_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                       state: torch.Tensor, out: torch.Tensor, scale: float, state_slots: torch.Tensor | None = None,
                       stream=None) -> None:
    """One token of each sequence: q (B, H, Dk), k (B, Hk, Dk), v (B, Hk, Dv) -> out (B, H, Dv), state in place."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and v must have 3 dimensions")
    (B, H, Dk), (_, Hk, Dv), device = q.shape, v.shape, q.device
    _rows_tensor(q, "q", q, (B, H, Dk))
    _rows_tensor(k, "k", q, (B, Hk, Dk))
    _rows_tensor(v, "v", q, (B, Hk, Dv))
    _rows_tensor(out, "out", q, (B, H, Dv))
    _plain_tensor(log_decay, "log_decay", torch.float32, (H,), device)
    n_slots = 0
    if state_slots is not None:
        _plain_tensor(state_slots, "state_slots", torch.int32, (B,), device)
        n_slots = state.shape[0]
    _plain_tensor(state, "state", torch.float32, (B if state_slots is None else n_slots, H, Dk, Dv), device)
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous()):
        strides = _strides_of[8](*q.stride()[:2], *k.stride()[:2], *v.stride()[:2], *out.stride()[:2])
    _check((_lib or _load()).fftconv_decay_step(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state.data_ptr(), out.data_ptr(), strides,
        _at(state_slots), n_slots, B, H, Hk, Dk, Dv, scale, _DTYPE_CODE[q.dtype], _raw_stream(stream, device)))


def fftconv_decay_bwd_workspace_bytes(B: int, T: int, H: int, Hk: int, Dk: int, Dv: int, dtype) -> int:
    return int(_load().fftconv_decay_bwd_workspace_bytes(B, T, H, Hk, Dk, Dv, _dtype_of(dtype)))


def fftconv_decay_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                      dq: torch.Tensor | None, dk: torch.Tensor | None, dv: torch.Tensor | None, scale: float,
                      state_in: torch.Tensor | None = None, dstate_out: torch.Tensor | None = None,
                      dstate_in: torch.Tensor | None = None, cu_seqlens: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of fftconv_decay_fwd into dq, dk, dv, dstate_in (None = skip)."""
    B, N, H, Hk, Dk, Dv = _decay_shapes(q, k, v, log_decay, cu_seqlens)
    _rows_tensor(dout, "dout", q, (*q.shape[:-1], Dv))
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _rows_tensor(t, name, q, like.shape)
    for name, t in (("state_in", state_in), ("dstate_out", dstate_out), ("dstate_in", dstate_in)):
        _plain_tensor(t, name, torch.float32, (B, H, Dk, Dv), q.device)
    _dev_tensor(workspace, "workspace")
    _check((_lib or _load()).fftconv_decay_bwd(
        dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _at(dq), _at(dk), _at(dv),
        _strides((dout, q, k, v, dq, dk, dv), cu_seqlens is not None), _at(state_in), _at(dstate_out),
        _at(dstate_in), _at(cu_seqlens), B, N, H, Hk, Dk, Dv, scale, _DTYPE_CODE[q.dtype], _at(workspace),
        _nbytes(workspace), _raw_stream(stream, q.device)))


def _scratch(nbytes, device):
    return None if nbytes == 0 else torch.empty(nbytes, dtype=torch.uint8, device=device)


def decay_attention(q, k, v, log_decay, scale=None, state_in=None, cu_seqlens=None, stream=None):
    """Decay attention of whole sequences (allocations by torch); returns (out, final states).  scale: Dk^-0.5.

    Packed tokens of no sequence (before cu_seqlens[0], from its last value on) have no result: their rows are not set.
    """
    if stream is not None:
        with torch.cuda.stream(stream):      # the scratch memory and the results are that stream's, too
            return decay_attention(q, k, v, log_decay, scale, state_in, cu_seqlens)
    B, N, H, Hk, Dk, Dv = _decay_shapes(q, k, v, log_decay, cu_seqlens)
    T = N if cu_seqlens is not None else B * N
    out = torch.empty((*q.shape[:-1], Dv), dtype=q.dtype, device=q.device)
    state_out = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device)
    ws = _scratch(fftconv_decay_fwd_workspace_bytes(B, T, H, Dk, Dv, q.dtype), q.device)
    fftconv_decay_fwd(q, k, v, log_decay, out, Dk ** -0.5 if scale is None else scale, state_in, state_out,
                      cu_seqlens=cu_seqlens, workspace=ws)
    return out, state_out


def decay_attention_bwd(q, k, v, log_decay, dout, scale=None, state_in=None, dstate_out=None, cu_seqlens=None,
                        stream=None):
    """Gradients of decay_attention; returns (dq, dk, dv, dstate_in), the last None without state_in.

    Rows of packed tokens that belong to no sequence are not set.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return decay_attention_bwd(q, k, v, log_decay, dout, scale, state_in, dstate_out, cu_seqlens)
    B, N, H, Hk, Dk, Dv = _decay_shapes(q, k, v, log_decay, cu_seqlens)
    T = N if cu_seqlens is not None else B * N
    dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
    dstate_in = None if state_in is None else torch.empty_like(state_in)
    ws = _scratch(fftconv_decay_bwd_workspace_bytes(B, T, H, Hk, Dk, Dv, q.dtype), q.device)
    fftconv_decay_bwd(dout, q, k, v, log_decay, dq, dk, dv, Dk ** -0.5 if scale is None else scale, state_in,
                      dstate_out, dstate_in, cu_seqlens, ws)
    return dq, dk, dv, dstate_in


# ---------------------------------------------------------------- linear product
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, not {name!r}")
    return ACTIVATIONS[name]


def _row_strides(*tensors):
    """Row strides of the matrices, None where all are dense."""
    if all(t is None or t.is_contiguous() for t in tensors):
        return None
    return _strides_of[len(tensors)](*(0 if t is None else t.stride(0) for t in tensors))


def _linear_shapes(x, W):
    if x.dim() != 2 or W.dim() != 2:
        raise ValueError("x and W must have 2 dimensions")
    (M, K), N = x.shape, W.shape[0]
    _rows_tensor(x, "x", x, (M, K))
    _rows_tensor(W, "W", x, (N, K))
    return M, N, K


def fftconv_linear_fwd_workspace_bytes(M: int, N: int, K: int, dtype) -> int:
    return int(_load().fftconv_linear_fwd_workspace_bytes(M, N, K, _dtype_of(dtype)))


def fftconv_linear_fwd(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None, residual: torch.Tensor | None,
                       out: torch.Tensor, pre: torch.Tensor | None = None, activation: str = "none",
                       workspace: torch.Tensor | None = None, stream=None) -> None:
    """out <- act(x W^T + bias) + residual for x (M, K), W (N, K); pre (optional) <- x W^T + bias."""
    M, N, K = _linear_shapes(x, W)
    _rows_tensor(out, "out", x, (M, N))
    if bias is not None:
        _rows_tensor(bias, "bias", x, (N,))
    if residual is not None:
        _rows_tensor(residual, "residual", x, (M, N))
    if pre is not None:
        _rows_tensor(pre, "pre", x, (M, N))
    _dev_tensor(workspace, "workspace")
    _check((_lib or _load()).fftconv_linear_fwd(
        x.data_ptr(), W.data_ptr(), _at(bias), _at(residual), out.data_ptr(), _at(pre),
        _row_strides(x, W, residual, out, pre), M, N, K, _activation(activation), _DTYPE_CODE[x.dtype],
        _at(workspace), _nbytes(workspace), _raw_stream(stream, x.device)))


def fftconv_linear_bwd_workspace_bytes(M: int, N: int, K: int, dtype) -> int:
    return int(_load().fftconv_linear_bwd_workspace_bytes(M, N, K, _dtype_of(dtype)))


def fftconv_linear_bwd(dout: torch.Tensor, x: torch.Tensor, W: torch.Tensor, pre: torch.Tensor | None,
                       dx: torch.Tensor | None, dW: torch.Tensor | None, dbias: torch.Tensor | None,
                       activation: str = "none", workspace: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of fftconv_linear_fwd into dx, dW, dbias (None = skip); the residual's is dout."""
    M, N, K = _linear_shapes(x, W)
    for name, t, shape in (("dout", dout, (M, N)), ("pre", pre, (M, N)), ("dx", dx, (M, K)), ("dW", dW, (N, K)),
                           ("dbias", dbias, (N,))):
        if t is not None:
            _rows_tensor(t, name, x, shape)
    _dev_tensor(workspace, "workspace")
    _check((_lib or _load()).fftconv_linear_bwd(
        _at(dout), x.data_ptr(), W.data_ptr(), _at(pre), _at(dx), _at(dW), _at(dbias),
        _row_strides(dout, x, W, pre, dx, dW), M, N, K, _activation(activation), _DTYPE_CODE[x.dtype],
        _at(workspace), _nbytes(workspace), _raw_stream(stream, x.device)))


def linear_act(x, W, bias=None, residual=None, activation="none", keep_pre=False, stream=None):
    """act(x W^T + bias) + residual (allocations by torch); with keep_pre also x W^T + bias for linear_act_bwd."""
    if stream is not None:
        with torch.cuda.stream(stream):      # the scratch memory and the results are that stream's, too
            return linear_act(x, W, bias, residual, activation, keep_pre)
    M, N, K = _linear_shapes(x, W)
    out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    pre = torch.empty_like(out) if keep_pre else None
    ws = _scratch(fftconv_linear_fwd_workspace_bytes(M, N, K, x.dtype), x.device)
    fftconv_linear_fwd(x, W, bias, residual, out, pre, activation, ws)
    return (out, pre) if keep_pre else out


def linear_act_bwd(dout, x, W, pre=None, activation="none", bias=True, stream=None):
    """Gradients of linear_act; returns (dx, dW, dbias), dbias None without a bias."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_act_bwd(dout, x, W, pre, activation, bias)
    M, N, K = _linear_shapes(x, W)
    dx, dW = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (x, W))
    dbias = torch.empty(N, dtype=x.dtype, device=x.device) if bias else None
    ws = _scratch(fftconv_linear_bwd_workspace_bytes(M, N, K, x.dtype), x.device)
    fftconv_linear_bwd(dout, x, W, pre, dx, dW, dbias, activation, ws)
    return dx, dW, dbias


# ---------------------------------------------------------------- gated delta rule
def _delta_shapes(q, k, v, log_decay, beta, cu_seqlens):
    qs, ks, vs = q.shape, k.shape, v.shape
    dims = 4 if cu_seqlens is None else 3
    if len(qs) != dims or len(ks) != dims or len(vs) != dims:
        raise ValueError(f"q, k and v must have {dims} dimensions, not {len(qs)}, {len(ks)} and {len(vs)}")
    H, Hk, Dk, Dv = vs[-2], qs[-2], qs[-1], vs[-1]
    _rows_tensor(q, "q", q, qs)
    _rows_tensor(k, "k", q, qs)
    _rows_tensor(v, "v", q, (*qs[:-2], H, Dv))
    _plain_tensor(log_decay, "log_decay", torch.float32, (*qs[:-2], H), q.device)
    _plain_tensor(beta, "beta", torch.float32, (*qs[:-2], H), q.device)
    if cu_seqlens is None:
        return qs[0], qs[1], H, Hk, Dk, Dv
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold B + 1 values")
    _plain_tensor(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, q.device)
    return cu_seqlens.numel() - 1, qs[0], H, Hk, Dk, Dv


def fftconv_delta_fwd_workspace_bytes(B: int, T: int, H: int, Hk: int, Dk: int, Dv: int, dtype) -> int:
    return int(_load().fftconv_delta_fwd_workspace_bytes(B, T, H, Hk, Dk, Dv, _dtype_of(dtype)))


def fftconv_delta_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, beta: torch.Tensor,
                      out: torch.Tensor, scale: float, state_in: torch.Tensor | None = None,
                      state_out: torch.Tensor | None = None, state_slots: torch.Tensor | None = None,
                      cu_seqlens: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> None:
    """out <- gated delta rule over q, k (B, N, Hk, Dk), v (B, N, H, Dv), or packed (T, heads, width) with cu_seqlens.

    log_decay, beta: fp32 (B, N, H).  state_in / state_out: fp32 (B, H, Dk, Dv), or pools of such matrices with
    state_slots (B) int32.
    """
    B, N, H, Hk, Dk, Dv = _delta_shapes(q, k, v, log_decay, beta, cu_seqlens)
    _rows_tensor(out, "out", q, v.shape)
    n_slots, device = 0, q.device
    if state_slots is not None:
        _plain_tensor(state_slots, "state_slots", torch.int32, (B,), device)
        pool = state_in if state_in is not None else state_out
        n_slots = pool.shape[0] if pool is not None else 0
    states = (B if state_slots is None else n_slots, H, Dk, Dv)
    _plain_tensor(state_in, "state_in", torch.float32, states, device)
    _plain_tensor(state_out, "state_out", torch.float32, states, device)
    _dev_tensor(workspace, "workspace")
    with _on(device):
        _check((_lib or _load()).fftconv_delta_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), beta.data_ptr(), out.data_ptr(),
            _strides((q, k, v, out), cu_seqlens is not None), _at(state_in), _at(state_out), _at(state_slots), n_slots,
            _at(cu_seqlens), B, N, H, Hk, Dk, Dv, scale, _DTYPE_CODE[q.dtype], _at(workspace), _nbytes(workspace),
            _raw_stream(stream, device)))


def fftconv_delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, beta: torch.Tensor,
                       state: torch.Tensor, out: torch.Tensor, scale: float, state_slots: torch.Tensor | None = None,
                       stream=None) -> None:
    """One token of each sequence: q, k (B, Hk, Dk), v (B, H, Dv), log_decay, beta (B, H) -> out, state in place."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and v must have 3 dimensions")
    (B, Hk, Dk), (_, H, Dv), device = q.shape, v.shape, q.device
    _rows_tensor(q, "q", q, (B, Hk, Dk))
    _rows_tensor(k, "k", q, (B, Hk, Dk))
    _rows_tensor(v, "v", q, (B, H, Dv))
    _rows_tensor(out, "out", q, (B, H, Dv))
    _plain_tensor(log_decay, "log_decay", torch.float32, (B, H), device)
    _plain_tensor(beta, "beta", torch.float32, (B, H), device)
    n_slots = 0
    if state_slots is not None:
        _plain_tensor(state_slots, "state_slots", torch.int32, (B,), device)
        n_slots = state.shape[0]
    _plain_tensor(state, "state", torch.float32, (B if state_slots is None else n_slots, H, Dk, Dv), device)
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous()):
        strides = _strides_of[8](*q.stride()[:2], *k.stride()[:2], *v.stride()[:2], *out.stride()[:2])
    with _on(device):
        _check((_lib or _load()).fftconv_delta_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), beta.data_ptr(), state.data_ptr(),
            out.data_ptr(), strides, _at(state_slots), n_slots, B, H, Hk, Dk, Dv, scale, _DTYPE_CODE[q.dtype],
            _raw_stream(stream, device)))


def delta_attention(q, k, v, log_decay, beta, scale=None, state_in=None, cu_seqlens=None, stream=None):
    """Gated delta rule over whole sequences (allocations by torch); returns (out, final states).  scale: Dk^-0.5.

    Packed tokens of no sequence (before cu_seqlens[0], from its last value on) have no result: their rows are not set.
    """
    if stream is not None:
        with torch.cuda.stream(stream):      # the scratch memory and the results are that stream's, too
            return delta_attention(q, k, v, log_decay, beta, scale, state_in, cu_seqlens)
    B, N, H, Hk, Dk, Dv = _delta_shapes(q, k, v, log_decay, beta, cu_seqlens)
    T = N if cu_seqlens is not None else B * N
    out = torch.empty(v.shape, dtype=q.dtype, device=q.device)
    state_out = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device)
    ws = _scratch(fftconv_delta_fwd_workspace_bytes(B, T, H, Hk, Dk, Dv, q.dtype), q.device)
    fftconv_delta_fwd(q, k, v, log_decay, beta, out, Dk ** -0.5 if scale is None else scale, state_in, state_out,
                      cu_seqlens=cu_seqlens, workspace=ws)
    return out, state_out


def fftconv_delta_bwd_workspace_bytes(B: int, T: int, H: int, Hk: int, Dk: int, Dv: int, dtype) -> int:
    return int(_load().fftconv_delta_bwd_workspace_bytes(B, T, H, Hk, Dk, Dv, _dtype_of(dtype)))


def fftconv_delta_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                      beta: torch.Tensor, dq: torch.Tensor | None, dk: torch.Tensor | None, dv: torch.Tensor | None,
                      dlog_decay: torch.Tensor | None, dbeta: torch.Tensor | None, scale: float,
                      state_in: torch.Tensor | None = None, dstate_out: torch.Tensor | None = None,
                      dstate_in: torch.Tensor | None = None, cu_seqlens: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of fftconv_delta_fwd into dq, dk, dv, dlog_decay, dbeta, dstate_in (None = skip)."""
    B, N, H, Hk, Dk, Dv = _delta_shapes(q, k, v, log_decay, beta, cu_seqlens)
    _rows_tensor(dout, "dout", q, v.shape)
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _rows_tensor(t, name, q, like.shape)
    for name, t in (("dlog_decay", dlog_decay), ("dbeta", dbeta)):
        _plain_tensor(t, name, torch.float32, log_decay.shape, q.device)
    for name, t in (("state_in", state_in), ("dstate_out", dstate_out), ("dstate_in", dstate_in)):
        _plain_tensor(t, name, torch.float32, (B, H, Dk, Dv), q.device)
    _dev_tensor(workspace, "workspace")
    with _on(q.device):
        _check((_lib or _load()).fftconv_delta_bwd(
            dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), beta.data_ptr(), _at(dq),
            _at(dk), _at(dv), _at(dlog_decay), _at(dbeta), _strides((dout, q, k, v, dq, dk, dv), cu_seqlens is not None),
            _at(state_in), _at(dstate_out), _at(dstate_in), _at(cu_seqlens), B, N, H, Hk, Dk, Dv, scale,
            _DTYPE_CODE[q.dtype], _at(workspace), _nbytes(workspace), _raw_stream(stream, q.device)))


def delta_attention_bwd(q, k, v, log_decay, beta, dout, scale=None, state_in=None, dstate_out=None, cu_seqlens=None,
                        stream=None):
    """Gradients of delta_attention; returns (dq, dk, dv, dlog_decay, dbeta, dstate_in), the last None without state_in.

    Rows of packed tokens that belong to no sequence are not set.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return delta_attention_bwd(q, k, v, log_decay, beta, dout, scale, state_in, dstate_out, cu_seqlens)
    B, N, H, Hk, Dk, Dv = _delta_shapes(q, k, v, log_decay, beta, cu_seqlens)
    T = N if cu_seqlens is not None else B * N
    grads = [torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v, log_decay, beta)]
    dstate_in = None if state_in is None else torch.empty_like(state_in)
    ws = _scratch(fftconv_delta_bwd_workspace_bytes(B, T, H, Hk, Dk, Dv, q.dtype), q.device)
    fftconv_delta_bwd(dout, q, k, v, log_decay, beta, *grads, Dk ** -0.5 if scale is None else scale, state_in,
                      dstate_out, dstate_in, cu_seqlens, ws)
    return (*grads, dstate_in)


# ---------------------------------------------------------------- root-mean-square norm
def _on(device):
    """The tensors' device as the current one for the call (the library launches on the current device)."""
    return torch.cuda.device(device) if device.index != torch.cuda.current_device() else _here


_here = contextlib.nullcontext()


def _row_groups(shape, tensors):
    """M, G, D of rows (..., D) and the (row, group) strides of each tensor, None where all are dense.

    Leading dimensions beyond two are folded where every tensor's strides allow it.
    """
    D, lead = shape[-1], tuple(shape[:-1])
    M = math.prod(lead)
    if all(t is None or t.is_contiguous() for t in tensors):
        return M, 1, D, None
    if M == 0:
        return M, 1, D, None
    dims = [i for i, n in enumerate(lead) if n != 1]
    # an outer run of dimensions and an inner one, each of which steps evenly in every tensor
    def runs(t):
        return {j for j in range(1, len(dims)) if t.stride(dims[j - 1]) != t.stride(dims[j]) * lead[dims[j]]}

    cuts = set().union(*(runs(t) for t in tensors if t is not None))
    if len(cuts) > 1:
        raise ValueError("leading dimensions must fold into two evenly strided ones")
    cut = cuts.pop() if cuts else 0
    outer, inner = dims[:cut], dims[cut:]
    G = math.prod(lead[i] for i in inner)
    flat = []
    for t in tensors:
        if t is None:
            flat += (0, 0)
        else:
            flat += (t.stride(outer[-1]) if outer else 0, t.stride(inner[-1]) if inner else 0)
    return M // max(G, 1), G, D, _strides_of[8](*flat)


def _weight_tensor(t, name, x):
    if t is not None:
        _plain_tensor(t, name, x.dtype, (x.shape[-1],), x.device)


def fftconv_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None, out: torch.Tensor, eps: float,
                     residual: torch.Tensor | None = None, sum: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, stream=None) -> None:
    """out <- (x + residual) / rms * weight over the last dimension; sum (optional) <- x + residual.

    With scales (fp32, one a row) out is torch.float8_e4m3fn and holds y / scale.
    """
    _rows_tensor(x, "x", x, x.shape)
    if x.dim() == 0:
        raise ValueError("x must have a dimension")
    _weight_tensor(weight, "weight", x)
    for name, t in (("residual", residual), ("sum", sum)):
        if t is not None:
            _rows_tensor(t, name, x, x.shape)
    if scales is None:
        _rows_tensor(out, "out", x, x.shape)
    else:
        _plain_tensor(scales, "scales", torch.float32, x.shape[:-1], x.device)
        if out.dtype is not torch.float8_e4m3fn:
            raise ValueError(f"out must have dtype {torch.float8_e4m3fn} with scales")
        if out.device != x.device or out.shape != x.shape or (out.stride(-1) != 1 and out.shape[-1] > 1):
            raise ValueError(f"out must be on {x.device}, of shape {tuple(x.shape)}, contiguous along its last dimension")
    M, G, D, strides = _row_groups(x.shape, (x, residual, out, sum))
    with _on(x.device):
        _check((_lib or _load()).fftconv_norm_fwd(
            x.data_ptr(), _at(residual), _at(weight), out.data_ptr(), _at(sum), _at(scales), strides, M, G, D, eps,
            _DTYPE_CODE[x.dtype], _raw_stream(stream, x.device)))


def fftconv_norm_bwd_workspace_bytes(rows: int, D: int) -> int:
    return int(_load().fftconv_norm_bwd_workspace_bytes(rows, D))


def fftconv_norm_bwd(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None, dx: torch.Tensor | None,
                     dweight: torch.Tensor | None, eps: float, dsum: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of fftconv_norm_fwd into dx and dweight (None = skip); x is the sum that was normed, dsum its own gradient."""
    _rows_tensor(x, "x", x, x.shape)
    if x.dim() == 0:
        raise ValueError("x must have a dimension")
    _weight_tensor(weight, "weight", x)
    _weight_tensor(dweight, "dweight", x)
    for name, t in (("dout", dout), ("dx", dx), ("dsum", dsum)):
        if t is not None:
            _rows_tensor(t, name, x, x.shape)
    _dev_tensor(workspace, "workspace")
    M, G, D, strides = _row_groups(x.shape, (dout, x, dsum, dx))
    with _on(x.device):
        _check((_lib or _load()).fftconv_norm_bwd(
            dout.data_ptr(), x.data_ptr(), _at(weight), _at(dsum), _at(dx), _at(dweight), strides, M, G, D, eps,
            _DTYPE_CODE[x.dtype], _at(workspace), _nbytes(workspace), _raw_stream(stream, x.device)))


def rms_norm(x, weight=None, eps=1e-6, residual=None, eight_bits=False, stream=None):
    """(x + residual) / rms * weight over the last dimension (allocations by torch).

    Returns out, with eight_bits out (float8_e4m3fn) and its scales, and with a residual x + residual behind them.
    """
    if stream is not None:
        with torch.cuda.stream(stream):      # the results are that stream's, too
            return rms_norm(x, weight, eps, residual, eight_bits)
    _rows_tensor(x, "x", x, x.shape)
    out = torch.empty(x.shape, dtype=torch.float8_e4m3fn if eight_bits else x.dtype, device=x.device)
    scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if eight_bits else None
    total = torch.empty(x.shape, dtype=x.dtype, device=x.device) if residual is not None else None
    fftconv_norm_fwd(x, weight, out, eps, residual, total, scales)
    got = [t for t in (out, scales, total) if t is not None]
    return got[0] if len(got) == 1 else tuple(got)


def rms_norm_bwd(dout, x, weight=None, eps=1e-6, dsum=None, stream=None):
    """Gradients of rms_norm, x being the sum that it normed; returns (dx, dweight), dweight None without a weight."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rms_norm_bwd(dout, x, weight, eps, dsum)
    _rows_tensor(x, "x", x, x.shape)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dweight = None if weight is None else torch.empty_like(weight)
    ws = _scratch(fftconv_norm_bwd_workspace_bytes(x.numel() // max(1, x.shape[-1]), x.shape[-1]), x.device)
    fftconv_norm_bwd(dout, x, weight, dx, dweight, eps, dsum, ws)
    return dx, dweight


def alloc_filter(H: int, N: int, dtype: torch.dtype, device="cuda") -> torch.Tensor:
    """Device buffer for K_f (torch allocation; the library never allocates it)."""
    return torch.empty(fftconv_filter_bytes(H, N, dtype), dtype=torch.uint8, device=device)


def alloc_workspace(B: int, H: int, N: int, dtype: torch.dtype, device="cuda"):
    n = fftconv_workspace_bytes(B, H, N, dtype)
    return None if n == 0 else torch.empty(n, dtype=torch.uint8, device=device)


def causal_conv(u, k, w=None, v=None, sparsity_mask=None, stream=None):
    """Prepare k and run one forward call (allocations by torch)."""
    B, H, N = u.shape
    L = k.shape[1]
    K_f = alloc_filter(H, N, u.dtype, u.device)
    ws_p = alloc_workspace(1, H, N, u.dtype, u.device)
    fftconv_prepare_filter(k, N, K_f, ws_p, stream)
    ws = alloc_workspace(B, H, N, u.dtype, u.device)
    out = torch.empty_like(u)
    fftconv_fwd(u, K_f, w, v, out, L, sparsity_mask, ws, stream)
    return out


def causal_conv_bwd(u, k, dy, w=None, v=None, sparsity_mask=None, stream=None):
    """Prepare k and run one backward call; returns (du, dk, dw, dv), None for absent gates."""
    B, H, N = u.shape
    L = k.shape[1]
    K_f = alloc_filter(H, N, u.dtype, u.device)
    ws_p = alloc_workspace(1, H, N, u.dtype, u.device)
    fftconv_prepare_filter(k, N, K_f, ws_p, stream)
    ws = torch.empty(fftconv_bwd_workspace_bytes(B, H, N, u.dtype), dtype=torch.uint8, device=u.device)
    du = torch.empty_like(u)
    dk = torch.empty((H, L), dtype=u.dtype, device=u.device)
    dw = torch.empty_like(u) if w is not None else None
    dv = torch.empty_like(u) if v is not None else None
    fftconv_bwd(dy, u, K_f, w, v, du, dk, dw, dv, L, sparsity_mask, ws, stream)
    return du, dk, dw, dv
