"""Python binding of ``liblh.so``, the MI355X local-Hessian NVFP4 weight-scale calibration library and
the decode-step operators on the formats it calibrates.

The functions carry the names of the C entry points in ``include/lh.h`` and only marshal
arguments: they check dtypes, shapes and devices of torch tensors, allocate missing outputs with
torch, and pass raw device pointers plus torch's current HIP stream to the library.  Every step of
the computation runs in the HIP kernels.  Importing this package fails loudly when the library has
not been built (``python -m nvfp4_scale_calibration_lh_amd.build``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# The library built next to this file; LH_LIBRARY may name another build of the same library.
LIB_PATH = os.environ.get("LH_LIBRARY") or os.path.join(_PKG, "liblh.so")

LH_OK, LH_ERR_INVALID_ARGUMENT, LH_ERR_UNSUPPORTED, LH_ERR_HIP = 0, 1, 2, 3
LH_DTYPE_F32, LH_DTYPE_BF16, LH_DTYPE_E4M3 = 0, 1, 2
LH_CACHE_E4M3, LH_CACHE_FP4 = 0, 1

EXPORTED = ("lh_accumulate", "lh_accumulate_noalloc", "lh_accumulate_act_aware", "lh_accumulate_act_aware_fq", "lh_activation_fake_quant",
            "lh_accumulate_sweep", "lh_dequantize", "lh_dequantize_ex", "lh_scale_sweep", "lh_scale_sweep_ex", "lh_scale_sweep_diag",
            "lh_scale_sweep_diag_ex", "lh_scale_sweep_mse", "lh_absmax", "lh_rms_norm_quant", "lh_matvec", "lh_cache_write",
            "lh_cache_read", "lh_paged_attention", "lh_paged_attention_workspace", "lh_last_error", "lh_version")
MAX_MULTIPLIERS = 128


class SweepOptions(ctypes.Structure):
    """lh_sweep_options: scale_norm (448 or 256 for "4/6"), the amax multipliers (host array)."""
    _fields_ = [("scale_norm", ctypes.c_float), ("n_multipliers", ctypes.c_int32),
                ("multipliers", ctypes.POINTER(ctypes.c_float))]


class CacheStruct(ctypes.Structure):
    """lh_cache: the format, sizes and device pointers of a paged key-value cache."""
    _fields_ = ([("format", ctypes.c_int)] + [(n, ctypes.c_int64) for n in ("n_pages", "page_size", "n_heads", "head_dim")]
                + [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "k_amax", "v_amax")])


class LHError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"liblh error {code}: {message}")
        self.code = code
        self.message = message


_lib_handle = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it is missing)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m nvfp4_scale_calibration_lh_amd.build`")
        h = ctypes.CDLL(LIB_PATH)
        vp, i64, f32, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
        h.lh_accumulate.argtypes = [vp, i32, i64, i64, vp, i64, f32, vp, vp, vp]
        h.lh_accumulate_noalloc.argtypes = [vp, i32, i64, i64, vp, i64, f32, vp, vp, vp]
        h.lh_accumulate_act_aware.argtypes = [vp, vp, i32, i64, i64, vp, i64, f32, vp, vp, vp]
        h.lh_accumulate_act_aware_fq.argtypes = [vp, i32, i64, i64, vp, i64, vp, f32, vp, vp, vp]
        h.lh_activation_fake_quant.argtypes = [vp, i32, i64, i64, vp, i64, vp, vp, vp]
        h.lh_scale_sweep.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp]
        h.lh_scale_sweep_diag.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, vp]
        h.lh_scale_sweep_ex.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]
        h.lh_scale_sweep_diag_ex.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp]
        h.lh_dequantize_ex.argtypes = [vp, vp, i32, i64, i64, i64, vp, f32, vp, vp, vp]
        h.lh_accumulate_sweep.argtypes = [vp, vp, i32, i64, i64, vp, i64, i64, vp, vp, vp, vp, vp, vp]
        h.lh_scale_sweep_mse.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, vp]
        h.lh_absmax.argtypes = [vp, i32, i64, i64, vp, vp]
        h.lh_dequantize.argtypes = [vp, vp, i32, i64, i64, i64, vp, vp, vp, vp]
        h.lh_rms_norm_quant.argtypes = [vp, vp, i32, i64, i64, vp, f32, i64, vp, vp, vp, vp]
        h.lh_matvec.argtypes = [vp, i32, vp, i64, i64, i64, vp, i64, i64, vp, vp, vp, f32, vp, vp]
        h.lh_cache_write.argtypes = [vp, vp, i64, vp, i64, i32, i64, vp, vp]
        h.lh_cache_read.argtypes = [vp, vp, i64, i32, vp, vp, vp]
        h.lh_paged_attention.argtypes = [vp, vp, i64, i32, i64, i64, vp, i64, vp, f32, vp, vp, i64, vp]
        h.lh_paged_attention_workspace.argtypes = [vp, i64, i64, i64]
        for f in ("lh_accumulate", "lh_accumulate_noalloc", "lh_accumulate_act_aware", "lh_accumulate_act_aware_fq",
                  "lh_activation_fake_quant", "lh_scale_sweep", "lh_scale_sweep_ex", "lh_scale_sweep_diag_ex",
                  "lh_dequantize_ex", "lh_accumulate_sweep",
                  "lh_scale_sweep_diag", "lh_scale_sweep_mse", "lh_absmax", "lh_dequantize", "lh_rms_norm_quant",
                  "lh_matvec", "lh_cache_write", "lh_cache_read", "lh_paged_attention"):
            getattr(h, f).restype = ctypes.c_int
        h.lh_paged_attention_workspace.restype = ctypes.c_int64
        h.lh_last_error.argtypes = []
        h.lh_last_error.restype = ctypes.c_char_p
        h.lh_version.argtypes = []
        h.lh_version.restype = ctypes.c_int
        _lib_handle = h
    return _lib_handle


def lh_last_error() -> str:
    return lib().lh_last_error().decode()


def lh_version() -> int:
    return int(lib().lh_version())


def _check(code: int):
    if code != LH_OK:
        raise LHError(code, lh_last_error())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LH_DTYPE_BF16
    if t.dtype == torch.float32:
        return LH_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    """Handle of torch's current stream on the device (0.1 us; the torch.cuda.Stream object costs 1.8 us a call)."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device.index is None else device.index)


def _need(t: torch.Tensor, name: str, shape=None, dtype=None):
    if t.is_cuda and (shape is None or t.shape == shape) and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _offsets(offsets: Optional[torch.Tensor], X: torch.Tensor):
    if offsets is None:
        return None, 1
    _need(offsets, "offsets", dtype=torch.int64)
    return offsets, offsets.numel() - 1


def lh_accumulate(X: torch.Tensor, H: Optional[torch.Tensor] = None, imp: Optional[torch.Tensor] = None,
                  offsets: Optional[torch.Tensor] = None, beta: float = 0.0, *, want_h: bool = True,
                  want_imp: bool = False) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Per-block Hessian H [G, cin/16, 16, 16] and importance imp [G, cin] of X [rows, cin]."""
    _need(X, "X")
    rows, cin = X.shape
    offsets, G = _offsets(offsets, X)
    if H is None and want_h:
        H = torch.empty((G, cin // 16, 16, 16), dtype=torch.float32, device=X.device)
    if imp is None and want_imp:
        imp = torch.empty((G, cin), dtype=torch.float32, device=X.device)
    if H is not None:
        _need(H, "H", (G, cin // 16, 16, 16), torch.float32)
    if imp is not None:
        _need(imp, "imp", (G, cin), torch.float32)
    _check(lib().lh_accumulate(_ptr(X), _dtype_code(X), rows, cin, _ptr(offsets), G, float(beta),
                               _ptr(H), _ptr(imp), _stream(X.device)))
    return H, imp


def lh_accumulate_noalloc(X: torch.Tensor, H: torch.Tensor = None, imp: Optional[torch.Tensor] = None,
                          offsets: Optional[torch.Tensor] = None, beta: float = 0.0):
    """lh_accumulate that allocates nothing (no output allocation here either: H and/or imp are
    required), its scratch in the library's fixed per-device array; overlapping calls on one
    device race."""
    _need(X, "X")
    rows, cin = X.shape
    offsets, G = _offsets(offsets, X)
    if H is None and imp is None:
        raise ValueError("H and/or imp must be given")
    if H is not None:
        _need(H, "H", (G, cin // 16, 16, 16), torch.float32)
    if imp is not None:
        _need(imp, "imp", (G, cin), torch.float32)
    _check(lib().lh_accumulate_noalloc(_ptr(X), _dtype_code(X), rows, cin, _ptr(offsets), G, float(beta),
                                       _ptr(H), _ptr(imp), _stream(X.device)))
    return H, imp


def lh_accumulate_act_aware(X: torch.Tensor, Xq: torch.Tensor, H: Optional[torch.Tensor] = None,
                            P: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                            beta: float = 0.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """H = X_q^T X_q / T and P = X_q^T (X_q - X) / T per 16-channel block."""
    _need(X, "X")
    _need(Xq, "Xq", X.shape, X.dtype)
    rows, cin = X.shape
    offsets, G = _offsets(offsets, X)
    shape = (G, cin // 16, 16, 16)
    if H is None:
        H = torch.empty(shape, dtype=torch.float32, device=X.device)
    if P is None:
        P = torch.empty(shape, dtype=torch.float32, device=X.device)
    _need(H, "H", shape, torch.float32)
    _need(P, "P", shape, torch.float32)
    _check(lib().lh_accumulate_act_aware(_ptr(X), _ptr(Xq), _dtype_code(X), rows, cin, _ptr(offsets), G,
                                         float(beta), _ptr(H), _ptr(P), _stream(X.device)))
    return H, P


def lh_accumulate_act_aware_fq(X: torch.Tensor, x_amax: torch.Tensor, H: Optional[torch.Tensor] = None,
                               P: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                               beta: float = 0.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """As lh_accumulate_act_aware, with X_q the NVFP4 fake-quant of X made in the kernel from the
    input quantizer's amax per group (x_amax [G] fp32)."""
    _need(X, "X")
    rows, cin = X.shape
    offsets, G = _offsets(offsets, X)
    _need(x_amax, "x_amax", (G,), torch.float32)
    shape = (G, cin // 16, 16, 16)
    if H is None:
        H = torch.empty(shape, dtype=torch.float32, device=X.device)
    if P is None:
        P = torch.empty(shape, dtype=torch.float32, device=X.device)
    _need(H, "H", shape, torch.float32)
    _need(P, "P", shape, torch.float32)
    _check(lib().lh_accumulate_act_aware_fq(_ptr(X), _dtype_code(X), rows, cin, _ptr(offsets), G, _ptr(x_amax),
                                            float(beta), _ptr(H), _ptr(P), _stream(X.device)))
    return H, P


def lh_activation_fake_quant(X: torch.Tensor, x_amax: torch.Tensor, Xq: Optional[torch.Tensor] = None,
                             offsets: Optional[torch.Tensor] = None) -> torch.Tensor:
    """X_q [rows, cin]: the NVFP4 fake-quant of X with the input quantizer's amax per group
    (x_amax [G] fp32), as lh_accumulate_act_aware_fq applies it inside its kernel."""
    _need(X, "X")
    rows, cin = X.shape
    offsets, G = _offsets(offsets, X)
    _need(x_amax, "x_amax", (G,), torch.float32)
    if Xq is None:
        Xq = torch.empty_like(X)
    _need(Xq, "Xq", X.shape, X.dtype)
    _check(lib().lh_activation_fake_quant(_ptr(X), _dtype_code(X), rows, cin, _ptr(offsets), G, _ptr(x_amax),
                                          _ptr(Xq), _stream(X.device)))
    return Xq


def _sweep_outputs(W, code, fp4, loss, want_fp4, want_loss):
    G, cout, cin = W.shape
    dev = W.device
    if code is None:
        code = torch.empty((G, cout, cin // 16), dtype=torch.uint8, device=dev)
    if fp4 is None and want_fp4:
        fp4 = torch.empty((G, cout, cin // 2), dtype=torch.uint8, device=dev)
    if loss is None and want_loss:
        loss = torch.empty((G, cout, cin // 16), dtype=torch.float32, device=dev)
    _need(code, "code", (G, cout, cin // 16), torch.uint8)
    if fp4 is not None:
        _need(fp4, "fp4", (G, cout, cin // 2), torch.uint8)
    if loss is not None:
        _need(loss, "loss", (G, cout, cin // 16), torch.float32)
    return code, fp4, loss


def _as3d(W: torch.Tensor) -> torch.Tensor:
    return W.unsqueeze(0) if W.dim() == 2 else W


def lh_scale_sweep(W: torch.Tensor, amax: torch.Tensor, H: torch.Tensor, P: Optional[torch.Tensor] = None,
                   code: Optional[torch.Tensor] = None, fp4: Optional[torch.Tensor] = None,
                   loss: Optional[torch.Tensor] = None, *, want_fp4: bool = True, want_loss: bool = True):
    """126-candidate E4M3 scale sweep scored by e^T H e + 2 e^T (P w): (code, fp4, loss)."""
    W = _as3d(W)
    _need(W, "W")
    G, cout, cin = W.shape
    _need(amax, "amax", (G,), torch.float32)
    _need(H, "H", (G, cin // 16, 16, 16), torch.float32)
    if P is not None:
        _need(P, "P", (G, cin // 16, 16, 16), torch.float32)
    code, fp4, loss = _sweep_outputs(W, code, fp4, loss, want_fp4, want_loss)
    _check(lib().lh_scale_sweep(_ptr(W), _dtype_code(W), G, cout, cin, _ptr(amax), _ptr(H), _ptr(P),
                                _ptr(code), _ptr(fp4), _ptr(loss), _stream(W.device)))
    return code, fp4, loss


def lh_scale_sweep_diag(W: torch.Tensor, amax: torch.Tensor, imp: torch.Tensor,
                        code: Optional[torch.Tensor] = None, fp4: Optional[torch.Tensor] = None,
                        loss: Optional[torch.Tensor] = None, *, want_fp4: bool = True, want_loss: bool = True):
    """126-candidate E4M3 scale sweep scored by sum_i imp_i e_i^2: (code, fp4, loss)."""
    W = _as3d(W)
    _need(W, "W")
    G, cout, cin = W.shape
    _need(amax, "amax", (G,), torch.float32)
    _need(imp, "imp", (G, cin), torch.float32)
    code, fp4, loss = _sweep_outputs(W, code, fp4, loss, want_fp4, want_loss)
    _check(lib().lh_scale_sweep_diag(_ptr(W), _dtype_code(W), G, cout, cin, _ptr(amax), _ptr(imp),
                                     _ptr(code), _ptr(fp4), _ptr(loss), _stream(W.device)))
    return code, fp4, loss


def lh_scale_sweep_mse(W: torch.Tensor, amax: torch.Tensor, code: Optional[torch.Tensor] = None,
                       fp4: Optional[torch.Tensor] = None, loss: Optional[torch.Tensor] = None, *,
                       want_fp4: bool = True, want_loss: bool = True):
    """126-candidate E4M3 scale sweep scored by the plain sum_i e_i^2: (code, fp4, loss)."""
    W = _as3d(W)
    _need(W, "W")
    G, cout, cin = W.shape
    _need(amax, "amax", (G,), torch.float32)
    code, fp4, loss = _sweep_outputs(W, code, fp4, loss, want_fp4, want_loss)
    _check(lib().lh_scale_sweep_mse(_ptr(W), _dtype_code(W), G, cout, cin, _ptr(amax),
                                    _ptr(code), _ptr(fp4), _ptr(loss), _stream(W.device)))
    return code, fp4, loss


def _options(norm: float, multipliers):
    """(ctypes options, keep-alive array) for the *_ex entry points."""
    import array
    m = array.array("f", [] if multipliers is None else [float(x) for x in multipliers])
    buf = (ctypes.c_float * max(1, len(m)))(*m) if len(m) else None
    opt = SweepOptions(float(norm), len(m), ctypes.cast(buf, ctypes.POINTER(ctypes.c_float)) if buf else None)
    return opt, buf


def lh_scale_sweep_ex(W: torch.Tensor, amax: torch.Tensor, H: torch.Tensor, P: Optional[torch.Tensor] = None,
                      code: Optional[torch.Tensor] = None, fp4: Optional[torch.Tensor] = None,
                      loss: Optional[torch.Tensor] = None, *, norm: float = 448.0, multipliers=None,
                      want_fp4: bool = True, want_loss: bool = True):
    """lh_scale_sweep with the global scale normalized to `norm` (448, or 256 for "4/6") and, when
    `multipliers` is given (at most 128 positive values), the amax-multiplier search."""
    W = _as3d(W)
    _need(W, "W")
    G, cout, cin = W.shape
    _need(amax, "amax", (G,), torch.float32)
    _need(H, "H", (G, cin // 16, 16, 16), torch.float32)
    if P is not None:
        _need(P, "P", (G, cin // 16, 16, 16), torch.float32)
    code, fp4, loss = _sweep_outputs(W, code, fp4, loss, want_fp4, want_loss)
    opt, keep = _options(norm, multipliers)
    _check(lib().lh_scale_sweep_ex(_ptr(W), _dtype_code(W), G, cout, cin, _ptr(amax), _ptr(H), _ptr(P),
                                   ctypes.byref(opt), _ptr(code), _ptr(fp4), _ptr(loss), _stream(W.device)))
    del keep
    return code, fp4, loss


def lh_accumulate_sweep(X: torch.Tensor, W: torch.Tensor, amax: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                        code: Optional[torch.Tensor] = None, fp4: Optional[torch.Tensor] = None,
                        loss: Optional[torch.Tensor] = None, *, norm: float = 448.0, multipliers=None,
                        want_fp4: bool = True, want_loss: bool = True):
    """Per-expert Hessians of X's grouped rows and the scale search of W [G, cout, cin] against
    them in one launch, H never written to memory: (code, fp4, loss) as lh_scale_sweep_ex."""
    _need(X, "X")
    W = _as3d(W)
    _need(W, "W")
    rows, cin = X.shape
    offsets, G = _offsets(offsets, X)
    if W.shape[0] != G or W.shape[2] != cin or W.dtype != X.dtype:
        raise ValueError(f"W must be [{G}, cout, {cin}] of X's dtype")
    _need(amax, "amax", (G,), torch.float32)
    code, fp4, loss = _sweep_outputs(W, code, fp4, loss, want_fp4, want_loss)
    opt, keep = _options(norm, multipliers)
    _check(lib().lh_accumulate_sweep(_ptr(X), _ptr(W), _dtype_code(X), rows, cin, _ptr(offsets), G, W.shape[1],
                                     _ptr(amax), ctypes.byref(opt), _ptr(code), _ptr(fp4), _ptr(loss),
                                     _stream(X.device)))
    del keep
    return code, fp4, loss


def lh_scale_sweep_diag_ex(W: torch.Tensor, amax: torch.Tensor, imp: Optional[torch.Tensor],
                           code: Optional[torch.Tensor] = None, fp4: Optional[torch.Tensor] = None,
                           loss: Optional[torch.Tensor] = None, *, norm: float = 448.0, multipliers=None,
                           want_fp4: bool = True, want_loss: bool = True):
    """lh_scale_sweep_diag (imp None: plain MSE) with the options of lh_scale_sweep_ex."""
    W = _as3d(W)
    _need(W, "W")
    G, cout, cin = W.shape
    _need(amax, "amax", (G,), torch.float32)
    if imp is not None:
        _need(imp, "imp", (G, cin), torch.float32)
    code, fp4, loss = _sweep_outputs(W, code, fp4, loss, want_fp4, want_loss)
    opt, keep = _options(norm, multipliers)
    _check(lib().lh_scale_sweep_diag_ex(_ptr(W), _dtype_code(W), G, cout, cin, _ptr(amax), _ptr(imp),
                                        ctypes.byref(opt), _ptr(code), _ptr(fp4), _ptr(loss), _stream(W.device)))
    del keep
    return code, fp4, loss


def lh_dequantize(code: torch.Tensor, fp4: torch.Tensor, amax: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                  Wq: Optional[torch.Tensor] = None, block_amax: Optional[torch.Tensor] = None,
                  want_wq: bool = True, want_block_amax: bool = True, norm: float = 448.0):
    """Fake-quantized weights Wq [G, cout, cin] (bf16 or fp32) and per-block amax [G, cout, cin/16]
    from the sweep's scale codes and FP4 nibbles (norm: the sweep's scale normalization, through
    lh_dequantize_ex when it is not 448)."""
    if code.dim() != 3:
        raise ValueError("code must be [G, cout, cin/16]")
    G, cout, nb = code.shape
    cin = nb * 16
    _need(code, "code", (G, cout, nb), torch.uint8)
    _need(fp4, "fp4", (G, cout, cin // 2), torch.uint8)
    _need(amax, "amax", (G,), torch.float32)
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    if Wq is None and want_wq:
        Wq = torch.empty((G, cout, cin), dtype=dtype, device=code.device)
    if block_amax is None and want_block_amax:
        block_amax = torch.empty((G, cout, nb), dtype=torch.float32, device=code.device)
    if Wq is not None:
        _need(Wq, "Wq", (G, cout, cin), dtype)
    if block_amax is not None:
        _need(block_amax, "block_amax", (G, cout, nb), torch.float32)
    if norm == 448.0:
        _check(lib().lh_dequantize(_ptr(code), _ptr(fp4), 1 if dtype == torch.bfloat16 else 0, G, cout, cin,
                                   _ptr(amax), _ptr(Wq), _ptr(block_amax), _stream(code.device)))
    else:
        _check(lib().lh_dequantize_ex(_ptr(code), _ptr(fp4), 1 if dtype == torch.bfloat16 else 0, G, cout, cin,
                                      _ptr(amax), float(norm), _ptr(Wq), _ptr(block_amax), _stream(code.device)))
    return Wq, block_amax


def lh_absmax(W: torch.Tensor, amax: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Per-group max |W| for W [G, ...] (a 2-D W is one group)."""
    W = _as3d(W) if W.dim() == 2 else W
    _need(W, "W")
    G = W.shape[0]
    per = W.numel() // G if G else 0
    if amax is None:
        amax = torch.empty((G,), dtype=torch.float32, device=W.device)
    _need(amax, "amax", (G,), torch.float32)
    _check(lib().lh_absmax(_ptr(W), _dtype_code(W), G, per, _ptr(amax), _stream(W.device)))
    return amax


def _scales(cin: int, group: int) -> int:
    """Scales of one row of cin channels."""
    if group == 0:
        return 1
    if group != 128:
        raise ValueError("the group of a scale must be 0 (the row) or 128")
    return (cin + 127) // 128


# New outputs are made with empty(*sizes) or empty_like, the cheapest of torch's forms, and only outputs that the
# caller gave are checked: at one token these calls are bound by the host.
_empty = torch.empty


def lh_rms_norm_quant(X: torch.Tensor, gamma: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
                      eps: float = 1e-6, group: int = 0, q: Optional[torch.Tensor] = None,
                      scale: Optional[torch.Tensor] = None, summed: Optional[torch.Tensor] = None):
    """(q, scale, summed): the RMS norm of X + residual times gamma, X [rows, cin], as E4M3 q [rows, cin]
    (torch.float8_e4m3fn) with scale [rows, 1], or [rows, ceil(cin/128)] for group = 128, and the
    sum itself in X's dtype (None without a residual; it may be X or residual for an update in place)."""
    _need(X, "X")
    if X.dim() != 2:
        raise ValueError("X must be [rows, cin]")
    shape, dtype, device = X.shape, X.dtype, X.device
    rows, cin = shape
    n = _scales(cin, group)
    _need(gamma, "gamma", (cin,), dtype)
    if residual is not None:
        _need(residual, "residual", shape, dtype)
        if summed is None:
            summed = torch.empty_like(X)
        else:
            _need(summed, "summed", shape, dtype)
    elif summed is not None:
        raise ValueError("summed is for a residual")
    if q is None:
        q = _empty(rows, cin, dtype=torch.float8_e4m3fn, device=device)
    else:
        _need(q, "q", shape, torch.float8_e4m3fn)
    if scale is None:
        scale = _empty(rows, n, dtype=torch.float32, device=device)
    else:
        _need(scale, "scale", (rows, n), torch.float32)
    _check(lib().lh_rms_norm_quant(X.data_ptr(), _ptr(residual), _dtype_code(X), rows, cin, gamma.data_ptr(), eps, group,
                                   _ptr(summed), q.data_ptr(), scale.data_ptr(), _stream(device)))
    return q, scale, summed


def lh_matvec(X: torch.Tensor, code: torch.Tensor, fp4: torch.Tensor, amax: torch.Tensor, Y: Optional[torch.Tensor] = None, *,
              x_scale: Optional[torch.Tensor] = None, x_group: int = 0, offsets: Optional[torch.Tensor] = None,
              norm: float = 448.0) -> torch.Tensor:
    """Y [rows, cout]: X [rows, cin] times the NVFP4 weights (code [G, cout, cin/16], fp4 [G, cout, cin/2], amax
    [G]) of a scale sweep with normalization `norm`, the rows of each group (offsets [G+1]) against its
    matrix.  X is fp32, bf16, or torch.float8_e4m3fn with x_scale as lh_rms_norm_quant gives it (x_group 0:
    [rows, 1], 128: [rows, ceil(cin/128)]; without effect for the other types); Y is fp32 for fp32 X,
    otherwise bf16."""
    _need(X, "X")
    if X.dim() != 2 or code.dim() != 3:
        raise ValueError("X must be [rows, cin] and code [G, cout, cin/16]")
    rows, cin = X.shape
    device = X.device
    G = 1
    if offsets is not None:
        offsets, G = _offsets(offsets, X)
    cout = code.shape[1]
    _need(code, "code", (G, cout, cin // 16), torch.uint8)
    _need(fp4, "fp4", (G, cout, cin // 2), torch.uint8)
    _need(amax, "amax", (G,), torch.float32)
    if X.dtype == torch.float8_e4m3fn:
        dtype = LH_DTYPE_E4M3
        if x_scale is None:
            raise ValueError("x_scale is required for E4M3 rows")
        _need(x_scale, "x_scale", (rows, _scales(cin, x_group)), torch.float32)
    else:
        dtype = _dtype_code(X)
        if x_scale is not None:
            raise ValueError("x_scale is for E4M3 rows")
        _scales(cin, x_group)
        x_group = 0                        # it says how x_scale is grouped, and there is none
    y_dtype = torch.float32 if dtype == LH_DTYPE_F32 else torch.bfloat16
    if Y is None:
        Y = _empty(rows, cout, dtype=y_dtype, device=device)
    else:
        _need(Y, "Y", (rows, cout), y_dtype)
    _check(lib().lh_matvec(X.data_ptr(), dtype, _ptr(x_scale), x_group, rows, cin, _ptr(offsets), G, cout, code.data_ptr(),
                           fp4.data_ptr(), amax.data_ptr(), norm, Y.data_ptr(), _stream(device)))
    return Y


class Cache:
    """A paged key-value cache: its code tensors k, v [n_pages, n_heads, page_size, head_dim] uint8 (E4M3) or
    [..., head_dim/2] with block scales k_scale, v_scale [..., head_dim/16] uint8 (NVFP4), and the calibrated
    amax per head k_amax, v_amax [n_heads] fp32.  `Cache.empty` makes the tensors.

    The tensors' addresses are read here once (reading them at each call would cost it 0.6 us), so the attributes cannot be
    assigned or deleted afterwards: copy into the tensors, or make another Cache, which costs no device work."""

    _FIXED = frozenset(("k", "v", "k_amax", "v_amax", "k_scale", "v_scale", "n_pages", "n_heads", "page_size", "head_dim", "struct", "ref"))

    def __setattr__(self, name, value):
        if name in self._FIXED and name in self.__dict__:
            raise AttributeError(f"{name} of a Cache is fixed; copy into its tensors, or make another Cache")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        if name in self._FIXED:
            raise AttributeError(f"{name} of a Cache is fixed; make another Cache")
        object.__delattr__(self, name)

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_amax: torch.Tensor, v_amax: torch.Tensor,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None):
        if k.dim() != 4:
            raise ValueError("k must be [n_pages, n_heads, page_size, head_dim (or half of it)]")
        if (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale must be given together")
        four = k_scale is not None
        shape = k.shape
        pages, heads, page_size, width = shape
        dim = 2 * width if four else width
        if dim % 16:
            raise ValueError("head_dim must be a multiple of 16")
        _need(k, "k", dtype=torch.uint8)
        _need(v, "v", shape, torch.uint8)
        _need(k_amax, "k_amax", (heads,), torch.float32)
        _need(v_amax, "v_amax", (heads,), torch.float32)
        if four:
            scales = (pages, heads, page_size, dim // 16)
            _need(k_scale, "k_scale", scales, torch.uint8)
            _need(v_scale, "v_scale", scales, torch.uint8)
        struct = CacheStruct(LH_CACHE_FP4 if four else LH_CACHE_E4M3, pages, page_size, heads, dim, k.data_ptr(),
                             v.data_ptr(), _ptr(k_scale), _ptr(v_scale), k_amax.data_ptr(), v_amax.data_ptr())
        # past __setattr__, which would cost a microsecond
        self.__dict__.update(k=k, v=v, k_amax=k_amax, v_amax=v_amax, k_scale=k_scale, v_scale=v_scale, n_pages=pages,
                             n_heads=heads, page_size=page_size, head_dim=dim, struct=struct, ref=ctypes.byref(struct))

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_heads: int, head_dim: int, k_amax: torch.Tensor, v_amax: torch.Tensor, *,
              four_bit: bool) -> "Cache":
        """A cache of zeros on the device of k_amax."""
        def new(n):
            return torch.zeros((n_pages, n_heads, page_size, n), dtype=torch.uint8, device=k_amax.device)
        if four_bit:
            return cls(new(head_dim // 2), new(head_dim // 2), k_amax, v_amax, new(head_dim // 16), new(head_dim // 16))
        return cls(new(head_dim), new(head_dim), k_amax, v_amax)


def _heads(t: torch.Tensor, name: str, heads: int, dim: int, dtype=None, tokens=None) -> int:
    """Checks a [tokens, heads, dim] tensor whose tokens may lie apart; its stride between tokens."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    shape = t.shape
    n = shape[0] if tokens is None else tokens
    if shape != (n, heads, dim):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected ({'tokens' if tokens is None else n}, {heads}, {dim})")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    a, b, c = t.stride()
    if (dim > 1 and c != 1) or (heads > 1 and b != dim):
        raise ValueError(f"{name} must hold each token's heads in one run of memory")
    return a if n > 1 else heads * dim


def lh_cache_write(cache: Cache, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantizes K, V [tokens, n_heads, head_dim] (fp32 or bf16; tokens may lie apart, as parts of a projection's
    rows do) into the cache at slots [tokens] int64 (page * page_size + place; outside the cache: skipped; named
    twice in a call: contents unspecified)."""
    ks = _heads(K, "K", cache.n_heads, cache.head_dim)
    tokens = K.shape[0]
    vs = _heads(V, "V", cache.n_heads, cache.head_dim, K.dtype, tokens)
    _need(slots, "slots", (tokens,), torch.int64)
    _check(lib().lh_cache_write(cache.ref, K.data_ptr(), ks, V.data_ptr(), vs, _dtype_code(K), tokens, slots.data_ptr(),
                                _stream(K.device)))


def lh_cache_read(cache: Cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, K: Optional[torch.Tensor] = None,
                  V: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(K, V) [tokens, n_heads, head_dim] of dtype (bf16 or fp32): the values held at slots [tokens] int64."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    if slots.dim() != 1:
        raise ValueError("slots must be [tokens]")
    _need(slots, "slots", dtype=torch.int64)
    tokens, heads, dim, device = slots.shape[0], cache.n_heads, cache.head_dim, slots.device
    if K is None:
        K = _empty(tokens, heads, dim, dtype=dtype, device=device)
    else:
        _need(K, "K", (tokens, heads, dim), dtype)
    if V is None:
        V = torch.empty_like(K)
    else:
        _need(V, "V", (tokens, heads, dim), dtype)
    _check(lib().lh_cache_read(cache.ref, slots.data_ptr(), tokens, LH_DTYPE_BF16 if dtype == torch.bfloat16 else LH_DTYPE_F32,
                               K.data_ptr(), V.data_ptr(), _stream(device)))
    return K, V


def lh_paged_attention_workspace(cache: Cache, batch: int, n_q_heads: int, max_pages: int) -> int:
    """Bytes of workspace that lh_paged_attention needs for these sizes."""
    return int(lib().lh_paged_attention_workspace(cache.ref, batch, n_q_heads, max_pages))


def lh_paged_attention(Q: torch.Tensor, cache: Cache, block_table: torch.Tensor, lengths: torch.Tensor, O: Optional[torch.Tensor] = None, *,
                       scale: float, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """O [batch, n_q_heads, head_dim]: one new token's attention per sequence, Q [batch, n_q_heads, head_dim] (fp32 or
    bf16; sequences may lie apart) over tokens t < lengths[b] in pages block_table[b] (int32 [batch, max_pages]).
    workspace (uint8) is allocated on the current stream when needed and not given."""
    if block_table.dim() != 2 or Q.dim() != 3:
        raise ValueError("block_table must be [batch, max_pages] and Q [batch, n_q_heads, head_dim]")
    batch, heads, dim = Q.shape
    device = Q.device
    stride = _heads(Q, "Q", heads, cache.head_dim)
    pages = block_table.shape[1]
    _need(block_table, "block_table", (batch, pages), torch.int32)
    _need(lengths, "lengths", (batch,), torch.int32)
    if O is None:
        O = _empty(batch, heads, dim, dtype=Q.dtype, device=device)
    else:
        _need(O, "O", (batch, heads, dim), Q.dtype)
    nbytes = 0
    if workspace is not None:
        _need(workspace, "workspace", dtype=torch.uint8)
        nbytes = workspace.numel()
    else:
        nbytes = lib().lh_paged_attention_workspace(cache.ref, batch, heads, pages)
        if nbytes:
            workspace = _empty(nbytes, dtype=torch.uint8, device=device)
    _check(lib().lh_paged_attention(cache.ref, Q.data_ptr(), stride, _dtype_code(Q), batch, heads, block_table.data_ptr(), pages,
                                    lengths.data_ptr(), scale, O.data_ptr(), _ptr(workspace), nbytes, _stream(device)))
    return O
