"""Python binding of libfairy2i.so (the C ABI declared in include/fairy2i.h).

Argument marshalling only: every step of the hot path runs in the library's HIP kernels.
PyTorch supplies device memory and the current HIP stream.  The functions carry the C names
and take torch tensors; output tensors are allocated here when the caller passes none.

The library is built in-tree by `python -m widely_linear_gemv_amd.build`.  If it is missing,
every call raises -- there is no fallback implementation.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# FAIRY2I_LIB selects another build of the same library (the host-sanitized one, for instance).
LIB_PATH = os.environ.get("FAIRY2I_LIB") or os.path.join(_HERE, "libfairy2i.so")

FAIRY2I_OK = 0
STATUS_NAMES = {0: "OK", 1: "ERR_NULL", 2: "ERR_SHAPE", 3: "ERR_STAGES", 4: "ERR_DTYPE",
                5: "ERR_ALIGN", 6: "ERR_WORKSPACE", 7: "ERR_HIP"}
F32, BF16, I8, I32, X_DIGITS, X_DIGITS_F6 = 0, 1, 2, 3, 4, 5
GEMV_AUTO, GEMV_VALU, GEMV_MFMA, GEMV_MFMA_BF16, GEMV_MFMA_I8, GEMV_MFMA_F4 = 0, 1, 2, 3, 4, 5

_DTYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8, torch.int32: I32}

# Every symbol include/fairy2i.h declares: name -> (restype, argtypes)
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_SZ = ctypes.c_size_t
SIGNATURES = {
    "fairy2i_quantize": (_INT, [_P, _I64, _I64, _INT, _P, _P, _P, _P, _P]),
    "fairy2i_quantize_bf16": (_INT, [_P, _I64, _I64, _INT, _P, _P, _P, _P, _P]),
    "fairy2i_quantize_tensor_workspace_bytes": (_SZ, [_I64, _I64, _INT]),
    "fairy2i_quantize_tensor": (_INT, [_P, _INT, _I64, _I64, _INT, _P, _SZ, _P, _P, _P, _P, _P]),
    "fairy2i_pack": (_INT, [_P, _I64, _I64, _INT, _P, _P]),
    "fairy2i_packed_bytes": (_SZ, [_I64, _I64, _INT]),
    "fairy2i_dequantize": (_INT, [_P, _P, _I64, _I64, _INT, _P, _INT, _P]),
    "fairy2i_x_digits_bytes": (_SZ, [_I64, _I64]),
    "fairy2i_x_digits": (_INT, [_P, _INT, _I64, _I64, _P, _P]),
    "fairy2i_x_digits_f6_bytes": (_SZ, [_I64, _I64]),
    "fairy2i_x_digits_f6": (_INT, [_P, _INT, _I64, _I64, _P, _P]),
    "fairy2i_gemv": (_INT, [_P, _P, _I64, _I64, _INT, _P, _INT, _I64, _P, _INT, _INT, _P]),
    "fairy2i_act_quant": (_INT, [_P, _INT, _I64, _I64, _P, _P, _P]),
    "fairy2i_gemm_workspace_bytes": (_SZ, [_I64, _I64, _INT, _I64, _INT]),
    "fairy2i_gemm": (_INT, [_P, _P, _I64, _I64, _INT, _P, _INT, _P, _I64, _P, _INT, _P, _SZ, _P]),
    "fairy2i_gemm_noalloc_max_bytes": (_SZ, []),
    "fairy2i_gemm_noalloc": (_INT, [_P, _P, _I64, _I64, _INT, _P, _INT, _P, _I64, _P, _INT, _P]),
    "fairy2i_status_string": (ctypes.c_char_p, [_INT]),
    "fairy2i_last_error": (ctypes.c_char_p, []),
    "fairy2i_abi_version": (_INT, []),
}



class GemvItem(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("n", ctypes.c_int64)]


SIGNATURES["fairy2i_quantize_grouped"] = (_INT, [_INT, ctypes.POINTER(ctypes.c_void_p), _INT, _I64, _I64, _INT,
                                                  ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_void_p),
                                                  ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_void_p),
                                                  _P])
SIGNATURES["fairy2i_gemv_grouped"] = (_INT, [ctypes.POINTER(GemvItem), _INT, _I64, _INT, _INT, _I64,
                                              _INT, _INT, _P])
SIGNATURES["fairy2i_gemv_strided"] = (_INT, [_P, _I64, _P, _I64, _I64, _I64, _INT, _P, _INT, _I64, _P, _I64,
                                              _INT, _I64, _INT, _P])



class LoraItem(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
                ("base", ctypes.c_void_p), ("y", ctypes.c_void_p), ("n", ctypes.c_int64)]


_F32 = ctypes.c_float
SIGNATURES["fairy2i_lora_workspace_bytes"] = (_SZ, [_INT, _I64, _I64, _INT, _I64])
SIGNATURES["fairy2i_lora"] = (_INT, [_P, _INT, _I64, _I64, _P, _P, _P, _I64, _INT, _I64, _P, _P, _I64, _P, _P, _INT,
                                     _P, _SZ, _P])
SIGNATURES["fairy2i_lora_grouped"] = (_INT, [ctypes.POINTER(LoraItem), _INT, _P, _INT, _I64, _I64, _I64, _INT, _P, _P,
                                             _I64, _INT, _P, _SZ, _P])
SIGNATURES["fairy2i_lora_backward_workspace_bytes"] = (_SZ, [_I64, _I64, _I64, _I64, _INT, _I64, _INT])
SIGNATURES["fairy2i_lora_backward"] = (_INT, [_P, _P, _INT, _I64, _I64, _P, _P, _P, _I64, _INT, _I64, _P, _P, _I64, _P,
                                              _P, _INT, _P, _P, _P, _SZ, _P])
SIGNATURES["fairy2i_vocab_loss_workspace_bytes"] = (_SZ, [_I64, _I64, _I64, _INT])
SIGNATURES["fairy2i_vocab_loss"] = (_INT, [_P, _P, _INT, _I64, _I64, _I64, _P, _P, _P, _P, _SZ, _P])
SIGNATURES["fairy2i_vocab_loss_backward_workspace_bytes"] = (_SZ, [_I64, _I64, _I64, _INT])
SIGNATURES["fairy2i_vocab_loss_backward"] = (_INT, [_P, _P, _INT, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P])
SIGNATURES["fairy2i_clip_grads_workspace_bytes"] = (_SZ, [_INT, ctypes.POINTER(_I64)])
SIGNATURES["fairy2i_clip_grads"] = (_INT, [_INT, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_I64),
                                           ctypes.POINTER(_INT), _F32, _P, _P, _SZ, _P])

SIGNATURES["fairy2i_packed_bytes_w4"] = (_SZ, [_I64, _I64, _INT, _INT])
SIGNATURES["fairy2i_pack_w4"] = (_INT, [_P, _P, _INT, _P, _I64, _I64, _INT, _P, _P])
SIGNATURES["fairy2i_gemv_w4"] = (_INT, [_P, _I64, _I64, _INT, _INT, _P, _INT, _I64, _P, _INT, _P])
SIGNATURES["fairy2i_distill_workspace_bytes"] = (_SZ, [_I64, _I64, _I64, _INT, _INT])
SIGNATURES["fairy2i_distill"] = (_INT, [_P, _P, _INT, _I64, _I64, _I64, _P, _P, _INT, _INT, _F32, _P, _P, _P, _SZ, _P])
SIGNATURES["fairy2i_distill_backward_workspace_bytes"] = (_SZ, [_I64, _I64, _I64, _INT, _INT])
SIGNATURES["fairy2i_distill_backward"] = (_INT, [_P, _P, _INT, _I64, _I64, _I64, _P, _P, _INT, _INT, _F32, _P, _P, _P, _P,
                                                 _P, _SZ, _P])
SIGNATURES["fairy2i_verify_draft_workspace_bytes"] = (_SZ, [_I64, _I64, _I64])
SIGNATURES["fairy2i_verify_draft"] = (_INT, [_P, _P, _INT, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _SZ, _P])

_lib = None


class Fairy2iError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m widely_linear_gemv_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(status: int) -> None:
    if status != FAIRY2I_OK:
        msg = lib().fairy2i_last_error().decode(errors="replace")
        raise Fairy2iError(status, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# ---- argument checks --------------------------------------------------------------------
# The C ABI takes bare device pointers and no buffer sizes: its kernels size every access from the
# call's n, m, T and B.  So before a pointer is passed on, each tensor is checked here for being a
# contiguous GPU tensor of the right dtype, shape and size; a mismatch raises ValueError and nothing
# is launched.  (Checks run dtype -> shape -> size -> layout -> device, so a CPU tensor that is
# otherwise right fails on the device check.)

def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    return t


def _dtype(t, name, *allowed):
    if t.dtype not in allowed:
        raise ValueError(f"{name}: dtype {t.dtype}, need one of {', '.join(str(a) for a in allowed)}")


def _shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, need {tuple(shape)}")


def _min_bytes(t, name, nbytes):
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name}: {have} bytes, need at least {nbytes}")


def _on_gpu(t, name, dev=None, contiguous=True):
    """Layout now; the device check is left to _gpu, after every other check of the call."""
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _gpu(*named):
    """(tensor, name) pairs: all on one GPU.  The last check before a call enters the library."""
    dev = None
    for t, name in named:
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{name}: must be on the GPU (got {t.device})")
        if dev is not None and t.device != dev:
            raise ValueError(f"{name}: on {t.device}, the other operands are on {dev}")
        dev = t.device


def _scales_nT(scales, name="scales"):
    """(n, T) of an fp32 scales tensor [n][T][2][2]."""
    _tensor(scales, name)
    _dtype(scales, name, torch.float32)
    if scales.dim() != 4 or tuple(scales.shape[2:]) != (2, 2):
        raise ValueError(f"{name}: shape {tuple(scales.shape)}, need [n][T][2][2]")
    return scales.shape[0], scales.shape[1]


def _check_x(x, name="x", dtypes=(torch.float32, torch.bfloat16)):
    """Checks a GEMV activation argument (a [B][2m] tensor or an XDigits) up to its device."""
    if isinstance(x, XDigits):
        _tensor(x.buf, name + ".buf")
        _dtype(x.buf, name + ".buf", torch.uint8)
        nbytes = (fairy2i_x_digits_f6_bytes if x.dtype == X_DIGITS_F6 else fairy2i_x_digits_bytes)(x.m, x.B)
        _min_bytes(x.buf, name + ".buf", nbytes)
        _on_gpu(x.buf, name + ".buf")
        return x.buf.device
    _tensor(x, name)
    _dtype(x, name, *dtypes)
    if x.dim() != 2 or x.shape[1] % 2:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, need [B][2m]")
    _on_gpu(x, name)
    return x.device


def _check_layer(packed, scales, m, dev, pname="packed", sname="scales"):
    """packed bytes and scales of an n x m layer, on device dev; returns (n, T)."""
    n, T = _scales_nT(scales, sname)
    _tensor(packed, pname)
    _dtype(packed, pname, torch.uint8)
    _min_bytes(packed, pname, fairy2i_packed_bytes(n, m, T))
    _on_gpu(packed, pname, dev)
    _on_gpu(scales, sname, dev)
    return n, T


def fairy2i_abi_version() -> int:
    return lib().fairy2i_abi_version()


def fairy2i_status_string(status: int) -> str:
    return lib().fairy2i_status_string(status).decode()


def fairy2i_last_error() -> str:
    return lib().fairy2i_last_error().decode(errors="replace")


def fairy2i_packed_bytes(n: int, m: int, T: int) -> int:
    return int(lib().fairy2i_packed_bytes(n, m, T))


def fairy2i_quantize_tensor_workspace_bytes(n: int, m: int, T: int) -> int:
    return int(lib().fairy2i_quantize_tensor_workspace_bytes(n, m, T))


def _check_weight(R, name="R"):
    _tensor(R, name)
    _dtype(R, name, torch.float32, torch.bfloat16)
    if R.dim() != 2 or R.shape[0] % 2 or R.shape[1] % 2:
        raise ValueError(f"{name}: shape {tuple(R.shape)}, need [2n][2m]")
    _on_gpu(R, name)
    return R.shape[0] // 2, R.shape[1] // 2, R.device


def _quant_outputs(packed, scales, n, m, T, dev):
    """The quantizers' packed and scales outputs: allocated when None, checked otherwise."""
    if packed is None:
        packed = torch.empty((fairy2i_packed_bytes(n, m, T),), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((n, T, 2, 2), dtype=torch.float32, device=dev)
    _tensor(scales, "scales")
    _dtype(scales, "scales", torch.float32)
    _shape(scales, "scales", (n, T, 2, 2))
    _check_layer(packed, scales, m, dev)
    return packed, scales


def fairy2i_quantize(R: torch.Tensor, T: int, *, want_scales64: bool = False,
                     want_codes: bool = False, packed=None, scales=None, stream=None):
    """R fp32 or bf16 [2n][2m] on the GPU -> dict(packed (flat uint8), scales[, scales64][, codes])."""
    n, m, dev = _check_weight(R)
    packed, scales = _quant_outputs(packed, scales, n, m, T, dev)
    s64 = torch.empty((n, T, 2, 2), dtype=torch.float64, device=dev) if want_scales64 else None
    codes = torch.empty((T, 2, n, m), dtype=torch.uint8, device=dev) if want_codes else None
    fn = lib().fairy2i_quantize_bf16 if R.dtype == torch.bfloat16 else lib().fairy2i_quantize
    _gpu((R, "R"), (packed, "packed"), (scales, "scales"), (s64, "scales64"), (codes, "codes"))
    _check(fn(_ptr(R), 2 * n, 2 * m, T, _ptr(packed), _ptr(scales), _ptr(s64), _ptr(codes), _stream(stream)))
    out = {"packed": packed, "scales": scales}
    if s64 is not None:
        out["scales64"] = s64
    if codes is not None:
        out["codes"] = codes
    return out


def fairy2i_quantize_grouped(Rs, T: int, *, want_scales64: bool = False, want_codes: bool = False,
                             packed=None, scales=None, stream=None):
    """fairy2i_quantize on a list of layers of one shape and dtype (fp32 or bf16 [2n][2m] on one
    GPU), in shared launches; each layer's result equals its own fairy2i_quantize call.  packed and
    scales: None (allocated) or lists of one output per layer.  Returns a list of dicts like
    fairy2i_quantize."""
    Rs = list(Rs)
    if not Rs:
        return []
    n, m, dev = _check_weight(Rs[0], "R[0]")
    for k, R in enumerate(Rs):
        nk, mk, _ = _check_weight(R, f"R[{k}]")
        if (nk, mk) != (n, m) or R.dtype != Rs[0].dtype:
            raise ValueError(f"R[{k}]: {R.dtype} [{2 * nk}][{2 * mk}], the group is {Rs[0].dtype} [{2 * n}][{2 * m}]")
    count = len(Rs)
    for name, given in (("packed", packed), ("scales", scales)):
        if given is not None and len(given) != count:
            raise ValueError(f"{name}: {len(given)} outputs for {count} layers")
    outs = [_quant_outputs(None if packed is None else packed[k], None if scales is None else scales[k], n, m, T, dev)
            for k in range(count)]
    s64 = [torch.empty((n, T, 2, 2), dtype=torch.float64, device=dev) for _ in range(count)] if want_scales64 else None
    codes = [torch.empty((T, 2, n, m), dtype=torch.uint8, device=dev) for _ in range(count)] if want_codes else None
    named = [(R, f"R[{k}]") for k, R in enumerate(Rs)]
    named += [(t, f"{name}[{k}]") for k, (pk, sc) in enumerate(outs) for t, name in ((pk, "packed"), (sc, "scales"))]
    named += [(t, f"scales64[{k}]") for k, t in enumerate(s64 or [])] + [(t, f"codes[{k}]") for k, t in enumerate(codes or [])]
    _gpu(*named)
    arr = lambda ts: (ctypes.c_void_p * count)(*[t.data_ptr() for t in ts])
    _check(lib().fairy2i_quantize_grouped(count, arr(Rs), _DTYPE[Rs[0].dtype], 2 * n, 2 * m, T,
                                          arr([o[0] for o in outs]), arr([o[1] for o in outs]),
                                          arr(s64) if s64 else None, arr(codes) if codes else None, _stream(stream)))
    res = []
    for k, (pk, sc) in enumerate(outs):
        d = {"packed": pk, "scales": sc}
        if s64:
            d["scales64"] = s64[k]
        if codes:
            d["codes"] = codes[k]
        res.append(d)
    return res


def fairy2i_quantize_tensor(R: torch.Tensor, T: int, *, want_scales64: bool = False,
                            want_codes: bool = False, workspace=None, packed=None, scales=None,
                            stream=None):
    """fairy2i_quantize with per-tensor axis scales (every row of scales holds the same pairs)."""
    n, m, dev = _check_weight(R)
    two_n, two_m = 2 * n, 2 * m
    if workspace is None:
        workspace = torch.empty((fairy2i_quantize_tensor_workspace_bytes(n, m, T),), dtype=torch.uint8, device=dev)
    _tensor(workspace, "workspace")
    _min_bytes(workspace, "workspace", fairy2i_quantize_tensor_workspace_bytes(n, m, T))
    _on_gpu(workspace, "workspace", dev)
    packed, scales = _quant_outputs(packed, scales, n, m, T, dev)
    s64 = torch.empty((n, T, 2, 2), dtype=torch.float64, device=dev) if want_scales64 else None
    codes = torch.empty((T, 2, n, m), dtype=torch.uint8, device=dev) if want_codes else None
    _gpu((R, "R"), (workspace, "workspace"), (packed, "packed"), (scales, "scales"), (s64, "scales64"),
         (codes, "codes"))
    _check(lib().fairy2i_quantize_tensor(_ptr(R), _DTYPE[R.dtype], two_n, two_m, T, _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _ptr(packed),
                                         _ptr(scales), _ptr(s64), _ptr(codes), _stream(stream)))
    out = {"packed": packed, "scales": scales}
    if s64 is not None:
        out["scales64"] = s64
    if codes is not None:
        out["codes"] = codes
    return out


def fairy2i_pack(codes: torch.Tensor, packed=None, stream=None) -> torch.Tensor:
    """codes uint8 [T][2][n][m] -> the packed form (flat uint8, fairy2i_packed_bytes)."""
    _tensor(codes, "codes")
    _dtype(codes, "codes", torch.uint8)
    if codes.dim() != 4 or codes.shape[1] != 2:
        raise ValueError(f"codes: shape {tuple(codes.shape)}, need [T][2][n][m]")
    _on_gpu(codes, "codes")
    T, _, n, m = codes.shape
    packed = packed if packed is not None else torch.empty((fairy2i_packed_bytes(n, m, T),), dtype=torch.uint8, device=codes.device)
    _tensor(packed, "packed")
    _dtype(packed, "packed", torch.uint8)
    _min_bytes(packed, "packed", fairy2i_packed_bytes(n, m, T))
    _on_gpu(packed, "packed", codes.device)
    _gpu((codes, "codes"), (packed, "packed"))
    _check(lib().fairy2i_pack(_ptr(codes), n, m, T, _ptr(packed), _stream(stream)))
    return packed


def fairy2i_dequantize(packed: torch.Tensor, scales: torch.Tensor, m: int, *, R_dtype=torch.float32,
                       R=None, stream=None) -> torch.Tensor:
    """packed form + scales [n][T][2][2] -> the real layer R^ [2n][2m] (fp32 or bf16)."""
    _tensor(packed, "packed")
    n, T = _check_layer(packed, scales, m, packed.device)
    if R is None:
        R = torch.empty((2 * n, 2 * m), dtype=R_dtype, device=packed.device)
    _tensor(R, "R")
    _dtype(R, "R", torch.float32, torch.bfloat16)
    _shape(R, "R", (2 * n, 2 * m))
    _on_gpu(R, "R", packed.device)
    _gpu((packed, "packed"), (scales, "scales"), (R, "R"))
    _check(lib().fairy2i_dequantize(_ptr(packed), _ptr(scales), n, m, T, _ptr(R), _DTYPE[R.dtype],
                                    _stream(stream)))
    return R


class XDigits:
    """A digit form of decode-GEMV activations: the uint8 buffer, the B and m it was made with,
    and its dtype code (X_DIGITS: int8 digits of fairy2i_x_digits; X_DIGITS_F6: fp6 digits of
    fairy2i_x_digits_f6)."""

    def __init__(self, buf: torch.Tensor, B: int, m: int, dtype: int = X_DIGITS):
        self.buf, self.B, self.m, self.dtype = buf, B, m, dtype

    @property
    def device(self):
        return self.buf.device


def _x_tensor(x):
    """The device tensor of a GEMV activation argument."""
    return x.buf if isinstance(x, XDigits) else x


def _x_cols(x) -> int:
    """Complex columns m of a GEMV/GEMM activation argument."""
    return x.m if isinstance(x, XDigits) else x.shape[1] // 2


def _x_args(x):
    """(pointer, x_dtype, B) of a GEMV activation argument: a [B][2m] tensor or an XDigits."""
    if isinstance(x, XDigits):
        return _ptr(x.buf), x.dtype, x.B
    return _ptr(x), _DTYPE[x.dtype], x.shape[0]


def _check_digits_out(out, B, m, dtype, dev):
    if not isinstance(out, XDigits):
        raise TypeError("out: expected an XDigits")
    if out.B != B or out.m != m or out.dtype != dtype:
        raise ValueError(f"out: made for B={out.B}, m={out.m}, dtype {out.dtype}; this x needs B={B}, m={m}, "
                         f"dtype {dtype}")
    _check_x(out, "out")
    if out.buf.device != dev:
        raise ValueError(f"out: on {out.buf.device}, x is on {dev}")


def fairy2i_x_digits_bytes(m: int, B: int) -> int:
    return int(lib().fairy2i_x_digits_bytes(m, B))


def fairy2i_x_digits(x: torch.Tensor, out: XDigits | None = None, stream=None) -> XDigits:
    """x [B][2m] (bf16 / fp32, B <= 2) -> its exact int8 digit form for the int8 MFMA GEMV."""
    _check_x(x)
    B, two_m = x.shape
    m = two_m // 2
    if out is None:
        out = XDigits(torch.empty((fairy2i_x_digits_bytes(m, B),), dtype=torch.uint8, device=x.device), B, m)
    _check_digits_out(out, B, m, X_DIGITS, x.device)
    _gpu((x, "x"), (out.buf, "out"))
    _check(lib().fairy2i_x_digits(_ptr(x), _DTYPE[x.dtype], m, B, _ptr(out.buf), _stream(stream)))
    return out


def fairy2i_x_digits_f6_bytes(m: int, B: int) -> int:
    return int(lib().fairy2i_x_digits_f6_bytes(m, B))


def fairy2i_x_digits_f6(x: torch.Tensor, out: XDigits | None = None, stream=None) -> XDigits:
    """x [B][2m] (bf16 / fp32, B <= 2) -> its exact fp6 digit form for the fp4 MFMA GEMV."""
    _check_x(x)
    B, two_m = x.shape
    m = two_m // 2
    if out is None:
        out = XDigits(torch.empty((fairy2i_x_digits_f6_bytes(m, B),), dtype=torch.uint8, device=x.device),
                      B, m, X_DIGITS_F6)
    _check_digits_out(out, B, m, X_DIGITS_F6, x.device)
    _gpu((x, "x"), (out.buf, "out"))
    _check(lib().fairy2i_x_digits_f6(_ptr(x), _DTYPE[x.dtype], m, B, _ptr(out.buf), _stream(stream)))
    return out


def _check_y(y, shape, dev, name="y"):
    _tensor(y, name)
    _dtype(y, name, torch.float32, torch.bfloat16)
    _shape(y, name, shape)
    _on_gpu(y, name, dev)


def fairy2i_gemv(packed: torch.Tensor, scales: torch.Tensor, x, *,
                 y_dtype=torch.float32, algo: int = GEMV_AUTO, y=None, stream=None) -> torch.Tensor:
    """packed form, scales [n][T][2][2], x [B][2m] (or its XDigits) -> y [B][2n].  n and T come
    from the scales, m from x."""
    dev = _check_x(x)
    m = _x_cols(x)
    n, T = _check_layer(packed, scales, m, dev)
    xp, xdt, B = _x_args(x)
    if y is None:
        y = torch.empty((B, 2 * n), dtype=y_dtype, device=dev)
    _check_y(y, (B, 2 * n), dev)
    _gpu((packed, "packed"), (scales, "scales"), (_x_tensor(x), "x"), (y, "y"))
    _check(lib().fairy2i_gemv(_ptr(packed), _ptr(scales), n, m, T, xp, xdt, B,
                              _ptr(y), _DTYPE[y.dtype], algo, _stream(stream)))
    return y


def fairy2i_gemv_grouped(items, *, algo: int = GEMV_AUTO, stream=None):
    """items: sequence of (packed, scales, x, y) tensor tuples sharing m, T, B and dtypes; each y
    [B][2n] is preallocated by the caller.  Returns the list of y."""
    items = list(items)
    if not items:
        raise ValueError("fairy2i_gemv_grouped: no items")
    arr = (GemvItem * len(items))()
    _, scales0, x0, y0 = items[0]
    dev = _check_x(x0, "items[0].x")
    m0 = _x_cols(x0)
    _, xdt0, B0 = _x_args(x0)
    T0 = _scales_nT(scales0, "items[0].scales")[1]
    _tensor(y0, "items[0].y")
    for k, (packed, scales, x, y) in enumerate(items):
        if _check_x(x, f"items[{k}].x") != dev:
            raise ValueError(f"items[{k}]: on another device than items[0]")
        if _x_cols(x) != m0 or _x_args(x)[1:] != (xdt0, B0):
            raise ValueError(f"items[{k}]: x has m = {_x_cols(x)}, dtype {_x_args(x)[1]}, B = {_x_args(x)[2]}; "
                             f"items[0] has m = {m0}, dtype {xdt0}, B = {B0}")
        n, T = _check_layer(packed, scales, m0, dev, f"items[{k}].packed", f"items[{k}].scales")
        if T != T0:
            raise ValueError(f"items[{k}]: T = {T}, items[0] has T = {T0}")
        _check_y(y, (B0, 2 * n), dev, f"items[{k}].y")
        if y.dtype != y0.dtype:
            raise ValueError(f"items[{k}].y: dtype {y.dtype}, items[0].y has {y0.dtype}")
        arr[k] = GemvItem(packed.data_ptr(), scales.data_ptr(), _x_args(x)[0], y.data_ptr(), n)
    T = scales0.shape[1]
    _, xdt, B = _x_args(x0)
    _gpu(*[(t, f"items[{k}]") for k, it in enumerate(items) for t in (it[0], it[1], _x_tensor(it[2]), it[3])])
    _check(lib().fairy2i_gemv_grouped(arr, len(items), _x_cols(x0), T, xdt, B,
                                      _DTYPE[y0.dtype], algo, _stream(stream)))
    return [it[3] for it in items]


def fairy2i_gemv_strided(packed: torch.Tensor, scales: torch.Tensor, x, y: torch.Tensor, *,
                         algo: int = GEMV_AUTO, stream=None):
    """A strided batch of GEMVs sharing x: packed [batch][bytes] uint8, scales [batch][n][T][2][2]
    (or [n][T][2][2], shared by all), y [batch][B][2n] preallocated; the strides are those of the
    tensors' first dimension (each matrix's slice contiguous).  Returns y."""
    if packed.dim() != 2 or y.dim() != 3 or scales.dim() not in (4, 5):
        raise ValueError("fairy2i_gemv_strided: packed [batch][bytes], scales [batch][n][T][2][2] or "
                         "[n][T][2][2], y [batch][B][2n]")
    batch = packed.shape[0]
    dev = _check_x(x)
    m = _x_cols(x)
    xp, xdt, B = _x_args(x)
    n, T = _scales_nT(scales[0] if scales.dim() == 5 else scales)
    _dtype(packed, "packed", torch.uint8)
    if packed.shape[1] < fairy2i_packed_bytes(n, m, T):
        raise ValueError(f"packed: {packed.shape[1]} bytes per matrix, need at least {fairy2i_packed_bytes(n, m, T)}")
    if scales.dim() == 5 and scales.shape[0] != batch:
        raise ValueError(f"scales: {scales.shape[0]} matrices, packed has {batch}")
    _dtype(y, "y", torch.float32, torch.bfloat16)
    if tuple(y.shape) != (batch, B, 2 * n):
        raise ValueError(f"y: shape {tuple(y.shape)}, need {(batch, B, 2 * n)}")
    # each matrix's slice must be contiguous; the first dimension may have any stride >= 0
    if packed.stride(1) != 1 or not y[0].is_contiguous() or not (scales[0] if scales.dim() == 5 else scales).is_contiguous():
        raise ValueError("fairy2i_gemv_strided: each matrix's packed bytes, scales and outputs must be contiguous")
    if batch > 1 and y.stride(0) < y[0].numel():
        raise ValueError("y: the outputs of different matrices overlap")
    for t, name in ((packed, "packed"), (scales, "scales"), (y, "y")):
        _on_gpu(t, name, dev, contiguous=False)
    s_stride = scales.stride(0) if scales.dim() == 5 else 0
    _gpu((packed, "packed"), (scales, "scales"), (_x_tensor(x), "x"), (y, "y"))
    _check(lib().fairy2i_gemv_strided(_ptr(packed), packed.stride(0), _ptr(scales), s_stride, n,
                                      _x_cols(x), T, xp, xdt, B, _ptr(y), y.stride(0), _DTYPE[y.dtype],
                                      batch, algo, _stream(stream)))
    return y


def fairy2i_act_quant(x: torch.Tensor, q=None, delta=None, stream=None):
    """x [N][2m] (fp32 / bf16) -> (q int8 [N][2m], delta fp32 [N])."""
    dev = _check_x(x)
    N, two_m = x.shape
    q = q if q is not None else torch.empty((N, two_m), dtype=torch.int8, device=dev)
    delta = delta if delta is not None else torch.empty((N,), dtype=torch.float32, device=dev)
    _tensor(q, "q")
    _dtype(q, "q", torch.int8)
    _shape(q, "q", (N, two_m))
    _on_gpu(q, "q", dev)
    _tensor(delta, "delta")
    _dtype(delta, "delta", torch.float32)
    _shape(delta, "delta", (N,))
    _on_gpu(delta, "delta", dev)
    _gpu((x, "x"), (q, "q"), (delta, "delta"))
    _check(lib().fairy2i_act_quant(_ptr(x), _DTYPE[x.dtype], N, two_m, _ptr(q), _ptr(delta), _stream(stream)))
    return q, delta


def fairy2i_gemm_workspace_bytes(n: int, m: int, T: int, N: int, x_dtype: int) -> int:
    return int(lib().fairy2i_gemm_workspace_bytes(n, m, T, N, x_dtype))


def fairy2i_gemm(packed: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, *,
                 x_scale=None, y_dtype=torch.float32, y=None, workspace=None, stream=None):
    """Prefill over N tokens.  x [N][2m] bf16/fp32 (x_scale receives delta if given) or int8
    (x_scale = delta input).  y_dtype float32/bfloat16 -> y [N][2n]; int32 -> raw
    accumulators [T][2][2][2][N][n]."""
    dev = _check_x(x, dtypes=(torch.float32, torch.bfloat16, torch.int8))
    m = x.shape[1] // 2
    N = x.shape[0]
    n, T = _check_layer(packed, scales, m, dev)
    if x_scale is not None or x.dtype == torch.int8:
        _tensor(x_scale, "x_scale")
        _dtype(x_scale, "x_scale", torch.float32)
        _shape(x_scale, "x_scale", (N,))
        _on_gpu(x_scale, "x_scale", dev)
    if y is None:
        shape = (T, 2, 2, 2, N, n) if y_dtype == torch.int32 else (N, 2 * n)
        y = torch.empty(shape, dtype=y_dtype, device=dev)
    _tensor(y, "y")
    _dtype(y, "y", torch.float32, torch.bfloat16, torch.int32)
    _shape(y, "y", (T, 2, 2, 2, N, n) if y.dtype == torch.int32 else (N, 2 * n))
    _on_gpu(y, "y", dev)
    nbytes = fairy2i_gemm_workspace_bytes(n, m, T, N, _DTYPE[x.dtype])
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _tensor(workspace, "workspace")
        _min_bytes(workspace, "workspace", nbytes)
        _on_gpu(workspace, "workspace", dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _gpu((packed, "packed"), (scales, "scales"), (x, "x"), (x_scale, "x_scale"), (y, "y"), (workspace, "workspace"))
    _check(lib().fairy2i_gemm(_ptr(packed), _ptr(scales), n, m, T, _ptr(x), _DTYPE[x.dtype],
                              _ptr(x_scale), N, _ptr(y), _DTYPE[y.dtype], _ptr(workspace), ws_bytes,
                              _stream(stream)))
    return y


def fairy2i_gemm_noalloc_max_bytes() -> int:
    return int(lib().fairy2i_gemm_noalloc_max_bytes())


def fairy2i_gemm_noalloc(packed: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, *,
                         x_scale=None, y: torch.Tensor, stream=None):
    """fairy2i_gemm without a workspace: the activation staging lives in the library's static
    device array (calls on one GPU must not overlap).  y is preallocated by the caller (no
    allocation at all here): float32/bfloat16 [N][2n], or int32 [T][2][2][2][N][n]."""
    dev = _check_x(x, dtypes=(torch.float32, torch.bfloat16, torch.int8))
    m = x.shape[1] // 2
    N = x.shape[0]
    n, T = _check_layer(packed, scales, m, dev)
    if x_scale is not None or x.dtype == torch.int8:
        _tensor(x_scale, "x_scale")
        _dtype(x_scale, "x_scale", torch.float32)
        _shape(x_scale, "x_scale", (N,))
        _on_gpu(x_scale, "x_scale", dev)
    _tensor(y, "y")
    _dtype(y, "y", torch.float32, torch.bfloat16, torch.int32)
    _shape(y, "y", (T, 2, 2, 2, N, n) if y.dtype == torch.int32 else (N, 2 * n))
    _on_gpu(y, "y", dev)
    _gpu((packed, "packed"), (scales, "scales"), (x, "x"), (x_scale, "x_scale"), (y, "y"))
    _check(lib().fairy2i_gemm_noalloc(_ptr(packed), _ptr(scales), n, m, T, _ptr(x), _DTYPE[x.dtype],
                                      _ptr(x_scale), N, _ptr(y), _DTYPE[y.dtype], _stream(stream)))
    return y



# ---- beside the packed layers: low-rank adapters, the vocabulary loss, gradient clipping ----
# These calls take stream= too (_on_stream adds it): they run, and allocate what the caller gives no
# tensor for, on that stream of the operands' device.

_FLOATS = {torch.float32, torch.bfloat16}
_HERE_SCOPE = contextlib.nullcontext()


def _scope(t, stream):
    """Context of a call on t's device and the given stream, or the device's current one.  What the
    call allocates then belongs to the stream that uses it."""
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        return _HERE_SCOPE                              # the argument checks refuse it
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"stream: on {stream.device}, the operands are on {t.device}")
        return torch.cuda.stream(stream)
    if t.get_device() != torch.cuda.current_device():
        return torch.cuda.device(t.device)
    return _HERE_SCOPE


def _on_stream(fn):
    """Runs fn(first, ...) in the _scope of its first tensor and its stream argument."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if not args and name not in kwargs:
            return fn(**kwargs)                         # raises for the missing argument
        first, args = (args[0], args[1:]) if args else (kwargs.pop(name), args)
        if not isinstance(first, torch.Tensor) and first is not None:
            first = list(first)
        scope = _scope(first[0] if isinstance(first, list) and first else first, stream)
        if scope is _HERE_SCOPE:
            return fn(first, *args, **kwargs)
        with scope:
            return fn(first, *args, **kwargs)
    return call


# The current stream of GPU number dev, as the C calls take it (torch.cuda.current_stream makes an object first:
# 2.7 us of a call's host time against 0.1).
_here = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _fits(t, dtype, shape, dev):
    """Whether t is what a call needs: a contiguous tensor of this dtype and shape on GPU number dev.
    The calls test all their arguments with it at once; only if one fails does the matching _refuse_
    function look for the reason (its checks in their fixed order) and raise."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == dev)


def _room(workspace, nbytes, dev):
    """(pointer, bytes, tensor) of the call's workspace: allocated when None, checked otherwise."""
    if workspace is None:
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
    else:
        _workspace(workspace, nbytes, dev)
        _gpu((workspace, "workspace"))
        if workspace.device != dev:
            raise ValueError(f"workspace: on {workspace.device}, the other operands are on {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _workspace(workspace, nbytes, dev):
    """The call's workspace: allocated when None, checked otherwise."""
    if workspace is None:
        return torch.empty((nbytes,), dtype=torch.uint8, device=dev)
    _tensor(workspace, "workspace")
    _min_bytes(workspace, "workspace", nbytes)
    _on_gpu(workspace, "workspace")
    return workspace


def _check_plain(t, name, dtypes, shape):
    _tensor(t, name)
    _dtype(t, name, *dtypes)
    _shape(t, name, shape)
    _on_gpu(t, name)


def _overlap(a, b):
    """Whether two contiguous tensors share memory without being the same range."""
    a0, b0 = a.data_ptr(), b.data_ptr()
    a1, b1 = a0 + a.numel() * a.element_size(), b0 + b.numel() * b.element_size()
    return a0 < b1 and b0 < a1 and (a0, a1) != (b0, b1)


def _check_segments(seg_start, seg_adapter):
    _tensor(seg_adapter, "seg_adapter")
    _dtype(seg_adapter, "seg_adapter", torch.int32)
    if seg_adapter.dim() != 1 or seg_adapter.shape[0] < 1:
        raise ValueError(f"seg_adapter: shape {tuple(seg_adapter.shape)}, need [S] with S >= 1")
    S = seg_adapter.shape[0]
    _on_gpu(seg_adapter, "seg_adapter")
    _check_plain(seg_start, "seg_start", (torch.int32,), (S + 1,))
    return S


def _check_adapters(x, A, B, alpha, name=""):
    """A [L][r][2m], B [L][2n][r] of x's dtype and alpha [L]; returns (L, r, 2n)."""
    _tensor(A, name + "A")
    _tensor(B, name + "B")
    _dtype(A, name + "A", x.dtype)
    _dtype(B, name + "B", x.dtype)
    if A.dim() != 3 or A.shape[2] != x.shape[1]:
        raise ValueError(f"{name}A: shape {tuple(A.shape)}, need [L][r][{x.shape[1]}]")
    L, r = A.shape[0], A.shape[1]
    if B.dim() != 3 or B.shape[0] != L or B.shape[2] != r or B.shape[1] % 2:
        raise ValueError(f"{name}B: shape {tuple(B.shape)}, need [{L}][2n][{r}]")
    _on_gpu(A, name + "A")
    _on_gpu(B, name + "B")
    _check_plain(alpha, name + "alpha", (torch.float32,), (L,))
    return L, r, B.shape[1]


def fairy2i_lora_workspace_bytes(count: int, N: int, m: int, r: int, S: int) -> int:
    return int(lib().fairy2i_lora_workspace_bytes(count, N, m, r, S))


@_on_stream
def fairy2i_lora_grouped(x: torch.Tensor, items, seg_start: torch.Tensor, seg_adapter: torch.Tensor, *, workspace=None):
    """Low-rank adapters beside projections that read the same x [N][2m].  items: sequence of
    (A [L][r][2m], B [L][2n][r], alpha [L], base [N][2n], y [N][2n] or None for base itself); L, r and
    the dtypes are shared.  Segment s is rows seg_start[s] .. seg_start[s+1]-1 and uses adapter
    seg_adapter[s] (int32 on the GPU); y = base + alpha B A x on its rows, other rows of y are not
    written.  Returns the list of y."""
    items = list(items)
    arr = (LoraItem * max(len(items), 1))()
    ys = []
    try:
        dt, dev = x.dtype, x.get_device()
        N, two_m = x.shape
        S, = seg_adapter.shape
        L, r, _ = items[0][0].shape
        ydt = items[0][3].dtype
        good = (dt in _FLOATS and ydt in _FLOATS and dev >= 0 and two_m % 2 == 0 and x.is_contiguous() and S > 0
                and _fits(seg_adapter, torch.int32, (S,), dev) and _fits(seg_start, torch.int32, (S + 1,), dev))
        for k, (A, B, alpha, base, y) in enumerate(items):
            two_n = B.shape[1]
            here = base.data_ptr()
            there = here if y is None or y is base else y.data_ptr()
            good = (good and two_n % 2 == 0 and _fits(A, dt, (L, r, two_m), dev) and _fits(B, dt, (L, two_n, r), dev)
                    and _fits(alpha, torch.float32, (L,), dev) and _fits(base, ydt, (N, two_n), dev)
                    and (there == here or abs(there - here) >= N * two_n * ydt.itemsize)
                    and (y is None or y is base or _fits(y, ydt, (N, two_n), dev)))
            arr[k] = (A.data_ptr(), B.data_ptr(), alpha.data_ptr(), here, there, two_n // 2)
            ys.append(base if y is None else y)
    except (AttributeError, IndexError, TypeError, ValueError):
        good = False
    if not good:
        _refuse_lora(x, items, seg_start, seg_adapter, workspace)
    ws, nbytes, keep = _room(workspace, fairy2i_lora_workspace_bytes(len(items), N, two_m // 2, r, S), x.device)
    _check(lib().fairy2i_lora_grouped(arr, len(items), x.data_ptr(), _DTYPE[dt], N, two_m // 2, L, r, seg_start.data_ptr(),
                                      seg_adapter.data_ptr(), S, _DTYPE[ydt], ws, nbytes, _stream()))
    return ys


def _refuse_lora(x, items, seg_start, seg_adapter, workspace):
    """Raises for the first argument of fairy2i_lora_grouped that does not fit."""
    if not items:
        raise ValueError("fairy2i_lora_grouped: no items")
    _check_x(x)
    N, two_m = x.shape
    S = _check_segments(seg_start, seg_adapter)
    named = [(x, "x"), (seg_start, "seg_start"), (seg_adapter, "seg_adapter")]
    for k, (A, B, alpha, base, y) in enumerate(items):
        name = f"items[{k}]." if len(items) > 1 else ""
        Lk, rk, two_n = _check_adapters(x, A, B, alpha, name)
        if k == 0:
            L, r = Lk, rk
        elif (Lk, rk) != (L, r):
            raise ValueError(f"{name}A: {Lk} adapters of rank {rk}, items[0] has {L} of rank {r}")
        y = base if y is None else y
        _check_y(base, (N, two_n), x.device, name + "base")
        _check_plain(y, name + "y", (base.dtype,), (N, two_n))
        if base.dtype != items[0][3].dtype:
            raise ValueError(f"{name}base: dtype {base.dtype}, items[0] has {items[0][3].dtype}")
        if _overlap(y, base):
            raise ValueError(f"{name}y: overlaps base without being base")
        named += [(A, name + "A"), (B, name + "B"), (alpha, name + "alpha"), (base, name + "base"), (y, name + "y")]
    if workspace is not None:
        _workspace(workspace, fairy2i_lora_workspace_bytes(len(items), N, two_m // 2, r, S), x.device)
    _gpu(*named, (workspace, "workspace"))
    raise ValueError("fairy2i_lora: the arguments do not fit together")


def fairy2i_lora(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: torch.Tensor, seg_start: torch.Tensor,
                 seg_adapter: torch.Tensor, base: torch.Tensor, *, y=None, workspace=None, stream=None) -> torch.Tensor:
    """fairy2i_lora_grouped for one projection; y None writes base in place.  Returns y."""
    return fairy2i_lora_grouped(x, [(A, B, alpha, base, y)], seg_start, seg_adapter, workspace=workspace,
                                stream=stream)[0]


def fairy2i_lora_backward_workspace_bytes(N: int, m: int, n: int, L: int, r: int, S: int, x_dtype: int) -> int:
    return int(lib().fairy2i_lora_backward_workspace_bytes(N, m, n, L, r, S, x_dtype))


@_on_stream
def fairy2i_lora_backward(dy: torch.Tensor, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: torch.Tensor,
                          seg_start: torch.Tensor, seg_adapter: torch.Tensor, *, dx_base=None, dx=None, dA=None, dB=None,
                          workspace=None):
    """Gradient of fairy2i_lora.  dy [N][2n] (x's dtype); dx_base [N][2m] is the gradient through the
    shared projection: dx = dx_base + A^T dh on rows with an adapter (dx None: in place; dx_base None:
    no dx).  Returns (dx or None, dA fp32 [L][r][2m], dB fp32 [L][2n][r])."""
    f32 = torch.float32
    out = dx_base if dx is None else dx
    try:
        dt, dev = x.dtype, x.get_device()
        N, two_m = x.shape
        S, = seg_adapter.shape
        L, r, _ = A.shape
        two_n = B.shape[1]
        good = (dt in _FLOATS and dev >= 0 and two_m % 2 == 0 and two_n % 2 == 0 and x.is_contiguous() and S > 0
                and _fits(dy, dt, (N, two_n), dev) and _fits(A, dt, (L, r, two_m), dev) and _fits(B, dt, (L, two_n, r), dev)
                and _fits(alpha, f32, (L,), dev) and _fits(seg_adapter, torch.int32, (S,), dev)
                and _fits(seg_start, torch.int32, (S + 1,), dev)
                and (dA is None or _fits(dA, f32, (L, r, two_m), dev)) and (dB is None or _fits(dB, f32, (L, two_n, r), dev))
                and (dx is None if dx_base is None else
                     dx_base.dtype in _FLOATS and _fits(dx_base, dx_base.dtype, (N, two_m), dev)
                     and (out is dx_base or _fits(out, dx_base.dtype, (N, two_m), dev) and not _overlap(out, dx_base))))
    except (AttributeError, IndexError, TypeError, ValueError):
        good = False
    if not good:
        _refuse_lora_backward(dy, x, A, B, alpha, seg_start, seg_adapter, dx_base, dx, dA, dB, workspace)
    dA = torch.empty((L, r, two_m), dtype=f32, device=x.device) if dA is None else dA
    dB = torch.empty((L, two_n, r), dtype=f32, device=x.device) if dB is None else dB
    ws, nbytes, keep = _room(workspace, fairy2i_lora_backward_workspace_bytes(N, two_m // 2, two_n // 2, L, r, S, _DTYPE[dt]),
                             x.device)
    _check(lib().fairy2i_lora_backward(dy.data_ptr(), x.data_ptr(), _DTYPE[dt], N, two_m // 2, A.data_ptr(), B.data_ptr(),
                                       alpha.data_ptr(), L, r, two_n // 2, seg_start.data_ptr(), seg_adapter.data_ptr(), S,
                                       None if out is None else dx_base.data_ptr(), None if out is None else out.data_ptr(),
                                       F32 if out is None else _DTYPE[out.dtype], dA.data_ptr(), dB.data_ptr(), ws, nbytes,
                                       _stream()))
    return out, dA, dB


def _refuse_lora_backward(dy, x, A, B, alpha, seg_start, seg_adapter, dx_base, dx, dA, dB, workspace):
    """Raises for the first argument of fairy2i_lora_backward that does not fit."""
    _check_x(x)
    N, two_m = x.shape
    S = _check_segments(seg_start, seg_adapter)
    L, r, two_n = _check_adapters(x, A, B, alpha)
    _check_plain(dy, "dy", (x.dtype,), (N, two_n))
    if dx_base is None and dx is not None:
        raise ValueError("dx: needs dx_base")
    if dx_base is not None:
        dx = dx_base if dx is None else dx
        _check_y(dx_base, (N, two_m), x.device, "dx_base")
        _check_plain(dx, "dx", (dx_base.dtype,), (N, two_m))
        if _overlap(dx, dx_base):
            raise ValueError("dx: overlaps dx_base without being dx_base")
    for t, name, shape in ((dA, "dA", (L, r, two_m)), (dB, "dB", (L, two_n, r))):
        if t is not None:
            _check_plain(t, name, (torch.float32,), shape)
    _gpu((x, "x"), (dy, "dy"), (A, "A"), (B, "B"), (alpha, "alpha"), (seg_start, "seg_start"),
         (seg_adapter, "seg_adapter"), (dx_base, "dx_base"), (dx, "dx"), (dA, "dA"), (dB, "dB"), (workspace, "workspace"))
    raise ValueError("fairy2i_lora_backward: the arguments do not fit together")


def _check_head(h, W, target):
    """h [N][K], W [V][K] of one dtype and target int64 [N]; returns (N, V, K)."""
    _tensor(h, "h")
    _tensor(W, "W")
    _dtype(h, "h", torch.float32, torch.bfloat16)
    _dtype(W, "W", h.dtype)
    if h.dim() != 2:
        raise ValueError(f"h: shape {tuple(h.shape)}, need [N][K]")
    if W.dim() != 2 or W.shape[1] != h.shape[1]:
        raise ValueError(f"W: shape {tuple(W.shape)}, need [V][{h.shape[1]}]")
    _on_gpu(h, "h")
    _on_gpu(W, "W")
    _check_plain(target, "target", (torch.int64,), (h.shape[0],))
    return h.shape[0], W.shape[0], h.shape[1]


def fairy2i_vocab_loss_workspace_bytes(N: int, V: int, K: int, x_dtype: int) -> int:
    return int(lib().fairy2i_vocab_loss_workspace_bytes(N, V, K, x_dtype))


@_on_stream
def fairy2i_vocab_loss(h: torch.Tensor, W: torch.Tensor, target: torch.Tensor, *, loss=None, lse=None, workspace=None):
    """Per-token cross entropy of the vocabulary projection l = h W^T, h [N][K], W [V][K], without
    storing l: (loss, lse) fp32 [N].  Tokens whose target (int64) is outside [0, V) get loss 0."""
    N, V, K = _check_head(h, W, target)
    f32 = torch.float32
    if loss is not None:
        _check_plain(loss, "loss", (f32,), (N,))
    if lse is not None:
        _check_plain(lse, "lse", (f32,), (N,))
    _gpu((h, "h"), (W, "W"), (target, "target"), (loss, "loss"), (lse, "lse"))
    loss = torch.empty((N,), dtype=f32, device=h.device) if loss is None else loss
    lse = torch.empty((N,), dtype=f32, device=h.device) if lse is None else lse
    code = _DTYPE[h.dtype]
    ws, nbytes, keep = _room(workspace, fairy2i_vocab_loss_workspace_bytes(N, V, K, code), h.device)
    _check(lib().fairy2i_vocab_loss(h.data_ptr(), W.data_ptr(), code, N, V, K, target.data_ptr(), loss.data_ptr(),
                                    lse.data_ptr(), ws, nbytes, _stream()))
    return loss, lse


def fairy2i_vocab_loss_backward_workspace_bytes(N: int, V: int, K: int, x_dtype: int) -> int:
    return int(lib().fairy2i_vocab_loss_backward_workspace_bytes(N, V, K, x_dtype))


@_on_stream
def fairy2i_vocab_loss_backward(h: torch.Tensor, W: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                                g: torch.Tensor, *, want_dh: bool = True, want_dW: bool = True, dh=None, dW=None,
                                workspace=None):
    """Gradient of fairy2i_vocab_loss: lse from the forward call, g fp32 [N] the gradient of each
    token's loss.  Returns (dh [N][K] or None, dW [V][K] or None), h's dtype; want_dh / want_dW False
    skip one of them (a frozen W needs no dW)."""
    N, V, K = _check_head(h, W, target)
    _check_plain(lse, "lse", (torch.float32,), (N,))
    _check_plain(g, "g", (torch.float32,), (N,))
    if not want_dh and not want_dW:
        raise ValueError("fairy2i_vocab_loss_backward: nothing to compute")
    if (dh is not None and not want_dh) or (dW is not None and not want_dW):
        raise ValueError("an output was given for a gradient that is not wanted")
    if dh is not None:
        _check_plain(dh, "dh", (h.dtype,), (N, K))
    if dW is not None:
        _check_plain(dW, "dW", (h.dtype,), (V, K))
    _gpu((h, "h"), (W, "W"), (target, "target"), (lse, "lse"), (g, "g"), (dh, "dh"), (dW, "dW"))
    dh = torch.empty_like(h) if want_dh and dh is None else dh
    dW = torch.empty_like(W) if want_dW and dW is None else dW
    code = _DTYPE[h.dtype]
    ws, nbytes, keep = _room(workspace, fairy2i_vocab_loss_backward_workspace_bytes(N, V, K, code), h.device)
    _check(lib().fairy2i_vocab_loss_backward(h.data_ptr(), W.data_ptr(), code, N, V, K, target.data_ptr(), lse.data_ptr(),
                                             g.data_ptr(), _ptr(dh), _ptr(dW), ws, nbytes, _stream()))
    return dh, dW


def fairy2i_clip_grads_workspace_bytes(numels) -> int:
    numels = list(numels)
    return int(lib().fairy2i_clip_grads_workspace_bytes(len(numels), (_I64 * len(numels))(*numels)))


_dtype_of = operator.attrgetter("dtype")


@_on_stream
def fairy2i_clip_grads(grads, max_norm: float, *, out=None, norm=None, workspace=None) -> torch.Tensor:
    """Global norm of a list of gradients (fp32 or bf16 each, on one GPU) and clipping to max_norm:
    each gradient times min(1, max_norm / (norm + 1e-6)), in place or into the list `out`.  Returns
    the norm, fp32 [1]."""
    Tensor, n = torch.Tensor, len(grads)
    outs = grads if out is None else list(out)
    # a stack's adapters are hundreds of tensors: each property is read once, in a loop of its own
    try:
        ptrs, counts, dtypes = list(map(Tensor.data_ptr, grads)), list(map(Tensor.numel, grads)), list(map(_dtype_of, grads))
        dev = grads[0].get_device()
        good = (max_norm >= 0 and dev >= 0 and set(dtypes) <= _FLOATS and all(map(Tensor.is_contiguous, grads))
                and set(map(Tensor.get_device, grads)) == {dev} and (norm is None or _fits(norm, torch.float32, (1,), dev)))
        to = ptrs
        if out is not None:
            to = list(map(Tensor.data_ptr, outs))
            good = (good and list(map(_dtype_of, outs)) == dtypes and all(map(Tensor.is_contiguous, outs))
                    and set(map(Tensor.get_device, outs)) == {dev} and list(map(Tensor.numel, outs)) == counts)
    except (AttributeError, IndexError, TypeError):
        good = False
    if not good:
        _refuse_clip(grads, outs, max_norm, norm)
    numel = array.array("q", counts)
    one = dtypes.count(dtypes[0]) == n
    codes = array.array("i", [_DTYPE[dtypes[0]]]) * n if one else array.array("i", [_DTYPE[d] for d in dtypes])
    address = lambda a, kind: ctypes.cast(a.buffer_info()[0], ctypes.POINTER(kind))
    from_, to_ = array.array("Q", ptrs), array.array("Q", to)
    norm = torch.empty((1,), dtype=torch.float32, device=grads[0].device) if norm is None else norm
    sizes = address(numel, _I64)
    ws, nbytes, keep = _room(workspace, lib().fairy2i_clip_grads_workspace_bytes(n, sizes), norm.device)
    _check(lib().fairy2i_clip_grads(n, address(from_, _P), None if out is None else address(to_, _P), sizes,
                                    address(codes, _INT), max_norm, norm.data_ptr(), ws, nbytes, _stream()))
    return norm


def _refuse_clip(grads, outs, max_norm, norm):
    """Raises for the first argument of fairy2i_clip_grads that does not fit."""
    if not grads:
        raise ValueError("fairy2i_clip_grads: no gradients")
    if len(outs) != len(grads):
        raise ValueError(f"out: {len(outs)} outputs for {len(grads)} gradients")
    for k, (g, o) in enumerate(zip(grads, outs)):
        _tensor(g, f"grads[{k}]")
        _dtype(g, f"grads[{k}]", torch.float32, torch.bfloat16)
        _on_gpu(g, f"grads[{k}]")
        if o is not g:
            _tensor(o, f"out[{k}]")
            _dtype(o, f"out[{k}]", g.dtype)
            if o.numel() != g.numel():
                raise ValueError(f"out[{k}]: {o.numel()} elements, its gradient has {g.numel()}")
            _on_gpu(o, f"out[{k}]")
            if _overlap(o, g):
                raise ValueError(f"out[{k}]: overlaps its gradient without being it")
    if not max_norm >= 0:
        raise ValueError(f"max_norm: {max_norm}, need at least 0")
    if norm is not None:
        _check_plain(norm, "norm", (torch.float32,), (1,))
    _gpu(*[(g, f"grads[{k}]") for k, g in enumerate(grads)], *[(o, f"out[{k}]") for k, o in enumerate(outs)], (norm, "norm"))
    raise ValueError("fairy2i_clip_grads: the arguments do not fit together")


# ---- a packed layer beside the model it came from: layers kept at four bits ----

class W4Layer:
    """A layer kept at four bits, as fairy2i_pack_w4 lays it out: the uint8 buffer, its rows, columns and
    group, and the dtype its scales are held in."""

    def __init__(self, buf: torch.Tensor, rows: int, cols: int, group: int, scales_dtype=torch.bfloat16):
        _tensor(buf, "buf")
        _dtype(buf, "buf", torch.uint8)
        if scales_dtype not in _FLOATS:
            raise ValueError(f"scales_dtype: {scales_dtype}, need torch.float32 or torch.bfloat16")
        nbytes = fairy2i_packed_bytes_w4(rows, cols, group, scales_dtype)
        if nbytes == 0:
            raise ValueError(f"rows = {rows}, cols = {cols}, group = {group}: sizes out of range")
        _min_bytes(buf, "buf", nbytes)
        _on_gpu(buf, "buf")
        self.buf, self.rows, self.cols, self.group, self.scales_dtype = buf, rows, cols, group, scales_dtype

    @property
    def device(self):
        return self.buf.device


def fairy2i_packed_bytes_w4(rows: int, cols: int, group: int, scales_dtype=torch.bfloat16) -> int:
    return int(lib().fairy2i_packed_bytes_w4(rows, cols, group, _DTYPE[scales_dtype]))


@_on_stream
def fairy2i_pack_w4(codes: torch.Tensor, scales: torch.Tensor, group: int, zeros=None, *, packed=None) -> W4Layer:
    """codes uint8 [rows][cols] (0..15, one a byte), scales [rows][ceil(cols / group)] (fp32 or bf16) and zero
    points uint8 of the same shape (None: 8) -> the layer W = scale (code - zero), laid out for
    fairy2i_gemv_w4.  packed: a uint8 buffer to fill (allocated when None)."""
    _tensor(codes, "codes")
    _dtype(codes, "codes", torch.uint8)
    if codes.dim() != 2:
        raise ValueError(f"codes: shape {tuple(codes.shape)}, need [rows][cols]")
    if group not in (32, 64, 128):
        raise ValueError(f"group: {group}, need 32, 64 or 128")
    rows, cols = codes.shape
    _on_gpu(codes, "codes")
    _check_plain(scales, "scales", (torch.float32, torch.bfloat16), (rows, -(-cols // group)))
    if zeros is not None:
        _check_plain(zeros, "zeros", (torch.uint8,), (rows, -(-cols // group)))
    if packed is None:
        packed = torch.empty((fairy2i_packed_bytes_w4(rows, cols, group, scales.dtype),), dtype=torch.uint8, device=codes.device)
    layer = W4Layer(packed, rows, cols, group, scales.dtype)
    _gpu((codes, "codes"), (scales, "scales"), (zeros, "zeros"), (packed, "packed"))
    _check(lib().fairy2i_pack_w4(codes.data_ptr(), scales.data_ptr(), _DTYPE[scales.dtype], _ptr(zeros), rows, cols, group,
                                 packed.data_ptr(), _stream()))
    return layer


def fairy2i_gemv_w4(layer: W4Layer, x: torch.Tensor, *, y_dtype=torch.float32, y=None, stream=None) -> torch.Tensor:
    """y = x W^T of a layer kept at four bits: x [B][cols] fp32 or bf16, B <= 16 -> y [B][rows]."""
    if not isinstance(layer, W4Layer):
        raise TypeError(f"layer: expected a W4Layer, got {type(layer).__name__}")
    scope = _scope(x, stream)
    if scope is _HERE_SCOPE:
        return _gemv_w4(layer, x, y_dtype, y)
    with scope:
        return _gemv_w4(layer, x, y_dtype, y)


def _gemv_w4(layer, x, y_dtype, y):
    dev = layer.buf.get_device()
    if not (isinstance(x, torch.Tensor) and x.dtype in _FLOATS and x.dim() == 2 and x.shape[1] == layer.cols
            and x.is_contiguous() and x.get_device() == dev >= 0
            and (y is None or isinstance(y, torch.Tensor) and y.dtype in _FLOATS
                 and _fits(y, y.dtype, (x.shape[0], layer.rows), dev))):
        _refuse_gemv_w4(layer, x, y)
    B = x.shape[0]
    if y is None:
        if y_dtype not in _FLOATS:
            raise ValueError(f"y_dtype: {y_dtype}, need torch.float32 or torch.bfloat16")
        y = x.new_empty((B, layer.rows), dtype=y_dtype)
    _check(lib().fairy2i_gemv_w4(layer.buf.data_ptr(), layer.rows, layer.cols, layer.group, _DTYPE[layer.scales_dtype],
                                 x.data_ptr(), _DTYPE[x.dtype], B, y.data_ptr(), _DTYPE[y.dtype], _here(dev)))
    return y


def _refuse_gemv_w4(layer, x, y):
    """Raises for the first argument of fairy2i_gemv_w4 that does not fit."""
    _tensor(x, "x")
    _dtype(x, "x", torch.float32, torch.bfloat16)
    if x.dim() != 2 or x.shape[1] != layer.cols:
        raise ValueError(f"x: shape {tuple(x.shape)}, need [B][{layer.cols}]")
    _on_gpu(x, "x")
    if y is not None:
        _check_y(y, (x.shape[0], layer.rows), x.device)
    _gpu((layer.buf, "layer"), (x, "x"), (y, "y"))
    raise ValueError("fairy2i_gemv_w4: the arguments do not fit together")


# ---- distillation from a teacher's top logits ----

def _check_lists(h, W, top_index, top_logit):
    """h [N][K], W [V][K] of one dtype and lists [N][top]; returns (N, V, K, top)."""
    _tensor(h, "h")
    _tensor(W, "W")
    _dtype(h, "h", torch.float32, torch.bfloat16)
    _dtype(W, "W", h.dtype)
    if h.dim() != 2:
        raise ValueError(f"h: shape {tuple(h.shape)}, need [N][K]")
    if W.dim() != 2 or W.shape[1] != h.shape[1]:
        raise ValueError(f"W: shape {tuple(W.shape)}, need [V][{h.shape[1]}]")
    _on_gpu(h, "h")
    _on_gpu(W, "W")
    _tensor(top_index, "top_index")
    _dtype(top_index, "top_index", torch.int64)
    if top_index.dim() != 2 or top_index.shape[0] != h.shape[0]:
        raise ValueError(f"top_index: shape {tuple(top_index.shape)}, need [{h.shape[0]}][top]")
    _on_gpu(top_index, "top_index")
    _check_plain(top_logit, "top_logit", (torch.float32, torch.bfloat16), tuple(top_index.shape))
    return h.shape[0], W.shape[0], h.shape[1], top_index.shape[1]


def fairy2i_distill_workspace_bytes(N: int, V: int, K: int, x_dtype: int, top: int) -> int:
    return int(lib().fairy2i_distill_workspace_bytes(N, V, K, x_dtype, top))


@_on_stream
def fairy2i_distill(h: torch.Tensor, W: torch.Tensor, top_index: torch.Tensor, top_logit: torch.Tensor,
                    temperature: float = 1.0, *, loss=None, lse=None, workspace=None):
    """Per-token divergence of the student's softmax(h W^T / temperature), h [N][K], W [V][K], from the
    teacher's, known by its top logits: top_index int64 [N][top] (outside [0, V): unused slot), top_logit fp32
    or bf16.  Returns (loss, lse) fp32 [N]; tokens with an empty list get loss 0."""
    N, V, K, top = _check_lists(h, W, top_index, top_logit)
    f32 = torch.float32
    if loss is not None:
        _check_plain(loss, "loss", (f32,), (N,))
    if lse is not None:
        _check_plain(lse, "lse", (f32,), (N,))
    _gpu((h, "h"), (W, "W"), (top_index, "top_index"), (top_logit, "top_logit"), (loss, "loss"), (lse, "lse"))
    loss = torch.empty((N,), dtype=f32, device=h.device) if loss is None else loss
    lse = torch.empty((N,), dtype=f32, device=h.device) if lse is None else lse
    code = _DTYPE[h.dtype]
    ws, nbytes, keep = _room(workspace, fairy2i_distill_workspace_bytes(N, V, K, code, top), h.device)
    _check(lib().fairy2i_distill(h.data_ptr(), W.data_ptr(), code, N, V, K, top_index.data_ptr(), top_logit.data_ptr(),
                                 _DTYPE[top_logit.dtype], top, temperature, loss.data_ptr(), lse.data_ptr(), ws, nbytes,
                                 _here(h.get_device())))
    return loss, lse


def fairy2i_distill_backward_workspace_bytes(N: int, V: int, K: int, x_dtype: int, top: int) -> int:
    return int(lib().fairy2i_distill_backward_workspace_bytes(N, V, K, x_dtype, top))


@_on_stream
def fairy2i_distill_backward(h: torch.Tensor, W: torch.Tensor, top_index: torch.Tensor, top_logit: torch.Tensor,
                             lse: torch.Tensor, g: torch.Tensor, temperature: float = 1.0, *, want_dh: bool = True,
                             want_dW: bool = True, dh=None, dW=None, workspace=None):
    """Gradient of fairy2i_distill: lse from the forward call, g fp32 [N] the gradient of each token's loss.
    Returns (dh [N][K] or None, dW [V][K] or None), h's dtype; want_dh / want_dW False skip one of them."""
    N, V, K, top = _check_lists(h, W, top_index, top_logit)
    _check_plain(lse, "lse", (torch.float32,), (N,))
    _check_plain(g, "g", (torch.float32,), (N,))
    if not want_dh and not want_dW:
        raise ValueError("fairy2i_distill_backward: nothing to compute")
    if (dh is not None and not want_dh) or (dW is not None and not want_dW):
        raise ValueError("an output was given for a gradient that is not wanted")
    if dh is not None:
        _check_plain(dh, "dh", (h.dtype,), (N, K))
    if dW is not None:
        _check_plain(dW, "dW", (h.dtype,), (V, K))
    _gpu((h, "h"), (W, "W"), (top_index, "top_index"), (top_logit, "top_logit"), (lse, "lse"), (g, "g"), (dh, "dh"),
         (dW, "dW"))
    dh = torch.empty_like(h) if want_dh and dh is None else dh
    dW = torch.empty_like(W) if want_dW and dW is None else dW
    code = _DTYPE[h.dtype]
    ws, nbytes, keep = _room(workspace, fairy2i_distill_backward_workspace_bytes(N, V, K, code, top), h.device)
    _check(lib().fairy2i_distill_backward(h.data_ptr(), W.data_ptr(), code, N, V, K, top_index.data_ptr(),
                                          top_logit.data_ptr(), _DTYPE[top_logit.dtype], top, temperature, lse.data_ptr(),
                                          g.data_ptr(), _ptr(dh), _ptr(dW), ws, nbytes, _stream()))
    return dh, dW


# ---- verification of drafted tokens ----

def fairy2i_verify_draft_workspace_bytes(S: int, D: int, V: int) -> int:
    return int(lib().fairy2i_verify_draft_workspace_bytes(S, D, V))


@_on_stream
def fairy2i_verify_draft(p: torch.Tensor, q, draft: torch.Tensor, u: torch.Tensor, r: torch.Tensor, *, draft_len=None,
                         tokens=None, accepted=None, workspace=None):
    """Drafted tokens against the target's probabilities: p [S][D + 1][V] of the target, q [S][D][V] of the
    draft (None: it was greedy), fp32 or bf16, draft int64 [S][D] and, if they differ, draft_len int32 [S], u
    fp32 [S][D] and r fp32 [S] uniform in [0, 1).  Returns (tokens int64 [S][D + 1]: the kept drafts, the
    next token, then -1; accepted int32 [S])."""
    i64, i32, f32 = torch.int64, torch.int32, torch.float32
    try:
        dt, dev = p.dtype, p.get_device()
        S, D1, V = p.shape
        D = D1 - 1
        good = (dt in _FLOATS and dev >= 0 and p.is_contiguous() and (q is None or _fits(q, dt, (S, D, V), dev))
                and _fits(draft, i64, (S, D), dev) and _fits(u, f32, (S, D), dev) and _fits(r, f32, (S,), dev)
                and (draft_len is None or _fits(draft_len, i32, (S,), dev))
                and (tokens is None or _fits(tokens, i64, (S, D1), dev))
                and (accepted is None or _fits(accepted, i32, (S,), dev)))
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _refuse_verify(p, q, draft, u, r, draft_len, tokens, accepted)
    tokens = p.new_empty((S, D1), dtype=i64) if tokens is None else tokens
    accepted = p.new_empty((S,), dtype=i32) if accepted is None else accepted
    nbytes = lib().fairy2i_verify_draft_workspace_bytes(S, D, V)
    ws = None
    if nbytes or workspace is not None:
        ws, nbytes, keep = _room(workspace, nbytes, p.device)
    _check(lib().fairy2i_verify_draft(p.data_ptr(), None if q is None else q.data_ptr(), _DTYPE[dt], S, D, V, draft.data_ptr(),
                                      None if draft_len is None else draft_len.data_ptr(), u.data_ptr(), r.data_ptr(),
                                      tokens.data_ptr(), accepted.data_ptr(), ws, nbytes, _here(dev)))
    return tokens, accepted


def _refuse_verify(p, q, draft, u, r, draft_len, tokens, accepted):
    """Raises for the first argument of fairy2i_verify_draft that does not fit."""
    _tensor(p, "p")
    _dtype(p, "p", torch.float32, torch.bfloat16)
    if p.dim() != 3 or p.shape[1] < 2:
        raise ValueError(f"p: shape {tuple(p.shape)}, need [S][D + 1][V]")
    _on_gpu(p, "p")
    S, D, V = p.shape[0], p.shape[1] - 1, p.shape[2]
    if q is not None:
        _check_plain(q, "q", (p.dtype,), (S, D, V))
    _check_plain(draft, "draft", (torch.int64,), (S, D))
    _check_plain(u, "u", (torch.float32,), (S, D))
    _check_plain(r, "r", (torch.float32,), (S,))
    for t, name, dt, shape in ((draft_len, "draft_len", torch.int32, (S,)), (tokens, "tokens", torch.int64, (S, D + 1)),
                               (accepted, "accepted", torch.int32, (S,))):
        if t is not None:
            _check_plain(t, name, (dt,), shape)
    _gpu((p, "p"), (q, "q"), (draft, "draft"), (u, "u"), (r, "r"), (draft_len, "draft_len"), (tokens, "tokens"),
         (accepted, "accepted"))
    raise ValueError("fairy2i_verify_draft: the arguments do not fit together")
