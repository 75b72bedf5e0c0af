"""Python binding of the microscaled 4-bit matrices (``include/nf4_mx.h``): E2M1
elements with a power of two for each 32 of a row, and products of two such
matrices. Argument marshalling only, as in the package's other calls.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DT, _check, _lib_functions, _workspace

_P = ctypes.c_void_p
_I32, _I64 = ctypes.c_int32, ctypes.c_int64


class MXMatrixDesc(ctypes.Structure):
    """ctypes mirror of ``nf4_mx_matrix``."""

    _fields_ = [("codes", _P), ("scales", _P), ("rows", _I64), ("cols", _I64)]


_MATRIX = ctypes.POINTER(MXMatrixDesc)
# (name, restype, argtypes) of every entry point of nf4_mx.h
_SIGNATURES = [
    ("nf4_mx_padded", _I64, [_I64]),
    ("nf4_mx_quantize", _I32, [_P, _I32, _I64, _I64, _I64, _P, _P, _P]),
    ("nf4_mx_dequantize", _I32, [_MATRIX, _I32, _P, _I64, _P]),
    ("nf4_mx_matmul_workspace_bytes", _I64, [_I64] * 3),
    ("nf4_mx_linear_workspace_bytes", _I64, [_I64] * 3),
    ("nf4_mx_matmul", _I32, [_MATRIX, _MATRIX, _P, _I32, _P, _I64, _P, _I64, _P]),
    ("nf4_mx_linear", _I32, [_P, _I32, _I64, _I64, _MATRIX, _P, _I32, _P, _I64, _P, _I64, _P]),
]

_fns = None


def _lib():
    global _fns
    if _fns is None:
        _fns = _lib_functions(_SIGNATURES)
    return _fns


def mx_exported_names() -> list[str]:
    return [s[0] for s in _SIGNATURES]


def mx_padded(cols: int) -> int:
    """Columns that rows of ``cols`` elements are padded to."""
    return -(-cols // 128) * 128


class MXTensor:
    """A microscaled 4-bit matrix of ``shape`` [rows, cols]: uint8 ``codes`` [rows,
    padded / 2] and ``scales`` [padded / 128, rows, 4] on one GPU, contiguous, with
    padded = mx_padded(cols); nf4_mx.h says what they hold."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, shape):
        rows, cols = shape
        padded = -(-cols // 128) * 128
        u8 = torch.uint8
        if codes.dtype is not u8 or scales.dtype is not u8 or codes.shape != (rows, padded // 2) or \
                scales.shape != (padded // 128, rows, 4):
            raise ValueError("MXTensor expects uint8 codes [rows, padded / 2] and scales "
                             "[padded / 128, rows, 4]")
        if not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("MXTensor expects contiguous codes and scales")
        index = codes.get_device()
        if index < 0 or scales.get_device() != index:
            raise TypeError("MXTensor expects two tensors on one GPU")
        self._set(codes, scales, rows, cols, index)

    def _set(self, codes, scales, rows, cols, index):
        self.codes, self.scales, self.shape = codes, scales, (rows, cols)
        self.index = index  # of the GPU
        self.desc = MXMatrixDesc(codes.data_ptr(), scales.data_ptr(), rows, cols)

    @classmethod
    def _like(cls, x: torch.Tensor, rows: int, cols: int, index: int) -> "MXTensor":
        """An uninitialised matrix beside x, on the GPU ``index``."""
        padded = -(-cols // 128) * 128
        t = cls.__new__(cls)
        t._set(x.new_empty((rows, padded // 2), dtype=torch.uint8),
               x.new_empty((padded // 128, rows, 4), dtype=torch.uint8), rows, cols, index)
        return t

    @property
    def device(self) -> torch.device:
        return self.codes.device

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "MXTensor":
        """An uninitialised matrix."""
        padded = mx_padded(cols)
        return cls(torch.empty(rows, padded // 2, dtype=torch.uint8, device=device),
                   torch.empty(padded // 128, rows, 4, dtype=torch.uint8, device=device),
                   (rows, cols))

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


# a device's current stream and the current device, without the objects around them
_stream_of = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice


def _call(index: int, name: str, *args) -> None:
    """The entry point `name` with the GPU ``index`` current, on its current stream."""
    fn = getattr(_lib(), name)
    if index == _current():
        status = fn(*args, _stream_of(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _stream_of(index))
    if status:
        _check(status, name)


def _input(x: torch.Tensor, what: str):
    """(tensor, rows, cols, row stride) of x as [rows, cols] with unit element stride."""
    if x.dtype not in _DT or not x.is_cuda:
        raise TypeError(f"{what} expects bf16 / fp16 / fp32 values on the GPU")
    if x.dim() == 2:
        rows, cols = x.shape
        ld, one = x.stride()
        if (one == 1 or cols <= 1) and (ld >= cols or rows <= 1):
            return x, rows, cols, ld if rows > 1 else cols
    if x.dim() == 0:
        raise ValueError(f"{what} expects rows of values")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    return x.reshape(rows, cols).contiguous(), rows, cols, cols


def _output(out, rows: int, cols: int, index: int, what: str) -> int:
    """The row stride of an output that the caller gives."""
    if out.dtype not in _DT or out.get_device() != index or out.shape != (rows, cols) or \
            (cols > 1 and out.stride(1) != 1) or (rows > 1 and out.stride(0) < cols):
        raise ValueError(f"{what}: out must be a [{rows}, {cols}] view with unit column stride "
                         "on the same GPU")
    return out.stride(0) if rows > 1 else cols


def mx_quantize(x: torch.Tensor, out: MXTensor | None = None) -> MXTensor:
    """nf4_mx_quantize: x [..., cols] (bf16 / fp16 / fp32, rows of any stride) as a
    microscaled matrix of its rows, into ``out`` where given."""
    x, rows, cols, ld = _input(x, "mx_quantize")
    index = x.get_device()
    if out is None:
        out = MXTensor._like(x, rows, cols, index)
    elif out.shape != (rows, cols) or out.index != index:
        raise ValueError("mx_quantize: out must be of x's shape, on its GPU")
    _call(index, "nf4_mx_quantize", x.data_ptr(), _DT[x.dtype], rows, cols, ld, out.desc.codes,
          out.desc.scales)
    return out


def mx_dequantize(m: MXTensor, dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """nf4_mx_dequantize: the values [rows, cols] in ``dtype`` (or into ``out``, in its dtype)."""
    rows, ld = m.shape
    if out is None:
        if dtype not in _DT:
            raise TypeError("mx_dequantize gives bf16, fp16 or fp32")
        out = m.codes.new_empty(m.shape, dtype=dtype)
    else:
        ld = _output(out, rows, ld, m.index, "mx_dequantize")
    _call(m.index, "nf4_mx_dequantize", m.desc, _DT[out.dtype], out.data_ptr(), ld)
    return out


def mx_workspace_bytes(M: int, N: int, K: int, quantized: bool = False) -> int:
    """nf4_mx_linear_workspace_bytes, or nf4_mx_matmul_workspace_bytes (``quantized``), on the
    current device."""
    fn = _lib().nf4_mx_matmul_workspace_bytes if quantized else _lib().nf4_mx_linear_workspace_bytes
    return fn(M, N, K)


def mx_linear(x, w: MXTensor, bias: torch.Tensor | None = None, out_dtype=None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """y[M, N] = MX(x)[M, K] . W^T (+ bias[N]) with W = w of shape (N, K), both sides in
    microscaled 4 bits and summed in fp32. x [..., K] is quantized in the call
    (nf4_mx_linear), or is an MXTensor itself (nf4_mx_matmul); the workspace is allocated
    here. out_dtype defaults to x's, for an MXTensor to bf16; the bias is of that type, and is
    added before the rounding to it."""
    N, K = w.shape
    index = w.index
    quantized = isinstance(x, MXTensor)
    if quantized:
        M, cols = x.shape
        dtype = torch.bfloat16
    else:
        x, M, cols, ldx = _input(x, "mx_linear")
        dtype = x.dtype
    if out is not None:
        dtype = out.dtype
    elif out_dtype is not None:
        dtype = out_dtype
    if dtype not in _DT:
        raise TypeError("mx_linear gives bf16, fp16 or fp32")
    if cols != K or (x.index if quantized else x.get_device()) != index:
        raise ValueError("mx_linear expects x [..., K] and w (N, K) on one GPU")
    bp = None
    if bias is not None:
        if bias.dtype != dtype or bias.get_device() != index or bias.numel() != N:
            raise ValueError("mx_linear expects a bias of N elements of the output's dtype on the "
                             "same GPU")
        bias = bias.reshape(-1).contiguous()
        bp = bias.data_ptr()
    ldy = N
    if out is None:
        out = w.codes.new_empty((M, N), dtype=dtype)
    else:
        ldy = _output(out, M, N, index, "mx_linear")
    if index == _current():
        need = mx_workspace_bytes(M, N, K, quantized)
    else:
        with torch.cuda.device(index):
            need = mx_workspace_bytes(M, N, K, quantized)
    ws, nbytes, _keep = _workspace(need, out.device) if need > 0 else (None, 0, None)
    if quantized:
        _call(index, "nf4_mx_matmul", x.desc, w.desc, bp, _DT[dtype], out.data_ptr(), ldy, ws, nbytes)
    else:
        _call(index, "nf4_mx_linear", x.data_ptr(), _DT[x.dtype], ldx, M, w.desc, bp, _DT[dtype],
              out.data_ptr(), ldy, ws, nbytes)
    return out


__all__ = ["MXTensor", "MXMatrixDesc", "mx_padded", "mx_quantize", "mx_dequantize", "mx_linear",
           "mx_workspace_bytes", "mx_exported_names"]
