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
        padded = mx_padded(cols)
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
        self.codes, self.scales, self.shape = codes, scales, (rows, cols)
        self.index = index  # of the GPU
        self.desc = MXMatrixDesc(codes.data_ptr(), scales.data_ptr(), rows, cols)

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


def _call(index: int, run) -> None:
    """run(stream) -> (status, name) with the GPU ``index`` current, on its current stream."""
    if index == torch.cuda.current_device():
        status, name = run(torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status, name = run(torch._C._cuda_getCurrentRawStream(index))
    if status:
        _check(status, name)


def _input(x: torch.Tensor, what: str):
    """(tensor, row stride) of x as [rows, cols] with unit element stride."""
    if x.dtype not in _DT or not x.is_cuda:
        raise TypeError(f"{what} expects bf16 / fp16 / fp32 values on the GPU")
    if x.dim() == 0:
        raise ValueError(f"{what} expects rows of values")
    cols = x.shape[-1]
    if x.dim() != 2 or (cols > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < cols):
        x = x.reshape(x.numel() // cols if cols else 0, cols).contiguous()
    return x, (x.stride(0) if x.shape[0] > 1 else cols)


def _output(out, shape, dtype, index: int, what: str):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index)), shape[1]
    if out.dtype not in _DT or out.get_device() != index or out.shape != shape or \
            (shape[1] > 1 and out.stride(1) != 1) or (shape[0] > 1 and out.stride(0) < shape[1]):
        raise ValueError(f"{what}: out must be a [{shape[0]}, {shape[1]}] view with unit column "
                         "stride on the same GPU")
    return out, (out.stride(0) if shape[0] > 1 else shape[1])


def mx_quantize(x: torch.Tensor, out: MXTensor | None = None) -> MXTensor:
    """nf4_mx_quantize: x [..., cols] (bf16 / fp16 / fp32, rows of any stride) as a
    microscaled matrix of its rows, into ``out`` where given."""
    x, ld = _input(x, "mx_quantize")
    rows, cols = x.shape
    index = x.get_device()
    if out is None:
        out = MXTensor.empty(rows, cols, x.device)
    elif out.shape != (rows, cols) or out.index != index:
        raise ValueError("mx_quantize: out must be of x's shape, on its GPU")
    _call(index, lambda stream: (_lib().nf4_mx_quantize(
        x.data_ptr(), _DT[x.dtype], rows, cols, ld, out.desc.codes, out.desc.scales, stream),
        "nf4_mx_quantize"))
    return out


def mx_dequantize(m: MXTensor, dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """nf4_mx_dequantize: the values [rows, cols] in ``dtype`` (or into ``out``, in its dtype)."""
    if out is None and dtype not in _DT:
        raise TypeError("mx_dequantize gives bf16, fp16 or fp32")
    out, ld = _output(out, m.shape, dtype, m.index, "mx_dequantize")
    _call(m.index, lambda stream: (_lib().nf4_mx_dequantize(
        m.desc, _DT[out.dtype], out.data_ptr(), ld, stream), "nf4_mx_dequantize"))
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
    quantized = isinstance(x, MXTensor)
    if quantized:
        ldx, index = 0, x.index
        dtype = out_dtype or torch.bfloat16
    else:
        x, ldx = _input(x, "mx_linear")
        index, dtype = x.get_device(), out_dtype or x.dtype
    if out is not None:
        dtype = out.dtype
    if dtype not in _DT:
        raise TypeError("mx_linear gives bf16, fp16 or fp32")
    M = x.shape[0]
    if x.shape[1] != K or index != w.index:
        raise ValueError("mx_linear expects x [..., K] and w (N, K) on one GPU")
    if bias is not None:
        if bias.dtype != dtype or bias.get_device() != index or bias.numel() != N:
            raise ValueError("mx_linear expects a bias of N elements of the output's dtype on the "
                             "same GPU")
        bias = bias.reshape(-1).contiguous()
    out, ldy = _output(out, (M, N), dtype, index, "mx_linear")
    bp = None if bias is None else bias.data_ptr()

    def run(stream):
        lib = _lib()
        need = mx_workspace_bytes(M, N, K, quantized)
        ws, nbytes, _keep = _workspace(need, out.device)
        if quantized:
            return lib.nf4_mx_matmul(x.desc, w.desc, bp, _DT[dtype], out.data_ptr(), ldy, ws,
                                     nbytes, stream), "nf4_mx_matmul"
        return lib.nf4_mx_linear(x.data_ptr(), _DT[x.dtype], ldx, M, w.desc, bp, _DT[dtype],
                                 out.data_ptr(), ldy, ws, nbytes, stream), "nf4_mx_linear"

    _call(index, run)
    return out


__all__ = ["MXTensor", "MXMatrixDesc", "mx_padded", "mx_quantize", "mx_dequantize", "mx_linear",
           "mx_workspace_bytes", "mx_exported_names"]
