"""Python binding of the 4-bit key/value cache (``include/nf4_kv.h``): keys and
values quantized as they are written into a paged cache, read back, and attended
to in their 4 bits. Argument marshalling only, as in the package's other calls.

The sequences of a call are given by ``block_table`` (int32 [batch, pages of a
sequence], -1 for none), ``kv_lens`` (int32 [batch], positions cached, the ones
written in the same call included) and ``row_offsets`` (int32 [batch + 1], or
None where every sequence has equally many rows). Rows row_offsets[b] ...
row_offsets[b + 1] - 1 of the row tensors are sequence b's last positions.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DT, _QT, _check, _lib_functions

_P = ctypes.c_void_p
_I32, _I64 = ctypes.c_int32, ctypes.c_int64


class KVCacheDesc(ctypes.Structure):
    """ctypes mirror of ``nf4_kv_cache``."""

    _fields_ = [("k_packed", _P), ("k_absmax", _P), ("v_packed", _P), ("v_absmax", _P),
                ("num_pages", _I64), ("packed_page_stride", _I64), ("absmax_page_stride", _I64),
                ("page_size", _I32), ("num_kv_heads", _I32), ("head_dim", _I32),
                ("blocksize", _I32), ("quant_type", _I32)]


class KVRowsDesc(ctypes.Structure):
    """ctypes mirror of ``nf4_kv_rows``."""

    _fields_ = [("block_table", _P), ("kv_lens", _P), ("row_offsets", _P),
                ("table_stride", _I64), ("table_cols", _I32), ("batch", _I32),
                ("total_rows", _I32)]


_CACHE, _ROWS = ctypes.POINTER(KVCacheDesc), ctypes.POINTER(KVRowsDesc)
# (name, restype, argtypes) of every entry point of nf4_kv.h
_SIGNATURES = [
    ("nf4_kv_write", _I32, [_CACHE, _ROWS, _P, _P, _I64, _I64, _I32, _P, _P, _P]),
    ("nf4_kv_read", _I32, [_CACHE, _ROWS, _I32, _P, _P, _I64, _I64, _P]),
    ("nf4_kv_attention_workspace_bytes", _I64, [_I32] * 8),
    ("nf4_kv_attention", _I32,
     [_CACHE, _ROWS, _P, _I64, _I64, _I32, _I32, ctypes.c_float, _I32, _I32, _I32, _I32, _P, _I64,
      _I64, _P, _I64, _P]),
]

_fns = None


def _lib():
    global _fns
    if _fns is None:
        _fns = _lib_functions(_SIGNATURES)
    return _fns


def kv_exported_names() -> list[str]:
    return [s[0] for s in _SIGNATURES]


def _page_stride(shape, stride) -> int:
    """Elements between pages of [pages, heads, positions, width], -1 where a page is not
    contiguous. A dimension of one element may have any stride: it addresses nothing."""
    pages, heads, n, w = shape
    if pages and not ((stride[1] == n * w or heads == 1) and (stride[2] == w or n == 1) and
                      (stride[3] == 1 or w == 1)):
        return -1
    return stride[0] if pages > 1 else heads * n * w


class KVCache:
    """A paged 4-bit key/value cache: uint8 ``k_packed`` and ``v_packed`` [pages,
    kv heads, page_size, head_dim / 2] and fp32 ``k_absmax`` and ``v_absmax``
    [pages, kv heads, page_size, head_dim / blocksize] on the GPU, contiguous
    within a page (pages may lie further apart, keys' and values' equally far).
    The layout of the codes within a head of a page is nf4_kv.h's."""

    def __init__(self, k_packed: torch.Tensor, k_absmax: torch.Tensor, v_packed: torch.Tensor,
                 v_absmax: torch.Tensor, blocksize: int = 64, quant_type: str = "nf4"):
        shape, sshape = k_packed.shape, k_absmax.shape
        if len(shape) != 4 or k_packed.dtype is not torch.uint8 or \
                v_packed.dtype is not torch.uint8:
            raise ValueError("KVCache expects uint8 codes [pages, kv heads, page_size, head_dim / 2]")
        pages, heads, page_size, half = shape
        nb = 2 * half // blocksize if blocksize > 0 else 0
        if v_packed.shape != shape:
            raise ValueError("KVCache expects codes of one shape, contiguous in a page")
        stride = _page_stride(shape, k_packed.stride())
        if stride < 0 or _page_stride(shape, v_packed.stride()) != stride:
            raise ValueError("KVCache expects codes of one shape, contiguous in a page")
        if k_absmax.dtype is not torch.float32 or v_absmax.dtype is not torch.float32 or \
                sshape != (pages, heads, page_size, nb) or v_absmax.shape != sshape:
            raise ValueError("KVCache expects fp32 scales [pages, kv heads, page_size, "
                             "head_dim / blocksize]")
        sstride = _page_stride(sshape, k_absmax.stride())
        if sstride < 0 or _page_stride(sshape, v_absmax.stride()) != sstride:
            raise ValueError("KVCache expects scales contiguous in a page, keys' and values' "
                             "pages equally far apart")
        index = k_packed.get_device()
        if index < 0 or k_absmax.get_device() != index or v_packed.get_device() != index or \
                v_absmax.get_device() != index:
            raise TypeError("KVCache expects four tensors on one GPU")
        self.k_packed, self.k_absmax = k_packed, k_absmax
        self.v_packed, self.v_absmax = v_packed, v_absmax
        self.blocksize, self.quant_type = blocksize, quant_type
        self.num_pages, self.num_kv_heads, self.page_size = pages, heads, page_size
        self.head_dim = 2 * half
        self.index = index  # of the GPU
        self.desc = KVCacheDesc(k_packed.data_ptr(), k_absmax.data_ptr(), v_packed.data_ptr(),
                                v_absmax.data_ptr(), pages, stride, sstride, page_size, heads,
                                2 * half, blocksize, _QT[quant_type])

    @property
    def device(self) -> torch.device:
        return self.k_packed.device

    @classmethod
    def empty(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int,
              blocksize: int = 64, quant_type: str = "nf4", device="cuda") -> "KVCache":
        """A cache of uninitialised pages."""
        shape = (num_pages, num_kv_heads, page_size)
        t = [torch.empty(*shape, head_dim // 2, dtype=torch.uint8, device=device)
             if i % 2 == 0 else
             torch.empty(*shape, head_dim // blocksize, dtype=torch.float32, device=device)
             for i in range(4)]
        return cls(*t, blocksize, quant_type)

    def nbytes(self) -> int:
        return 2 * (self.k_packed.numel() + 4 * self.k_absmax.numel())


def _rows(cache: KVCache, total: int, block_table, kv_lens, row_offsets, what: str) -> KVRowsDesc:
    int32 = torch.int32
    if block_table.dtype is not int32 or kv_lens.dtype is not int32 or \
            block_table.dim() != 2 or kv_lens.dim() != 1:
        raise TypeError(f"{what} expects int32 block_table [batch, pages] and kv_lens [batch]")
    batch, cols = block_table.shape
    stride, inner = block_table.stride()
    if kv_lens.shape[0] != batch or not kv_lens.is_contiguous() or \
            (cols > 1 and inner != 1) or (batch > 1 and stride < cols):
        raise ValueError(f"{what}: block_table needs unit column stride, kv_lens [batch]")
    index = cache.index
    if block_table.get_device() != index or kv_lens.get_device() != index:
        raise TypeError(f"{what} expects every tensor on the cache's GPU")
    off = None
    if row_offsets is not None:
        if row_offsets.dtype is not int32 or row_offsets.shape != (batch + 1,) or \
                not row_offsets.is_contiguous() or row_offsets.get_device() != index:
            raise ValueError(f"{what} expects int32 row_offsets [batch + 1] on the cache's GPU")
        off = row_offsets.data_ptr()
    return KVRowsDesc(block_table.data_ptr(), kv_lens.data_ptr(), off,
                      stride if batch > 1 else cols, cols, batch, total)


def _strides(t: torch.Tensor):
    """(row, head) strides of [rows, heads, head_dim] for the ABI, None where it does not
    take the tensor as it is. The stride of a single row or head addresses nothing and may
    be anything."""
    r, h, e = t.stride()
    n, heads, d = t.shape
    if n <= 1:
        r = heads * d
    if heads <= 1:
        h = d
    es = t.element_size()
    if e == 1 and r >= d and h >= d and not (r * es | h * es | t.data_ptr()) & 15:
        return r, h
    return None


def _empty_rows(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _check_rows(t: torch.Tensor, cache: KVCache, what: str) -> None:
    if t.dtype not in _DT or t.get_device() != cache.index:
        raise TypeError(f"{what} expects bf16 / fp16 / fp32 rows on the cache's GPU")
    if t.dim() != 3 or t.shape[2] != cache.head_dim:
        raise ValueError(f"{what} expects rows [rows, heads, head_dim]")


def _aligned_copy(t: torch.Tensor) -> torch.Tensor:
    u = t.contiguous()  # t itself where it was
    dense = t.shape[1] * t.shape[2], t.shape[2]
    return u if _strides(u) == dense else t.clone(memory_format=torch.contiguous_format)


# the raw handle of a device's current stream: building a Stream object takes longer
# than the launch itself
_stream_of = torch._C._cuda_getCurrentRawStream


def _call(cache: KVCache, run) -> None:
    """run(stream) -> (status, name) with the cache's device current, on its current
    stream."""
    index = cache.index
    if index == torch.cuda.current_device():
        status, name = run(_stream_of(index))
    else:
        with torch.cuda.device(index):
            status, name = run(_stream_of(index))
    if status:
        _check(status, name)


def kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
             kv_lens: torch.Tensor, row_offsets: torch.Tensor | None = None, values: bool = False):
    """nf4_kv_write: quantizes k and v [rows, kv heads, head_dim] into the cache.
    With ``values`` returns (k, v) as the cache now holds them, rounded to their
    dtype, for a computation that is to see what later reads will see."""
    for t in (k, v):
        _check_rows(t, cache, "kv_write")
    if k.dtype != v.dtype or k.shape != v.shape or k.shape[1] != cache.num_kv_heads:
        raise ValueError("kv_write expects k and v [rows, kv heads, head_dim] of one dtype")
    strides = _strides(k)
    if strides is None or _strides(v) != strides:
        k, v = _aligned_copy(k), _aligned_copy(v)
        strides = _strides(k)
    rows = _rows(cache, k.shape[0], block_table, kv_lens, row_offsets, "kv_write")
    kq, vq = (_empty_rows(k), _empty_rows(k)) if values else (None, None)
    rs, hs = strides
    _call(cache, lambda stream: (_lib().nf4_kv_write(
        cache.desc, rows, k.data_ptr(), v.data_ptr(), rs, hs, _DT[k.dtype],
        kq.data_ptr() if values else None, vq.data_ptr() if values else None, stream),
        "nf4_kv_write"))
    return (kq, vq) if values else None


def kv_read(cache: KVCache, rows: int, block_table: torch.Tensor, kv_lens: torch.Tensor,
            row_offsets: torch.Tensor | None = None, dtype=torch.bfloat16, out=None):
    """nf4_kv_read: the last positions of each sequence, ``rows`` in all, as (k, v)
    [rows, kv heads, head_dim] (or into the pair ``out``). Rows behind the last
    offset are left as they are: unspecified without ``out``."""
    shape = (rows, cache.num_kv_heads, cache.head_dim)
    if out is None:
        if dtype not in _DT:
            raise TypeError("kv_read gives bf16, fp16 or fp32")
        k = torch.empty(shape, dtype=dtype, device=cache.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        for t in out:
            _check_rows(t, cache, "kv_read")
            if t.shape != shape or t.dtype != k.dtype or _strides(t) is None or \
                    _strides(t) != _strides(k):
                raise ValueError("kv_read: out must be two [rows, kv heads, head_dim] tensors of "
                                 "one dtype and layout, with 16-byte aligned heads")
    desc = _rows(cache, rows, block_table, kv_lens, row_offsets, "kv_read")
    rs, hs = _strides(k)
    _call(cache, lambda stream: (_lib().nf4_kv_read(
        cache.desc, desc, _DT[k.dtype], k.data_ptr(), v.data_ptr(), rs, hs, stream),
        "nf4_kv_read"))
    return k, v


def _int32(n: int) -> int:
    """A size as the C calls take it (ctypes would drop the upper bits): the largest one is
    past every position."""
    return n if 0 <= n < 0x7ff00000 else (0x7ff00000 if n > 0 else -1)


def kv_attention_workspace_bytes(batch: int, max_rows: int, max_len: int, num_heads: int,
                                 num_kv_heads: int, head_dim: int, dtype=torch.bfloat16,
                                 window: int = 0) -> int:
    """nf4_kv_attention_workspace_bytes on the current device."""
    sizes = map(_int32, (batch, max_rows, max_len, num_heads, num_kv_heads, head_dim))
    return _lib().nf4_kv_attention_workspace_bytes(*sizes, _DT[dtype], _int32(window))


def kv_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                 row_offsets: torch.Tensor | None = None, max_rows: int = 0, max_len: int = 0,
                 scale: float | None = None, causal: bool = True, window: int = 0,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """nf4_kv_attention (with a workspace this call allocates): attention of q
    [rows, heads, head_dim] to the cache, in q's dtype. ``max_rows`` is the most
    rows of a sequence where row_offsets is given (0: that many as there are
    rows), ``max_len`` about the longest of kv_lens (0: what the table can hold);
    both only size the launch, but rows of a sequence past max_rows stay
    unwritten, and a batch of many sequences without max_rows takes several times
    as long. ``scale`` defaults to head_dim ** -0.5. Rows behind the last
    offset are left as they are: unspecified without ``out``."""
    _check_rows(q, cache, "kv_attention")
    total, heads, d = q.shape
    if out is None:
        out = _empty_rows(q)
        out_strides = heads * d, d
    else:
        _check_rows(out, cache, "kv_attention")
        out_strides = _strides(out)
        if out.shape != q.shape or out.dtype != q.dtype or out_strides is None:
            raise ValueError("kv_attention: out must be like q, with 16-byte aligned heads")
    strides = _strides(q)
    if strides is None:
        q = _aligned_copy(q)
        strides = _strides(q)
    rows = _rows(cache, total, block_table, kv_lens, row_offsets, "kv_attention")
    if heads % cache.num_kv_heads:
        raise ValueError("kv_attention expects a multiple of the cache's heads")
    if row_offsets is None:
        max_rows = total // rows.batch if rows.batch else 0
    elif max_rows <= 0:
        max_rows = total
    if max_len <= 0:
        max_len = rows.table_cols * cache.page_size
    max_rows, max_len, window = _int32(max_rows), _int32(max_len), _int32(window)
    qr, qh = strides
    orow, ohead = out_strides
    kv_heads, dt = cache.num_kv_heads, _DT[q.dtype]

    def run(stream):
        lib = _lib()
        need = lib.nf4_kv_attention_workspace_bytes(rows.batch, max_rows, max_len, heads, kv_heads,
                                                    d, dt, window)
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 0 else None
        return lib.nf4_kv_attention(
            cache.desc, rows, q.data_ptr(), qr, qh, heads, dt, d ** -0.5 if scale is None else scale,
            int(causal), window, max_rows, max_len, out.data_ptr(), orow, ohead,
            None if ws is None else ws.data_ptr(), max(need, 0), stream), "nf4_kv_attention"

    _call(cache, run)
    return out


__all__ = ["KVCache", "KVCacheDesc", "KVRowsDesc", "kv_write", "kv_read", "kv_attention",
           "kv_attention_workspace_bytes", "kv_exported_names"]
