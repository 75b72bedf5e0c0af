"""The C ABI of the key/value cache without a GPU: exports, and the refusals of
every entry point before any device work. Fake pointers are only passed to calls
that must fail validation or do nothing."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED, DEVICE, SCRATCH = 0, 1, 2, 3, 4, 5
A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000
MIS = 0x10008


@pytest.fixture(scope="module")
def kv():
    import bit_weight_quantization_nf4_amd as m
    from bit_weight_quantization_nf4_amd import kv as k

    if not os.path.exists(m.LIB_PATH):
        from bit_weight_quantization_nf4_amd.build import build

        build()
    return k


def cache(kv, **over):
    f = dict(k_packed=A, k_absmax=B, v_packed=C, v_absmax=D, num_pages=4, packed_page_stride=0,
             absmax_page_stride=0, page_size=16, num_kv_heads=2, head_dim=128, blocksize=64,
             quant_type=0)
    f.update(over)
    n = f["num_kv_heads"] * f["page_size"]
    if not f["packed_page_stride"]:
        f["packed_page_stride"] = n * f["head_dim"] // 2
    if not f["absmax_page_stride"]:
        f["absmax_page_stride"] = n * (f["head_dim"] // max(1, f["blocksize"]))
    return kv.KVCacheDesc(**f)


def rows(kv, **over):
    f = dict(block_table=A, kv_lens=B, row_offsets=None, table_stride=3, table_cols=3, batch=2,
             total_rows=4)
    f.update(over)
    return kv.KVRowsDesc(**f)


def calls(kv):
    """Every entry point over a cache and rows, the rest of its arguments valid."""
    L = kv._lib()
    return [
        lambda c, r, dt=0: L.nf4_kv_write(c, r, A, B, 256, 128, dt, None, None, None),
        lambda c, r, dt=0: L.nf4_kv_read(c, r, dt, A, B, 256, 128, None),
        lambda c, r, dt=0: L.nf4_kv_attention(c, r, A, 512, 128, 4, dt, 0.1, 1, 0, 2, 48, B, 512,
                                              128, C, 1 << 30, None),
    ]


def test_exports_every_declared_symbol(kv):
    text = open(os.path.join(ROOT, "include", "nf4_kv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = sorted(set(re.findall(r"\b(nf4_kv_[a-z0-9_]+)\s*\(", text)))
    assert sorted(kv.kv_exported_names()) == declared
    from bit_weight_quantization_nf4_amd import LIB_PATH

    handle = ctypes.CDLL(LIB_PATH)
    for name in declared:
        assert hasattr(handle, name), name


@pytest.mark.parametrize("which", [0, 1, 2])
def test_cache_refusals(kv, which):
    call = calls(kv)[which]
    r = rows(kv)
    assert call(None, r) == INVALID
    for over in (dict(num_pages=-1), dict(page_size=0), dict(page_size=-16), dict(num_kv_heads=0),
                 dict(head_dim=0), dict(quant_type=2), dict(blocksize=48), dict(blocksize=16),
                 dict(k_packed=None), dict(v_absmax=None), dict(packed_page_stride=16),
                 dict(absmax_page_stride=1)):
        assert call(cache(kv, **over), r) == INVALID, over
    for over in (dict(head_dim=80, blocksize=32), dict(head_dim=512), dict(head_dim=32, blocksize=32),
                 dict(head_dim=96, blocksize=64), dict(head_dim=64, blocksize=128),
                 dict(head_dim=256, blocksize=256), dict(page_size=24), dict(page_size=8),
                 dict(page_size=1 << 26), dict(num_kv_heads=70000), dict(num_pages=1 << 31)):
        assert call(cache(kv, **over), r) == UNSUPPORTED, over
    for over in (dict(k_packed=MIS), dict(v_packed=MIS), dict(k_absmax=MIS), dict(v_absmax=MIS),
                 dict(packed_page_stride=2 * 16 * 64 + 8)):
        assert call(cache(kv, **over), r) == MISALIGNED, over


@pytest.mark.parametrize("which", [0, 1, 2])
def test_rows_refusals(kv, which):
    call = calls(kv)[which]
    c = cache(kv)
    assert call(c, None) == INVALID
    for over in (dict(batch=-1), dict(total_rows=-1), dict(table_cols=-1), dict(table_stride=2),
                 dict(kv_lens=None), dict(block_table=None), dict(total_rows=5),
                 dict(batch=0)):
        assert call(c, rows(kv, **over)) == INVALID, over
    assert call(c, rows(kv, batch=70000, total_rows=70000)) == UNSUPPORTED
    for over in (dict(kv_lens=MIS + 1), dict(block_table=A + 2), dict(row_offsets=A + 1)):
        assert call(c, rows(kv, **over)) == MISALIGNED, over
    assert call(c, rows(kv), 3) == INVALID
    # nothing to do
    assert call(c, rows(kv, batch=0, total_rows=0)) == OK
    assert call(c, rows(kv, total_rows=0, block_table=None, kv_lens=None)) == OK
    assert call(c, rows(kv, batch=0, total_rows=3, row_offsets=A)) == OK


def test_row_tensor_refusals(kv):
    L = kv._lib()
    c, r = cache(kv), rows(kv)

    def write(k=A, v=B, rs=256, hs=128, kq=None, vq=None):
        return L.nf4_kv_write(c, r, k, v, rs, hs, 0, kq, vq, None)

    def read(k=A, v=B, rs=256, hs=128):
        return L.nf4_kv_read(c, r, 0, k, v, rs, hs, None)

    for call in (write, read):
        assert call(k=None) == INVALID and call(v=None) == INVALID
        assert call(rs=127) == INVALID and call(hs=64) == INVALID
        assert call(rs=1 << 60) == INVALID and call(hs=-128) == INVALID
        assert call(k=MIS) == MISALIGNED and call(v=MIS) == MISALIGNED
        assert call(rs=260) == MISALIGNED and call(hs=132) == MISALIGNED
    assert write(kq=A) == INVALID and write(vq=A) == INVALID
    assert write(kq=MIS, vq=A) == MISALIGNED


def test_attention_refusals(kv):
    L = kv._lib()
    c = cache(kv)

    def att(q=A, qrs=512, qhs=128, heads=4, scale=0.1, window=0, max_rows=2, max_len=48, out=B,
            ors=512, ohs=128, ws=C, wb=1 << 30, r=rows(kv)):
        return L.nf4_kv_attention(c, r, q, qrs, qhs, heads, 0, scale, 1, window, max_rows, max_len,
                                  out, ors, ohs, ws, wb, None)

    for over in (dict(q=None), dict(out=None), dict(qrs=100), dict(qhs=100), dict(ors=100),
                 dict(ohs=100), dict(heads=3), dict(heads=0), dict(heads=-2), dict(window=-1),
                 dict(max_rows=-1), dict(max_len=-1), dict(scale=float("nan")),
                 dict(scale=float("inf")), dict(ws=None), dict(wb=-1)):
        assert att(**over) == INVALID, over
    for over in (dict(q=MIS), dict(out=MIS), dict(qrs=516), dict(qhs=132), dict(ors=516),
                 dict(ohs=132), dict(ws=MIS)):
        assert att(**over) == MISALIGNED, over
    # more rows than a launch can hold
    big = rows(kv, batch=1, total_rows=1 << 30)
    assert att(r=big) == UNSUPPORTED


def test_workspace_query(kv):
    q = kv.kv_attention_workspace_bytes
    for bad in ((-1, 1, 1, 8, 8, 128), (1, -1, 1, 8, 8, 128), (1, 1, -1, 8, 8, 128),
                (1, 1, 1, 8, 3, 128), (1, 1, 1, 0, 8, 128), (1, 1, 1, 8, 0, 128),
                (1, 1, 1, 8, 8, 100), (70000, 1, 1, 8, 8, 128)):
        assert q(*bad) == -1, bad
    assert q(1, 1, 1, 8, 8, 128, window=-1) == -1
    assert kv._lib().nf4_kv_attention_workspace_bytes(1, 1, 1, 8, 8, 128, 3, 0) == -1
    assert q(1, 1, 1, 65536, 1, 128) == -1 and q(1, 1, 1, 65535, 1, 128) >= 0
    assert q(0, 1, 100, 8, 8, 128) == 0 and q(1, 0, 100, 8, 8, 128) == 0
    assert q(1, 1, 1, 8, 8, 128) == 0
    # a long sequence and few heads is split: fp32 sums of 128 columns and two statistics a row
    n = q(1, 1, 1 << 17, 8, 8, 128)
    assert n > 0 and n % 256 == 0
    assert q(4096, 1, 1 << 17, 8, 8, 128) == 0  # enough sequences: no split
    assert q(1, 1, 1 << 17, 8, 8, 128, window=100) == 0  # nor for what a window shows


def test_binding_refuses_cpu_tensors(kv):
    p = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    a = torch.zeros(2, 2, 16, 2)
    with pytest.raises(TypeError):
        kv.KVCache(p, a, p.clone(), a.clone(), 64, "nf4")
    with pytest.raises(ValueError):
        kv.KVCache(p, a, p.clone(), torch.zeros(2, 2, 16, 1), 64, "nf4")
    with pytest.raises(ValueError):
        kv.KVCache(p.float(), a, p, a)


def test_workspace_query_of_sizes_past_32_bits(kv):
    """The query's sizes are C ints: larger ones are taken as the largest, not modulo 2^32,
    and negative ones stay negative."""
    q = kv.kv_attention_workspace_bytes
    most = 0x7ff00000
    assert q(1, 1, most, 8, 8, 128) > 0
    for n in (1 << 32, (1 << 40) + 5, most + 1):
        assert q(1, 1, n, 8, 8, 128) == q(1, 1, most, 8, 8, 128)
        assert q(1, 1, 1 << 17, 8, 8, 128, window=n) == q(1, 1, 1 << 17, 8, 8, 128)
    low = -(1 << 32)
    assert q(1, 1, low + 9, 8, 8, 128) == -1 and q(1, 1, 100, 8, 8, 128, window=low) == -1
    assert q((1 << 32) + 1, 1, 1, 8, 8, 128) == -1 and q(1, 1, 1, (1 << 32) + 8, 8, 128) == -1
