"""Every attention kernel that a call can choose, against float64: each head_dim and
blocksize in each element type, in the three shapes of workgroup (one tile of 16 (row,
head) pairs shared by the waves; two, or several blocks of one; waves with rows of their
own), with the positions in one range and in several. The bound is test_gpu_kv.py's,
element by element.
"""
import pytest
import torch

import kv_reference as ref
from test_gpu_kv import (check_attention, dense, device_cache, gpu_call, nf4,  # noqa: F401
                         queries, run_attention)
from test_gpu_kv_limits import check_rows, largest_seen

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 32), (192, 64),
          (256, 32), (256, 64), (256, 128)]
# name, heads, kv heads, lengths, rows
ROWS = [
    ("one row", 8, 2, [70, 33], [1, 1]),       # 4 pairs a kv head: decoding
    ("one tile", 8, 2, [75, 41], [4, 2]),      # 16
    ("tiles", 8, 2, [75, 41], [9, 5]),         # 36
    # 128 pairs, in 256 workgroups (two blocks of the wider heads), so that two ranges fit
    ("rows apart", 512, 128, [75, 40], [32, 9]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,bs", SHAPES)
def test_every_instance(nf4, orc, d, bs, dtype):  # noqa: F811
    for name, heads, kvh, lens, rows in ROWS:
        if name == "rows apart" and d > 128:
            heads, kvh = heads // 2, kvh // 2
        case = (dtype, "nf4", d, bs, heads, kvh, 16, lens, rows, True, 0)
        out, want, (call, cache, q, nat) = run_attention(nf4, orc, case, 1000 + d, 1)
        where = [t.cuda() for t in (call.table, torch.tensor(lens, dtype=torch.int32), call.offsets)]
        print(name, d, bs, dtype, flush=True)
        check_attention(out, *want, dtype, "nf4", d, max(lens), nat, norm=False)
        many = nf4.kv_attention(q.cuda(), cache, *where, max_rows=max(rows), max_len=1 << 17)
        check_attention(many, *want, dtype, "nf4", d, max(lens), nat, norm=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,bs", SHAPES)
def test_every_instance_with_scales_of_its_rows_own(nf4, orc, d, bs, dtype):  # noqa: F811
    """The same kernels where the rows of a block see value scales of very different size:
    each new position's, block by block in turn, is up to 2^12 (fp16) or 2^40 times the
    last one's, and the last but one is 0. The bound is test_gpu_kv_limits.py's."""
    for name, heads, kvh, lens, rows in ROWS:
        if name == "rows apart" and d > 128:
            heads, kvh = heads // 2, kvh // 2
        call, pages = ref.make_call(lens, rows, 16, 1100 + d)
        book = ref.codebook(orc, "nf4")
        nat = ref.random_cache(book, pages, kvh, 16, d, bs, "nf4", 1101 + d)
        q = queries(call.total, heads, d, dtype, 1102)
        codes, a = nat[1]
        for _, b, p, pg, at in call.places():
            i = p - (lens[b] - rows[b])
            grow = [1.0, 2.0 ** 12, 0.0, 2.0 ** -9][i % 4] if dtype == "fp16" else \
                2.0 ** min(100, 40 * i) if i != rows[b] - 2 else 0.0
            a[pg, :, at, i % a.shape[-1]] *= grow
        cache = device_cache(nf4, (nat[0], (codes, a)), bs, "nf4")
        want = ref.attention(call, q, dense(book, *nat[0], bs), dense(book, codes, a, bs),
                             ref.sqrt_scale(d), True, 0)
        seen = largest_seen(call, a, heads, True, 0)
        for max_len in (1, 1 << 17):
            print(name, d, bs, dtype, max_len, flush=True)
            out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=max(rows),
                                   max_len=max_len)
            check_rows(out, *want, seen, dtype, "nf4", d, max(lens))
