"""Every attention kernel that a call can choose, against float64: each head_dim and
blocksize in each element type, in the three shapes of workgroup (one tile of 16 (row,
head) pairs shared by the waves; two, or several blocks of one; waves with rows of their
own), with the positions in one range and in several. The bound is test_gpu_kv.py's,
element by element.
"""
import pytest
import torch

from test_gpu_kv import check_attention, nf4, run_attention  # noqa: F401  (nf4: fixture)

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
