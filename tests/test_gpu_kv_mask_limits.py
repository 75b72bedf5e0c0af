"""The masked attention to a 4-bit cache where lengths pass the table: positions past its last
column are not there, and the first positions stay visible behind a window wherever that lies.
Bounds are test_gpu_kv.py's, whose sums run over the positions that the table has."""
import pytest
import torch

import kv_mask_reference as mref
import kv_reference as ref
from test_gpu_kv import check_attention, dense, device_cache, nf4, queries  # noqa: F401


def seen_in_table(lens, rows, capacity, window, sinks, masks):
    """kv_mask_reference.visible() of the positions below `capacity` (lengths may be any)."""
    out, t = [], 0
    for n, r in zip(lens, rows):
        base = n - r
        for i in range(r):
            mine = [] if masks is None else [j for j in masks[t] if j < r]
            place = base + (i if masks is None else len(mine) - 1)
            last = min(place + 1, capacity) if masks is None else min(base, place + 1, capacity)
            low = max(0, place - window + 1) if window else 0
            see = set(range(low, max(low, last))) | set(range(min(sinks, low, max(0, last))))
            out.append(see | {base + j for j in mine if 0 <= base + j < capacity})
            t += 1
    return out


CASES = [
    # dtype, quant, D, bs, heads, kv heads, page, columns, rows, window, sinks
    ("bf16", "nf4", 64, 32, 8, 2, 16, 3, [5, 5, 1], 7, 4),
    ("bf16", "nf4", 128, 64, 8, 2, 16, 2, [3, 9, 2], 16, 4),
    ("fp16", "nf4", 128, 64, 6, 2, 48, 3, [20, 7, 33], 40, 33),
    ("fp32", "fp4", 96, 32, 4, 1, 16, 5, [9, 1, 4], 25, 200),
    # windows long enough that positions are cut into ranges, first positions of one and of several
    ("fp32", "nf4", 256, 128, 4, 2, 16, 30, [9, 4, 1], 300, 100),
    ("fp32", "nf4", 256, 64, 4, 2, 16, 60, [9, 4, 1], 400, 700),
    # waves with rows of their own
    ("bf16", "nf4", 128, 64, 64, 64, 16, 6, [128, 100, 97, 128], 20, 9),
    ("fp16", "fp4", 64, 32, 64, 64, 16, 7, [128, 31, 97, 64], 30, 64),
    ("fp32", "nf4", 256, 128, 32, 32, 16, 5, [128, 100, 128, 77], 33, 10),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["sinks", "tree"])
@pytest.mark.parametrize("past", [1, 20, 60, 150, 500, 1 << 30])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_first_positions_of_sequences_past_the_table(nf4, orc, case, past, kind):  # noqa: F811
    """The first sequence ends `past` positions behind the table, the others within it or a
    little behind: windows that begin in the table, at its end and past it, for some rows of a
    block and for all."""
    dtype, quant, d, bs, heads, kvh, page, cols, rows, window, sinks = case
    capacity = page * cols
    lens = [capacity + past, capacity - 3, capacity + window, capacity + window // 2][:len(rows)]
    book = ref.codebook(orc, quant)
    g = torch.Generator().manual_seed(past % 1000)
    pages = len(rows) * cols
    table = torch.randperm(pages, generator=g).to(torch.int32).view(len(rows), cols)
    nat = ref.random_cache(book, pages, kvh, page, d, bs, quant, 700 + d)
    cache = device_cache(nf4, nat, bs, quant)
    total = sum(rows)
    q = queries(total, heads, d, dtype, 701)
    off = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32)
    masks = mref.random_trees(rows, 12) if kind == "tree" else None
    see = seen_in_table(lens, rows, capacity, window, sinks, masks)
    call = ref.Call(table, [capacity] * len(rows), rows, off, page)
    want = mref.attention(call, q, *(dense(book, *x, bs) for x in nat), ref.sqrt_scale(d), see)
    kw = dict(max_rows=max(rows), window=window, sinks=sinks)
    if kind == "tree":
        kw["tree"] = mref.tree_words(masks, -(-max(rows) // 32), total).cuda()
    where = (torch.tensor(lens, dtype=torch.int32).cuda(), off.cuda())
    longer = torch.cat([table, torch.full((len(rows), 40), -1, dtype=torch.int32)], 1)
    for max_len in (1, 1 << 17):
        out = nf4.kv_attention(q.cuda(), cache, table.cuda(), *where, max_len=max_len, **kw)
        check_attention(out, *want, dtype, quant, d, capacity, nat, norm=False)
        assert torch.all(out.cpu()[want[1].sum(-1) == 0] == 0)
        # as if the table went on with pages of -1
        more = nf4.kv_attention(q.cuda(), cache, longer.cuda(), *where, max_len=max_len, **kw)
        check_attention(more, *want, dtype, quant, d, capacity, nat, norm=False)


def test_the_reference_agrees_with_the_masks_spelled_out():
    rows, capacity = [5, 3, 7], 48
    masks = mref.random_trees(rows, 3)
    for lens in ([60, 40, 9], [48, 49, 130], [3, 1, 7]):
        call = ref.Call(None, lens, rows, None, 16)
        for window, sinks in ((0, 0), (7, 4), (20, 60), (1, 1)):
            for m in (None, masks):
                want = [{p for p in s if p < capacity} for s in mref.visible(call, window, sinks, m)]
                assert seen_in_table(lens, rows, capacity, window, sinks, m) == want
