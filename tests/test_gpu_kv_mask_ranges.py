"""The masked attention to a 4-bit cache where positions are cut into ranges, whose results a
second kernel joins, against 64 bits. Which cases are cut, and where, goes by the workspace that
the library asks for: every case says of its sequences in how many ranges they come, so that a
change of the rule shows here. The bound is test_gpu_kv.py's, element by element: a join is a few
roundings of fp32 more, which that of the sums over positions holds room for."""
import pytest
import torch

import kv_mask_reference as mref
import kv_reference as ref
from bit_weight_quantization_nf4_amd import kv
from test_gpu_kv import (DT, check_attention, dense, device_cache, gpu_call, nf4,  # noqa: F401
                         queries, same)

STEP = 256  # ranges are multiples: 8 waves take steps of 32 positions in turn


def range_length(case, max_len, window, sinks):
    """Positions of a range in a call of sequences no longer than max_len (0: not cut)."""
    dtype, _, d, _, heads, kvh, _, lens, rows = case
    pairs = max(rows) * (heads // kvh)
    block = 16 if pairs <= 16 or d > 128 else 32
    results = len(lens) * kvh * -(-pairs // block) * min(pairs, block)  # of a range
    need = kv._lib().nf4_kv_attention_masked_workspace_bytes(
        len(lens), max(rows), max_len, heads, kvh, d, kv._DT[DT[dtype]], window, sinks)
    count = need // (results * (4 * d + 8))
    if count < 2:
        return 0
    assert need - count * results * (4 * d + 8) < 256
    span = min(max_len, window + sinks + max(rows)) if window else max_len
    return -(-(-(-span // count)) // STEP) * STEP


def pieces(case, max_len, window, sinks, see):
    """Ranges of each sequence, by the positions that its rows see."""
    length, out, first = range_length(case, max_len, window, sinks), [], 0
    for n in case[8]:
        seen = set().union(*see[first:first + n]) if n else set()
        out.append(-(-len(seen) // length) if length else 1)
        first += n
    return out


CASES = [
    # (dtype, quant, D, bs, heads, kv heads, page, lens, rows), window, sinks, trees, ranges
    # the whole of each sequence, and trees
    (("bf16", "nf4", 128, 64, 8, 2, 16, [3000, 2500, 700, 300, 0, 1000], [4, 3, 4, 1, 2, 2]), 0, 0, True,
     [6, 5, 2, 1, 0, 2]),
    (("bf16", "nf4", 128, 64, 8, 2, 64, [3000, 2500, 700, 300, 0, 1000], [40, 13, 33, 7, 2, 1]), 0, 0, True,
     [4, 4, 1, 1, 0, 2]),
    (("bf16", "fp4", 96, 32, 5, 1, 48, [4000, 2900, 20], [11, 9, 11]), 0, 0, True, [6, 4, 1]),
    (("fp16", "nf4", 64, 32, 6, 2, 16, [9000, 4000, 1200, 100], [7, 3, 5, 1]), 0, 0, True, [9, 4, 2, 1]),
    (("fp16", "fp4", 192, 64, 4, 2, 16, [3000, 1500, 300], [6, 9, 1]), 0, 0, True, [6, 3, 1]),
    (("fp32", "nf4", 256, 128, 4, 2, 16, [900, 500, 201, 40, 0], [9, 4, 6, 1, 3]), 0, 0, True, [4, 2, 1, 1, 0]),
    (("fp32", "fp4", 128, 64, 8, 2, 32, [2000, 900, 200], [20, 1, 9]), 0, 0, True, [8, 4, 1]),
    # windows: first positions in one range with the window's, in several of their own, and none
    (("bf16", "nf4", 128, 64, 8, 2, 16, [5000, 3000, 900, 30], [4, 2, 3, 1]), 2100, 600, False, [6, 6, 2, 1]),
    (("bf16", "nf4", 128, 64, 8, 2, 16, [5000, 3000, 900, 30], [30, 12, 20, 1]), 2100, 600, True, [6, 6, 2, 1]),
    (("bf16", "nf4", 128, 32, 40, 1, 64, [6000, 2300], [1, 1]), 600, 1600, False, [5, 5]),
    (("bf16", "nf4", 128, 64, 8, 2, 48, [2720, 2690, 2750], [3, 3, 3]), 2100, 600, True, [6, 6, 6]),
    (("fp16", "nf4", 128, 64, 8, 8, 16, [4000, 2400, 500], [5, 2, 17]), 2300, 33, False, [5, 5, 1]),
    (("fp16", "nf4", 64, 64, 4, 2, 16, [9000, 6000], [9, 3]), 4500, 1, True, [5, 5]),
    (("fp32", "nf4", 256, 64, 4, 2, 16, [900, 500, 301, 40, 0], [9, 4, 6, 1, 3]), 300, 300, False, [3, 2, 2, 1, 0]),
    (("fp32", "nf4", 256, 128, 4, 2, 32, [900, 700, 301, 20], [9, 4, 6, 2]), 100, 700, True, [4, 3, 2, 1]),
    (("fp32", "nf4", 96, 32, 4, 1, 16, [3000, 1100], [5, 20]), 1000, 70, True, [5, 5]),
]
IDS = ["-".join(map(str, (*c[0], c[1], c[2], "tree" if c[3] else "chain"))).replace(" ", "") for c in CASES]


def masks_of(case, trees, seed):
    return mref.random_trees(case[8], seed) if trees else None


@pytest.mark.parametrize("case,window,sinks,trees,ranges", CASES, ids=IDS)
def test_cases_are_cut(case, window, sinks, trees, ranges):
    """(On the CPU, for a device of 256 CUs.)"""
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("another number of CUs")
    call, _ = ref.make_call(case[7], case[8], case[6], 1)
    see = mref.visible(call, window, sinks, masks_of(case, trees, 21))
    assert pieces(case, max(case[7]), window, sinks, see) == ranges


@pytest.mark.gpu
@pytest.mark.parametrize("part", [1.0, 0.8])
@pytest.mark.parametrize("case,window,sinks,trees,ranges", CASES, ids=IDS)
def test_ranges(nf4, orc, case, window, sinks, trees, ranges, part):  # noqa: F811
    """max_len as it is, and less; pages missing at the front, where ranges meet and
    before the last rows; scales of infinity and NaN that no row looks at."""
    dtype, quant, d, bs, heads, kvh, page, lens, rows = case
    book = ref.codebook(orc, quant)
    masks = masks_of(case, trees, 21)
    for holes in ((), tuple((0, at // page) for at in (page, 512, 600, max(lens) - 40))):
        call, pages = ref.make_call(lens, rows, page, 800 + d, holes=holes)
        nat = ref.random_cache(book, pages, kvh, page, d, bs, quant, 801)
        cache = device_cache(nf4, nat, bs, quant)
        q = queries(call.total, heads, d, dtype, 802)
        see = mref.visible(call, window, sinks, masks)
        want = mref.attention(call, q, *(dense(book, *x, bs) for x in nat), ref.sqrt_scale(d), see)
        kw = dict(max_rows=max(rows), max_len=int(part * max(lens)), window=window, sinks=sinks)
        if trees:
            kw["tree"] = mref.tree_words(masks, -(-max(rows) // 32), call.total).cuda()
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), **kw)
        check_attention(out, *want, dtype, quant, d, max(lens), nat, norm=False)
        assert torch.all(out.cpu()[want[1].sum(-1) == 0] == 0)
        assert same(nf4.kv_attention(q.cuda(), cache, *gpu_call(call), **kw), out)
        unseen = torch.ones(cache.num_pages, page, dtype=torch.bool)
        row = 0
        for b, n in enumerate(rows):
            for p in set().union(*see[row:row + n]) if n else ():
                if int(call.table[b, p // page]) >= 0:
                    unseen[call.table[b, p // page], p % page] = False
            row += n
        bad = torch.tensor([float("inf"), float("nan"), 3e38]).repeat(unseen.numel() // 3 + 1)
        bad = bad[:unseen.numel()].view(unseen.shape)[:, None, :, None].cuda()
        for t in (cache.k_absmax, cache.v_absmax):
            t.copy_(torch.where(unseen.cuda()[:, None, :, None], bad, t))
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), **kw)
        check_attention(out, *want, dtype, quant, d, max(lens), nat, norm=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_chains_and_windows_that_hide_nothing(nf4, orc, dtype):  # noqa: F811
    """A tree of one branch, and a window with first positions that together hide nothing: causal
    attention, cut into ranges or not."""
    case = (dtype, "nf4", 128, 64, 8, 2, 16, [3400, 1700, 90], [40, 9, 20])
    book = ref.codebook(orc, "nf4")
    call, pages = ref.make_call(case[7], case[8], 16, 820)
    nat = ref.random_cache(book, pages, 2, 16, 128, 64, "nf4", 821)
    cache = device_cache(nf4, nat, 64, "nf4")
    q = queries(call.total, 8, 128, dtype, 822)
    chain = [set(range(i + 1)) for n in case[8] for i in range(n)]
    want = mref.attention(call, q, *(dense(book, *x, 64) for x in nat), ref.sqrt_scale(128),
                          mref.visible(call))
    tree = mref.tree_words(chain, 2, call.total).cuda()
    assert range_length(case, 3400, 0, 0) > 0 and range_length(case, 3400, 2500, 1000) > 0
    for max_len in (1, 3400):
        for kw in (dict(tree=tree), dict(tree=tree, window=2500, sinks=1000), dict(window=2500, sinks=1000),
                   dict(window=3400, sinks=1), dict()):
            out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=40, max_len=max_len, **kw)
            check_attention(out, *want, dtype, "nf4", 128, 3400, nat, norm=False)
