"""The masked attention to a 4-bit cache against 64 bits: a window with first positions that
stay visible, and trees of drafted rows. The kernels are those of nf4_kv_attention but for
which positions a row sees, so the bound of a result is test_gpu_kv.py's, element by element."""
import pytest
import torch

import kv_mask_reference as mref
import kv_reference as ref
from test_gpu_kv import (check_attention, dense, device_cache, gpu_call, nf4,  # noqa: F401
                         queries, same)
from test_gpu_kv_instances import SHAPES

pytestmark = pytest.mark.gpu


def setup(nf4, orc, case, seed, holes=()):  # noqa: F811
    dtype, quant, d, bs, heads, kvh, page, lens, rows = case
    call, pages = ref.make_call(lens, rows, page, seed, holes=holes)
    book = ref.codebook(orc, quant)
    nat = ref.random_cache(book, pages, kvh, page, d, bs, quant, seed + 1)
    cache = device_cache(nf4, nat, bs, quant)
    q = queries(call.total, heads, d, dtype, seed + 2)
    k64, v64 = (dense(book, *x, bs) for x in nat)
    return call, cache, q, nat, k64, v64


def run(nf4, orc, case, seed, window=0, sinks=0, masks=None, words=None, max_len=1, holes=(),  # noqa: F811
        norm=False, **kw):
    call, cache, q, nat, k64, v64 = setup(nf4, orc, case, seed, holes)
    tree = None
    if masks is not None:
        words = words if words is not None else max(1, -(-max(max(case[8]), 1) // 32))
        tree = mref.tree_words([{j for j in m if j < 32 * words} for m in masks], words,
                               call.total).cuda()
    out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=max(case[8]), max_len=max_len,
                           window=window, sinks=sinks, tree=tree, **kw)
    see = mref.visible(call, window, sinks, masks, words if words is not None else 1 << 20)
    want = mref.attention(call, q, k64, v64, ref.sqrt_scale(case[2]), see)
    check_attention(out, *want, case[0], case[1], case[2], max(case[7]), nat, norm=norm)
    assert torch.all(out.cpu()[want[1].sum(-1) == 0] == 0)
    return out, want, (call, cache, q, nat, tree, see)


SPLITS = {"one": 1, "many": 1 << 17}  # max_len: positions in one range, or in many

SINKS = [
    # dtype, quant, D, bs, heads, kv heads, page, lens, rows, window, sinks
    ("bf16", "nf4", 128, 64, 4, 1, 16, [1], [1], 4, 2),
    ("bf16", "nf4", 128, 64, 8, 2, 16, [31, 32, 33, 64, 65, 300], [1] * 6, 16, 4),
    ("bf16", "nf4", 128, 128, 8, 2, 48, [500, 256, 257, 1000], [1, 1, 1, 1], 100, 33),
    ("bf16", "nf4", 128, 32, 4, 4, 64, [513, 70], [1, 1], 31, 64),
    ("fp16", "nf4", 64, 64, 6, 2, 16, [400, 47, 5], [7, 3, 5], 1, 1),
    ("fp16", "nf4", 64, 32, 16, 1, 32, [900, 29], [2, 1], 64, 31),
    ("fp32", "nf4", 128, 64, 8, 2, 16, [333, 64], [3, 1], 40, 32),
    ("fp32", "nf4", 256, 128, 4, 2, 16, [529, 300], [5, 9], 40, 100),
    ("fp32", "nf4", 96, 32, 4, 1, 16, [411], [9], 32, 5),
    ("bf16", "fp4", 256, 64, 8, 1, 48, [401, 9], [5, 2], 3, 65),
    ("fp16", "fp4", 192, 64, 4, 2, 16, [587], [6], 96, 7),
    ("bf16", "nf4", 128, 64, 8, 2, 64, [700, 512], [130, 64], 50, 20),
    ("bf16", "nf4", 128, 64, 4, 2, 16, [600], [100], 133, 129),
    ("fp16", "nf4", 128, 32, 2, 1, 16, [280], [60], 1, 40),
    # sinks past the window, past the length, and 2^31 - 1; windows past the length
    ("bf16", "nf4", 128, 64, 4, 2, 16, [100, 20], [2, 1], 10, 90),
    ("bf16", "nf4", 128, 64, 4, 2, 16, [100, 20], [2, 1], 10, 2 ** 31 - 1),
    ("bf16", "nf4", 128, 64, 4, 2, 16, [100, 20], [2, 1], 300, 4),
    # rows that see nothing: more rows than positions, empty sequences, no rows
    ("bf16", "nf4", 128, 64, 4, 2, 16, [3, 0, 140, 8], [7, 2, 0, 8], 2, 1),
    ("fp32", "nf4", 64, 64, 4, 2, 16, [0, 200], [1, 40], 3, 2),
    # waves with rows of their own
    ("bf16", "nf4", 128, 64, 64, 64, 16, [250, 131, 297, 128], [128, 100, 97, 3], 40, 9),
    ("fp16", "fp4", 64, 32, 96, 32, 48, [170, 61, 243, 99, 0, 12, 50, 43],
     [43, 40, 1, 43, 7, 12, 33, 43], 20, 40),
    ("fp32", "nf4", 256, 128, 32, 32, 16, [329, 140, 128, 277], [128, 100, 128, 77], 70, 33),
    ("bf16", "nf4", 128, 64, 64, 64, 16, [250, 131, 297, 128], [128, 100, 97, 3], 150, 100),
]


@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("case", SINKS, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_sinks(nf4, orc, case, split):  # noqa: F811
    run(nf4, orc, case[:9], 100 + case[2], case[9], case[10], max_len=SPLITS[split])


TREES = [
    # dtype, quant, D, bs, heads, kv heads, page, lens, rows
    ("bf16", "nf4", 128, 64, 4, 1, 16, [1], [1]),
    ("bf16", "nf4", 128, 64, 8, 2, 16, [40, 33, 17, 90], [8, 1, 17, 13]),
    ("bf16", "nf4", 128, 128, 8, 2, 48, [255, 256, 257], [31, 32, 33]),
    ("fp16", "nf4", 64, 64, 6, 2, 16, [100, 47, 5], [7, 3, 5]),
    ("fp16", "nf4", 64, 32, 16, 1, 32, [300, 29], [65, 29]),
    ("fp32", "nf4", 128, 64, 8, 2, 16, [333, 64], [64, 10]),
    ("fp32", "fp4", 256, 128, 4, 2, 16, [129, 300], [5, 90]),
    ("bf16", "nf4", 96, 32, 5, 1, 16, [140, 33], [11, 1]),
    ("fp16", "fp4", 192, 64, 4, 2, 16, [87], [6]),
    ("bf16", "nf4", 128, 64, 8, 2, 64, [700, 512], [130, 64]),
    # more rows than positions, empty sequences, no rows
    ("bf16", "nf4", 128, 64, 4, 2, 16, [3, 0, 40, 8], [7, 2, 0, 8]),
    # waves with rows of their own
    ("bf16", "nf4", 128, 64, 64, 64, 16, [250, 131, 297, 128], [128, 100, 97, 3]),
    ("fp16", "fp4", 64, 32, 96, 32, 48, [170, 61, 243, 99, 0, 12, 50, 43],
     [43, 40, 1, 43, 7, 12, 33, 43]),
]


@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("window,sinks", [(0, 0), (25, 3), (3, 40)])
@pytest.mark.parametrize("case", TREES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_tree(nf4, orc, case, window, sinks, split):  # noqa: F811
    masks = mref.random_trees(case[8], 7)
    run(nf4, orc, case, 300 + case[2], window, sinks, masks, max_len=SPLITS[split])


@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("case", [
    ("bf16", "nf4", 128, 64, 8, 2, 16, [140, 70, 50], [40, 70, 3]),
    ("fp32", "nf4", 64, 32, 64, 64, 16, [190, 70, 90, 131], [64, 64, 90, 128])],
    ids=["shared", "apart"])
@pytest.mark.parametrize("kind", ["none", "bits", "later", "short", "long", "everything"])
def test_any_bits_are_a_mask(nf4, orc, case, kind, split):  # noqa: F811
    """Rows without themselves or without any row, later rows, bits past the sequence's last
    row, masks of fewer words than rows, and of more."""
    total = sum(case[8])
    g = torch.Generator().manual_seed(5)
    masks, words = [], -(-max(case[8]) // 32)
    for t in range(total):
        if kind == "none":
            masks.append(set())
        elif kind == "later":
            masks.append(set(range(t % 11, 32 * words)))
        elif kind == "everything":
            masks.append(set(range(32 * words)))
        else:
            masks.append({j for j in range(32 * words) if torch.rand(1, generator=g) < 0.3})
    words = {"short": 1, "long": words + 2}.get(kind, words)
    for window, sinks in ((0, 0), (30, 2)):
        run(nf4, orc, case, 400, window, sinks, masks, words, SPLITS[split])


def test_no_words_and_strided_trees(nf4, orc):  # noqa: F811
    """A tree without words hides every row of the call; a slice of a wider tree's columns is
    taken as it is."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [40, 9], [8, 9])
    out, _, _ = run(nf4, orc, case, 500, 0, 0, [set()] * 17, 0)
    assert torch.all(out[8:] == 0) and bool((out[:8] != 0).any())
    masks = mref.random_trees(case[8], 8)
    out, _, (call, cache, q, _, tree, _) = run(nf4, orc, case, 501, 0, 0, masks)
    wide = torch.full((17, 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:3] = tree
    for t in (wide[:, 2:3], tree.expand(17, 1)):
        assert same(nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=9, max_len=1, tree=t),
                    out)
    two = torch.stack((tree[:, 0], torch.zeros_like(tree[:, 0]))).T  # column stride other than 1
    assert same(nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=9, max_len=1, tree=two), out)


@pytest.mark.parametrize("split", list(SPLITS))
def test_a_chain_is_causal_attention(nf4, orc, split):  # noqa: F811
    """A tree of one branch, and a window that hides nothing, give causal attention's bits: the
    same positions in the same steps."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [340, 170], [40, 70])
    chain = [set(range(i + 1)) for n in case[8] for i in range(n)]
    out, _, (call, cache, q, _, _, _) = run(nf4, orc, case, 520, 0, 0, chain, max_len=SPLITS[split])
    plain = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=70, max_len=SPLITS[split])
    assert torch.allclose(out.float(), plain.float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    kept = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=70, max_len=SPLITS[split], sinks=5)
    assert same(kept, plain)


def test_missing_pages_and_what_is_not_there(nf4, orc):  # noqa: F811
    """Pages missing among the first positions and inside the window; scales of NaN and
    infinity where no row looks: past the lengths, and in pages that no sequence has."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [300, 133], [3, 1])
    out, want, (call, cache, q, nat, _, _) = run(nf4, orc, case, 540, 60, 40, holes=[(0, 1), (0, 17), (1, 0)])
    used = torch.zeros(cache.num_pages, 16, dtype=torch.bool)
    for b, n in enumerate(call.lens):
        for p in range(n):
            pg = int(call.table[b, p // 16])
            if pg >= 0:
                used[pg, p % 16] = True
    for bad in (float("nan"), float("inf"), 3e38):
        for t in (cache.k_absmax, cache.v_absmax):
            t.masked_fill_(~used.cuda()[:, None, :, None], bad)
        again = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=3, max_len=1, window=60, sinks=40)
        assert same(again, out), bad


@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("kind", ["sinks", "tree"])
@pytest.mark.parametrize("shape", [("bf16", 128, 64, 8, 2), ("fp16", 64, 32, 4, 1), ("fp32", 96, 32, 4, 2)])
def test_positions_affect_only_rows_that_see_them(nf4, orc, shape, kind, split):  # noqa: F811
    """Scales of infinity and NaN at positions that the mask hides from some rows or all of
    them: between the first positions and the window, at another branch's draft."""
    dtype, d, bs, heads, kvh = shape
    case = (dtype, "nf4", d, bs, heads, kvh, 16, [290, 175], [9, 6])
    masks = mref.random_trees(case[8], 3) if kind == "tree" else None
    window, sinks = (0, 0) if kind == "tree" else (40, 5)
    out, want, (call, _, q, nat, tree, see) = run(nf4, orc, case, 560, window, sinks, masks,
                                                  max_len=SPLITS[split])
    spots = [285, 289, 284] if kind == "tree" else [5, 6, 31, 32, 100, 243, 244, 4]
    for p in spots:
        hit = torch.tensor([p in s and r < 9 for r, s in enumerate(see)])
        for which in (0, 1):
            for bad in (float("inf"), float("nan")):
                cache = device_cache(nf4, nat, bs, "nf4")
                (cache.k_absmax, cache.v_absmax)[which][int(call.table[0, p // 16]), :, p % 16] = bad
                got = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=9,
                                       max_len=SPLITS[split], window=window, sinks=sinks, tree=tree).cpu()
                check_attention(got[~hit], *(t[~hit] for t in want), dtype, "nf4", d, 290, nat, norm=False)
                assert not bool(torch.isfinite(got[hit]).all(-1).all(-1).any()) or not bool(hit.any())


@pytest.mark.parametrize("split", list(SPLITS))
def test_uneven_scales_of_hidden_positions(nf4, orc, split):  # noqa: F811
    """Value scales 2^60 times the others' at positions that some rows do not see: these rows
    keep their precision, whose bound is that of the largest scale that they see."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [260, 90], [12, 5])
    masks = mref.random_trees(case[8], 4)
    for kind in ("tree", "sinks"):
        call, cache, q, nat, k64, v64 = setup(nf4, orc, case, 580)
        kw = dict(window=50, sinks=6) if kind == "sinks" else dict(masks=masks)
        see = mref.visible(call, **kw)
        p = 253 if kind == "tree" else 20
        pg = int(call.table[0, p // 16])
        cache.v_absmax[pg, :, p % 16] *= 2.0 ** 60
        if kind == "tree":
            kw = dict(tree=mref.tree_words(masks, 1, call.total).cuda())
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=12, max_len=SPLITS[split], **kw)
        want = mref.attention(call, q, k64, v64, ref.sqrt_scale(128), see)
        rows = torch.tensor([not (r < 12 and p in s) for r, s in enumerate(see)])
        assert bool(rows.any()) and (kind == "sinks" or not bool(rows.all()))
        check_attention(out.cpu()[rows], *(t[rows] for t in want), "bf16", "nf4", 128, 260, nat, norm=False)


@pytest.mark.parametrize("page", [16, 48, 256])
def test_a_long_sequence_past_its_window(nf4, orc, page):  # noqa: F811
    """120000 positions of which few are seen; where the others lie does not matter."""
    n, window, sinks = 120007, 200, 37
    cols = -(-n // page)
    g = torch.Generator().manual_seed(page)
    few = 12 * 256 // page
    table = torch.randint(0, few, (1, cols), generator=g).to(torch.int32)
    table[0, 100 // page + 1:(n - 300) // page] = -1  # not there: nobody looks
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, few, 2, page, 128, 64, "nf4", 5)
    cache = device_cache(nf4, nat, 64, "nf4")
    q = queries(5, 8, 128, "bf16", 6)
    call = ref.Call(table, [n], [5], torch.tensor([0, 5], dtype=torch.int32), page)
    see = []
    for i in range(5):
        place = n - 5 + i
        see.append(set(range(sinks)) | set(range(place - window + 1, place + 1)))
    want = mref.attention(call, q, *(dense(book, *x, 64) for x in nat), ref.sqrt_scale(128), see)
    for max_len in (1, n):
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=5, max_len=max_len,
                               window=window, sinks=sinks)
        check_attention(out, *want, "bf16", "nf4", 128, 300, nat)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,bs", SHAPES)
def test_every_instance(nf4, orc, d, bs, dtype):  # noqa: F811
    """Each kernel that a masked call can choose: workgroups of one tile of rows, of two, and
    of waves with rows of their own, with one range of positions and several."""
    for name, heads, kvh, lens, rows in (("one tile", 8, 2, [105, 71], [4, 2]),
                                         ("tiles", 8, 2, [105, 71], [9, 5]),
                                         ("rows apart", 512, 128, [105, 70], [32, 9])):
        if name == "rows apart" and d > 128:
            heads, kvh = heads // 2, kvh // 2
        case = (dtype, "nf4", d, bs, heads, kvh, 16, lens, rows)
        masks = mref.random_trees(rows, 9)
        for max_len in SPLITS.values():
            print(name, d, bs, dtype, max_len, flush=True)
            run(nf4, orc, case, 1000 + d, 30, 3, masks, max_len=max_len)
            run(nf4, orc, case, 1000 + d, 30, 3, max_len=max_len)


def test_outputs_rows_and_reproducibility(nf4, orc):  # noqa: F811
    """Strided queries and outputs, rows behind the last offset and past max_rows, uniform
    rows without offsets; the same bits each time."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [200, 133, 160], [6, 2, 3])
    masks = mref.random_trees(case[8], 5)
    kw = dict(window=50, sinks=4)
    out, want, (call, cache, q, nat, tree, _) = run(nf4, orc, case, 600, 50, 4, masks)
    where = gpu_call(call)
    big = torch.full((14, 12, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    big[:11, 2:10, 64:192] = q.cuda()
    o = torch.full((14, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.cat((tree, torch.full((3, 1), -1, dtype=torch.int32, device="cuda")))
    got = nf4.kv_attention(big[:, 2:10, 64:192], cache, *where, max_rows=6, max_len=1, out=o, tree=wide, **kw)
    assert got is o and same(o[:11], out) and torch.all(o[11:] == 3.0)
    o.fill_(3.0)
    nf4.kv_attention(q.cuda(), cache, *where, max_rows=3, max_len=1, out=o[:11], tree=tree, **kw)
    kept = [0, 1, 2, 6, 7, 8, 9, 10]
    assert torch.all(o[3:6] == 3.0)
    check_attention(o[:11][kept], *(t[kept] for t in want), "bf16", "nf4", 128, 200, nat, norm=False)
    equal = ("bf16", "nf4", 128, 64, 8, 2, 16, [200, 133, 160], [4, 4, 4])
    masks = mref.random_trees(equal[8], 6)
    out, _, (call, cache, q, _, tree, _) = run(nf4, orc, equal, 601, 50, 4, masks, max_len=200)
    table, lens, _ = gpu_call(call)
    for _ in range(3):
        assert same(nf4.kv_attention(q.cuda(), cache, table, lens, max_len=200, tree=tree, **kw), out)


def test_streams_and_graphs(nf4, orc):  # noqa: F811
    """Split calls on streams of their own at once, and a captured step whose lengths and tree
    change in place between replays, beside eager work."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [3000, 2500], [6, 6])
    call, cache, q, nat, k64, v64 = setup(nf4, orc, case, 620)
    table, lens, off = gpu_call(call)
    tree = mref.tree_words(mref.random_trees(case[8], 1), 1, 12).cuda()
    qd = q.cuda()

    def step():
        return [nf4.kv_attention(qd, cache, table, lens, off, max_rows=6, max_len=3000, tree=tree),
                nf4.kv_attention(qd, cache, table, lens, off, max_rows=6, max_len=3000, window=900,
                                 sinks=70, tree=tree),
                nf4.kv_attention(qd, cache, table, lens, off, max_rows=6, max_len=3000, window=900, sinks=70)]

    eager = step()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(step())
    torch.cuda.synchronize()
    for out in outs:
        assert all(same(a, b) for a, b in zip(eager, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        lens -= 17
        tree.copy_(mref.tree_words(mref.random_trees(case[8], 10 + i), 1, 12))
        graph.replay()
        again = step()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(held, again)), i


def test_binding_refusals(nf4, orc):  # noqa: F811
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [40], [4])
    call, cache, q, _, _, _ = setup(nf4, orc, case, 640)
    q, where = q.cuda(), gpu_call(call)
    tree = torch.full((4, 1), 15, dtype=torch.int32, device="cuda")

    def call_with(**kw):
        return nf4.kv_attention(q, cache, *where, max_rows=4, **kw)

    call_with(tree=tree)
    for kw in (dict(tree=tree, causal=False), dict(sinks=3, window=5, causal=False),
               dict(tree=tree[:3]), dict(tree=tree[0])):
        with pytest.raises(ValueError):
            call_with(**kw)
    for kw in (dict(tree=tree.long()), dict(tree=tree.cpu())):
        with pytest.raises(TypeError):
            call_with(**kw)
    with pytest.raises(nf4.Nf4Error):
        call_with(sinks=-1, window=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_many_blocks_at_long_tables(nf4, orc, dtype):  # noqa: F811
    """Blocks enough for waves with rows of their own where max_len is long (each is then whole),
    and as many as are just shared."""
    for kvh in (96, 256):
        case = (dtype, "nf4", 64, 32, 4 * kvh, kvh, 16, [105, 70, 0], [32, 9, 0])
        masks = mref.random_trees(case[8], 17)
        for window, sinks, trees in ((0, 0, masks), (40, 3, masks), (40, 3, None)):
            for max_len in (1, 1 << 17):
                print(kvh, window, max_len, flush=True)
                run(nf4, orc, case, 1700 + kvh, window, sinks, trees, max_len=max_len)
