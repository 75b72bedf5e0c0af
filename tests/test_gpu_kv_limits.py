"""The 4-bit key/value cache at the ends of what include/nf4_kv.h promises. Bounds are
test_gpu_kv.py's; the floor of a row (a position's weight in fp16 steps of 2^-32 of the
largest value scale) is taken from the scales that this row sees.
"""
import pytest
import torch

import kv_reference as ref
from test_gpu_kv import (DT, HALF, dense, device_cache, gpu_call, natural, nf4,  # noqa: F401
                         queries, row_values, same)

pytestmark = pytest.mark.gpu


def largest_seen(call, a, heads, causal, window):
    """[rows, heads, 1]: the largest scale of the positions that a row sees; a: the value
    scales [pages, kv heads, page, blocks]."""
    kvh = a.shape[1]
    top = a.double().amax(-1)[..., None]
    out = torch.zeros(call.total, kvh, 1, dtype=torch.float64)
    row = 0
    for b, n in enumerate(call.rows):
        s, there = ref.sequence(call, top, b, kvh)
        for i in range(n):
            hi = call.lens[b] - n + i + 1 if causal else call.lens[b]
            lo = max(0, hi - window) if window else 0
            if hi > lo and there[lo:hi].any():
                out[row] = s[:, lo:hi][:, there[lo:hi]].amax(1)
            row += 1
    return out.repeat_interleave(heads // kvh, 1)


def check_rows(got, want, spread, reach, seen, dtype, quant, d, longest, rows=slice(None)):
    """test_gpu_kv.py's bound element by element, with each row's own floor, and 2^-16 more
    of a score: where value scales differ by powers of two, so may the reference that a
    row's exponents are taken from, by less than 2^7, and four roundings of numbers below
    that are half of 2^-17 each at most."""
    c = 0.0 if quant == "fp4" else {"bf16": 2.0 ** -11, "fp16": 2.0 ** -22, "fp32": 2.0 ** -22}[dtype]
    w = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    r = (c + (d + 16) * 2.0 ** -24) * reach + 2.0 ** -21 + 2.0 ** -16
    if dtype == "fp32":
        r = r + 2.0 ** -22 * reach
    bound = spread * (2 * r + w + 2.0 ** -22 + 2 * (longest + 64) * 2.0 ** -24) + HALF[dtype] * want.abs()
    if dtype == "fp16":
        bound = bound + 2.0 ** -25
    bound = bound + longest * 2.0 ** -32 * seen
    got = got.double().cpu()
    err = (got - want).abs()
    assert torch.isfinite(got[rows]).all()
    assert torch.all(err[rows] <= bound[rows]), ((err - bound)[rows]).max().item()


# dtype, D, bs, heads, kv heads, lens, rows: waves that share a block of one tile, of two,
# and waves with rows of their own
BLOCKS = [
    ("bf16", 128, 64, 4, 2, [75, 40], [5, 3]),
    ("fp16", 64, 32, 4, 1, [90], [4]),
    ("fp32", 128, 64, 4, 2, [75, 40], [5, 3]),
    ("fp32", 256, 128, 2, 1, [60], [6]),
    ("bf16", 128, 128, 8, 2, [170], [40]),
    ("fp16", 96, 32, 4, 1, [100, 37], [37, 33]),
    ("bf16", 128, 128, 64, 64, [140, 150, 131, 40], [128, 128, 100, 3]),
    ("fp32", 64, 32, 64, 32, [90, 70] * 2, [64, 64] * 2),
]


@pytest.mark.parametrize("split", ["one", "many"])
@pytest.mark.parametrize("case", BLOCKS, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_large_value_scales_reach_only_rows_that_see_them(nf4, orc, case, split):  # noqa: F811
    """A value scale of 2^20, 2^40 or 3e38 at the newest position, which only the last row
    of its sequence sees, and at one that a window has left behind for all but the first:
    all other rows stay within the bounds of what they see. So does the row itself where
    its type holds the result."""
    dtype, d, bs, heads, kvh, lens, rows = case
    call, pages = ref.make_call(lens, rows, 16, 920)
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, pages, kvh, 16, d, bs, "nf4", 921)
    k64 = dense(book, *nat[0], bs)
    q = queries(call.total, heads, d, dtype, 922)
    b, window = len(lens) - 1, 19
    kw = dict(max_rows=max(rows), max_len=1 if split == "one" else 1 << 17, window=window)
    first, last = call.total - rows[b], call.total - 1
    for pos, row in ((lens[b] - 1, last), (lens[b] - rows[b] + 1 - window, first)):
        if pos < 0:
            continue
        keep = [r for r in range(call.total) if r != row]
        for big in (2.0 ** 20, 2.0 ** 40, 3e38):
            codes, a = nat[1]
            a = a.clone()
            a[int(call.table[b, pos // 16]), :, pos % 16] = big
            cache = device_cache(nf4, (nat[0], (codes, a)), bs, "nf4")
            out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), **kw).cpu()
            want = ref.attention(call, q, k64, dense(book, codes, a, bs), ref.sqrt_scale(d), True, window)
            seen = largest_seen(call, a, heads, True, window)
            check_rows(out, *want, seen, dtype, "nf4", d, max(lens), keep)
            if dtype != "fp16" and big < 1e30:
                check_rows(out, *want, seen, dtype, "nf4", d, max(lens), [row])


@pytest.mark.parametrize("split", ["one", "many"])
@pytest.mark.parametrize("case", BLOCKS, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_value_scales_that_grow_from_row_to_row(nf4, orc, case, split):  # noqa: F811
    """The positions of the call's rows have scales that grow by 2^9 (or fall, or are zero
    for some) from one to the next: every row is within the bounds of what it sees."""
    dtype, d, bs, heads, kvh, lens, rows = case
    call, pages = ref.make_call(lens, rows, 16, 930)
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, pages, kvh, 16, d, bs, "nf4", 931)
    k64 = dense(book, *nat[0], bs)
    q = queries(call.total, heads, d, dtype, 932)
    top = 12 if dtype == "fp16" else 108
    for kind in ("grow", "fall", "zeros first"):
        codes, a = nat[1]
        a = a.clone()
        for _, b, p, pg, at in call.places():
            if pg < 0:
                continue
            i = p - (lens[b] - rows[b])
            step = {"grow": 9 * i, "fall": -9 * i, "zeros first": 9 * i - 27}[kind]
            a[pg, :, at] *= 2.0 ** max(-top, min(top, step))
        if kind == "zeros first":  # what lies before the rows of the call
            for b in range(len(lens)):
                for p in range(lens[b] - rows[b] + 1):
                    a[int(call.table[b, p // 16]), :, p % 16] = 0.0
        cache = device_cache(nf4, (nat[0], (codes, a)), bs, "nf4")
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=max(rows),
                               max_len=1 if split == "one" else 1 << 17)
        want = ref.attention(call, q, k64, dense(book, codes, a, bs), ref.sqrt_scale(d), True, 0)
        check_rows(out, *want, largest_seen(call, a, heads, True, 0), dtype, "nf4", d, max(lens))


@pytest.mark.parametrize("case", BLOCKS, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_large_value_scales_beside_scores_of_any_size(nf4, orc, case):  # noqa: F811
    """Scores of 2^28, whose neighbours in fp32 are 32 apart, and value scales that grow
    with the rows: every row is finite, and the value of its nearest key where the next one
    is 1e-2 of the largest score away (keys' codes and fp32 sums: 2^-10 of it at most)."""
    dtype, d, bs, heads, kvh, lens, rows = case
    if dtype == "fp16":
        dtype = "bf16"  # (fp16's range ends before such queries)
    call, pages = ref.make_call(lens, rows, 16, 980)
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, pages, kvh, 16, d, bs, "nf4", 981)
    k64 = dense(book, *nat[0], bs)
    q = (queries(call.total, heads, d, "fp32", 982) * 2.0 ** 28).to(DT[dtype])
    codes, a = nat[1]
    for _, b, p, pg, at in call.places():
        if pg >= 0:
            a[pg, :, at] *= 2.0 ** min(100, 20 * (p - lens[b] + rows[b]))
    v64 = dense(book, codes, a, bs)
    sure = torch.zeros(call.total, heads, dtype=torch.bool)
    row = 0
    for b, n in enumerate(call.rows):
        k, _ = ref.sequence(call, k64, b, kvh)
        for i in range(n):
            qr = q[row].double().reshape(kvh, heads // kvh, d)
            ks = k[:, :lens[b] - n + i + 1]
            two = torch.einsum("hgd,htd->hgt", qr, ks).topk(2, -1).values
            reach = torch.einsum("hgd,htd->hgt", qr.abs(), ks.abs()).amax(-1)
            sure[row] = (two[..., 0] - two[..., 1] >= 1e-2 * reach).reshape(heads)
            row += 1
    assert sure.sum() >= sure.numel() // 2
    want, spread, reach = ref.attention(call, q, k64, v64, ref.sqrt_scale(d), True, 0)
    cache = device_cache(nf4, (nat[0], (codes, a)), bs, "nf4")
    seen = largest_seen(call, a, heads, True, 0)
    for max_len in (1, 1 << 17):
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=max(rows), max_len=max_len)
        assert torch.isfinite(out).all()
        got = torch.where(sure[..., None].cuda(), out, want.to(out.dtype).cuda())
        check_rows(got, want, spread, torch.zeros_like(reach), seen, dtype, "nf4", d, max(lens))


@pytest.mark.parametrize("d,bs,heads,kvh,rows,window,lens", [
    (64, 32, 8, 2, 5, 600, list(range(700, 733))),  # waves that share a block of two tiles
    (128, 64, 4, 2, 3, 600, list(range(700, 733))),  # of one
    (64, 64, 512, 128, 32, 100, [201, 219, 230]),  # rows of a wave's own
])
def test_windows_that_begin_anywhere_in_a_step(nf4, orc, d, bs, heads, kvh, rows, window, lens):  # noqa: F811
    """Windows whose first positions are seen by some rows of a block alone, at every place
    in a step; some of these positions have value scales of 2^30."""
    call, pages = ref.make_call(lens, [rows] * len(lens), 16, 970)
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, pages, kvh, 16, d, bs, "nf4", 971)
    q = queries(call.total, heads, d, "bf16", 972)
    k64 = dense(book, *nat[0], bs)
    codes, a = nat[1]
    for big in (False, True):
        if big:
            a = a.clone()
            for b in range(0, len(lens), 2):
                p = lens[b] - rows + 1 - window
                a[int(call.table[b, p // 16]), :, p % 16] = 2.0 ** 30
        cache = device_cache(nf4, (nat[0], (codes, a)), bs, "nf4")
        want = ref.attention(call, q, k64, dense(book, codes, a, bs), ref.sqrt_scale(d), True, window)
        seen = largest_seen(call, a, heads, True, window)
        for max_len in (1, 1 << 17):
            out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=rows,
                                   max_len=max_len, window=window)
            check_rows(out, *want, seen, "bf16", "nf4", d, window)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_key_scales_near_the_ends_of_fp32(nf4, orc, dtype):  # noqa: F811
    """Keys of 2^n and queries of 2^-n (or the other way round) have ordinary scores. Keys
    of 2^110 under ordinary queries have scores far apart: a row is the value of its
    nearest key (E2M1 codes, whose products are exact, and a gap of 5e-4 of the largest
    score at least, against 160 2^-24 of it that fp32 sums can be off by)."""
    d, bs, heads, kvh, quant = 128, 64, 4, 2, "fp4"
    call, pages = ref.make_call([75, 40], [5, 3], 16, 940)
    book = ref.codebook(orc, quant)
    nat = ref.random_cache(book, pages, kvh, 16, d, bs, quant, 941)
    v64 = dense(book, *nat[1], bs)
    seen = largest_seen(call, nat[1][1], heads, True, 0)
    for n in (60, 100, 118, -60, -100):
        codes, a = nat[0]
        a = a * 2.0 ** n
        q = (queries(call.total, heads, d, "fp32", 942) * 2.0 ** -n).to(DT[dtype])
        cache = device_cache(nf4, ((codes, a), nat[1]), bs, quant)
        for max_len in (1, 1 << 17):
            out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=5, max_len=max_len)
            want = ref.attention(call, q, dense(book, codes, a, bs), v64, ref.sqrt_scale(d), True, 0)
            check_rows(out, *want, seen, dtype, quant, d, 75)
    q = queries(call.total, heads, d, dtype, 943)
    codes, a = nat[0]
    a = a * 2.0 ** 110
    k64 = dense(book, codes, a, bs)
    row = 0
    for b, n in enumerate(call.rows):  # the gaps, on the CPU
        k, _ = ref.sequence(call, k64, b, kvh)
        for i in range(n):
            qr = q[row].double().reshape(kvh, heads // kvh, d)
            ks = k[:, :call.lens[b] - n + i + 1]
            two = torch.einsum("hgd,htd->hgt", qr, ks).topk(2, -1).values
            reach = torch.einsum("hgd,htd->hgt", qr.abs(), ks.abs()).amax(-1)
            assert torch.all(two[..., 0] - two[..., 1] >= 5e-4 * reach)
            row += 1
    cache = device_cache(nf4, ((codes, a), nat[1]), bs, quant)
    want = ref.attention(call, q, k64, v64, ref.sqrt_scale(d), True, 0)
    for max_len in (1, 1 << 17):
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=5, max_len=max_len)
        check_rows(out, want[0], want[1], torch.zeros_like(want[2]), seen, dtype, quant, d, 75)


def test_strides_of_one_row_and_one_head_do_not_matter(nf4, orc):  # noqa: F811
    """A dimension of one element may have any stride: keys, values, queries, outputs and
    caches that differ there alone give what dense ones give, with no copy of an output."""
    d, bs, page, heads, kvh = 128, 64, 16, 4, 2
    call, pages = ref.make_call([20], [1], page, 960)
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, pages, kvh, page, d, bs, "nf4", 961)
    one, two = device_cache(nf4, nat, bs, "nf4"), device_cache(nf4, nat, bs, "nf4")
    where = gpu_call(call)

    def odd(t):  # the same elements, the row 3 elements off a multiple of 16 bytes
        room = torch.zeros(3 * (t.shape[1] * d + 3), dtype=t.dtype, device="cuda")
        view = room.as_strided((3, t.shape[1], d), (t.shape[1] * d + 3, d, 1))[:1]
        view.copy_(t)
        return view

    k, v = (row_values((1, kvh, d), "bf16", 962 + i).cuda() for i in range(2))
    q = queries(1, heads, d, "bf16", 964).cuda()
    want = nf4.kv_write(one, k, v, *where, values=True)
    got = nf4.kv_write(two, odd(k), odd(v), *where, values=True)
    assert all(same(a, b) for a, b in zip(want, got))
    for (c0, a0), (c1, a1) in zip(natural(one), natural(two)):
        assert torch.equal(c0, c1) and same(a0, a1)
    o = nf4.kv_attention(q, one, *where)
    assert same(nf4.kv_attention(odd(q), one, *where), o)
    out = odd(torch.zeros_like(q))
    assert nf4.kv_attention(q, one, *where, out=out) is out and same(out, o)
    pair = odd(torch.zeros_like(k)), torch.zeros_like(v)
    nf4.kv_read(one, 1, *where, out=pair)
    assert same(pair[0], want[0]) and same(pair[1], want[1])
    # one kv head: pages [pages, page_size, 1, ...] seen as [pages, 1, page_size, ...]
    nat = ref.random_cache(book, pages, 1, page, d, 128, "nf4", 965)
    plain = device_cache(nf4, nat, 128, "nf4")
    turned = nf4.KVCache(*(t.squeeze(1).unsqueeze(2).transpose(1, 2) for t in
                           (plain.k_packed, plain.k_absmax, plain.v_packed, plain.v_absmax)), 128, "nf4")
    assert turned.k_packed.stride(1) == d // 2
    assert same(nf4.kv_attention(q, turned, *where), nf4.kv_attention(q, plain, *where))
    # one head of queries, its stride odd
    q1 = q[:, :1]
    lone = torch.zeros(1, 1, d, dtype=q.dtype, device="cuda").as_strided((1, 1, d), (5, 3, 1))
    lone.copy_(q1)
    assert same(nf4.kv_attention(lone, plain, *where), nf4.kv_attention(q1.contiguous(), plain, *where))
    # one page
    single = nf4.KVCache.empty(1, page, kvh, d, bs)
    for t in (single.k_packed, single.v_packed):
        t.fill_(0x5a)
    for t in (single.k_absmax, single.v_absmax):
        t.fill_(0.5)
    loose = nf4.KVCache(*(t.as_strided(t.shape, (7, *t.stride()[1:])) for t in
                          (single.k_packed, single.k_absmax, single.v_packed, single.v_absmax)), bs, "nf4")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([9], dtype=torch.int32, device="cuda")
    assert same(nf4.kv_attention(q, loose, table, lens), nf4.kv_attention(q, single, table, lens))


@pytest.mark.parametrize("past", [1, 3, 20, 1 << 30])
def test_lengths_past_the_table(nf4, orc, past):  # noqa: F811
    """Positions that the table has no room for are not there, as if its rows went on with
    pages of -1: what is cached is not overwritten, reads give zeros, rows see the
    positions that there are. Bitwise the calls with such a longer table, and those of
    lengths that end within it for the other sequence."""
    heads, kvh, d, bs, page, cols = 8, 2, 64, 32, 16, 3
    lens, rows = [cols * page + past, 21], [5, 5]
    book = ref.codebook(orc, "nf4")
    table = torch.tensor([[3, 1, 5], [0, 4, -1]], dtype=torch.int32)
    pages = 6
    nat = ref.random_cache(book, pages, kvh, page, d, bs, "nf4", 951)
    off = torch.tensor([0, 5, 10], dtype=torch.int32)
    x = [row_values((10, kvh, d), "bf16", 952 + i).cuda() for i in range(2)]
    q = queries(10, heads, d, "bf16", 954).cuda()
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    where = (table.cuda(), lens_t, off.cuda())
    cache = device_cache(nf4, nat, bs, "nf4")
    kq, vq = nf4.kv_write(cache, *x, *where, values=True)
    got = natural(cache)
    # the rows of the first sequence that have a place, by the definition
    call = ref.Call(torch.cat([table, torch.full((2, 2), -1, dtype=torch.int32)], 1),
                    [min(lens[0], (cols + 2) * page), 21], rows, off, page)
    kept = {i for i in range(5) if lens[0] - 5 + i < cols * page}
    written = torch.zeros(pages, page, dtype=torch.bool)
    for i in range(5):
        if i in kept:
            p = lens[0] - 5 + i
            written[table[0, p // page], p % page] = True
        p = 16 + i
        written[table[1, p // page], p % page] = True
    for which in range(2):
        for new, old in zip(got[which], nat[which]):
            assert torch.equal(new[~written[:, None].expand(new.shape[:3])],
                               old[~written[:, None].expand(old.shape[:3])])
    k, v = nf4.kv_read(cache, 10, *where)
    for i in range(10):
        for t, val in ((k, kq), (v, vq)):
            if i >= 5 or i in kept:
                assert same(t[i], val[i]), i
            else:
                assert torch.all(t[i] == 0), i
    # attention: the longer table's where it can be written down, the definition besides
    k64, v64 = (dense(book, *t, bs) for t in got)
    for causal, window in ((True, 0), (False, 0), (True, 7), (False, 30)):
        kw = dict(max_rows=5, causal=causal, window=window)
        for max_len in (1, 1 << 17):
            out = nf4.kv_attention(q, cache, *where, max_len=max_len, **kw)
            if past < 1 << 20:
                longer = (call.table.cuda(), *where[1:])
                assert same(nf4.kv_attention(q, cache, *longer, max_len=max_len, **kw), out)
                want = ref.attention(call, q.cpu(), k64, v64, ref.sqrt_scale(d), causal, window)
                check_rows(out, *want, largest_seen(call, got[1][1], heads, causal, window),
                           "bf16", "nf4", d, 48)
            elif window:
                assert torch.all(out[:5] == 0)
            else:
                full = torch.tensor([cols * page, 21], dtype=torch.int32).cuda()
                again = nf4.kv_attention(q, cache, where[0], full, where[2], max_len=max_len,
                                         max_rows=5, causal=False)
                assert same(out[:5], again[:5])


def test_a_window_below_32_bits_is_refused(nf4):  # noqa: F811
    cache = nf4.KVCache.empty(1, 16, 1, 64)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    for window in (-1, -(1 << 32)):
        with pytest.raises(nf4.Nf4Error):
            nf4.kv_attention(q, cache, one[None] - 1, one, window=window)


def test_large_keys_beside_a_large_query(nf4, orc):  # noqa: F811
    """Keys of 2^118 under queries of 2^-118, one of which is of 2^80: the others' scores
    are ordinary."""
    d, bs, heads, kvh = 128, 64, 4, 2
    call, pages = ref.make_call([75, 40], [5, 3], 16, 990)
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, pages, kvh, 16, d, bs, "nf4", 991)
    codes, a = nat[0]
    a = a * 2.0 ** 118
    q = queries(call.total, heads, d, "fp32", 992) * 2.0 ** -118
    q[1] = queries(1, heads, d, "fp32", 993)[0] * 2.0 ** 80
    keep = [0, 2, 3, 4, 5, 6, 7]
    cache = device_cache(nf4, ((codes, a), nat[1]), bs, "nf4")
    want = ref.attention(call, q, dense(book, codes, a, bs), dense(book, *nat[1], bs),
                         ref.sqrt_scale(d), True, 0)
    seen = largest_seen(call, nat[1][1], heads, True, 0)
    for max_len in (1, 1 << 17):
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=5, max_len=max_len)
        check_rows(out, *want, seen, "fp32", "nf4", d, 75, keep)
