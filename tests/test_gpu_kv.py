"""The 4-bit key/value cache on the GPU, through the Python binding, against the
plain cache of kv_reference.py (64 bits) and the C oracle's quantization.

Writes are bit-exact: codes, scales and the values handed back. Reads are
bit-exact. Attention is held to two derived bounds per case:

 element by element,  |o - ref| <= S (2 r + w + 2^-22 + 2 (T + 64) 2^-24) + h |ref| + floor
   S = sum_p e_p |v_p|, the output's absolute attention; r = the largest error of
   a score: c (keys' code values) + (D + 16) 2^-24 (products, sums and scales in
   fp32) of the largest sum_d |q_d k_d| scale, plus 2^-21 for the exponential and
   its argument near the maximum; a softmax weight is off by twice that at most
   (numerator and denominator), w its own rounding; 2^-22 that of the values'
   codes (two fp16 parts); T positions are summed; h the rounding of the output
   (half a step). c: fp16's half step 2^-11 for bf16 rows (0 for E2M1 codes,
   which are exact), 2^-22 for fp16 rows and for fp32 rows, whose queries have two
   parts too. w:
   2^-11 for bf16 rows, 2^-22 (two parts) otherwise, and for these 2^-22 more: the
   product of the weights' and the values' second parts, each at most 2^-11 of the
   whole, is left out.
   A floor is added, which shows where the largest weights meet zeros. The weight
   of position p enters the matrix cores as w = 2^(t - m) a / A 2^8 in fp16, whose
   half step below 2^-14 (and that of the second part of a two-part weight) is
   2^-25. Undone, that is 2^-33 A, and divided by the sum of weights, which is at
   least 1 (the largest score is at least m), it is at most 2^-33 A |c| <= 2^-32 a_max
   for each of T positions (A is a power of two, at most twice the largest scale
   seen): T 2^-32 a_max;

 in the norm,  |o - ref| <= (h + 2^-10) |ref| for 16-bit rows (keys' code
   values 6e-5, weights 2^-12 rms, scores of size about 2: below 2^-10 together,
   independent from position to position), and 4e-6 for fp32 rows. The
   sums over positions are long enough there for signs to average.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module")
def nf4():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import bit_weight_quantization_nf4_amd as m

    assert m.lib().nf4_device_check() == 0, "device is not gfx950"
    return m


def bits(t):
    t = t.detach().cpu().contiguous()
    return t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32) \
        if t.dtype == torch.float32 else t


def same(a, b):
    return torch.equal(bits(a), bits(b))


def device_cache(nf4, nat, bs, quant_type, page_gap=0):
    """The natural-order cache laid out on the GPU; page_gap: bytes between pages."""
    out = []
    for which, (codes, a) in zip("kv", nat):
        for t in (ref.lay_out(codes, which), a):
            if not page_gap:
                out.append(t.cuda())
                continue
            n = t[0].numel()
            room = torch.zeros(t.shape[0], n + page_gap // t.element_size(), dtype=t.dtype,
                               device="cuda")
            view = room[:, :n].view(t.shape[0], *t.shape[1:]) if False else \
                room.as_strided(t.shape, (room.stride(0), *t.stride()[1:]))
            view.copy_(t)
            out.append(view)
    kp, ka, vp, va = out
    return nf4.KVCache(kp, ka, vp, va, bs, quant_type)


def natural(cache):
    return [(ref.codes_of(p.cpu().contiguous(), w), a.cpu().clone()) for w, p, a in
            (("k", cache.k_packed, cache.k_absmax), ("v", cache.v_packed, cache.v_absmax))]


def gpu_call(call):
    lens = torch.tensor(call.lens, dtype=torch.int32).cuda()
    return call.table.cuda(), lens, call.offsets.cuda()


# ------------------------------------------------------------ write and read

WRITES = [
    # dtype, quant, D, bs, heads, page, lens, rows
    ("bf16", "nf4", 128, 64, 2, 16, [1], [1]),
    ("bf16", "nf4", 128, 64, 3, 16, [5, 16, 40, 17], [5, 1, 33, 2]),
    ("fp16", "nf4", 64, 32, 1, 48, [100, 3], [77, 3]),
    ("fp32", "nf4", 256, 128, 2, 32, [64, 31, 9], [64, 30, 1]),
    ("bf16", "fp4", 96, 32, 2, 16, [21, 22, 23], [6, 7, 8]),
    ("fp16", "fp4", 192, 64, 2, 16, [19], [18]),
    ("fp32", "fp4", 128, 32, 2, 64, [70, 2], [5, 2]),
    ("bf16", "nf4", 256, 32, 1, 16, [37], [37]),
    ("bf16", "nf4", 192, 32, 5, 16, [33, 1], [13, 1]),
    ("fp16", "nf4", 64, 64, 8, 16, [18] * 9, [1] * 9),
    ("fp32", "nf4", 128, 128, 4, 16, [300], [290]),
]


def row_values(shape, dtype, seed):
    """Rows with what quantization meets: normal values, whole blocks of zeros,
    tiny and huge blocks (past the fast division's range), ties, the type's
    largest and smallest magnitudes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    n = x.shape[0]
    d = shape[-1]
    x[n // 2, 0, :32] = 0
    x[0, 0, d - 32:] *= 1e-4 if dtype == "fp16" else 1e-36
    if dtype == "fp32":
        x[n // 3, -1, 32:64] *= 1e37
        x[n - 1, 0, :32] *= 1e-41
    elif dtype == "bf16":
        x[n // 3, -1, 32:64] *= 1e37
        x[n - 1, 0, :32] *= 1e-40
    else:
        x[n // 3, -1, 32:64] *= 1e4
        x[n - 1, 0, :32] *= 1e-6
    x[n - 1, -1, 32:48] = torch.linspace(-1, 1, 16)
    return x.to(DT[dtype])


def expected_write(orc, x, dtype, bs, quant_type):
    """codes [rows, heads, D], absmax [rows, heads, D / bs], values as x's dtype."""
    host = x.numpy() if dtype == "fp32" else x.view(torch.int16).numpy().view(np.uint16)
    p, a = orc.quantize_typed(np.ascontiguousarray(host), dtype, bs, quant_type)
    p = torch.from_numpy(np.asarray(p).reshape(-1).copy())
    codes = torch.stack((p >> 4, p & 15), -1).reshape(x.shape)
    a = torch.from_numpy(np.asarray(a).copy()).reshape(*x.shape[:-1], -1)
    book = torch.from_numpy(orc.codebook(quant_type))
    vals = (book[codes.long()] * a.repeat_interleave(bs, -1)).to(DT[dtype])
    return codes, a, vals


@pytest.mark.parametrize("dtype,quant,d,bs,heads,page,lens,rows", WRITES)
def test_write_and_read_bitwise(nf4, orc, dtype, quant, d, bs, heads, page, lens, rows):
    call, pages = ref.make_call(lens, rows, page, 11 + d)
    book = ref.codebook(orc, quant)
    before = ref.random_cache(book, pages, heads, page, d, bs, quant, 12)
    cache = device_cache(nf4, before, bs, quant)
    x = [row_values((call.total, heads, d), dtype, 13 + i) for i in range(2)]
    # a row behind the last sequence stays out of everything
    pad = [torch.cat([t, torch.full((3, heads, d), 7.0, dtype=t.dtype)]).cuda() for t in x]
    kq, vq = nf4.kv_write(cache, *pad, *gpu_call(call), values=True)
    torch.cuda.synchronize()
    got = natural(cache)
    for which in range(2):
        codes, a, vals = expected_write(orc, x[which], dtype, bs, quant)
        want_c, want_a = before[which][0].clone(), before[which][1].clone()
        for row, _, _, pg, at in call.places():
            want_c[pg, :, at] = codes[row]
            want_a[pg, :, at] = a[row]
        assert torch.equal(got[which][0], want_c), "codes"
        assert same(got[which][1], want_a), "scales"
        assert same((kq, vq)[which][:call.total], vals), "values"
    # read the written rows back in every type; rows behind the last are untouched
    for out_dt in ("bf16", "fp16", "fp32"):
        out = [torch.full((call.total + 3, heads, d), 5.0, dtype=DT[out_dt], device="cuda")
               for _ in range(2)]
        nf4.kv_read(cache, call.total + 3, *gpu_call(call), out=out)
        fbook = torch.from_numpy(orc.codebook(quant))
        for which in range(2):
            codes, a = got[which]
            full = fbook[codes.long()] * a.repeat_interleave(bs, -1)
            want = torch.stack([full[pg, :, at] for _, _, _, pg, at in call.places()])
            assert same(out[which][:call.total], want.to(DT[out_dt])), out_dt
            assert torch.all(out[which][call.total:] == 5.0)
    # whole sequences from the start
    whole, _ = ref.make_call(lens, lens, page, 11 + d)
    k, v = nf4.kv_read(cache, whole.total, *gpu_call(whole), dtype=torch.float32)
    for which, t in enumerate((k, v)):
        codes, a = got[which]
        full = fbook[codes.long()] * a.repeat_interleave(bs, -1)
        want = torch.stack([full[pg, :, at] for _, _, _, pg, at in whole.places()])
        assert same(t, want)


def test_write_without_values_strided_and_uniform(nf4, orc):
    """Keys and values as slices of one projection's output, no offsets, pages of a
    larger allocation; and head-major rows. Bitwise the contiguous call."""
    heads, d, bs, page = 2, 128, 64, 16
    lens, rows = [20, 9, 33], [4, 4, 4]
    call, pages = ref.make_call(lens, rows, page, 21)
    book = ref.codebook(orc, "nf4")
    before = ref.random_cache(book, pages, heads, page, d, bs, "nf4", 22)
    proj = row_values((call.total, 8, d), "bf16", 23).cuda()  # query heads 0..3, then K, V
    k, v = proj[:, 4:6], proj[:, 6:8]
    table, lens_t, off = gpu_call(call)
    one = device_cache(nf4, before, bs, "nf4")
    nf4.kv_write(one, k.contiguous(), v.contiguous(), table, lens_t, off)
    two = device_cache(nf4, before, bs, "nf4", page_gap=4096)
    assert nf4.kv_write(two, k, v, table, lens_t) is None
    head_major = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (k, v)]
    three = device_cache(nf4, before, bs, "nf4")
    nf4.kv_write(three, *head_major, table, lens_t, off)
    for other in (two, three):
        for (c0, a0), (c1, a1) in zip(natural(one), natural(other)):
            assert torch.equal(c0, c1) and same(a0, a1)
    # an unaligned view is copied, keys and values of different strides too
    odd = torch.empty(call.total * heads * d + 1, dtype=torch.bfloat16, device="cuda")
    odd = odd[1:].view(call.total, heads, d)
    odd.copy_(k)
    four = device_cache(nf4, before, bs, "nf4")
    nf4.kv_write(four, odd, v, table, lens_t, off)
    for (c0, a0), (c1, a1) in zip(natural(one), natural(four)):
        assert torch.equal(c0, c1) and same(a0, a1)


def test_rows_without_a_place(nf4, orc):
    """Pages that are not there, positions before the first, lengths of zero and past
    the table: nothing is written, reads give zeros, values are handed back."""
    heads, d, bs, page = 2, 64, 32, 16
    call, pages = ref.make_call([40, 20, 3], [40, 20, 3], page, 31, holes=[(0, 1)])
    call.table[1, 1] = 10 ** 6  # past the cache
    call.lens = [40, 20, 2]     # the third sequence has more rows than positions
    book = ref.codebook(orc, "nf4")
    before = ref.random_cache(book, pages, heads, page, d, bs, "nf4", 32)
    cache = device_cache(nf4, before, bs, "nf4")
    x = [row_values((call.total, heads, d), "bf16", 33 + i) for i in range(2)]
    kq, vq = nf4.kv_write(cache, x[0].cuda(), x[1].cuda(), *gpu_call(call), values=True)
    got = natural(cache)
    places = [(r, pg if 0 <= pg < pages else -1, at) for r, _, _, pg, at in call.places()]
    for which in range(2):
        codes, a, vals = expected_write(orc, x[which], "bf16", bs, "nf4")
        want_c, want_a = before[which][0].clone(), before[which][1].clone()
        for r, pg, at in places:
            if pg >= 0:
                want_c[pg, :, at] = codes[r]
                want_a[pg, :, at] = a[r]
        assert torch.equal(got[which][0], want_c) and same(got[which][1], want_a)
        assert same((kq, vq)[which], vals)
    k, v = nf4.kv_read(cache, call.total, *gpu_call(call))
    for which, t in enumerate((k, v)):
        _, _, vals = expected_write(orc, x[which], "bf16", bs, "nf4")
        for r, pg, _ in places:
            if pg < 0:
                assert torch.all(t[r] == 0)
            else:
                assert same(t[r], vals[r])
    assert sum(pg < 0 for _, pg, _ in places) == 16 + 4 + 1
    # an empty cache, and lengths past the table
    none = nf4.KVCache.empty(0, page, heads, d, bs)
    kv0 = nf4.kv_read(none, 2, torch.full((1, 3), 5, dtype=torch.int32).cuda(),
                      torch.tensor([9], dtype=torch.int32).cuda())
    assert all(torch.all(t == 0) for t in kv0)
    long = torch.tensor([1 << 30, 40, 40], dtype=torch.int32).cuda()
    call.table[1, 1] = call.table[1, 0]
    k, v = nf4.kv_read(cache, call.total, call.table.cuda(), long, call.offsets.cuda())
    torch.cuda.synchronize()


# ------------------------------------------------------------------ attention

ATTENTION = [
    # dtype, quant, D, bs, heads, kv heads, page, lens, rows, causal, window
    ("bf16", "nf4", 128, 64, 4, 1, 16, [1], [1], True, 0),
    ("bf16", "nf4", 128, 64, 8, 2, 16, [15, 16, 17, 31, 32, 33], [1] * 6, True, 0),
    ("bf16", "nf4", 128, 128, 8, 2, 48, [255, 256, 257, 1000], [1, 1, 1, 1], True, 0),
    ("bf16", "nf4", 128, 32, 4, 4, 64, [513, 70], [1, 1], True, 0),
    ("fp16", "nf4", 64, 64, 6, 2, 16, [100, 47, 5], [7, 3, 5], True, 0),
    ("fp16", "nf4", 64, 32, 16, 1, 32, [300, 29], [2, 1], True, 0),
    ("fp16", "nf4", 128, 64, 3, 3, 16, [90], [20], False, 0),
    ("fp32", "nf4", 128, 64, 8, 2, 16, [333, 64], [3, 1], True, 0),
    ("fp32", "nf4", 256, 128, 4, 2, 16, [129, 300], [5, 9], True, 40),
    ("fp32", "fp4", 64, 32, 2, 2, 16, [77], [70], True, 0),
    ("fp32", "nf4", 192, 32, 2, 1, 16, [50, 50], [4, 17], False, 0),
    ("fp32", "nf4", 96, 32, 4, 1, 16, [211], [9], True, 0),
    ("bf16", "fp4", 256, 64, 8, 1, 16, [401, 9], [5, 2], True, 0),
    ("bf16", "nf4", 256, 32, 2, 2, 16, [65], [33], True, 0),
    ("fp16", "nf4", 256, 128, 4, 4, 64, [200, 150], [1, 1], True, 0),
    ("bf16", "nf4", 96, 32, 5, 1, 16, [140, 33], [11, 1], True, 17),
    ("fp16", "fp4", 192, 64, 4, 2, 16, [87], [6], True, 0),
    ("bf16", "nf4", 192, 32, 16, 2, 32, [190, 63], [1, 4], True, 0),
    ("bf16", "nf4", 64, 32, 40, 1, 16, [75, 200], [1, 3], True, 64),
    ("bf16", "nf4", 128, 64, 8, 2, 64, [700, 512], [130, 64], True, 0),
    ("bf16", "nf4", 128, 64, 4, 2, 16, [600], [100], True, 33),
    ("fp16", "nf4", 128, 32, 2, 1, 16, [280], [60], True, 1),
    # rows that see nothing: more rows than positions, empty sequences, no rows
    ("bf16", "nf4", 128, 64, 4, 2, 16, [3, 0, 40, 8], [7, 2, 0, 8], True, 0),
    ("fp32", "nf4", 64, 64, 4, 2, 16, [0, 2], [1, 40], True, 3),
    ("fp16", "nf4", 128, 128, 2, 2, 16, [0, 5], [3, 3], False, 0),
]


def queries(total, heads, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(total, heads, d, generator=g).to(DT[dtype])


def check_attention(got, want, spread, reach, dtype, quant, d, longest, nat, norm=True):
    c = {"bf16": 2.0 ** -11, "fp16": 2.0 ** -22, "fp32": 2.0 ** -22}[dtype]
    c = 0.0 if quant == "fp4" else c
    w = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    r = (c + (d + 16) * 2.0 ** -24) * reach + 2.0 ** -21
    if dtype == "fp32":
        r = r + 2.0 ** -22 * reach  # the queries' two parts
    bound = spread * (2 * r + w + 2.0 ** -22 + 2 * (longest + 64) * 2.0 ** -24) + HALF[dtype] * want.abs()
    if dtype == "fp16":
        bound = bound + 2.0 ** -25  # subnormal outputs
    bound = bound + longest * 2.0 ** -32 * nat[1][1].max().item()
    err = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all()
    assert torch.all(err <= bound), (err - bound).max().item()
    if norm and want.norm() > 0:
        rel = ((got.double().cpu() - want).norm() / want.norm()).item()
        assert rel <= (4e-6 if dtype == "fp32" else HALF[dtype] + 2.0 ** -10), rel


def run_attention(nf4, orc, case, seed, max_len=0, **kw):
    dtype, quant, d, bs, heads, kvh, page, lens, rows, causal, window = case
    call, pages = ref.make_call(lens, rows, page, seed, holes=kw.pop("holes", ()))
    book = ref.codebook(orc, quant)
    nat = ref.random_cache(book, pages, kvh, page, d, bs, quant, seed + 1)
    cache = device_cache(nf4, nat, bs, quant)
    q = queries(call.total, heads, d, dtype, seed + 2)
    out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=max(rows), max_len=max_len,
                           causal=causal, window=window, **kw)
    k64, v64 = (dense(*x) for x in ((book, *nat[0], bs), (book, *nat[1], bs)))
    want = ref.attention(call, q, k64, v64, kw.get("scale") or ref.sqrt_scale(d), causal, window)
    return out, want, (call, cache, q, nat)


def dense(book, codes, a, bs):
    return ref.dense(book, codes, a, bs)


@pytest.mark.parametrize("split", ["one", "many"])
@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_attention(nf4, orc, case, split):
    """split many: max_len far past the lengths, so positions are spread over as many
    workgroups as the device has room for and joined; one: no workspace."""
    out, want, (_, _, _, nat) = run_attention(nf4, orc, case, 100 + case[2],
                                              1 if split == "one" else 1 << 17)
    check_attention(out, *want, case[0], case[1], case[2], max(case[7]), nat)
    empty = want[1].sum(-1) == 0
    assert torch.all(out.cpu()[empty] == 0)


# Rows of a workgroup's waves are their own from 128 (row, head) pairs a kv head and 256
# workgroups on; positions are then split where max_len is large and workgroups few.
MANY_ROWS = [
    ("bf16", "nf4", 128, 64, 64, 64, 16, [150, 131, 97, 128], [128, 100, 97, 3], True, 0),
    ("fp16", "fp4", 64, 32, 96, 32, 48, [70, 61, 43, 99, 0, 12, 50, 43], [43, 40, 1, 43, 7, 12, 33, 43], True, 0),
    ("fp32", "nf4", 256, 128, 32, 32, 16, [129, 140, 128, 77], [128, 100, 128, 77], True, 0),
    ("bf16", "nf4", 192, 64, 64, 32, 16, [90, 101, 64, 150], [64, 33, 64, 1], True, 20),
    ("fp16", "nf4", 96, 32, 64, 64, 32, [128, 60, 200, 5], [128, 60, 90, 9], False, 0),
    ("fp32", "nf4", 128, 32, 64, 64, 16, [128, 300, 33, 64], [128, 64, 33, 64], True, 0),
    ("bf16", "fp4", 256, 32, 32, 32, 16, [128, 140, 1, 90], [128, 128, 1, 40], True, 0),
]


@pytest.mark.parametrize("split", ["one", "many"])
@pytest.mark.parametrize("case", MANY_ROWS, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_attention_of_many_rows(nf4, orc, case, split):
    """As test_attention; rows of sequences shorter than their rows see nothing."""
    out, want, (_, _, _, nat) = run_attention(nf4, orc, case, 150 + case[2],
                                              1 if split == "one" else 1 << 17)
    check_attention(out, *want, case[0], case[1], case[2], max(case[7]), nat)
    assert torch.all(out.cpu()[want[1].sum(-1) == 0] == 0)


def test_attention_is_reproducible_and_split_by_its_arguments(nf4, orc):
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [1500, 700], [1, 1], True, 0)
    a, want, (call, cache, q, nat) = run_attention(nf4, orc, case, 200)
    for _ in range(3):
        b = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=1)
        assert same(a, b)
    # every split is within the bound
    for max_len in (1, 256, 1500, 4096, 10000, 1 << 15, 1 << 20):
        b = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=1, max_len=max_len)
        check_attention(b, *want, "bf16", "nf4", 128, 1500, nat)


def test_attention_strides_and_outputs(nf4, orc):
    """Queries as a slice of a fused projection and head-major, an output window,
    rows behind the last sequence and past max_rows left as they were."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [90, 33, 60], [5, 2, 9], True, 0)
    a, want, (call, cache, q, nat) = run_attention(nf4, orc, case, 300)
    table, lens, off = gpu_call(call)
    fused = torch.randn(call.total + 4, 12, 128, device="cuda").bfloat16()
    fused[:call.total, :8] = q.cuda()
    out = torch.full((call.total + 4, 10, 128), 3.0, device="cuda").bfloat16()
    got = nf4.kv_attention(fused[:, :8], cache, table, lens, off, max_rows=9, out=out[:, 1:9])
    assert got.data_ptr() == out[:, 1:9].data_ptr()
    assert same(out[:call.total, 1:9], a)
    assert torch.all(out[:, 0] == 3.0) and torch.all(out[:, 9] == 3.0)
    assert torch.all(out[call.total:] == 3.0)
    hm = torch.empty(8, call.total, 128, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    hm.copy_(q.cuda())
    out = torch.empty_like(hm)
    nf4.kv_attention(hm, cache, table, lens, off, max_rows=9, out=out)
    assert same(out, a)
    # 5 of 9 rows at most: the others stay
    out = torch.full((call.total, 8, 128), 3.0, device="cuda").bfloat16()
    nf4.kv_attention(q.cuda(), cache, table, lens, off, max_rows=5, out=out)
    assert torch.all(out[12:] == 3.0)
    check_attention(out[:12], *(t[:12] for t in want), "bf16", "nf4", 128, 90, nat)
    # no offsets
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [90, 33, 60], [4, 4, 4], True, 0)
    a, want, (call, cache, q, nat) = run_attention(nf4, orc, case, 301)
    table, lens, off = gpu_call(call)
    assert same(nf4.kv_attention(q.cuda(), cache, table, lens), a)


def test_attention_ignores_what_is_not_there(nf4, orc):
    """Missing pages inside a sequence, scales of NaN and infinity in positions past
    the lengths and in pages that no sequence has."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [100, 33], [3, 1], True, 0)
    a, want, (call, cache, q, nat) = run_attention(nf4, orc, case, 400, holes=[(0, 2), (1, 0)])
    check_attention(a, *want, "bf16", "nf4", 128, 100, nat)
    used = torch.zeros(cache.num_pages, 16, dtype=torch.bool)
    for b, n in enumerate(call.lens):
        for p in range(n):
            pg = int(call.table[b, p // 16])
            if pg >= 0:
                used[pg, p % 16] = True
    for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
        for t in (cache.k_absmax, cache.v_absmax):
            t.masked_fill_(~used.cuda()[:, None, :, None], bad)
        b = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=3)
        assert same(a, b), bad
    # page indices past the cache are as absent as negative ones
    table = call.table.clone()
    table[table < 0] = 2 ** 31 - 1
    _, lens, off = gpu_call(call)
    assert same(nf4.kv_attention(q.cuda(), cache, table.cuda(), lens, off, max_rows=3), a)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_attention_of_uneven_scales(nf4, orc, dtype):
    """Scores of hundreds (the softmax is one position's), positions whose values differ
    by 2^24, blocks of zeros, queries of very different size in one call."""
    quant, d, bs, heads, kvh, page = "nf4", 128, 64, 4, 2, 16
    call, pages = ref.make_call([200, 150], [4, 4], page, 500)
    book = ref.codebook(orc, quant)
    nat = ref.random_cache(book, pages, kvh, page, d, bs, quant, 501)
    g = torch.Generator().manual_seed(502)
    (kc, ka), (vc, va) = nat
    ka *= torch.where(torch.rand(ka.shape[:-1], generator=g) < 0.1, 12.0, 1.0)[..., None]
    va *= torch.exp2(torch.randint(-12, 13, va.shape[:-1], generator=g).float())[..., None]
    va[torch.rand(va.shape, generator=g) < 0.1] = 0.0
    ka[torch.rand(ka.shape, generator=g) < 0.1] = 0.0
    q = torch.randn(call.total, heads, d, generator=g)
    q *= torch.exp2(torch.randint(-8, 3, (call.total, heads, 1), generator=g).float())
    q[1, 1] = 0
    q = q.to(DT[dtype])
    cache = device_cache(nf4, nat, bs, quant)
    k64, v64 = dense(book, kc, ka, bs), dense(book, vc, va, bs)
    want = ref.attention(call, q, k64, v64, ref.sqrt_scale(d), True, 0)
    for max_len in (1, 1 << 17):
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=4, max_len=max_len)
        check_attention(out, *want, dtype, quant, d, 200, nat, norm=False)


def test_attention_of_extreme_value_scales(nf4, orc):
    """Value scales near the ends of fp32: their reference is a power of two in range."""
    for factor in (2.0 ** 100, 2.0 ** -100, 2.0 ** -126):
        call, pages = ref.make_call([70], [2], 16, 510)
        book = ref.codebook(orc, "nf4")
        nat = ref.random_cache(book, pages, 1, 16, 64, 32, "nf4", 511)
        nat[1][1].mul_(factor)
        cache = device_cache(nf4, nat, 32, "nf4")
        q = queries(2, 2, 64, "fp32", 512)
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=2).cpu().double()
        k64, v64 = (dense(book, *x, 32) for x in nat)
        want, spread, _ = ref.attention(call, q, k64, v64, 0.125, True, 0)
        # 2^-126: results are subnormal in part, in steps of 2^-149
        assert torch.all((out - want).abs() <= 1e-5 * spread + 2.0 ** -140 * (factor < 1e-37))


def test_attention_scale_argument(nf4, orc):
    case = ("fp32", "nf4", 64, 64, 4, 2, 16, [120], [3], True, 0)
    for scale in (1.0, -0.3, 1e-3):
        out, want, (_, _, _, nat) = run_attention(nf4, orc, case, 600, scale=scale)
        check_attention(out, *want, "fp32", "nf4", 64, 120, nat)
    out, _, (call, cache, q, nat) = run_attention(nf4, orc, case, 600, scale=0.0)
    book = ref.codebook(orc, "nf4")
    k64, v64 = (dense(book, *x, 64) for x in nat)
    want = ref.attention(call, q, k64, v64, 0.0, True, 0)
    check_attention(out, *want, "fp32", "nf4", 64, 120, nat)


def test_offsets_past_32_bits(nf4, orc):
    """Pages more than 4 GiB apart: written, read and attended to."""
    heads, d, bs, page = 2, 128, 64, 16
    gap = 5 << 30
    codes = torch.zeros(gap + 16 * heads * d // 2, dtype=torch.uint8, device="cuda")
    shape = (2, heads, page, d // 2)
    inner = (page * d // 2, d // 2, 1)
    kp = codes.as_strided(shape, (gap, *inner))
    vcodes = torch.zeros_like(codes)
    vp = vcodes.as_strided(shape, (gap, *inner))
    sgap = (9 << 30) // 8  # floats: 4.5 GiB
    scales = torch.zeros(sgap + heads * page * 2, device="cuda")
    ka = scales.as_strided((2, heads, page, 2), (sgap, page * 2, 2, 1))
    vscales = torch.zeros_like(scales)
    va = vscales.as_strided((2, heads, page, 2), (sgap, page * 2, 2, 1))
    cache = nf4.KVCache(kp, ka, vp, va, bs, "nf4")
    call = ref.Call(torch.tensor([[0, 1]], dtype=torch.int32), [30], [30],
                    torch.tensor([0, 30], dtype=torch.int32), page)
    x = [row_values((30, heads, d), "bf16", 700 + i) for i in range(2)]
    kq, vq = nf4.kv_write(cache, x[0].cuda(), x[1].cuda(), *gpu_call(call), values=True)
    k, v = nf4.kv_read(cache, 30, *gpu_call(call))
    assert same(k, kq) and same(v, vq)
    for which, t in enumerate((k, v)):
        assert same(t, expected_write(orc, x[which], "bf16", bs, "nf4")[2])
    small = nf4.KVCache.empty(2, page, heads, d, bs)
    nf4.kv_write(small, x[0].cuda(), x[1].cuda(), *gpu_call(call))
    q = queries(30, 4, d, "bf16", 702).cuda()
    assert same(nf4.kv_attention(q, cache, *gpu_call(call), max_rows=30),
                nf4.kv_attention(q, small, *gpu_call(call), max_rows=30))


def test_long_sequence(nf4, orc):
    """A length in the tens of thousands against float64 on the GPU."""
    d, bs, n = 128, 128, 70001
    g = torch.Generator(device="cuda").manual_seed(800)
    cache = nf4.KVCache.empty(n // 256 + 1, 256, 2, d, bs)
    table = torch.randperm(cache.num_pages, generator=g, device="cuda").to(torch.int32)[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(n, 2, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    nf4.kv_write(cache, k, v, table, lens)
    k, v = nf4.kv_read(cache, n, table, lens, dtype=torch.float32)
    q = torch.randn(1, 8, d, generator=g, device="cuda")
    s = (q.double().view(2, 4, d) @ k.double().permute(1, 2, 0)) * d ** -0.5
    want = (torch.softmax(s, -1) @ v.double().transpose(0, 1)).view(1, 8, d)
    for dt, tol in ((torch.float32, 4e-6), (torch.float16, 2.0 ** -10), (torch.bfloat16, 2.0 ** -7)):
        qd = q.to(dt)
        if dt != torch.float32:
            s = (qd.double().view(2, 4, d) @ k.double().permute(1, 2, 0)) * d ** -0.5
            want = (torch.softmax(s, -1) @ v.double().transpose(0, 1)).view(1, 8, d)
        out = nf4.kv_attention(qd, cache, table, lens).double()
        assert ((out - want).norm() / want.norm()).item() <= tol


def test_streams_and_graphs(nf4, orc):
    """A decode step (write, attention, read) on another stream and captured in two
    graphs that share a pool, replayed with eager work between: bitwise the eager step."""
    heads, kvh, d, bs, page = 8, 2, 128, 64, 16
    call, pages = ref.make_call([700, 350], [1, 1], page, 900)
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, pages, kvh, page, d, bs, "nf4", 901)
    cache = device_cache(nf4, nat, bs, "nf4")
    where = gpu_call(call)
    q = queries(2, heads, d, "bf16", 902).cuda()
    x = [row_values((2, kvh, d), "bf16", 903 + i).cuda() for i in range(2)]

    def step():
        kq, vq = nf4.kv_write(cache, *x, *where, values=True)
        o = nf4.kv_attention(q, cache, *where, max_rows=1, max_len=700)
        k, v = nf4.kv_read(cache, 2, *where)
        return [kq, vq, o, k, v]

    eager = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(eager, other))
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, pool=graphs[0].pool() if graphs else None):
            outs.append(step())
        graphs.append(gr)
    for rep in range(3):
        for gr, out in zip(graphs, outs):
            for t in out:
                t.fill_(0)
            gr.replay()
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(eager, out)), rep
            again = step()
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(eager, again))


def test_binding_refusals(nf4):
    cache = nf4.KVCache.empty(4, 16, 2, 128)
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    k = torch.zeros(1, 2, 128, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 128, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nf4.kv_write(cache, k.double(), k, table, lens)
    with pytest.raises(ValueError):
        nf4.kv_write(cache, k, k.float(), table, lens)
    with pytest.raises(ValueError):
        nf4.kv_write(cache, q, q, table, lens)
    with pytest.raises(TypeError):
        nf4.kv_write(cache, k, k, table.long(), lens)
    with pytest.raises(TypeError):
        nf4.kv_write(cache, k, k, table, lens.cpu())
    with pytest.raises(ValueError):
        nf4.kv_write(cache, k, k, table, lens, lens)
    with pytest.raises(ValueError):
        nf4.kv_attention(q[:, :3], cache, table, lens)
    with pytest.raises(ValueError):
        nf4.kv_attention(q[..., :64], cache, table, lens)
    with pytest.raises(ValueError):
        nf4.kv_attention(q, cache, table, lens, out=q.float())
    with pytest.raises(nf4.Nf4Error):
        nf4.kv_attention(q, cache, table, lens, window=-1)
    with pytest.raises(nf4.Nf4Error):
        nf4.KVCache.empty(4, 24, 2, 128) and nf4.kv_read(nf4.KVCache.empty(4, 24, 2, 128), 1, table,
                                                         lens)
    with pytest.raises(ValueError):
        nf4.kv_read(cache, 1, table, lens, out=(k, k.half()))


def test_workspace_too_small_is_refused(nf4):
    """The C call reports a workspace that is smaller than the query says."""
    from bit_weight_quantization_nf4_amd import kv

    cache = nf4.KVCache.empty(64, 16, 2, 128)
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([1000], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 128, device="cuda", dtype=torch.bfloat16)
    need = nf4.kv_attention_workspace_bytes(1, 1, 1 << 17, 4, 2, 128)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    rows = kv._rows(cache, 1, table, lens, None, "")
    for n, want in ((need - 1, 5), (0, 5)):
        st = kv._lib().nf4_kv_attention(cache.desc, rows, q.data_ptr(), 512, 128, 4, 0, 0.1, 1, 0, 1,
                                        1 << 17, q.data_ptr(), 512, 128, ws.data_ptr(), n, None)
        assert st == want


ROWS_APART = [
    # dtype, D, bs, heads, kv heads, lens, rows: waves that share a block of one tile, of
    # two, several such blocks, and waves with rows of their own
    ("bf16", 128, 64, 4, 2, [75, 40], [5, 3]),
    ("fp16", 64, 32, 16, 2, [90], [4]),
    ("fp32", 256, 128, 2, 1, [60], [6]),
    ("bf16", 128, 128, 8, 2, [170], [40]),
    ("fp16", 96, 32, 4, 1, [100, 37], [37, 33]),
    ("bf16", 128, 128, 64, 64, [140, 150, 131, 40], [128, 128, 100, 3]),
    ("fp32", 64, 32, 64, 32, [90, 70] * 2, [64, 64] * 2),
]


@pytest.mark.parametrize("split", ["one", "many"])
@pytest.mark.parametrize("case", ROWS_APART, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_queries_do_not_affect_each_other(nf4, orc, case, split):
    """One query of infinities, NaN, or near the type's ends: every other row (of the
    same block, too) is within its bounds, and the odd one is where it is finite."""
    dtype, d, bs, heads, kvh, lens, rows = case
    call, pages = ref.make_call(lens, rows, 16, 900)
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, pages, kvh, 16, d, bs, "nf4", 901)
    cache = device_cache(nf4, nat, bs, "nf4")
    k64, v64 = (dense(book, *x, bs) for x in nat)
    info = torch.finfo(DT[dtype])
    odd = torch.zeros(call.total, heads, dtype=torch.bool)
    odd[1, 0] = odd[call.total - 1, heads - 1] = True
    for value in (float("inf"), float("nan"), info.max, -info.max / 3, info.tiny):
        q = queries(call.total, heads, d, dtype, 902)
        q[1, 0] = 0
        q[1, 0, 5] = value
        q[-1, -1, 3::2] = value
        out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=max(rows),
                               max_len=1 if split == "one" else 1 << 17).cpu()
        clean = torch.where(odd[..., None], torch.zeros((), dtype=DT[dtype]), q)
        want, spread, reach = ref.attention(call, clean, k64, v64, ref.sqrt_scale(d), True, 0)
        got = torch.where(odd[..., None], want.to(out.dtype), out)
        check_attention(got, want, spread, reach, dtype, "nf4", d, max(lens), nat, norm=False)
        if value == info.tiny:  # scores of about zero: the mean of the values
            check_attention(out[1:2, :1], *(t[1:2, :1] for t in (want, spread, reach)), dtype,
                            "nf4", d, max(lens), nat, norm=False)
        elif not np.isfinite(value):
            assert not torch.isfinite(out[1, 0]).all() and not torch.isfinite(out[-1, -1]).all()


@pytest.mark.parametrize("split", ["one", "many"])
@pytest.mark.parametrize("case", ROWS_APART, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_positions_affect_only_rows_that_see_them(nf4, orc, case, split):
    """Scales of infinity and NaN at the newest position, which only the last row of its
    sequence sees, and at one that a window has left behind for all but the first."""
    dtype, d, bs, heads, kvh, lens, rows = case
    call, pages = ref.make_call(lens, rows, 16, 910)
    book = ref.codebook(orc, "nf4")
    nat = ref.random_cache(book, pages, kvh, 16, d, bs, "nf4", 911)
    k64, v64 = (dense(book, *x, bs) for x in nat)
    q = queries(call.total, heads, d, dtype, 912)
    b, window = len(lens) - 1, 19
    kw = dict(max_rows=max(rows), max_len=1 if split == "one" else 1 << 17, window=window)
    want = ref.attention(call, q, k64, v64, ref.sqrt_scale(d), True, window)
    first, last = call.total - rows[b], call.total - 1  # rows of sequence b
    newest = lens[b] - 1
    oldest = lens[b] - rows[b] + 1 - window             # seen by its first row only
    for pos, row in ((newest, last), (oldest, first)):
        if pos < 0:
            continue
        keep = [r for r in range(call.total) if r != row]
        for which in (0, 1):
            for bad in (float("inf"), float("nan")):
                cache = device_cache(nf4, nat, bs, "nf4")
                a = (cache.k_absmax, cache.v_absmax)[which]
                a[int(call.table[b, pos // 16]), :, pos % 16] = bad
                out = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), **kw).cpu()
                check_attention(out[keep], *(t[keep] for t in want), dtype, "nf4", d, max(lens),
                                nat, norm=False)
                assert not torch.isfinite(out[row]).all()


def test_rows_past_max_rows_and_wide_arguments(nf4, orc):
    """Rows past max_rows stay as they are; windows and lengths past 32 bits are as good
    as none."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [100, 33, 60], [6, 2, 3], True, 0)
    a, want, (call, cache, q, nat) = run_attention(nf4, orc, case, 920)
    out = torch.full_like(q, 7.0).cuda()
    nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=3, out=out)
    kept = [0, 1, 2, 6, 7, 8, 9, 10]
    assert torch.all(out[3:6] == 7.0)
    check_attention(out[kept], *(t[kept] for t in want), "bf16", "nf4", 128, 100, nat)
    wide = nf4.kv_attention(q.cuda(), cache, *gpu_call(call), max_rows=6, max_len=1 << 40,
                            window=(1 << 32) + 5)
    check_attention(wide, *want, "bf16", "nf4", 128, 100, nat)


def test_a_captured_step_follows_its_lengths(nf4):
    """One captured step (write and attention) replayed while the lengths grow in place
    past page ends, with a sequence that is padding (no pages, length 0) and rows behind
    the last offset: bitwise the eager steps on another cache, padding rows zeros."""
    g = torch.Generator(device="cuda").manual_seed(950)
    caches = [nf4.KVCache.empty(40, 16, 2, 128) for _ in range(2)]
    wide = torch.full((4, 12), -1, dtype=torch.int32)
    wide[:3, 2:11] = torch.randperm(40)[:27].view(3, 9).to(torch.int32)
    table = wide.cuda()[:, 2:11]  # a slice of a wider table
    lens = torch.tensor([14, 100, 1, 0], dtype=torch.int32).cuda()
    grow = torch.tensor([1, 1, 1, 0], dtype=torch.int32).cuda()
    off = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32).cuda()
    k, v = (torch.empty(6, 2, 128, device="cuda", dtype=torch.float16) for _ in range(2))
    q = torch.empty(6, 8, 128, device="cuda", dtype=torch.float16)
    start = torch.randn(2, 115, 2, 128, generator=g, device="cuda").half()
    start_off = torch.tensor([0, 14, 114, 115, 115], dtype=torch.int32).cuda()
    for c in caches:
        nf4.kv_write(c, start[0], start[1], table, lens, start_off)
    outs = [torch.empty_like(q) for _ in caches]

    def step(i):
        nf4.kv_write(caches[i], k, v, table, lens, off)
        nf4.kv_attention(q, caches[i], table, lens, off, max_rows=1, max_len=1 << 14, out=outs[i])

    def inputs():
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    inputs()
    lens += grow
    step(0)
    step(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    for i in range(36):
        inputs()
        lens += grow
        for o in outs:
            o.fill_(5.0)
        graph.replay()
        step(1)
        torch.cuda.synchronize()
        assert same(*outs), i
        assert torch.all(outs[0][3] == 0) and torch.all(outs[0][4:] == 5.0)
        assert torch.isfinite(outs[0]).all()
    # the same pages in both caches (those of the table: others are uninitialised)
    used = table[:3].long().unique()
    n = torch.zeros(40, 16, dtype=torch.bool, device="cuda")
    for b in range(3):
        for p in range(int(lens[b])):
            n[table[b, p // 16].long(), p % 16] = True
    for name in ("k_absmax", "v_absmax"):
        a, b = (getattr(c, name) for c in caches)
        at = n[:, None, :, None].expand_as(a)
        assert same(a[at], b[at])
    assert len(used) == 27


def test_calls_at_once_on_one_cache(nf4, orc):
    """Several calls in flight on streams of their own, each split and with a workspace of
    its own: each is what it is alone."""
    case = ("bf16", "nf4", 128, 64, 8, 2, 16, [3000, 2500], [1, 1], True, 0)
    a, want, (call, cache, q, nat) = run_attention(nf4, orc, case, 960, max_len=3000)
    where = gpu_call(call)
    qs = [(q.float() * f).to(q.dtype).cuda() for f in (1.0, 0.5, 0.25, 2.0)]
    alone = [nf4.kv_attention(x, cache, *where, max_rows=1, max_len=3000) for x in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        got = []
        for s, x in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(nf4.kv_attention(x, cache, *where, max_rows=1, max_len=3000))
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(alone, got))
    assert same(alone[0], a)


@pytest.mark.parametrize("rows", [1, 3])
def test_the_longest_sequence(nf4, rows):
    """2^31 - 2^20 positions (the most) and a length past them, in a table that repeats one
    page and ends in another: every score is 0, values are 1 and in the last page 2^15.
    A lane adds up 2^31 / (512 ranges 8 waves 32) = 2^14 steps of 8 positions, each addition
    off by 2^-24 of the sum, so sums and their quotient by 2^-9 at most."""
    page, most = 1 << 16, (1 << 31) - (1 << 20)
    cols = most // page
    cache = nf4.KVCache.empty(2, page, 1, 64, 64)
    cache.k_packed.fill_(0x35)
    cache.k_absmax.fill_(1.0)
    cache.v_packed.fill_(0xff)  # twice the code of 1
    cache.v_absmax[0] = 1.0
    cache.v_absmax[1] = 2.0 ** 15
    table = torch.zeros(1, cols + 40, dtype=torch.int32, device="cuda")
    table[0, cols - 1:] = 1
    q = torch.zeros(rows, 1, 64, device="cuda")
    want = torch.tensor(((most - page) + page * 2.0 ** 15) / most)
    for n in (most, (1 << 31) - 1):
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        o = nf4.kv_attention(q, cache, table, lens, causal=False).cpu()
        assert torch.all((o - want).abs() <= 2.0 ** -9 * want), (n, o[0, 0, 0])
        # the window of the last positions alone
        o = nf4.kv_attention(q, cache, table, lens, causal=False, window=1000).cpu()
        assert torch.all((o - 2.0 ** 15).abs() <= 2.0 ** -9 * 2.0 ** 15)
    k, v = nf4.kv_read(cache, rows, table, lens, dtype=torch.float32)
    assert torch.all(v == 2.0 ** 15)
