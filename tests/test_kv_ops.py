"""The torch.library operators of the key/value cache, and the cache at work: a
decoder layer with Linear4bit projections that stores a ragged batch of prompts, then
takes one token a step, then several drafted ones.

CPU: registration and the fake implementations. GPU: opcheck, torch.compile, and the
layer against float64 on the values that its cache holds.
"""
import pytest
import torch

import kv_reference as ref
from bit_weight_quantization_nf4_amd.ops import Linear4bit  # registers the nf4:: operators


def meta_cache(pages=4, heads=2, page=16, d=128, bs=64):
    e = lambda *s, dt: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    return [e(pages, heads, page, d // 2, dt=torch.uint8), e(pages, heads, page, d // bs, dt=torch.float32)] * 2


def test_operators_registered_with_fake_impls():
    c = meta_cache()
    table = torch.empty(1, 4, dtype=torch.int32, device="meta")
    lens = torch.empty(1, dtype=torch.int32, device="meta")
    q = torch.empty(3, 8, 128, dtype=torch.float16, device="meta")
    o = torch.ops.nf4.kv_attention(q, *c, table, lens, None, 64, "nf4")
    assert o.shape == q.shape and o.dtype == torch.float16
    k, v = torch.ops.nf4.kv_read(*c, table, lens, None, 5, 64, "nf4", torch.bfloat16)
    assert k.shape == v.shape == (5, 2, 128) and k.dtype == torch.bfloat16
    x = torch.empty(3, 2, 128, dtype=torch.float16, device="meta")
    assert torch.ops.nf4.kv_write(x, x, *meta_cache()[:2], *meta_cache()[:2], table, lens, None, 64,
                                  "nf4") is None
    kq, vq = torch.ops.nf4.kv_write_values(x, x, *meta_cache()[:2], *meta_cache()[:2], table, lens,
                                           None, 64, "nf4")
    assert kq.shape == x.shape and vq.dtype == torch.float16


# --------------------------------------------------------------------- GPU


@pytest.fixture(scope="module")
def nf4():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import bit_weight_quantization_nf4_amd as m

    assert m.lib().nf4_device_check() == 0, "device is not gfx950"
    return m


def small(nf4, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = nf4.KVCache.empty(6, 16, 2, 64, 32)
    table = torch.tensor([[3, 1, 5], [0, 4, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([40, 21], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 40, 61], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(61, 2, 64, generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn(61, 4, 64, generator=g, device="cuda").to(dtype)
    return cache, (table, lens, off), k, v, q


def buffers(cache):
    return cache.k_packed, cache.k_absmax, cache.v_packed, cache.v_absmax


@pytest.mark.gpu
def test_operators_equal_the_binding(nf4):
    cache, where, k, v, q = small(nf4)
    kq, vq = nf4.kv_write(cache, k, v, *where, values=True)
    o = nf4.kv_attention(q, cache, *where, max_rows=40, max_len=40, window=9)
    other = nf4.KVCache.empty(6, 16, 2, 64, 32)
    for t, u in zip(buffers(other), buffers(cache)):
        t.copy_(u)
        t.zero_()
    torch.ops.nf4.kv_write(k, v, *buffers(other), *where, 32, "nf4")
    rk, rv = torch.ops.nf4.kv_read(*buffers(other), *where, 61, 32, "nf4", torch.bfloat16)
    assert torch.equal(rk, kq) and torch.equal(rv, vq)
    wk, wv = torch.ops.nf4.kv_write_values(k, v, *buffers(other), *where, 32, "nf4")
    assert torch.equal(wk, kq) and torch.equal(wv, vq)
    p = torch.ops.nf4.kv_attention(q, *buffers(other), *where, 32, "nf4", 40, 40, None, True, 9)
    assert torch.equal(o, p)


@pytest.mark.gpu
def test_opcheck_and_compile(nf4):
    cache, where, k, v, q = small(nf4)
    nf4.kv_write(cache, k, v, *where)
    checks = ("test_schema", "test_faketensor")
    torch.library.opcheck(torch.ops.nf4.kv_write.default,
                          (k, v, *buffers(cache), *where, 32, "nf4"), test_utils=checks)
    torch.library.opcheck(torch.ops.nf4.kv_write_values.default,
                          (k, v, *buffers(cache), *where, 32, "nf4"), test_utils=checks)
    torch.library.opcheck(torch.ops.nf4.kv_read.default,
                          (*buffers(cache), *where, 61, 32, "nf4", torch.float16), test_utils=checks)
    torch.library.opcheck(torch.ops.nf4.kv_attention.default,
                          (q, *buffers(cache), *where, 32, "nf4", 40), test_utils=checks)

    def step(q, k, v, *c):
        torch.ops.nf4.kv_write(k * 2, v, *c, *where, 32, "nf4")
        return torch.ops.nf4.kv_attention(q, *c, *where, 32, "nf4", 40) + 1

    want = step(q, k, v, *buffers(cache))
    got = torch.compile(step, backend="aot_eager", fullgraph=True)(q, k, v, *buffers(cache))
    assert torch.equal(got, want)


class Layer(torch.nn.Module):
    """Attention of a decoder layer over a 4-bit cache, with 4-bit projections."""

    def __init__(self, nf4, width, heads, kv_heads, head_dim, dtype, pages):
        super().__init__()
        self.shape = heads, kv_heads, head_dim
        rows = (heads + 2 * kv_heads) * head_dim
        self.qkv = Linear4bit(width, rows, bias=False, compute_dtype=dtype)
        self.out = Linear4bit(heads * head_dim, width, bias=False, compute_dtype=dtype)
        self.pages = pages
        self.nf4 = nf4

    def forward(self, x, where, max_rows):
        h, kvh, d = self.shape
        qkv = self.qkv(x).view(-1, h + 2 * kvh, d)
        q, k, v = qkv[:, :h], qkv[:, h:h + kvh], qkv[:, h + kvh:]
        self.nf4.kv_write(self.pages, k, v, *where)
        o = self.nf4.kv_attention(q, self.pages, *where, max_rows=max_rows)
        return self.out(o.reshape(len(x), h * d)), q, o


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_layer_decodes_a_ragged_batch(nf4, dtype):
    """Prompts of several lengths, single tokens, then drafts of several tokens; every
    output of the attention against float64 over what the cache holds then. The bound
    is the output's rounding, half a step, and as much again in the norm (keys' code
    values 6e-5 and bf16's weights 2^-12 are well below it)."""
    torch.manual_seed(0)
    heads, kv_heads, d, width, page = 8, 2, 64, 256, 16
    cache = nf4.KVCache.empty(30, page, kv_heads, d, 32)
    layer = Layer(nf4, width, heads, kv_heads, d, dtype, cache).to("cuda")
    order = torch.randperm(30).to(torch.int32)
    table = order.view(3, 10).cuda()
    lens = [0, 0, 0]
    for rows in ([37, 5, 90], [1, 1, 1], [1, 1, 1], [4, 1, 2], [0, 3, 1]):
        lens = [a + b for a, b in zip(lens, rows)]
        off = [0]
        for n in rows:
            off.append(off[-1] + n)
        where = (table, torch.tensor(lens, dtype=torch.int32).cuda(),
                 torch.tensor(off, dtype=torch.int32).cuda())
        x = torch.randn(off[-1], width, device="cuda", dtype=dtype)
        y, q, o = layer(x, where, max(rows))
        assert y.shape == x.shape and torch.isfinite(y).all()
        # all that is cached so far, read back whole
        total = sum(lens)
        upto = [0]
        for n in lens:
            upto.append(upto[-1] + n)
        k, v = nf4.kv_read(cache, total, table, where[1],
                           torch.tensor(upto, dtype=torch.int32).cuda(), dtype=torch.float32)
        call = ref.Call(torch.zeros(3, 1, dtype=torch.int32), lens, rows, None, 1 << 20)
        call.table = torch.arange(3, dtype=torch.int32)[:, None]
        dense = []
        for t in (k, v):  # one page a sequence
            room = torch.zeros(3, kv_heads, max(lens), d, dtype=torch.float64)
            for b, n in enumerate(lens):
                room[b, :, :n] = t[upto[b]:upto[b + 1]].double().cpu().transpose(0, 1)
            dense.append(room)
        want, _, _ = ref.attention(call, q.cpu(), *dense, ref.sqrt_scale(d), True, 0)
        rel = ((o.double().cpu() - want).norm() / want.norm()).item()
        assert rel <= torch.finfo(dtype).eps, (rows, rel)
