"""A plain 4-bit key/value cache in 64 bits, for the tests: codes in natural
order, the layout of include/nf4_kv.h spelled out element by element, and
attention by its definition. Shares nothing with the library."""
import math
from dataclasses import dataclass

import numpy as np
import torch


def codebook(orc, quant_type) -> torch.Tensor:
    return torch.from_numpy(orc.codebook(quant_type).astype(np.float64))


def byte_places(page_size: int, head_dim: int, which: str) -> torch.Tensor:
    """Byte offset of every (position, element pair) of a head of a page."""
    p_bytes = head_dim // 32
    pos = torch.arange(page_size)[:, None]
    pair = torch.arange(head_dim // 2)[None]
    k, m = pair // 16, pair % 16
    if which == "k":
        return pos * (16 * p_bytes) + m * p_bytes + k
    return pos // 4 * (64 * p_bytes) + m * (4 * p_bytes) + pos % 4 * p_bytes + k


def lay_out(codes: torch.Tensor, which: str) -> torch.Tensor:
    """uint8 codes [pages, heads, page_size, D] -> the cache's bytes."""
    pages, heads, ps, d = codes.shape
    pairs = (codes[..., 0::2] << 4) | codes[..., 1::2]
    out = torch.empty(pages, heads, ps * d // 2, dtype=torch.uint8)
    out[:, :, byte_places(ps, d, which).reshape(-1)] = pairs.reshape(pages, heads, -1)
    return out.reshape(pages, heads, ps, d // 2)


def codes_of(packed: torch.Tensor, which: str) -> torch.Tensor:
    """The inverse of lay_out."""
    pages, heads, ps, half = packed.shape
    b = packed.reshape(pages, heads, -1)[:, :, byte_places(ps, 2 * half, which).reshape(-1)]
    b = b.reshape(pages, heads, ps, half)
    return torch.stack((b >> 4, b & 15), -1).reshape(pages, heads, ps, 2 * half)


@dataclass
class Call:
    """Host copies of what a call takes besides the cache."""
    table: torch.Tensor      # int32 [batch, cols]
    lens: list
    rows: list               # rows of each sequence
    offsets: torch.Tensor    # int32 [batch + 1]
    page: int

    @property
    def total(self):
        return sum(self.rows)

    def places(self):
        """(row, sequence, position, page, index in page) of every row; page -1
        where the row is not in the cache."""
        out, row = [], 0
        for b, n in enumerate(self.rows):
            for i in range(n):
                p = self.lens[b] - n + i
                pg = int(self.table[b, p // self.page]) if p >= 0 else -1
                out.append((row, b, p, pg, p % self.page))
                row += 1
        return out


def make_call(lens, rows, page, seed, spare=2, holes=()):
    """Pages in random order; holes: (sequence, column) entries set to -1."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    for b, c in holes:
        table[b, c] = -1
    off = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
    return Call(table, list(lens), list(rows), off, page), pages


def random_cache(book, pages, heads, page, d, bs, quant_type, seed):
    """(codes, absmax) of keys and of values in natural order."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        codes = torch.randint(0, 16, (pages, heads, page, d), generator=g, dtype=torch.uint8)
        a = torch.rand(pages, heads, page, d // bs, generator=g) * 2 + 0.25
        out.append((codes, a * torch.exp(0.5 * torch.randn(pages, heads, page, 1, generator=g))))
    return out


def dense(book, codes, absmax, bs):
    """c[code] a in 64 bits."""
    return book[codes.long()] * absmax.double().repeat_interleave(bs, -1)


def sequence(call: Call, cache64, b, heads):
    """Keys or values of sequence b [heads, len, D] and which positions exist."""
    n, ps = call.lens[b], call.page
    d = cache64.shape[-1]
    out = torch.zeros(heads, n, d, dtype=torch.float64)
    there = torch.zeros(n, dtype=torch.bool)
    for c in range(-(-n // ps)):
        pg, lo, hi = int(call.table[b, c]), c * ps, min(n, (c + 1) * ps)
        if 0 <= pg < cache64.shape[0]:
            out[:, lo:hi] = cache64[pg, :, :hi - lo]
            there[lo:hi] = True
    return out, there


def attention(call: Call, q, k64, v64, scale, causal, window):
    """out, and per output element what a derived bound needs: sum_p p |v|, and
    per row the largest sum_d |q_d k_d| scale over the positions seen."""
    total, heads, d = q.shape
    kvh = k64.shape[1]
    group = heads // kvh
    out = torch.zeros(total, heads, d, dtype=torch.float64)
    spread = torch.zeros_like(out)
    reach = torch.zeros(total, heads, 1, dtype=torch.float64)
    row = 0
    for b, n in enumerate(call.rows):
        k, there = sequence(call, k64, b, kvh)
        v, _ = sequence(call, v64, b, kvh)
        for i in range(n):
            hi = call.lens[b] - n + i + 1 if causal else call.lens[b]
            lo = max(0, hi - window) if window else 0
            if hi > lo:
                see = there[lo:hi]
                ks, vs = k[:, lo:hi][:, see], v[:, lo:hi][:, see]
                if ks.shape[1]:
                    qr = q[row].double().reshape(kvh, group, d)
                    s = torch.einsum("hgd,htd->hgt", qr, ks) * scale
                    p = torch.softmax(s, -1)
                    out[row] = torch.einsum("hgt,htd->hgd", p, vs).reshape(heads, d)
                    spread[row] = torch.einsum("hgt,htd->hgd", p, vs.abs()).reshape(heads, d)
                    r = torch.einsum("hgd,htd->hgt", qr.abs(), ks.abs()).amax(-1) * abs(scale)
                    reach[row] = r.reshape(heads, 1)
            row += 1
    return out, spread, reach


def sqrt_scale(d):
    return 1.0 / math.sqrt(d)
