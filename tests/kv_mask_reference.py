"""The masks of include/nf4_kv_mask.h row by row, and attention under any mask in 64 bits,
for the tests. Shares nothing with the library."""
import torch

import kv_reference as ref


def tree_words(masks, words, total):
    """int32 [total, words] of a list of sets: masks[t] are the rows that row t sees."""
    out = torch.zeros(total, words, dtype=torch.int64)
    for t, seen in enumerate(masks):
        for j in seen:
            out[t, j // 32] |= 1 << (j % 32)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def visible(call, window=0, sinks=0, masks=None, words=1 << 20):
    """Of every row of the call, the set of positions that it sees by the mask."""
    out, t = [], 0
    for b, n in enumerate(call.rows):
        base = call.lens[b] - n
        for i in range(n):
            if masks is None:
                place, last = base + i, base + i + 1
                mine = []
            else:
                mine = [j for j in masks[t] if j < n and j < 32 * words]
                place, last = base + len(mine) - 1, base
            see = {p for p in range(0, min(last, place + 1))
                   if not window or p > place - window or p < sinks}
            see |= {base + j for j in mine if base + j >= 0}
            out.append(see)
            t += 1
    return out


def attention(call, q, k64, v64, scale, see):
    """As kv_reference.attention, of the positions in `see` that are in the cache."""
    total, heads, d = q.shape
    kvh = k64.shape[1]
    group = heads // kvh
    out = torch.zeros(total, heads, d, dtype=torch.float64)
    spread = torch.zeros_like(out)
    reach = torch.zeros(total, heads, 1, dtype=torch.float64)
    row = 0
    for b, n in enumerate(call.rows):
        k, there = ref.sequence(call, k64, b, kvh)
        v, _ = ref.sequence(call, v64, b, kvh)
        for _ in range(n):
            p = torch.tensor(sorted(see[row]), dtype=torch.long)
            p = p[there[p]]
            if len(p):
                qr = q[row].double().reshape(kvh, group, d)
                ks, vs = k[:, p], v[:, p]
                w = torch.softmax(torch.einsum("hgd,htd->hgt", qr, ks) * scale, -1)
                out[row] = torch.einsum("hgt,htd->hgd", w, vs).reshape(heads, d)
                spread[row] = torch.einsum("hgt,htd->hgd", w, vs.abs()).reshape(heads, d)
                r = torch.einsum("hgd,htd->hgt", qr.abs(), ks.abs()).amax(-1) * abs(scale)
                reach[row] = r.reshape(heads, 1)
            row += 1
    return out, spread, reach


def random_trees(rows, seed, chain=0.4):
    """Masks of random trees, a list of sets over all rows of the call: each row sees
    itself and its ancestors up to its sequence's first row."""
    g = torch.Generator().manual_seed(seed)
    masks = []
    for n in rows:
        first = len(masks)
        for i in range(n):
            u, w = torch.rand(2, generator=g).tolist()
            parent = i - 1 if u < chain else int(w * i)
            masks.append({i} | (masks[first + parent] if i else set()))
    return masks
