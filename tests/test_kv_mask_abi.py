"""The C ABI of the masked attention without a GPU: exports, refusals before any device work,
and the tests' own mask reference."""
import os
import re

import pytest
import torch

import kv_mask_reference as mref
import kv_reference as ref
from test_kv_abi import A, B, C, DEVICE, INVALID, MISALIGNED, OK, cache, kv, rows  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def call(kv, c=None, r=None, dtype=0, window=0, sinks=0, tree=None, stride=0, words=0, max_rows=2,  # noqa: F811
         scale=0.1, ws=C, size=1 << 30, q=A, out=B):
    return kv._lib().nf4_kv_attention_masked(
        c or cache(kv), r or rows(kv), q, 512, 128, 4, dtype, scale, window, sinks, tree, stride, words,
        max_rows, 48, out, 512, 128, ws, size, None)


def test_exports_every_declared_symbol(kv):  # noqa: F811
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "nf4_kv_mask.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(nf4_kv_[a-z0-9_]+)\s*\(", text)))
    assert sorted(kv.kv_mask_exported_names()) == declared and len(declared) == 2
    for name in declared:
        assert getattr(kv._lib(), name)


def test_refusals(kv):  # noqa: F811
    for over in (dict(sinks=-1), dict(window=-1), dict(dtype=9), dict(scale=float("nan")), dict(q=None),
                 dict(out=None), dict(max_rows=-1), dict(ws=None), dict(size=-1),
                 dict(tree=A, stride=1, words=2), dict(tree=A, stride=1, words=-1),
                 dict(tree=A, stride=1 << 61, words=1)):
        assert call(kv, **over) == INVALID, over
    assert call(kv, tree=A + 2, stride=1, words=1) == MISALIGNED
    assert call(kv, ws=C + 8) == MISALIGNED
    assert kv._lib().nf4_kv_attention_masked(None, rows(kv), A, 512, 128, 4, 0, 0.1, 0, 0, None, 0, 0, 2, 48,
                                             B, 512, 128, C, 1 << 30, None) == INVALID
    assert call(kv, r=rows(kv, batch=0, total_rows=0)) == OK
    if not torch.cuda.is_available():
        assert call(kv) == DEVICE and call(kv, tree=A, stride=3, words=2, window=5, sinks=9) == DEVICE


def test_workspace_query(kv):  # noqa: F811
    sizes = (4, 6, 8000, 32, 8, 128)
    for window in (1000, 6000):  # positions in one range; in several
        plain = kv.kv_attention_workspace_bytes(*sizes, window=window)
        assert kv.kv_attention_workspace_bytes(*sizes, window=window, sinks=1) >= plain
        assert (plain > 0) == (window == 6000)
    L = kv._lib()
    assert L.nf4_kv_attention_masked_workspace_bytes(*sizes, 0, 1000, -1) == -1
    assert L.nf4_kv_attention_masked_workspace_bytes(*sizes, 0, -1, 1) == -1
    assert L.nf4_kv_attention_masked_workspace_bytes(*sizes, 0, 2 ** 31 - 1, 2 ** 31 - 1) >= 0
    assert kv.kv_attention_workspace_bytes(*sizes, window=1 << 40, sinks=1 << 40) >= 0


def test_reference_masks():
    c, _ = ref.make_call([6, 4], [3, 2], 16, 1)
    assert mref.visible(c) == [set(range(4)), set(range(5)), set(range(6)), {0, 1, 2}, {0, 1, 2, 3}]
    assert mref.visible(c, 2, 1) == [{0, 2, 3}, {0, 3, 4}, {0, 4, 5}, {0, 1, 2}, {0, 2, 3}]
    masks = [{0}, {0, 1}, {0, 2}, {0}, {1}]
    assert mref.visible(c, masks=masks) == [{0, 1, 2, 3}, {0, 1, 2, 3, 4}, {0, 1, 2, 3, 5}, {0, 1, 2}, {0, 1, 3}]
    # places 3, 4, 4 and 2, 2
    assert mref.visible(c, 2, 1, masks) == [{0, 2, 3}, {0, 3, 4}, {0, 3, 5}, {0, 1, 2}, {0, 1, 3}]
    w = mref.tree_words([{0, 31}, {32, 33}], 2, 2)
    assert w.tolist() == [[1 - (1 << 31), 0], [0, 3]]


@pytest.mark.parametrize("chain", [0.0, 0.4, 1.0])
def test_reference_trees(chain):
    for rows_of in ([5], [40, 1, 33]):
        masks, first = mref.random_trees(rows_of, 2, chain), 0
        for n in rows_of:
            for i, m in enumerate(masks[first:first + n]):
                assert i in m and 0 in m and max(m) == i
                assert all(masks[first + j] <= m for j in m)
            first += n
