"""Products of microscaled matrices by the tiled kernel, in each of its forms: tiles of 256 and of
128, stages of 256 columns that are loaded again and again, last stages of one 128-wide step and of
two, ranges of K whose last one is shorter. Which form a size takes is read from the library's log.
Tolerances are test_gpu_mx.py's; 64-bit results are formed for some of the rows."""
import os
import re
import subprocess
import sys

import pytest
import torch

from test_gpu_mx import DTYPES, check_product, dense, nf4, rows_of, weight_of  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# M, N, K: side of the tiles, ranges of K, 128-wide steps of a range (of all: the last may be shorter)
TILES = {
    (3000, 3100, 2000): (256, 1, 16),
    (3000, 3100, 1900): (256, 1, 15),
    (4000, 7900, 1200): (256, 1, 10),  # more tiles than CUs
    (3900, 4050, 300): (256, 1, 3),
    (700, 1537, 640): (128, 1, 5),
    (333, 2801, 1003): (128, 1, 8),
    (1000, 1000, 2100): (128, 1, 17),
    (130, 300, 8300): (128, 17, 4),    # 65 steps: a last range of one
    (200, 300, 9000): (128, 12, 6),    # 71: of five
    (300, 260, 12000): (128, 16, 6),   # 94: of four
}
ONE_OF_EACH = [(3000, 3100, 1900), (700, 1537, 640), (200, 300, 9000)]

CHILD = """
import torch
import bit_weight_quantization_nf4_amd as nf4
for m, n, k in %r:
    nf4.mx_linear(nf4.MXTensor.empty(m, k), nf4.MXTensor.empty(n, k))
torch.cuda.synchronize()
"""


@pytest.fixture(autouse=True)
def cus():
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("another number of CUs: other forms")


def test_which_form_a_size_takes():
    env = dict(os.environ, NF4_LOG="1", PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", CHILD % list(TILES)], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    found = re.findall(r"mx product M=(\d+) N=(\d+) K=(\d+): mx_gemm_kernel, tiles of (\d+), (\d+) range\(s\) "
                       r"of (\d+) steps", r.stderr)
    found = [tuple(map(int, f)) for f in found]
    assert {f[:3]: f[3:] for f in found} == TILES


def some_rows(m):
    return torch.tensor(sorted({*range(0, min(m, 40)), *range(m // 2, min(m, m // 2 + 40)), *range(max(0, m - 40), m),
                                *range(0, m, 97)}))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", TILES)
def test_product(nf4, m, n, k, dtype):  # noqa: F811
    """Rows and columns that end inside a tile; a bias; outputs of any alignment, which keep what
    is beside them; the same bits when x is quantized in the call, and again."""
    w = weight_of(nf4, n, k, n + k)
    x = rows_of(m, k, dtype, m + k, 0.5).cuda()
    q = nf4.mx_quantize(x)
    bias = rows_of(1, n, dtype, 5)[0]
    room = torch.full((m + 2, n + 9), 9.0, dtype=dtype, device="cuda")
    y = nf4.mx_linear(q, w, bias.cuda(), out=room[1:-1, 5:n + 5])
    rows = some_rows(m)
    check_product(y.cpu()[rows], dense(q)[rows], dense(w), bias, k, (m, n, k))
    for _ in range(2):
        assert torch.equal(nf4.mx_linear(x, w, bias.cuda()), y)
    room[1:-1, 5:n + 5] = 9.0
    assert bool((room == 9.0).all())


@pytest.mark.parametrize("m,n,k", ONE_OF_EACH)
def test_blocks_that_are_not_finite_spoil_their_row_or_column_only(nf4, m, n, k):  # noqa: F811
    wd, x = rows_of(n, k, torch.float32, 1), rows_of(m, k, torch.float32, 2)
    clean = nf4.mx_linear(x.cuda(), nf4.mx_quantize(wd.cuda()))
    assert bool(torch.isfinite(clean).all())
    columns, rows = [0, n // 3, n - 1], [1, m // 2, m - 1]
    for c, at in zip(columns, (0, k // 2, k - 1)):
        wd[c, at] = torch.nan if at else torch.inf
    for r, at in zip(rows, (k - 1, 17, 300)):
        x[r, at] = -torch.inf if at == 17 else torch.nan
    y = nf4.mx_linear(x.cuda(), nf4.mx_quantize(wd.cuda()))
    lost = torch.zeros(m, n, dtype=torch.bool)
    lost[rows], lost[:, columns] = True, True
    assert torch.equal(y.isnan().cpu(), lost)
    assert torch.equal(y.cpu()[~lost], clean.cpu()[~lost])


@pytest.mark.parametrize("m,n,k", ONE_OF_EACH)
def test_large_and_small_scales(nf4, m, n, k):  # noqa: F811
    """Scales whose product passes fp32's range or falls below it, rows of unequal size."""
    rows = some_rows(m)
    for ex, ew in ((100, -100), (-100, 100), (60, 60), (-60, -60)):
        x = (rows_of(m, k, torch.float32, 5) * 2.0 ** ex).cuda()
        w = nf4.mx_quantize((rows_of(n, k, torch.float32, 6) * 2.0 ** ew).cuda())
        q = nf4.mx_quantize(x)
        fits = check_product(nf4.mx_linear(x, w).cpu()[rows], dense(q)[rows], dense(w), None, k, (ex, ew))
        assert bool(fits.all()) or (ex, ew) == (60, 60)
        assert bool(fits.any())


@pytest.mark.parametrize("m,n,k", TILES)
def test_what_lies_behind_a_matrix_has_no_part(nf4, m, n, k):  # noqa: F811
    """Matrices at the end of a buffer, with codes and NaN scales of no concern behind them."""
    x, w = nf4.mx_quantize(rows_of(m, k, torch.float32, 1).cuda()), weight_of(nf4, n, k, 2)
    want = nf4.mx_linear(x, w)

    def surrounded(t):
        out = []
        for a, fill in ((t.codes, 0x77), (t.scales, 255)):
            room = torch.full((a.numel() + 8192,), fill, dtype=torch.uint8, device="cuda")
            out.append(room[4096:4096 + a.numel()].view(a.shape).copy_(a))
        return nf4.MXTensor(*out, t.shape)

    assert bool(torch.isfinite(want).all())
    assert torch.equal(nf4.mx_linear(surrounded(x), surrounded(w)), want)


def test_streams_and_graphs(nf4):  # noqa: F811
    """Each form on streams of their own at once, and captured, replayed on other inputs beside
    eager work."""
    ws = [weight_of(nf4, n, k, n) for _, n, k in ONE_OF_EACH]
    xs = [[rows_of(m, k, torch.bfloat16, s).cuda() for m, _, k in ONE_OF_EACH] for s in (1, 2)]

    def step(x):
        return [nf4.mx_linear(a, w) for a, w in zip(x, ws)]

    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s, x in zip(streams, xs):
        with torch.cuda.stream(s):
            outs.append(step(x))
    torch.cuda.synchronize()
    for out, y in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, y))
    held = [x.clone() for x in xs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(held)
    for x, y in zip(xs * 2, want * 2):
        for a, b in zip(held, x):
            a.copy_(b)
        graph.replay()
        again = step(x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, y))
        assert all(torch.equal(a, b) for a, b in zip(again, y))
