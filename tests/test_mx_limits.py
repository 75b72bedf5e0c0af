"""Microscaled products of so many features that a workgroup for each 16 of them passes what a
launch can hold: other kernels take them, and what fits none is refused before any launch."""
import pytest
import torch

import bit_weight_quantization_nf4_amd as nf4
import mx_reference as ref
from test_mx_abi import B, C, D, DEVICE, UNSUPPORTED, linear, matmul, matrix, mx  # noqa: F401

# workgroups of 512 threads for 16 features (few rows), and for 64
FIRST_16, FIRST_64 = 1 << 27, 1 << 29


def test_workspaces_past_a_launch(mx):  # noqa: F811
    quantized = 128 * 17 // 32  # bytes of a row of x
    for m in (1, 3, 16):
        assert mx.mx_workspace_bytes(m, FIRST_16 - 16, 128) == 0  # x is quantized in the kernel
        assert mx.mx_workspace_bytes(m, FIRST_16, 128) >= m * quantized
        assert mx.mx_workspace_bytes(m, FIRST_16, 128, True) == 0
    for m in (17, 40, 64):
        for n in (FIRST_16, FIRST_64):
            assert mx.mx_workspace_bytes(m, n, 128) >= m * quantized
    # 256 x 256 tiles of 512 threads, 128 x 128 ones of 256
    for m, n in ((1, (1 << 31) - 1), (64, (1 << 31) - 256 + 1), (129, 1 << 30)):
        assert mx.mx_workspace_bytes(m, n, 128) == -1 and mx.mx_workspace_bytes(m, n, 128, True) == -1
    assert mx.mx_workspace_bytes(64, (1 << 31) - 256, 128) >= 64 * quantized


def test_refused_before_a_launch(mx):  # noqa: F811
    w = matrix(mx, rows=(1 << 31) - 1)
    assert linear(mx, m=1, w=w, ldy=1 << 31) == UNSUPPORTED
    assert matmul(mx, x=matrix(mx, rows=1), w=w, ldy=1 << 31) == UNSUPPORTED
    if not torch.cuda.is_available():
        w = matrix(mx, rows=FIRST_16)
        assert linear(mx, m=1, w=w, ldy=FIRST_16) == DEVICE
        assert matmul(mx, x=matrix(mx, rows=1), w=w, ldy=FIRST_16) == DEVICE


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 5])
def test_a_weight_of_more_rows_than_a_launch_has_workgroups(m):
    """2^27 + 40 rows of 128 elements, 9 GB, against 64 bits at its ends and in its middle. All
    scales are 1 and sums of 128 products multiples of 1/4 below 2^13: fp32 sums are exact."""
    n, k = FIRST_16 + 40, 128
    g = torch.Generator(device="cuda").manual_seed(m)
    codes = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    for part in codes.split(1 << 24):
        part.random_(0, 256, generator=g)
    w = nf4.MXTensor(codes, torch.full((1, n, 4), 127, dtype=torch.uint8, device="cuda"), (n, k))
    x = torch.randint(-6, 7, (m, k), generator=g, device="cuda").float()
    x[:, ::32] = 6.0  # blocks of scale 1
    q = nf4.mx_quantize(x)
    assert bool((q.scales == 127).all())
    y = nf4.mx_linear(x, w)
    assert torch.equal(nf4.mx_linear(q, w, out_dtype=torch.float32), y)
    x64 = ref.values(*ref.load(q.codes.cpu(), q.scales.cpu()), k)
    for lo in (0, n // 2 - 777, FIRST_16 - 500, n - 1000):
        part = ref.load(codes[lo:lo + 1000].cpu(), w.scales[:, lo:lo + 1000].cpu())
        want = x64 @ ref.values(*part, k).T
        assert torch.equal(y[:, lo:lo + 1000].cpu().double(), want), lo
