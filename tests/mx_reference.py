"""Microscaled 4-bit matrices in 64 bits, for the tests: quantisation by search over the
code values, the storage of include/nf4_mx.h spelled out. Shares nothing with the library."""
import torch

MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def padded(cols):
    return -(-cols // 128) * 128


def quantize(x):
    """(codes [rows, Kp], scales [rows, Kp / 32]) of x [rows, cols], as integers: one code an
    element, in order."""
    rows, cols = x.shape
    v = torch.zeros(rows, padded(cols), dtype=torch.float64)
    v[:, :cols] = x.double()
    negative = torch.zeros(rows, padded(cols), dtype=torch.bool)
    negative[:, :cols] = torch.signbit(x)
    v, negative = v.view(rows, -1, 32), negative.view(rows, -1, 32)
    bad = ~torch.isfinite(v).all(-1)
    v = torch.where(bad[..., None], 0.0, v)
    top = v.abs().amax(-1)
    # the largest power p in -127 .. 125 with 4 p <= top (floor(log2 top) = log2 p + 2)
    power = torch.full_like(top, 2.0 ** -127)
    for e in range(-126, 126):
        power = torch.where(top >= 4 * 2.0 ** e, 2.0 ** e, power)
    power = torch.where(top == 0, 1.0, power)
    m = v.abs() / power[..., None]  # exact
    code = torch.zeros_like(m, dtype=torch.int64)
    far = m.clone()
    for c, mag in enumerate(MAGNITUDES[1:], 1):
        d = (m - mag).abs()
        take = (d < far) | ((d == far) & (c % 2 == 0))
        code = torch.where(take, c, code)
        far = torch.minimum(far, d)
    code = torch.where(negative & ~bad[..., None], code + 8, code)
    scale = torch.where(bad, 255, torch.log2(power).round().long() + 127)
    return code.view(rows, -1), scale


def values(codes, scales, cols):
    """What codes stand for, in 64 bits: [rows, cols]."""
    book = torch.tensor(MAGNITUDES + [-m for m in MAGNITUDES], dtype=torch.float64)
    power = torch.where(scales == 255, torch.nan, 2.0 ** (scales.double() - 127))
    return (book[codes] * power.repeat_interleave(32, -1))[:, :cols]


def store(codes, scales):
    """The bytes of nf4_mx.h: (uint8 [rows, Kp / 2], uint8 [Kp / 128, rows, 4])."""
    rows = codes.shape[0]
    b = (codes[:, 0::2] * 16 + codes[:, 1::2]).to(torch.uint8)
    s = scales.to(torch.uint8).view(rows, -1, 4).transpose(0, 1).contiguous()
    return b, s


def load(b, s):
    """The inverse of store."""
    b = b.long()
    codes = torch.stack((b // 16, b % 16), -1).flatten(-2)
    return codes, s.long().transpose(0, 1).reshape(b.shape[0], -1)
