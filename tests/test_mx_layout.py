"""The layout in LDS of rows that a workgroup of the few rows' product quantizes itself, from the
kernel's own source: every 16-byte read of it is at a multiple of 16, and all rows have room."""
import os
import shutil
import subprocess

import pytest

from bit_weight_quantization_nf4_amd import build

SOURCE = r"""
#include "mx_gemv.hip"

namespace nf4 {
namespace {

constexpr bool aligned_rows() {
  for (int64_t padded = kMxStep; padded <= kRawElements; padded += kMxStep)
    if (raw_row_bytes(padded) % 16 != 0) return false;
  return true;
}
constexpr bool whole_rows() {  // codes, and a scale for each block behind them and a gap of 16
  for (int64_t padded = kMxStep; padded <= kRawElements; padded += kMxStep)
    if (raw_row_bytes(padded) < padded / 2 + 16 + padded / kMxBlock) return false;
  return true;
}
constexpr bool room() {
  for (int64_t padded = kMxStep; padded <= kRawElements; padded += kMxStep)
    for (int64_t rows = 1; rows <= 16 && rows * padded <= kRawElements; ++rows)
      if (rows * raw_row_bytes(padded) > kRawBytes) return false;
  return true;
}
static_assert(aligned_rows(), "rows 16 bytes aligned");
static_assert(whole_rows(), "rows that do not overlap");
static_assert(room(), "room for all rows");

}  // namespace
}  // namespace nf4
"""


def test_rows_quantized_in_lds(tmp_path):
    if shutil.which(build.HIPCC) is None:
        pytest.skip("no hipcc")
    src = tmp_path / "layout.hip"
    src.write_text(SOURCE)
    r = subprocess.run([build.HIPCC, *build.CXXFLAGS, "-fconstexpr-steps=10000000", f"-I{build.CSRC}", "--cuda-host-only", "-fsyntax-only",
                        str(src)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
