"""The element-to-row arithmetic of the compaction's copies (csrc/row_of.cuh), run
on the host for every row size that dsa_evict_compact takes."""
import ctypes
import os
import shutil
import subprocess

import pytest

from sparse_indexed_attention_b200 import build

CHECK = r"""
#include "row_of.cuh"
// Elements of `rows` rows of nv whose row or column is wrong: all of them, or the
// first and the last ones of each row (the quotient is monotone in i, so an element
// between two right ones of a row is right).
extern "C" int64_t wrong(uint32_t nv, uint32_t rows, int all) {
  const dsa::RowDivisor by = dsa::row_divisor(nv);
  const uint32_t edge = 4;
  int64_t bad = 0;
  for (uint32_t r = 0; r < rows; ++r)
    for (uint32_t c = 0; c < nv; ++c) {
      if (!all && c == edge && nv > 2 * edge) c = nv - edge;
      const dsa::RowColumn x = dsa::row_of(r * nv + c, by);
      bad += x.row != r || x.column != c;
    }
  return bad;
}
"""
ROWS = 32                                          # rows of a block


@pytest.fixture(scope="module")
def wrong(tmp_path_factory):
    d = tmp_path_factory.mktemp("row_of")
    src, lib = d / "check.cpp", d / "check.so"
    src.write_text(CHECK)
    cxx = os.environ.get("CXX") or shutil.which("g++")
    subprocess.run([cxx, "-O2", "-shared", "-fPIC", "-std=c++17", "-I", build.CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).wrong
    f.restype, f.argtypes = ctypes.c_int64, [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_int]
    return f


def _elements(row_bytes):
    return row_bytes // (16 if row_bytes % 16 == 0 else 8 if row_bytes % 8 == 0 else 4)


def test_every_row_size(wrong):
    bad = [n for n in range(4, 65537, 4) if wrong(_elements(n), ROWS, 0)]
    assert not bad, f"{len(bad)} sizes, {bad[:3]} .. {bad[-1]}"


@pytest.mark.parametrize("row_bytes", [4, 8, 12, 1152, 46508, 65528, 65532, 65536])
def test_every_element(wrong, row_bytes):
    assert wrong(_elements(row_bytes), ROWS, 1) == 0


@pytest.mark.parametrize("nv", [73, 577, 1000, 4096, 16383, 16384, 2 ** 20 - 1])
def test_every_element_number(wrong, nv):
    """Up to 2^33 / nv, where the argument of the divisor ends."""
    assert wrong(nv, max(1, min(2 ** 32 - 1, 2 ** 33 // nv) // nv), 0) == 0
