"""Rows of any width and alignment (csrc/tt_rows.h) on the host, with loads and stores checked against the alignment
that their types declare: groups of eight are read and written from every place that a row of every width has
them, for every type."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "tensor_train_compressed_ttembeddingbag_amd", "csrc")
# what of the HIP headers the file uses
HIP = """#pragma once
#include <algorithm>
#define __device__
#define __forceinline__ inline
using std::min;
"""
MAIN = """#include "tt_rows.h"
#include <stdio.h>
#include <string.h>
using namespace ttb;
template <class T, bool NARROW>
int rows(long d, int offset) {
  alignas(64) static T from[64], to[64];
  for (int i = 0; i < 64; ++i) from[i] = (T)(i + 1), to[i] = (T)0;
  for (long g = 0; g < (d + 7) / 8; ++g) {
    const long c = column<NARROW>(g, d);
    put8<NARROW>(to + offset + c, get8<NARROW>(from + offset + c, d), d);
  }
  for (int i = 0; i < 64; ++i)
    if (to[i] != (i >= offset && i < offset + d ? from[i] : (T)0)) return 1;
  return 0;
}
template <class T>
int all() {
  int bad = 0;
  for (int offset = 0; offset < 9; ++offset) {
    for (long d = 1; d < 8; ++d) bad += rows<T, true>(d, offset);
    for (long d = 8; d < 40; ++d) bad += rows<T, false>(d, offset);
  }
  return bad;
}
int main() { return all<signed char>() + all<_Float16>() + all<float>(); }
"""


@pytest.mark.parametrize("planted", [False, True])
def test_rows(tmp_path, planted):
    """planted: a copy of the file that declares too much must fail, or nothing was checked."""
    clang = next((c for c in ("/opt/rocm/llvm/bin/clang++", shutil.which("clang++")) if c and os.path.exists(c)), None)
    if clang is None:
        pytest.skip("clang++ not available")
    (tmp_path / "hip").mkdir()
    (tmp_path / "hip" / "hip_runtime.h").write_text(HIP)
    text = open(os.path.join(CSRC, "tt_rows.h")).read()
    if planted:
        assert "aligned(sizeof(T) < 2 ? 1 : 2)" in text
        text = text.replace("aligned(sizeof(T) < 2 ? 1 : 2)", "aligned(2)")
    (tmp_path / "tt_rows.h").write_text(text)
    (tmp_path / "main.cpp").write_text(MAIN)
    subprocess.check_call([clang, "-std=c++17", "-O1", "-fsanitize=alignment", "-fsanitize-trap=alignment",
                           "-I", str(tmp_path), str(tmp_path / "main.cpp"), "-o", str(tmp_path / "main")])
    code = subprocess.run([str(tmp_path / "main")]).returncode
    assert code < 0 if planted else code == 0
