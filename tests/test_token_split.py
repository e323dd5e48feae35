"""Which lanes write which of a row's items in the quantizer, checked on the CPU
for every length up to some 4,200 and every place of a row's first value: each
int8 value and each of the operand's items exactly once.

csrc/token_split.h is compiled with g++; the loops around it are the kernel's.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int8_quantized_q8ta_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "token_split.h"

// The first value or item of a row that is not written exactly once, or -1.
template <bool VEC, bool OP>
int wrong(int K, int t, int warps, int U) {
  using L = q8::RowLanes<VEC, OP>;
  const int chunks = (K + 63) / 64 * 8, items = L::items(K, chunks), step = L::step(warps);
  std::vector<int> q(K, 0), op(OP ? chunks : 0, 0);
  for (int warp = 0; warp < warps; ++warp)
    for (int lane = 0; lane < 32; ++lane) {
      const auto put = [&](int c) {
        if (!L::stores(lane)) return;
        for (int j = 0; j < 8; ++j) {
          const int k = c * 8 - t + j;
          if (k >= 0 && k < K) ++q[k];
        }
        if (OP && c < chunks) ++op[c];
      };
      const int c0 = L::first(warp, lane);
      for (int u = 0; u < U; ++u)
        if (c0 + u * step - lane < items) put(c0 + u * step);
      for (int c = c0 + U * step; c - lane < items; c += step) put(c);
    }
  for (int k = 0; k < K; ++k)
    if (q[k] != 1) return k;
  for (int c = 0; c < static_cast<int>(op.size()); ++c)
    if (op[c] != 1) return c;
  return -1;
}

int bad = 0;
void check(int at, bool vec, bool op, int K, int t, int warps, int U) {
  if (at >= 0 && bad++ < 10)
    std::printf("vec %d op %d K %d t %d warps %d U %d: %d\n", vec, op, K, t, warps, U, at);
}

int main() {
  for (int K = 1; K <= 4200; ++K)
    for (int U : {2, 4})
      for (int t = 0; t < 8; ++t) {
        // one warp a row, as many as hold all items, and what a CTA has at most
        const int fit = (K / 8 + 10 + 30) / 31;
        for (int warps : {1, 2, (fit + U - 1) / U, fit < 22 ? fit : 22, 22}) {
          check(wrong<false, true>(K, t, warps, U), 0, 1, K, t, warps, U);
          check(wrong<false, false>(K, t, warps, U), 0, 0, K, t, warps, U);
          if (t == 0 && K % 8 == 0) {
            check(wrong<true, true>(K, t, warps, U), 1, 1, K, t, warps, U);
            check(wrong<true, false>(K, t, warps, U), 1, 0, K, t, warps, U);
          }
        }
      }
  std::printf("%d\n", bad);
  return 0;
}
"""


def test_every_value_and_item_is_written_once(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "ts.cpp", tmp_path / "ts"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert out.splitlines() == ["0"], out
