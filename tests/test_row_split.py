"""The index arithmetic of the kernels for rows of one batch, checked on the CPU
against Python's integers at sizes whose products pass 32 bits.

The header's host form is compiled with g++ into a small program; the device
form is the same code.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int8_quantized_q8ta_gb300", "csrc")

PROGRAM = r"""
#include <cinttypes>
#include <cstdio>
#include <cstring>
#include "row_split.h"
int main() {
  char what[16];
  while (std::scanf("%15s", what) == 1) {
    long long a, b, c, d;
    if (std::strcmp(what, "items") == 0) {       // first, step, width, how many on
      if (std::scanf("%lld %lld %lld %lld", &a, &b, &c, &d) != 4) return 1;
      q8::RowItems at(static_cast<uint32_t>(a), static_cast<uint32_t>(b), static_cast<uint32_t>(c));
      for (long long i = 0; i < d; ++i) at.next();
      std::printf("%" PRId64 " %u\n", at.row, at.item);
    } else if (std::strcmp(what, "part") == 0) { // part, n, parts
      if (std::scanf("%lld %lld %lld", &a, &b, &c) != 3) return 1;
      std::printf("%d\n", q8::part_start(static_cast<int>(a), static_cast<int>(b),
                                         static_cast<int>(c)));
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def prog(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("row_split")
    src = d / "rs.cpp"
    src.write_text(PROGRAM)
    exe = d / "rs"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src),
                           "-o", str(exe)])

    def run(lines):
        out = subprocess.run([str(exe)], input="\n".join(lines) + "\n", capture_output=True,
                             text=True, check=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]
    return run


def test_items_of_rows(prog):
    """Up to 192 rows of (2^30 / 8) chunks: item numbers beyond 2^32."""
    cases = []
    for width in (8, 24, 512, 1000, 2 ** 22, 2 ** 25 - 8, 2 ** 27):
        for first, step in ((0, 256), (255, 1024), (311295, 311296), (7, width),
                            (1, 2 * width + 3)):
            for n in (0, 1, 5, 1000, 80000):
                cases.append((first, step, width, n))
    assert max((f + n * s) for f, s, _, n in cases) > 2 ** 34
    got = prog([f"items {f} {s} {w} {n}" for f, s, w, n in cases])
    for (f, s, w, n), pair in zip(cases, got, strict=True):
        assert pair == divmod(f + n * s, w), (f, s, w, n)


def test_parts_of_a_line(prog):
    """A unit's k-blocks, up to 2^30 inputs' worth, shared by up to all SMs: the
    product of the two passes 32 bits."""
    cases = [(part, n, parts) for n in (1, 4, 63, 64, 1000, 2 ** 24 - 1, 2 ** 24, 2 ** 31 - 1)
             for parts in (1, 2, 3, 38, 75, 151, 152, 1000) for part in range(0, parts + 1, 1)]
    assert max(part * n for part, n, _ in cases) > 2 ** 31
    got = prog([f"part {part} {n} {parts}" for part, n, parts in cases])
    for (part, n, parts), (at,) in zip(cases, got, strict=True):
        assert at == part * n // parts, (part, n, parts)
