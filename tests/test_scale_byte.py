"""The weights' scale bytes of the 8-bit attention, on the host, by a compiler that reports undefined
arithmetic: exponents of any size, with none (a block that a row does not see) and NaN among them."""
import os
import subprocess

from verify_gated_gqa_gb300 import build as build_mod

PROGRAM = r"""
#include <cmath>
#include <cstdio>
#include "ga_v8.cuh"
int main() {
  const float none[] = {ga::kNone, ga::kNone - 8.f, -INFINITY, -3e38f, -2147483904.f, -2147483648.f, -700.f, NAN};
  for (int v = ga::kQ8MinExp; v <= ga::kQ8MaxExp; ++v) {
    for (float x : none)
      if (ga::scale_byte(x, v) != 0u) return std::printf("%g %d\n", x, v), 1;
    // a block's weights are at most 2^64 past the reference
    for (int x = -300; x <= 56; ++x) {
      const int want = x + v + 127 < 0 ? 0 : x + v + 127;
      if (want > 254 || ga::scale_byte((float)x, v) != (unsigned)want) return std::printf("%d %d\n", x, v), 1;
    }
  }
  return std::puts("right"), 0;
}
"""


def test_scale_bytes_without_undefined_arithmetic(tmp_path):
    src, exe = tmp_path / "main.cu", tmp_path / "main"
    src.write_text(PROGRAM)
    subprocess.run([build_mod._nvcc(), *build_mod.ARCH, "-std=c++17", "-I", build_mod.CSRC, "-I",
                    os.path.join(build_mod.ROOT, "include"), "-Xcompiler",
                    "-fsanitize=undefined,-fsanitize=float-cast-overflow,-fno-sanitize-recover=all", "-o", exe, src],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert (r.returncode, r.stdout.strip(), r.stderr) == (0, "right", "")
