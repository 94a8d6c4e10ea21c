"""How the layer norm's rows fall into 16-byte vectors (csrc/rows.cuh), walked over on the host: what the kernels load as
a whole vector lies within the matrix, and every column of a row is in one vector.  No GPU needed."""

import subprocess

import pytest

from moe_grouped_gemm_block_gb300 import build as b

WALK = r"""
#include <cstdio>
#include <cstdlib>
#include "rows.cuh"
using namespace fp8g;

static int faults = 0;
static void fault(const char* what, int64_t M, int N, int64_t ld, int64_t m, int v) {
  if (++faults <= 5) printf("%s: M %lld N %d ld %lld row %lld vector %d\n", what, (long long)M, N, (long long)ld,
                            (long long)m, v);
}

// Every vector that may hold a column of a row.
static void walk(int64_t M, int N, int64_t ld) {
  const int64_t end = (M - 1) * ld + N;
  for (int64_t m = 0; m < M; ++m) {
    const RowShape<true> shape(N, m, ld);
    int columns = 0;
    for (int v = 0; v < shape.vectors(); ++v) {
      const uint32_t mask = shape.mask(v);
      for (int j = 0; j < 8; ++j) columns += mask >> j & 1u;
      const int64_t at = m * ld + shape.col(v);
      if (at % 8 != 0) fault("off the grid", M, N, ld, m, v);
      const bool inside = vector_inside(m, M, ld, N, shape.col(v));
      if ((mask == 0xFFu || inside) && (at < 0 || at + 8 > end)) fault("outside", M, N, ld, m, v);
    }
    if (columns != N) fault("columns", M, N, ld, m, columns);
    if (shape.mask(shape.vectors())) fault("past the row", M, N, ld, m, shape.vectors());
  }
}

int main() {
  for (int64_t M = 1; M <= 20; ++M)
    for (int N = 1; N <= 16; ++N)
      for (int64_t ld = N; ld <= N + 9; ++ld) walk(M, N, ld);
  for (int N : {17, 57, 58, 249, 250, 264, 8185, 16370})
    for (int64_t ld = N; ld <= N + 9; ++ld) walk(9, N, ld);
  printf("faults %d\n", faults);
  return faults != 0;
}
"""


def _host_program(tmp_path, source):
    """Compiles a host program that uses the library's headers, runs it and returns its output."""
    src, exe = tmp_path / "walk.cu", tmp_path / "walk"
    src.write_text(source)
    subprocess.run([b._nvcc(), *b.ARCH, "-std=c++17", "-I", b.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    return r.stdout


def test_vectors_stay_within_the_matrix(tmp_path):
    assert _host_program(tmp_path, WALK).strip() == "faults 0"
