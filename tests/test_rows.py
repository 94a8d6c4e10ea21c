"""How the layer norm's rows fall into 16-byte vectors (csrc/rows.cuh), walked over on the host: what the kernels load as
a whole vector lies within the matrix, every column of a row is in one vector, and what a ring's sum warps take as a
row's own whole vectors is that.  No GPU needed."""

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

// A ring's copies and the vectors that its sum warps take as whole ones, for every row and each CTA of a cluster.
template <bool SHIFT>
static void walk_ring(int64_t M, int N, int64_t ld, int ranks) {
  for (int64_t m = 0; m < M; ++m) {
    const RowShape<SHIFT> shape(N, m, ld);
    int taken = 0;
    for (int rank = 0; rank < ranks; ++rank) {
      const Share sh(shape, rank, ranks);
      const int n = copied(shape, sh, m + 1 == M);
      const int64_t at = m * ld + shape.col(sh.first);
      if (n && (at < 0 || at + 8 * n > (M - 1) * ld + N)) fault("copied from outside", M, N, ld, m, rank);
      const Inner<SHIFT> in(sh);
      if (in.heads() < 30 || in.heads() > 32) fault("heads", M, N, ld, m, in.heads());
      for (int v = in.lo; v < in.hi; ++v)
        if (shape.mask(sh.first + v) != 0xFFu || v >= n) fault("not whole", M, N, ld, m, v);
      if (in.lo + in.heads() > in.hi) fault("heads past the whole vectors", M, N, ld, m, in.heads());
      taken += sh.count;
    }
    if (taken != shape.vectors()) fault("shares", M, N, ld, m, taken);
  }
}

int main() {
  for (int64_t M = 1; M <= 20; ++M)
    for (int N = 1; N <= 16; ++N)
      for (int64_t ld = N; ld <= N + 9; ++ld) walk(M, N, ld);
  for (int N : {17, 57, 58, 249, 250, 264, 8185, 16370})
    for (int64_t ld = N; ld <= N + 9; ++ld) walk(9, N, ld);
  for (int N = 250; N <= 300; ++N)  // the shortest rows that the ring takes off the grid
    for (int64_t ld = N; ld <= N + 9; ++ld)
      for (int64_t M : {1, 2, 9, 20}) walk_ring<true>(M, N, ld, 1);
  for (int N : {520, 8184, 8192}) walk_ring<false>(9, N, N, 1);
  for (int N = 8180; N <= 8200; ++N) walk_ring<true>(9, N, N, N <= 8185 ? 1 : 2);
  for (int N = 16360; N <= 16377; ++N) walk_ring<true>(9, N, N + 1, 2);
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
