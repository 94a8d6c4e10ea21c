// rows.cuh -- how the rows of a matrix fall into vectors of 8 values on the 16-byte grid, for host and device (the host
// tests walk over every vector that a kernel may touch).
#pragma once

#include <algorithm>
#include <cstdint>

namespace fp8g {

// How a row falls into vectors of 8.  Where every row starts on the grid of its matrix's 8-value groups (SHIFT
// false), vector v holds columns 8 v .. 8 v + 7.  Else row m starts q = (m ld) mod 8 values after a group's start and
// vector v holds columns 8 v - q ..: its first and last vectors reach into the neighbouring rows, whose values are
// left out.  q repeats every 8 rows, so a thread that steps by multiples of 8 rows keeps its columns, and with
// them its weights and its sums of the weight gradients.  Every matrix of a call has the same q (the host checks).
template <bool SHIFT>
struct RowShape {
  int N, q;
  __host__ __device__ __forceinline__ RowShape(int n, int64_t m, int64_t ld)
      : N(n), q(SHIFT ? static_cast<int>((m & 7) * (ld & 7)) & 7 : 0) {}
  __host__ __device__ __forceinline__ int vectors() const { return (N + q + 7) >> 3; }
  __host__ __device__ __forceinline__ int col(int v) const { return 8 * v - q; }
  // The columns of vector v that exist, a bit each.
  __host__ __device__ __forceinline__ uint32_t mask(int v) const {
    const int c = col(v);
    if (!SHIFT) return c < N ? 0xFFu : 0u;
    uint32_t k = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) k |= (c + j >= 0 && c + j < N ? 1u : 0u) << j;
    return k;
  }
};

// Whether the 8 values from column c of row m on end within the matrix, neighbouring rows included.  (A row after this one
// is not enough: where ld < 7 a vector reaches over several rows.)
__host__ __device__ __forceinline__ bool vector_inside(int64_t m, int64_t M, int64_t ld, int N, int c) {
  return m * ld + c + 8 <= (M - 1) * ld + N;
}

// This CTA's share of every row: the vectors first .. first + count - 1 of the row's.
struct Share {
  int first, count;
  template <bool SHIFT>
  __host__ __device__ __forceinline__ Share(const RowShape<SHIFT>& shape, int rank, int ranks) {
    const int all = shape.vectors(), each = (all + ranks - 1) / ranks;
    first = rank * each;
    count = min(each, all - first);
  }
};

// The vectors of the share that a stage's copy holds: a last row's last vector may reach past the matrix, and is left
// out (the threads that need it read its values themselves).
template <bool SHIFT>
__host__ __device__ __forceinline__ int copied(const RowShape<SHIFT>& shape, const Share& sh, bool last_row) {
  const bool past = SHIFT && last_row && (shape.N + shape.q) % 8 != 0 && sh.first + sh.count == shape.vectors();
  return sh.count - (past ? 1 : 0);
}
// The vectors of a share that are whole in every row; off the grid its first and last one may not be.
template <bool SHIFT>
struct Inner {
  int lo, hi;
  __host__ __device__ __forceinline__ Inner(const Share& sh) : lo(SHIFT ? 1 : 0), hi(sh.count - (SHIFT ? 1 : 0)) {}
  // How many of them a warp sees at once: a short row off the grid has fewer than 32 (a ring's at least 30).
  __host__ __device__ __forceinline__ int heads() const { return SHIFT && hi - lo < 32 ? hi - lo : 32; }
};

}  // namespace fp8g
