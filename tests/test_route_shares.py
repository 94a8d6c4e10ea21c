"""How a CTA's warps share the rows that the router leaves for its end (csrc/shares.cuh), walked over on the host: a warp that
has a row adds up the sums of warps that there are, those of its row and no others; what is left over has none.  No GPU
needed."""

from tests.test_rows import _host_program

WALK = r"""
#include <cstdio>
#include "shares.cuh"
using namespace fp8g;

int main() {
  int faults = 0, left = 0;
  for (int warps = 1; warps <= 32; ++warps)
    for (int E = 1; E <= 2048; ++E) {
      int columns = 0, rows = 0;
      for (int w = 0; w < warps; ++w) {
        const RowShares s(E, warps, w);
        if (!s.some()) {
          ++left;
          continue;
        }
        for (int i = 0; i < s.parts; ++i) {
          const int from = s.first() + i;
          if (from < 0 || from >= warps || RowShares(E, warps, from).slot != s.slot) ++faults;
        }
        if (w != s.first() + s.part) ++faults;
        if (s.part == 0) ++rows;
        if (s.slot == 0) columns += (E - 32 * s.part + 32 * s.parts - 1) / (32 * s.parts) > 0;
      }
      const RowShares s(E, warps, 0);
      if (rows != s.at_once || columns != s.parts || s.at_once < 1) ++faults;
    }
  printf("faults %d left %d\n", faults, left);
  return faults != 0 || left == 0;
}
"""


def test_warps_add_up_the_sums_of_their_own_row(tmp_path):
    _host_program(tmp_path, WALK)
