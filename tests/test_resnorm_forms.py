"""Which form the norms around a block take for a row of any length (csrc/resnorm.cuh), walked over on the host: up to 16384
columns the forward call has a form that holds a row, whatever the types, and its CTAs fit an SM beside one another.  No
GPU needed."""

import os
import subprocess

from moe_grouped_gemm_block_gb300 import build as b

WALK = r"""
#include <cstdio>
#include "fp8gemm.h"
#include "resnorm.cuh"
using namespace fp8g;

int main() {
  int faults = 0, forms = 0;
  for (const ResMode mode : {kAligned, kShifted, kSingle})
    for (int64_t N = mode == kAligned ? 8 : 1; N <= (mode == kShifted ? 16384 - 7 : 16384); N += mode == kAligned ? 8 : 1)
      for (int64_t stream : {2, 4})
        for (int64_t block : {2, 4})
          for (const bool f : {false, true}) {
            const ResPlan p = res_forward_plan(N, mode, stream, block, f);
            const ResShared& s = p.shared;
            ++forms;
            const bool fits = s.stages >= 1 && s.stages <= kResMaxStages && s.stages_f >= 1 && p.per_sm >= 1 &&
                              p.per_sm * (s.bytes + 1024) <= 228 * 1024 && s.bytes + 1024 <= 227 * 1024 &&
                              p.per_sm * p.form.threads <= 2048;
            if (!fits && ++faults <= 5)
              printf("mode %d N %lld types %lld %lld f %d: stages %d, %d CTAs an SM\n", mode, (long long)N, (long long)stream,
                     (long long)block, f, s.stages, p.per_sm);
          }
  if (res_forward_plan(16385, kSingle, 2, 2, true).shared.stages != 0) ++faults;
  printf("faults %d of %d\n", faults, forms);
  return faults != 0;
}
"""


def test_rows_of_up_to_16384_columns_are_held(tmp_path):
    src, exe = tmp_path / "walk.cu", tmp_path / "walk"
    src.write_text(WALK)
    subprocess.run([b._nvcc(), *b.ARCH, "-std=c++17", "-I", b.CSRC, "-I", os.path.join(b.ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
