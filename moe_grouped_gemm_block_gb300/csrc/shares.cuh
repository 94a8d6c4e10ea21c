// shares.cuh -- how a CTA's warps share the rows of E experts that are left for its end: an expert a lane, so as many warps
// a row as it has 32 experts, and several rows at once.  Plain arithmetic, on the host as on the device.
#pragma once

namespace fp8g {

struct RowShares {
  int parts, at_once;  // warps a row, rows at once
  int slot, part;      // of this warp
  __host__ __device__ RowShares(int E, int warps, int warp) {
    parts = (E + 31) / 32 < warps ? (E + 31) / 32 : warps;
    at_once = warps / parts;
    slot = warp / parts;
    part = warp % parts;
  }
  // Warps that are left over where `parts` does not divide their number have no row, and no full set of warps beside them.
  __host__ __device__ bool some() const { return slot < at_once; }
  __host__ __device__ int first() const { return slot * parts; }  // of the row's warps
};

}  // namespace fp8g
