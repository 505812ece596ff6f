// Shared by the grouped-GEMM kernels: how a plan's entries are read.  Internal to the library.
#pragma once

#include <algorithm>

#include "pql_internal.hpp"

namespace pql {

// Expert e's assignments, inside 0 .. P whatever the offsets hold.
__device__ __forceinline__ void expert_range(const MoeGemmArgs& g, int e, int& lo, int& hi) {
  lo = std::min(std::max(g.offsets[e], 0), g.P);
  hi = std::min(std::max(g.offsets[e + 1], lo), g.P);
}

// The activation row of position p (inside the operand whatever the order holds).
__device__ __forceinline__ int64_t a_row(const MoeGemmArgs& g, int p) {
  const int64_t r = g.gather ? (int64_t)((uint32_t)std::max(g.order[p], 0) / (uint32_t)g.top_k) : (int64_t)p;
  return std::min<int64_t>(r, g.a_rows - 1);
}

}  // namespace pql
