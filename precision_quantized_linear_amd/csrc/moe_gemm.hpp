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

// The token of an order entry (inside 0 .. a_rows - 1 whatever it holds).  The magic is
// 2^32 / k + d with 0 < d <= 1, so the product is off by at most i 2^-32 < 2^-8 < 1 / k: exact.
__device__ __forceinline__ uint32_t token_of(const MoeGemmArgs& g, int32_t entry) {
  const uint32_t i = (uint32_t)std::min(std::max(entry, 0), (1 << 24) - 1);
  const uint32_t t = g.top_k == 1 ? i : __umulhi(i, g.top_k_magic);
  return std::min<uint32_t>(t, (uint32_t)g.a_rows - 1);
}

// The activation row of position p (inside the operand whatever the order holds).
__device__ __forceinline__ int64_t a_row(const MoeGemmArgs& g, int p) {
  return g.gather ? (int64_t)token_of(g, g.order[p]) : std::min<int64_t>(p, g.a_rows - 1);
}

}  // namespace pql
