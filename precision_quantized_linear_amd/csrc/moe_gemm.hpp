// Shared by the grouped-GEMM kernels: how a plan's entries are read.  Internal to the library.
#pragma once

#include <algorithm>

#include "pql_internal.hpp"

namespace pql {

// Expert e's assignments, inside 0 .. P whatever the offsets hold.
__host__ __device__ __forceinline__ void expert_range(const MoeGemmArgs& g, int e, int& lo, int& hi) {
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

// ---- the schedule of the tiles of BM rows by 256 columns: expert by expert, inside an expert in
// column walks kWalk row tiles tall.

// An expert's row tiles.
template <int BM>
__host__ __device__ __forceinline__ int row_tiles_of(const MoeGemmArgs& g, int e) {
  int lo, hi;
  expert_range(g, e, lo, hi);
  return (hi - lo + BM - 1) / BM;
}

// A plan has at most this many row tiles.  Wild offsets (ranges that overlap) are cut there, and so is
// every count of row tiles before an expert: at most 2^17 + 2^10, times at most 2^12 column tiles, it
// stays inside 32 bits, which 2^27 (2^17 row tiles for each of 1024 experts) would not.
template <int BM>
__host__ __device__ __forceinline__ int most_row_tiles(const MoeGemmArgs& g) { return g.P / BM + g.E; }

// Tile L of prefix[E] * tiles_n: its expert, first row, live rows (1 .. BM) and column tile.
// prefix[e]: the row tiles before expert e, cut at most_row_tiles.
struct TilePlace {
  int e, m0, rows, column;
};
template <int BM>
__host__ __device__ __forceinline__ TilePlace tile_place(const MoeGemmArgs& g, const int* prefix, int tiles_n, int L) {
  constexpr int kWalk = 4;
  int e = 0, above = g.E;   // prefix[e] * tiles_n <= L < prefix[above] * tiles_n
  while (above - e > 1) {
    const int mid = (e + above) >> 1;
    if (prefix[mid] * tiles_n <= L) e = mid;
    else above = mid;
  }
  int lo, hi;
  expert_range(g, e, lo, hi);
  const int tiles_m = (hi - lo + BM - 1) / BM;
  const int l = L - prefix[e] * tiles_n;
  const int group = l / (kWalk * tiles_n);
  const int gm = std::max(1, std::min(tiles_m - group * kWalk, kWalk));
  const int r = l - group * kWalk * tiles_n;
  const int m0 = lo + (group * kWalk + r % gm) * BM;
  return TilePlace{e, m0, std::max(0, std::min(BM, hi - m0)), r / gm};
}

}  // namespace pql
