// The tile schedule of the grouped products (csrc/moe_gemm.hpp) on the host, under
// UndefinedBehaviorSanitizer (test infrastructure): tiles of correct plans cover every row of every
// expert once; with wild offsets every tile stays inside 0 .. P, up to the largest sizes.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include <hip/hip_runtime.h>

#include "moe_gemm.hpp"

static long failures = 0;

template <int BM>
static void walk(const char* what, const std::vector<int32_t>& offsets, int P, int64_t N, bool plan) {
  const int E = (int)offsets.size() - 1, tiles_n = (int)((N + 255) / 256);
  pql::MoeGemmArgs g{};
  g.offsets = offsets.data();
  g.P = P;
  g.E = E;
  g.N = N;
  std::vector<int> prefix(E + 1);
  const int most = pql::most_row_tiles<BM>(g);
  int carry = 0;
  for (int e = 0; e <= E; ++e) {
    prefix[e] = std::min(carry, most);
    if (e < E) carry += pql::row_tiles_of<BM>(g, e);
  }
  const int total = prefix[E] * tiles_n;
  std::vector<int> seen(plan ? P : 0);
  const int step = plan ? 1 : std::max(1, total / 200000);
  auto look = [&](int L) {
    const pql::TilePlace t = pql::tile_place<BM>(g, prefix.data(), tiles_n, L);
    int lo = 0, hi = 0;
    if (t.e >= 0 && t.e < E) pql::expert_range(g, t.e, lo, hi);
    const bool good = t.e >= 0 && t.e < E && t.rows >= 1 && t.rows <= BM && t.m0 >= lo && t.m0 + t.rows <= hi &&
                      t.column >= 0 && t.column < tiles_n;
    if (!good && ++failures < 20)
      std::printf("FAIL %s BM=%d P=%d E=%d N=%lld: tile %d is expert %d, rows %d + %d, column %d\n", what, BM, P, E,
                  (long long)N, L, t.e, t.m0, t.rows, t.column);
    if (plan && good && t.column == tiles_n - 1)
      for (int i = 0; i < t.rows; ++i) ++seen[t.m0 + i];
  };
  for (int L = 0; L < total; L += step) look(L);
  if (total && !plan) look(total - 1);
  if (plan)
    for (int p = 0; p < P; ++p)
      if (seen[p] != (p < offsets[E]) && ++failures < 20) std::printf("FAIL %s: row %d is in %d tiles\n", what, p, seen[p]);
}

template <int BM>
static void both() {
  std::mt19937 rng(5);
  for (int E : {1, 3, 60, 1024})
    for (int P : {1, 37, 1000, 5003}) {
      std::vector<int32_t> at(E + 1, 0);
      for (int e = 1; e <= E; ++e) at[e] = std::min<int>(P, at[e - 1] + (int)(rng() % (2 * P / E + 2)));
      for (int64_t N : {128, 257, 4096}) walk<BM>("plan", at, P, N, true);
      for (int round = 0; round < 4; ++round) {
        for (int e = 0; e <= E; ++e) at[e] = (int32_t)rng() >> (round * 7);
        walk<BM>("wild", at, P, 640, false);
      }
    }
  // every expert claims all of the rows
  for (int P : {1 << 17, 1 << 20, (1 << 24) - 1})
    for (int64_t N : {int64_t(1) << 16, int64_t(1) << 20}) {
      std::vector<int32_t> at(1025);
      for (int e = 0; e <= 1024; ++e) at[e] = e & 1 ? INT32_MAX : INT32_MIN;
      walk<BM>("overlapping", at, P, N, false);
    }
}

int main() {
  both<128>();
  both<256>();
  std::printf("%s: %ld failures\n", failures ? "FAILED" : "ok", failures);
  return failures ? 1 : 0;
}
