// Grouped FP8 products for experts with more than a few rows, gfx950 (tiles of BM rows by 256
// columns).
//
// The mathematics is moe_gemm.hip's.  A tile belongs to one expert: BM = 128 or 256 of its rows
// and 256 of its columns.  8 waves, two per SIMD, as 2 x 4: wave w owns the (BM / 2) x 64
// part (w / 4, w % 4), as MI x 2 blocks of v_mfma_scale_f32_32x32x64_f8f6f4 with unit scales,
// the W fragment first, so lane l of a block holds row l % 32 and four quads of consecutive
// columns.  FP8_BLOCK128: a K-group's partial product is promoted into the fp32 sums with one
// FMA per element while the SIMD's other wave runs its MFMAs; FP8_ROW: the matrix core
// accumulates over all of K and the scales come in the epilogue.
//
// Pipeline: LDS holds S K-groups ("regions": BM activation rows and 256 weight rows of 128
// bytes, each row's 16-byte chunk c at c ^ ((r / 2) % 8), and the group's scales), S = 2 for
// BM = 256 and 3 below.  At the start of region R every wave waits for its own loads of R and
// meets the others at a barrier; the slot of region R - 1 is then free and each wave issues its
// share of region R + S - 1 into it, direct to LDS.  The load stream runs ahead over tile
// boundaries with a cursor of its own.
//
// Gathered rows cost nothing extra in the stream: each lane's row offset within the activation
// is formed once per tile from the plan's order and every load adds the K offset in the scalar
// operand.  Rows past the expert's last read zero (their offset lies outside the descriptor).
//
// Schedule: persistent, one workgroup per CU.  Tile counts per expert come from the plan's
// offsets (on the device: the host never learns them); every workgroup sums them into a prefix
// in LDS, and takes tiles XCD by XCD, expert by expert, in 4-tile-tall column walks, so that
// workgroups of an XCD share an expert's weight rows in its L2.
#include <algorithm>
#include <type_traits>

#include "gemm_common.hpp"
#include "moe_gemm.hpp"
#include "pql_device.hpp"
#include "pql_internal.hpp"

namespace pql {

namespace {

using namespace gemm;

constexpr int kThreads = 512;
constexpr int kWaves = 8;
constexpr int BN = 256;
constexpr int kRow = 128;                          // bytes of one K-group per row
constexpr int kPersistentCap = 256;
constexpr uint32_t kOutside = 0xFFFFFFF0u;         // a row offset outside every descriptor

typedef float v16f __attribute__((ext_vector_type(16)));

template <int MI, bool ROW>
struct Shape {
  static constexpr int BM = 64 * MI;
  static constexpr int kAOp = BM * kRow;
  static constexpr int kRegion = kAOp + BN * kRow;
  static constexpr int kSlots = MI == 4 ? 2 : 3;
  static constexpr int kSaBytes = ROW ? 0 : BM * 4;        // activation scales of one group
  static constexpr int kSwBytes = ROW ? 0 : 256;           // a weight block's scale, one copy per lane
  static constexpr int kScales = kSlots * kRegion;
  static constexpr int kPrefix = kScales + kSlots * (kSaBytes + 2 * kSwBytes);
  static constexpr int kTiles = kPrefix + 4 * (kMoeMaxExperts + 4);
  static constexpr int kLds = kTiles + 64 * 8;
  static_assert(kLds <= 160 * 1024, "a CU has 160 KB of LDS");
};

template <int MI, bool ROW>
__global__ __launch_bounds__(kThreads, 1) void k_moe_tile(MoeGemmArgs g) {
  using S = Shape<MI, ROW>;
  __shared__ __attribute__((aligned(16))) uint8_t smem[S::kLds];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int Kb = (int)g.K;
  const int G = Kb / kRow;                         // K-groups = regions per tile
  const int tiles_n = (int)((g.N + BN - 1) / BN);
  const int nblocks = (int)(g.N / 128);            // weight-scale blocks along N (block-128)

  // ---- row tiles before each expert: prefix[e], prefix[E] = all of them
  int* const prefix = reinterpret_cast<int*>(smem + S::kPrefix);
  if (wave == 0) {
    const int most = most_row_tiles<S::BM>(g);
    int carry = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
      const int e = e0 + lane;
      const int n = e < g.E ? row_tiles_of<S::BM>(g, e) : 0;
      int s = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o);
        if (lane >= o) s += u;
      }
      if (e < g.E) prefix[e] = std::min(carry + s - n, most);
      carry += __shfl(s, 63);
    }
    if (lane == 0) prefix[g.E] = std::min(carry, most);
  }
  __syncthreads();
  const int row_tiles = __builtin_amdgcn_readfirstlane(prefix[g.E]);
  Sched sched;
  sched.init(row_tiles * tiles_n, row_tiles, tiles_n);
  const int my_tiles = __builtin_amdgcn_readfirstlane(sched.count);
  if (my_tiles == 0) return;

  // The workgroup's tiles, 64 at a time in LDS: entry i holds tile tile_base + i as its first
  // row, and expert, column tile and live rows packed.
  struct Tile {
    int e, m0, rows, n0;   // rows: those of the expert from m0 on, at most BM
  };
  int* const tiles = reinterpret_cast<int*>(smem + S::kTiles);
  int tile_base = 0;
  auto fill_tiles = [&](int base) __attribute__((always_inline)) {
    tile_base = base;
    if (wave != 0) return;
    const int el = fresh_lane();
    const int L = sched.first + std::min(base + el, my_tiles - 1) * sched.stride;
    const TilePlace at = tile_place<S::BM>(g, prefix, tiles_n, L);
    tiles[2 * el] = at.m0;
    tiles[2 * el + 1] = (at.e * 4096 + at.column) * 512 + at.rows;
  };
  auto tile_at = [&](int k) __attribute__((always_inline)) {
    const int i = 2 * ((k - tile_base) & 63);
    const int m0 = __builtin_amdgcn_readfirstlane(tiles[i]);
    const int rest = __builtin_amdgcn_readfirstlane(tiles[i + 1]);
    return Tile{(int)((uint32_t)rest >> 21), m0, rest & 511, ((rest >> 9) & 4095) * BN};
  };
  fill_tiles(0);
  __syncthreads();

  // ---- load stream (see the file comment).  Load p of a wave covers activation rows
  // 8 MI w + 8 p .. + 7 and weight rows 32 w + 8 p .. + 7 of the tile, whole 128-byte lines.
  struct Cursor {
    v4i a, w, sa, sw;   // descriptors of the tile's codes and scales
    uint32_t voff_a[MI];
    uint32_t voff_sa;
    int k, rg;          // tile, region within it
  } cur;
  // block-128: waves 0 .. MI - 1 load the activation scales of 64 rows each, waves 4 and 6 the
  // weight scales of the tile's two 128-column blocks
  const bool sa_wave = !ROW && wave < MI, sw_wave = !ROW && (wave == 4 || wave == 6);
  // The cursor moves to a tile in two steps: start_tile sets the descriptors and, for gathered
  // rows, issues the loads of the plan's order; finish_tile turns those into offsets, a region
  // later, when they have landed behind that region's products.
  bool started = false;
  Tile ct;
  auto start_tile = [&](int k) __attribute__((always_inline)) {
    cur.k = k;
    cur.rg = 0;
    ct = tile_at(std::min(k, my_tiles - 1));
    const int64_t base = g.gather ? 0 : (int64_t)ct.m0;   // gathered rows are offset from the operand's start
    const uint64_t rows = g.gather ? (uint64_t)g.a_rows : (uint64_t)ct.rows;
    const int64_t n = (int64_t)ct.e * g.N + ct.n0;
    const int nr = (int)std::min<int64_t>(BN, g.N - ct.n0);
    cur.a = make_rsrc(g.a + base * Kb, (int)(uint32_t)(rows * (uint64_t)Kb));
    cur.w = make_rsrc(g.w + n * Kb, nr * Kb);
    if constexpr (!ROW) {
      // the wave's weight block; a wave wholly past N takes the last one (its sums are never stored)
      const int nb = std::min(ct.n0 / 128 + (wn >> 1), nblocks - 1);
      cur.sa = make_rsrc(g.a_scales + base * G, (int)(uint32_t)(rows * (uint64_t)(G * 4)));
      cur.sw = make_rsrc(g.w_scales + ((int64_t)ct.e * nblocks + nb) * G, G * 4);
    }
    auto row_of = [&](int m) __attribute__((always_inline)) {
      if (!g.gather) return (uint32_t)m;
      return (uint32_t)g.order[ct.m0 + std::max(0, std::min(m, ct.rows - 1))];
    };
#pragma unroll
    for (int p = 0; p < MI; ++p) cur.voff_a[p] = row_of(wave * 8 * MI + 8 * p + (lane >> 3));
    if constexpr (!ROW) cur.voff_sa = row_of((wave & (MI - 1)) * 64 + lane);
    started = true;
  };
  auto finish_tile = [&]() __attribute__((always_inline)) {
    auto row_of = [&](uint32_t raw) __attribute__((always_inline)) {   // inside the operand, whatever the order holds
      return g.gather ? token_of(g, (int32_t)raw) : raw;
    };
#pragma unroll
    for (int p = 0; p < MI; ++p) {
      const int m = wave * 8 * MI + 8 * p + (lane >> 3);
      const uint32_t off = row_of(cur.voff_a[p]) * (uint32_t)Kb + (uint32_t)(dma_chunk(lane, p & 1) << 4);
      cur.voff_a[p] = m < ct.rows ? off : kOutside;
    }
    if constexpr (!ROW) {
      const int m = (wave & (MI - 1)) * 64 + lane;
      cur.voff_sa = m < ct.rows ? row_of(cur.voff_sa) * (uint32_t)(G * 4) : kOutside;
    }
    started = false;
  };
  uint8_t* const sa_lds = smem + S::kScales;                            // [slot][BM] floats
  uint8_t* const sw_lds = sa_lds + S::kSlots * S::kSaBytes;             // [slot][block][64] floats
  // Loads per wave and region, which the waits count: these, and one of scales on some waves.
  constexpr int kLoads = MI + 4;
  // The next region of the stream into `slot` (past the last tile: that tile again, into slots
  // that are never read).
  auto issue = [&](int slot) __attribute__((always_inline)) {
    uint8_t* const base = smem + slot * S::kRegion;
    const int so = cur.rg * kRow;
    // weight rows 8 apart differ by 8 K bytes and the parity bit of the swizzle; formed afresh,
    // as the fragments' addresses are: kept, they would cost registers that the sums need
    const int fl = fresh_lane();
    const int voff_w = (wave * 32 + (fl >> 3)) * Kb + (dma_chunk(fl, 0) << 4);
    if constexpr (!ROW) {   // the scales first: a gather, one cache line per row
      if (sa_wave) lds_load4_so(cur.sa, sa_lds + slot * S::kSaBytes + wave * 256, (int)cur.voff_sa, cur.rg * 4);
      if (sw_wave) lds_load4_so(cur.sw, sw_lds + (slot * 2 + (wn >> 1)) * S::kSwBytes, 0, cur.rg * 4);
    }
#pragma unroll
    for (int p = 0; p < MI; ++p)
      lds_load16_so(cur.a, base + (wave * 8 * MI + 8 * p) * kRow, (int)cur.voff_a[p], so);
#pragma unroll
    for (int p = 0; p < 4; ++p)
      lds_load16_so(cur.w, base + S::kAOp + (wave * 32 + 8 * p) * kRow, (voff_w ^ ((p & 1) << 6)) + 8 * p * Kb, so);
    if (++cur.rg == G) start_tile(cur.k + 1);
  };

  // ---- fragments: 32x32x64 operands, lane row l % 32; slice h takes chunks 4 h + c and
  // 4 h + 2 + c (c = l / 32) of the row; rows + 32 i keep the swizzle.
  // Wave (wm, wn) takes row blocks wm, wm + 2, ..: a tile with few live rows then leaves both
  // waves of a SIMD about the same work.
  int a_base, w_base;
  uint4 fw[2][2][2];   // [j][slice][chunk]
  uint4 fa[2][2][2];   // [buffer][slice][chunk]: A block i in buffer i % 2
  auto read_w = [&](const uint8_t* region) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) fw[j][h][q] = lds16(region + (w_base ^ (h * 64 + q * 32)) + j * 32 * kRow);
  };
  auto read_a = [&](const uint8_t* region, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) fa[i & 1][h][q] = lds16(region + (a_base ^ (h * 64 + q * 32)) + i * 64 * kRow);
  };
  float sc[MI];   // s_a * s_w per 32-row block of this region
  auto read_scales = [&](int slot, int fl) __attribute__((always_inline)) {
    const float* sa = reinterpret_cast<const float*>(sa_lds + slot * S::kSaBytes) + wm * 32 + (fl & 31);
    const float sw = reinterpret_cast<const float*>(sw_lds + (slot * 2 + (wn >> 1)) * S::kSwBytes)[fl];
#pragma unroll
    for (int i = 0; i < MI; ++i) sc[i] = sa[i * 64] * sw;
  };

  v16f acc[MI][2];
  v16f P[2];   // partial products of consecutive blocks, alternating (block-128)
  auto promote = [&](int b, float s) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[b >> 1][b & 1][e] = __builtin_fmaf(P[b & 1][e], s, acc[b >> 1][b & 1][e]);
  };
  // The two MFMAs of block b.
  auto block = [&](int b) __attribute__((always_inline)) {
    const int i = b >> 1, j = b & 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v8i w8 = cat(fw[j][h][0], fw[j][h][1]), a8 = cat(fa[i & 1][h][0], fa[i & 1][h][1]);
      if constexpr (ROW)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, a8, acc[i][j], 0, 0, 0, 127, 0, 127);
      else
        P[b & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, a8, h ? P[b & 1] : v16f{}, 0, 0, 0, 127, 0, 127);
    }
  };
  // A region of a tile in which LIVE of this wave's row blocks hold rows: a block's promotion
  // runs behind the next block's MFMAs, the last one's behind the next region's first (carry).
  auto region = [&](auto live_c, const uint8_t* rgn, int slot) __attribute__((always_inline)) {
    constexpr int LIVE = decltype(live_c)::value;
    if constexpr (LIVE > 0) {
      const int fl = fresh_lane();
      a_base = swz128(wm * 32 + (fl & 31), fl >> 5);
      w_base = S::kAOp + swz128(wn * 64 + (fl & 31), fl >> 5);
      read_w(rgn);
      read_a(rgn, 0);
      if constexpr (!ROW) {
          promote(2 * LIVE - 1, sc[LIVE - 1]);   // the previous region's
        read_scales(slot, fl);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < 2 * LIVE; ++b) {
        const int i = b >> 1, j = b & 1;
        block(b);
        __builtin_amdgcn_sched_barrier(0);
        if (j == 0 && i + 1 < LIVE) read_a(rgn, i + 1);
        if constexpr (!ROW) {
          if (b > 0) promote(b - 1, sc[(b - 1) >> 1]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // ---- epilogue.  In block (i, j) lane (r, c) = (l % 32, l / 32) holds, per register quad rq,
  // columns 8 rq + 4 c .. + 3 of row 32 i + r.  One v_permlane32_swap per packed dword leaves the
  // lane 8 consecutive columns, and where rows of C start on 16 bytes and the wave's 64 columns
  // exist a v_permlane16_swap brings four lanes' pieces of a row together: each store writes 64
  // consecutive bytes of 16 rows.  (Staging whole 128-byte segments in LDS took 7100 of a tile's
  // 75000 cycles: its writes use a quarter of the lanes at a time, for want of LDS.)
  auto epilogue = [&](auto live_c, const Tile& tl) __attribute__((always_inline)) {
    constexpr int LIVE = decltype(live_c)::value;
    const int m0 = tl.m0 + wm * 32, hi = tl.m0 + tl.rows;
    const int64_t n0 = tl.n0 + wn * 64;
    const bool whole = g.vec_store && n0 + 64 <= g.N;   // wave-uniform
    const int el = fresh_lane();
    const int fr = el & 31, fk = el >> 5;
    float cs[2][16], row_s[LIVE > 0 ? LIVE : 1];   // FP8_ROW: the scales of the lane's columns and rows
    if constexpr (ROW) {
#pragma unroll
      for (int i = 0; i < LIVE; ++i) row_s[i] = g.a_scales[a_row(g, std::min(m0 + i * 64 + fr, hi - 1))];
      const float* sw = g.w_scales + (int64_t)tl.e * g.N;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int rq = 0; rq < 4; ++rq) {
          const int64_t n = n0 + j * 32 + rq * 8 + fk * 4;
          if (n0 + 64 <= g.N) {   // wave-uniform
            __builtin_memcpy(&cs[j][4 * rq], sw + n, 16);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) cs[j][4 * rq + q] = sw[std::min<int64_t>(n + q, g.N - 1)];
          }
        }
    }
#pragma unroll
    for (int i = 0; i < LIVE; ++i) {
      const float rs = ROW ? row_s[i] : 1.0f;
      uint4 u[2][2];   // [j][h]
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t d[4][2];
#pragma unroll
        for (int rq = 0; rq < 4; ++rq) {
          float v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = ROW ? acc[i][j][4 * rq + q] * rs * cs[j][4 * rq + q] : acc[i][j][4 * rq + q];
          d[rq][0] = pack_bf16x2(v[0], v[1]);
          d[rq][1] = pack_bf16x2(v[2], v[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const auto s0 = __builtin_amdgcn_permlane32_swap(d[2 * h][0], d[2 * h + 1][0], false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(d[2 * h][1], d[2 * h + 1][1], false, false);
          u[j][h] = uint4{s0[0], s1[0], s0[1], s1[1]};
        }
      }
      if (whole) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t lo[4], hi4[4];
          const uint32_t x[4] = {u[j][0].x, u[j][0].y, u[j][0].z, u[j][0].w}, y[4] = {u[j][1].x, u[j][1].y, u[j][1].z, u[j][1].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const auto sw2 = __builtin_amdgcn_permlane16_swap(x[q], y[q], false, false);
            lo[q] = sw2[0];
            hi4[q] = sw2[1];
          }
          const int row = m0 + i * 64 + (el & 15), g4 = el >> 4;
          uint16_t* dst = g.c + (int64_t)row * g.ldc + n0 + j * 32 + ((g4 & 1) * 2 + (g4 >> 1)) * 8;
          if (row < hi) *reinterpret_cast<uint4*>(dst) = uint4{lo[0], lo[1], lo[2], lo[3]};
          if (row + 16 < hi) *reinterpret_cast<uint4*>(dst + 16 * g.ldc) = uint4{hi4[0], hi4[1], hi4[2], hi4[3]};
        }
      } else {
        const int row = m0 + i * 64 + fr;
        if (row < hi) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int64_t col = n0 + j * 32 + h * 16 + 8 * fk;
              uint16_t* dst = g.c + (int64_t)row * g.ldc + col;
              const uint32_t wds[4] = {u[j][h].x, u[j][h].y, u[j][h].z, u[j][h].w};
#pragma unroll
              for (int c = 0; c < 8; ++c)
                if (col + c < g.N) dst[c] = (uint16_t)(wds[c >> 1] >> (16 * (c & 1)));
            }
        }
      }
      __builtin_amdgcn_sched_barrier(0);   // one accumulator block at a time
    }
  };

  // ---- the stream
  start_tile(0);
  finish_tile();
#pragma unroll
  for (int s = 0; s < S::kSlots - 1; ++s) {
    issue(s);
    if (started) finish_tile();
  }
  int slot = 0;
  auto walk = [&](auto live_c) __attribute__((always_inline)) {   // a tile's K-groups
    constexpr int LIVE = decltype(live_c)::value;
#pragma unroll
    for (int i = 0; i < LIVE; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = v16f{};
    if constexpr (!ROW && LIVE > 0) {   // the first region's carried promotion adds 0 * 0
      P[1] = v16f{};
      sc[LIVE - 1] = 0.f;
    }
    for (int r = 0; r < G; ++r) {
      // This wave's loads of the region; those of the S - 2 regions after it may be in flight.  (The
      // last tile's stores are waited for too: letting them run behind the first region, by
      // counting them, measured 10 % slower over the whole kernel.)
      if constexpr (S::kSlots == 2) __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
      else if (sa_wave || sw_wave) __builtin_amdgcn_s_waitcnt(waitcnt_imm((S::kSlots - 2) * (kLoads + 1), 0));
      else __builtin_amdgcn_s_waitcnt(waitcnt_imm((S::kSlots - 2) * kLoads, 0));
      __builtin_amdgcn_s_barrier();   // everyone's; the previous region's slot is free
      __builtin_amdgcn_sched_barrier(0);
      if (started) finish_tile();     // (after the region's products it would draw them below its branch)
      issue(slot == 0 ? S::kSlots - 1 : slot - 1);
      region(live_c, smem + slot * S::kRegion, slot);
      slot = slot + 1 == S::kSlots ? 0 : slot + 1;
    }
    if constexpr (!ROW && LIVE > 0) promote(2 * LIVE - 1, sc[LIVE - 1]);   // the tile's last block
  };
  for (int k = 0; k < my_tiles; ++k) {
    // while tile k runs the cursor reads up to tile k + kSlots (one K-group per tile)
    if (k + S::kSlots >= tile_base + 64) {
      __syncthreads();   // everyone has read its tiles
      fill_tiles(k);
      __syncthreads();
    }
    const Tile tl = tile_at(k);
    const int live = std::max(0, std::min(MI, (tl.rows - wm * 32 + 63) >> 6));
    using std::integral_constant;
    switch (live) {
      case 4: if constexpr (MI == 4) { walk(integral_constant<int, 4>{}); epilogue(integral_constant<int, 4>{}, tl); } break;
      case 3: if constexpr (MI == 4) { walk(integral_constant<int, 3>{}); epilogue(integral_constant<int, 3>{}, tl); } break;
      case 2: walk(integral_constant<int, 2>{}); epilogue(integral_constant<int, 2>{}, tl); break;
      case 1: walk(integral_constant<int, 1>{}); epilogue(integral_constant<int, 1>{}, tl); break;
      default: walk(integral_constant<int, 0>{});   // its share of the loads
    }
  }
  __builtin_amdgcn_s_waitcnt(0);
}

template <int MI, bool ROW>
hipError_t launch_shape(const MoeGemmArgs& g, hipStream_t st) {
  constexpr int BM = 64 * MI;
  const int64_t row_tiles = g.P / BM + std::min(g.P, g.E);
  const int64_t tiles = row_tiles * ((g.N + BN - 1) / BN);
  hipLaunchKernelGGL((k_moe_tile<MI, ROW>), dim3((unsigned)std::min<int64_t>(tiles, kPersistentCap)), dim3(kThreads), 0,
                     st, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_tile(bool row_scales, int bm, const MoeGemmArgs& g, hipStream_t st) {
  if (row_scales) return bm == 128 ? launch_shape<2, true>(g, st) : launch_shape<4, true>(g, st);
  return bm == 128 ? launch_shape<2, false>(g, st) : launch_shape<4, false>(g, st);
}

}  // namespace pql
