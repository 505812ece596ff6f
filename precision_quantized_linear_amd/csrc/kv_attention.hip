// Attention of a batch's new tokens over the paged cache of keys and values, gfx950.
//
// For a head of the cache, the G = H / Hk query heads of n new tokens are n G rows that share its keys and
// values.  A workgroup takes a tile of rows and a range of keys, forms
//   S^T = K Q^T,  w = 2^(scale log2 e S - m),  O^T = V^T w^T,  l = sum w
// with the running maximum m of a softmax, key tile by key tile, and either divides and stores, or leaves
// (O, m, l) of its range for k_attend_join.  Both products keep keys (then head values) along the rows of
// the matrix cores' results and the query rows along the lanes: the maximum, the sum and the correction
// of O are one lane's own numbers, and the registers that hold w are, as they stand, the second
// operand of the second product (its order along the keys is free, and V^T follows it).
//
// FP8 codes are multiplied as they are: keys in bf16 beside q, values in fp16 beside w, both exact.  With
// a scale per token, the score of key j is s_j = ks_j (code_j . q), and its value's scale goes into the weight as a
// power of two: w_j = 2^(s_j + log2 vs_j - m) is at most about 1 whatever the scales, O sums w_j code_j and l
// sums w_j / vs_j, so that O / l is the answer, at one exponential per score.  w is shifted up
// by 2^7 (and may rise 2^8 above the last m that was taken, below), so that fp16 keeps 11 bits of every weight
// down to 2^-21 of the largest.  bf16 caches have w in bf16; there l sums the rounded weights, so that a
// token that holds nearly all of the weight comes out without their rounding, and a second sum, of the weights
// before they are rounded, is kept for the logarithm where it is asked for.
// m follows the maximum only when that passes it by 2^8: O is rarely rescaled.
#include <algorithm>
#include <cmath>

#include "gemm_common.hpp"
#include "kv_common.hpp"
#include "pql_device.hpp"
#include "pql_internal.hpp"

namespace pql {

namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRise = 8.0f;       // m follows the maximum when that is so much higher
// l is at most 2^(90 + 15) times the number of keys.  Slight keys (below) make it so large by themselves, at an m of
// -90; where values with a scale of 2^36 or more join them, the factor between the two m is below fp32's range
// although the slight keys still count, so l is multiplied by the factor's root twice.
constexpr float kSmallestValueScale = 0x1p-90f, kSmallestLog = -90.0f, kNoShare = -200.0f;

template <int SCHEME>
constexpr float weight_shift() { return SCHEME == kKvBf16 ? 0.0f : 7.0f; }

// ---------------------------------------------------------------- work of a workgroup
// Tiles of BM rows; keys in tiles of 64.  A sequence's row tiles are each cut into `splits` ranges of `chunk`
// key tiles at most, the chunk chosen on the device so that all ranges of all heads are about `target`: long
// contexts are spread over the card whatever the others' lengths.  Every workgroup finds its own sequence by
// a scan over the batch, 4 sequences per lane and step.
constexpr int kKeyTile = 64;

struct Work {
  Seq s;
  int b, tile, split, chunk;
  uint32_t part;   // place of its range among those of a head
};

// Sums over the wave by data-parallel moves: within rows of 16, then row to row.
__device__ __forceinline__ uint32_t scan_add(uint32_t v) {   // inclusive
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true);   // from 1, 2, 4, 8 lanes below
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, true);   // row 0's and 2's last lane to the next row
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, true);   // row 1's last lane to rows 2 and 3
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#define PQL_ADD_DPP(ctrl, rows)                                                                      \
  v += __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), ctrl, rows, 0xF, true),    \
                        __builtin_amdgcn_update_dpp(0, __double2loint(v), ctrl, rows, 0xF, true))
  PQL_ADD_DPP(0x111, 0xF);
  PQL_ADD_DPP(0x112, 0xF);
  PQL_ADD_DPP(0x114, 0xF);
  PQL_ADD_DPP(0x118, 0xF);
  PQL_ADD_DPP(0x142, 0xA);
  PQL_ADD_DPP(0x143, 0xC);
#undef PQL_ADD_DPP
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), 63), __builtin_amdgcn_readlane(__double2loint(v), 63));
}

// The first token that a row at `pos` sees; a negative position comes of more new tokens than the cache holds.
__device__ __forceinline__ int window_begin(const AttendArgs& g, int pos) {
  return g.window ? std::max(0, std::max(0, pos) - g.window + 1) : 0;
}

__device__ __forceinline__ int splits_of(int kt, int chunk) { return kt <= chunk ? 1 : (kt + chunk - 1) / chunk; }

// Four consecutive sequences of a lane: their rows, row tiles and the key tiles that any of their rows sees.
// Row counts stay below 2^28 (T H D <= 2^34), key tiles below 2^25.
template <int BM>
struct Shapes {
  Seq s[4];
  int qt[4], kt[4];
  __device__ __forceinline__ void load(const AttendArgs& g, int b0) {
    const int lane = threadIdx.x & 63, G = g.H / g.Hk;
    const int64_t cap = g.width << g.page_shift;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int b = b0 + 4 * lane + r;
      s[r] = Seq{0, 0, 0};
      if (b < g.B) s[r] = sequence(g.starts, g.lens, b, g.T);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      qt[r] = (s[r].n * G + BM - 1) / BM;
      const int end = (int)std::min<int64_t>(s[r].len, cap);
      const int begin = window_begin(g, s[r].len - s[r].n);
      kt[r] = std::max(0, (end + kKeyTile - 1) / kKeyTile - begin / kKeyTile);
    }
  }
  // Whole numbers that fp64 holds exactly: every kernel gets the same sum, however its compiler fuses.
  __device__ __forceinline__ double work() const {
    return ((double)qt[0] * kt[0] + (double)qt[1] * kt[1]) + ((double)qt[2] * kt[2] + (double)qt[3] * kt[3]);
  }
};

// The range with number `idx` among a head's; with MULTI, of the row tiles of sequences that are cut, the
// tile with number idx.  The chunk is the same in every workgroup and in k_attend_join.
template <int BM, bool MULTI>
__device__ __forceinline__ bool find_work(const AttendArgs& g, uint32_t idx, Work& w) {
  const int lane = threadIdx.x & 63;
  Shapes<BM> x;
  x.load(g, 0);
  int chunk = INT32_MAX;
  if (g.target) {
    double total = x.work();
    for (int b0 = 256; b0 < g.B; b0 += 256) {
      x.load(g, b0);
      total += x.work();
    }
    if (g.B > 256) x.load(g, 0);
    const double want = __builtin_ceil(wave_sum(total) * (double)g.Hk / (double)g.target);
    chunk = std::max(g.min_chunk, (int)fmin(want, 1073741824.0));
    chunk = __builtin_amdgcn_readfirstlane(chunk);
  }
  uint32_t before = 0, parts_before = 0;
  for (int b0 = 0; b0 < g.B; b0 += 256) {
    if (b0) x.load(g, b0);
    uint32_t n[4], parts[4], mine = 0, my_parts = 0;
    int splits[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      splits[r] = splits_of(x.kt[r], chunk);
      const uint32_t items = (uint32_t)x.qt[r] * (uint32_t)splits[r];
      parts[r] = splits[r] > 1 ? items : 0u;
      n[r] = MULTI ? (splits[r] > 1 ? (uint32_t)x.qt[r] : 0u) : items;
      mine += n[r];
      my_parts += parts[r];
    }
    const uint32_t incl = scan_add(mine), incl_parts = scan_add(my_parts);
    uint32_t at = before + incl - mine, at_parts = parts_before + incl_parts - my_parts;
    const uint64_t hit = __ballot(idx >= at && idx - at < mine);
    if (hit) {
      const int who = __builtin_ctzll(hit);
      int found = 0, found_splits = 1, found_qt = 0, found_kt = 0;
      Seq found_s{0, 0, 0};
      uint32_t rest = 0, found_parts = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (idx >= at && idx - at < n[r]) {
          found = b0 + 4 * lane + r;
          found_splits = splits[r];
          found_qt = x.qt[r];
          found_kt = x.kt[r];
          found_s = x.s[r];
          rest = idx - at;
          found_parts = at_parts;
        }
        at += n[r];
        at_parts += parts[r];
      }
      w.b = __builtin_amdgcn_readlane(found, who);
      w.s = Seq{__builtin_amdgcn_readlane(found_s.first, who), __builtin_amdgcn_readlane(found_s.n, who),
                __builtin_amdgcn_readlane(found_s.len, who)};
      const uint32_t splits_b = (uint32_t)__builtin_amdgcn_readlane(found_splits, who);
      const int qt = __builtin_amdgcn_readlane(found_qt, who);
      rest = (uint32_t)__builtin_amdgcn_readlane((int)rest, who);
      found_parts = (uint32_t)__builtin_amdgcn_readlane((int)found_parts, who);
      const uint32_t kt = (uint32_t)__builtin_amdgcn_readlane(found_kt, who);
      w.chunk = splits_b == 1 ? chunk : (int)((kt + splits_b - 1) / splits_b);   // of equal length
      // the last tile sees most: it goes first
      const uint32_t j = MULTI || splits_b == 1 ? rest : rest / splits_b;
      w.tile = qt - 1 - (int)j;
      w.split = MULTI ? 0 : (int)(rest - j * splits_b);
      w.part = found_parts + j * splits_b + (uint32_t)w.split;
      return w.tile >= 0;
    }
    before += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
    parts_before += (uint32_t)__builtin_amdgcn_readlane((int)incl_parts, 63);
  }
  return false;
}

// What a tile's rows see: keys begin .. end - 1 in all, all_begin .. all_end - 1 by every row; its key tiles.
struct Sight {
  int begin, end, all_begin, all_end;
  int kt0, kt1;
};

template <int BM>
__device__ __forceinline__ Sight sight_of(const AttendArgs& g, const Seq& s, int tile) {
  const int G = g.H / g.Hk;
  const int rows = s.n * G, last_row = std::min(rows, (tile + 1) * BM) - 1;
  const int lo = s.len - s.n + tile * BM / G, hi = s.len - s.n + last_row / G;   // positions of the first and last row
  const int held = (int)std::min<int64_t>(s.len, g.width << g.page_shift);
  Sight v;
  v.end = g.causal ? std::max(0, std::min(held, hi + 1)) : held;
  v.all_end = g.causal ? std::max(0, std::min(held, lo + 1)) : held;
  v.begin = window_begin(g, lo);
  v.all_begin = window_begin(g, hi);
  v.kt0 = std::min(v.begin, v.end) / kKeyTile;   // a window past the end (a length past the pages) sees none
  v.kt1 = std::max(v.kt0, (v.end + kKeyTile - 1) / kKeyTile);
  return v;
}

// The first row of the cache (of [n_pages * Hk * page_size]) for 16 keys from `key` (a multiple of 16, on
// one page), and whether the cache holds them: a page outside it reads page 0, masked.
__device__ __forceinline__ int64_t rows_at(const AttendArgs& g, int b, int hk, int key, bool& held) {
  const int p = key >> g.page_shift, last = (int)g.width - 1;
  int page = g.pages[b * g.ldp + std::min(p, last)];
  held = page >= 0 && page < g.n_pages && p <= last;
  page = __builtin_amdgcn_readfirstlane(held ? page : 0);
  held = __builtin_amdgcn_readfirstlane(held);
  return (((int64_t)page * g.Hk + hk) << g.page_shift) + (key & ((1 << g.page_shift) - 1));
}

// ---------------------------------------------------------------- numbers
__device__ __forceinline__ float max32(float x) {   // with lane ^ 32
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max16(float x) {   // with lane ^ 16
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 8 codes -> 8 bf16 / 4 codes -> 4 fp16, exact.
__device__ __forceinline__ uint32_t bf16x2_of(uint32_t codes, bool high) {
  const v2b r = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, true)
                     : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, false);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes, bool high) {
  const v2h r = high ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, true)
                     : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 1.0f, false);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2h));
}

__device__ __forceinline__ uint4 bf16x8_of(uint2 codes) {
  return make_uint4(bf16x2_of(codes.x, false), bf16x2_of(codes.x, true), bf16x2_of(codes.y, false), bf16x2_of(codes.y, true));
}

// Two weights in 16 bits; under bf16 they become what they were rounded to.
template <int SCHEME>
__device__ __forceinline__ uint32_t pack_weights(float& a, float& b) {
  if constexpr (SCHEME == kKvBf16) {
    const uint32_t p = gemm::pack_bf16x2(a, b);
    a = bf16lo(p);
    b = bf16hi(p);
    return p;
  } else {
    return pack_f16x2(a, b);
  }
}

// 4 x 4 transposes of what four keys' loads hold: out[d] = the four keys' value d, 4 bytes (codes), or two
// words of 16-bit values.
__device__ __forceinline__ void transpose4(const uint32_t (&k)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(k[1], k[0], 0x05010400u), b = __builtin_amdgcn_perm(k[1], k[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(k[3], k[2], 0x05010400u), d = __builtin_amdgcn_perm(k[3], k[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}
__device__ __forceinline__ uint32_t low16s(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high16s(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Whether 4 codes hold a NaN (0x7F, 0xFF), or two bf16 values a NaN or an infinity.
__device__ __forceinline__ bool bad_codes(uint32_t c) {
  const uint32_t m = c & 0x7F7F7F7Fu;
  return ((m + 0x01010101u) & 0x80808080u) != 0;
}
__device__ __forceinline__ bool bad_bf16(uint32_t c) {
  return (c & 0x7F80u) == 0x7F80u || (c & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ uint32_t magnitude(uint32_t codes) { return codes & 0x7F7F7F7Fu; }
template <int SCHEME>
__device__ __forceinline__ bool bad_word(uint32_t c) { return SCHEME == kKvBf16 ? bad_bf16(c) : bad_codes(c); }

// A value scale as the weights take it: its logarithm and its reciprocal.  Slight keys, looked for only where a scale
// is 1 or below 2^-90, are rows of zeros (their scale of 1, by the quantizer's rule, says nothing about their
// size and would lift m above all weights that matter where the others' values are small) and keys whose scale's
// reciprocal l could not hold.  They have the logarithm -90 in m's sense, add 2^(s - m) to l by themselves, and their
// weight then goes down by share_log: the logarithm of what the scale is of 2^-90, kNoShare for zeros.  That stands
// in the reciprocal's place and marks them, being below 0; what it adds to l, times the weight, is below
// 2^-80 of what they have added.  Below about 2^-115 a scale leaves fp16's range, an error of 2^-113 at most in a
// value.  A negative scale counts as 0.
__device__ __forceinline__ void value_scale(float vs, float& lv, float& rv) {
  vs = vs < kSmallestValueScale ? kSmallestValueScale : vs;   // a NaN stays one
  lv = __builtin_amdgcn_logf(vs);
  rv = __builtin_amdgcn_rcpf(vs);
}
__device__ __forceinline__ float share_log(float vs) {
  return fminf(fmaxf(__builtin_amdgcn_logf(fmaxf(vs * 0x1p90f, 0.0f)), kNoShare), -0x1p-22f);
}

// 2^d, d <= 0, as a product: its root twice where slight keys can make l that large, so that l times both stays
// in range where 2^d does not.
struct Factor {
  float a, b;
  __device__ __forceinline__ float whole() const { return a * b; }
};
template <int SCHEME>
__device__ __forceinline__ Factor factor_of(float d) {
  if constexpr (SCHEME != kKvRow) return Factor{__builtin_amdgcn_exp2f(d), 1.0f};
  const float root = __builtin_amdgcn_exp2f(0.5f * d);
  return Factor{root, root};
}

// Lanes 0 .. 7 of each row of 16 lanes, in all of the row's lanes.
__device__ __forceinline__ void row_lanes8(float x, float (&out)[8]) {
#define PQL_ROW_LANE(n) \
  out[n] = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + n, 0xF, 0xF, true))
  PQL_ROW_LANE(0);
  PQL_ROW_LANE(1);
  PQL_ROW_LANE(2);
  PQL_ROW_LANE(3);
  PQL_ROW_LANE(4);
  PQL_ROW_LANE(5);
  PQL_ROW_LANE(6);
  PQL_ROW_LANE(7);
#undef PQL_ROW_LANE
}

// The second products' operands, as 16-byte words.
template <int SCHEME>
__device__ __forceinline__ v4f mfma16_pv(uint4 v, uint4 w, v4f acc) {
  if constexpr (SCHEME == kKvBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, v), __builtin_bit_cast(v8bf, w), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, v), __builtin_bit_cast(v8h, w), acc, 0, 0, 0);
}
template <int SCHEME>
__device__ __forceinline__ v16f mfma32_pv(uint4 v, uint4 w, v16f acc) {
  if constexpr (SCHEME == kKvBf16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, v), __builtin_bit_cast(v8bf, w), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, v), __builtin_bit_cast(v8h, w), acc, 0, 0, 0);
}

// What multiplies O / l at the end, and a score before its exponential.
template <int SCHEME>
__device__ __forceinline__ float final_scale(const AttendArgs& g) { return SCHEME == kKvTensor ? g.v_scales[0] : 1.0f; }
template <int SCHEME>
__device__ __forceinline__ float score_scale(const AttendArgs& g) {
  return g.scale * kLog2e * (SCHEME == kKvTensor ? g.k_scales[0] : 1.0f);
}

// log sum exp, natural, from m and l (l carries the weights' shift).
template <int SCHEME>
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : kLn2 * (m - weight_shift<SCHEME>() + __builtin_amdgcn_logf(l));
}

// ---------------------------------------------------------------- results
// 8 values of a row from their sums; a row that saw nothing is zeros.
template <int SCHEME>
__device__ __forceinline__ void store_row(const AttendArgs& g, const Seq& s, int row, int hk, int d, const float (&acc)[8],
                                          float m, float l, float le, float fin) {
  const int G = g.H / g.Hk;
  const int64_t t = s.first + row / G;
  const int h = hk * G + row % G;
  const float f = l == 0.0f ? 0.0f : fin / l;
  stg16(g.out + t * g.ldot + (int64_t)h * g.ldoh + d,
        make_uint4(gemm::pack_bf16x2(acc[0] * f, acc[1] * f), gemm::pack_bf16x2(acc[2] * f, acc[3] * f),
                   gemm::pack_bf16x2(acc[4] * f, acc[5] * f), gemm::pack_bf16x2(acc[6] * f, acc[7] * f)));
  if (g.lse && d == 0) g.lse[t * g.H + h] = lse_of<SCHEME>(m, SCHEME == kKvBf16 ? le : l);
}

// What the sums of a range with maximum m count for beside the highest one.  A range that saw nothing but
// NaN has no maximum; its sums are NaN and stay.
template <int SCHEME>
__device__ __forceinline__ Factor join_factor(float m, float l, float top) {
  if (m == -INFINITY) return l != 0.0f ? Factor{1.0f, 1.0f} : Factor{0.0f, 0.0f};
  return factor_of<SCHEME>(m - top);
}

// Parts, [Hk, parts, BM, D] sums and then [Hk, parts, BM] x (m, l, l of weights as they were, unused), fp32.
__device__ __forceinline__ float* part_sums(const AttendArgs& g, int BM, int D, int hk, uint32_t part, int row) {
  return g.ws + (((int64_t)hk * g.parts + part) * BM + row) * D;
}
__device__ __forceinline__ float4* part_ml(const AttendArgs& g, int BM, int D, int hk, uint32_t part, int row) {
  return reinterpret_cast<float4*>(g.ws + (int64_t)g.Hk * g.parts * BM * D) + ((int64_t)hk * g.parts + part) * BM + row;
}

// ---------------------------------------------------------------- few rows: keys stream past
// 16 NQ rows per workgroup.  Four waves take 32 keys each in turn, straight from memory into the
// registers that the 16 x 16 x 32 matrix instructions read: a lane's part of a key is D / 4 contiguous
// values (q is read in the same order), and of a value D / 16 contiguous ones of eight keys, transposed in
// registers.  Nothing is staged and no wave waits for another until the end, where the four (O, m, l)
// are joined through LDS.  A step's loads go into the registers that the last step has just used: a second set would
// leave half the waves, and several waves per SIMD hide the wait better (one token over 131000: 160 -> 78 us).
// A key's scale, its value scale's logarithm and reciprocal are formed by one lane and broadcast within rows of 16.
//
// Bound by reading the cache, with the unpacking of codes close behind: 64 sequences of up to 16384 tokens, 4 heads
// of 128 with a scale per token, 111 us and 7.5 for the join, 555 MB, 5.0 TB/s (reads alone reach 5.7 to 5.9);
// bf16, half the instructions per byte, 4.8 TB/s in all.  A single context of 6007 tokens, 7.8 + 4.5 us, is two launches'
// and one range's latency.
template <int SCHEME, int D>
struct StreamTile {
  static constexpr int EB = SCHEME == kKvBf16 ? 2 : 1;       // bytes of a value
  static constexpr int KW = D / 4 * EB / 16;                 // 16-byte loads of a lane per 16 keys
  static constexpr int VW = D / 16 * EB / 4;                 // words of a lane per key
  uint4 k[2][KW];
  uint32_t v[8][VW];
  float ks, vs;                                              // of key 16 (c / 4 % 2) + 4 q + c % 4
  int64_t row[2];
  bool held[2], next_held[2];

  __device__ __forceinline__ void find(const AttendArgs& g, int b, int hk, int key) {
#pragma unroll
    for (int t = 0; t < 2; ++t) row[t] = rows_at(g, b, hk, key + 16 * t, next_held[t]);
  }
  __device__ __forceinline__ void load_k(const AttendArgs& g, int lane) {
    const int c = lane & 15, q = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* p = static_cast<const uint8_t*>(g.k_codes) + row[t] * (D * EB) + (c * (D * EB) + q * (D / 4 * EB));
#pragma unroll
      for (int i = 0; i < KW; ++i) k[t][i] = ldg16(p + 16 * i);
    }
  }
  __device__ __forceinline__ void load_v(const AttendArgs& g, int lane) {
    const int c = lane & 15, q = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* p = static_cast<const uint8_t*>(g.v_codes) + row[t] * (D * EB) + (4 * q * (D * EB) + c * (VW * 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        struct W { uint32_t w[VW]; };
        const W x = *reinterpret_cast<const W*>(p + i * (D * EB));
#pragma unroll
        for (int j = 0; j < VW; ++j) v[4 * t + i][j] = x.w[j];
      }
    }
  }
  __device__ __forceinline__ void load_scales(const AttendArgs& g, int lane) {
    if constexpr (SCHEME == kKvRow) {
      const int64_t r = ((lane & 4) ? row[1] : row[0]) + (4 * (lane >> 4) + (lane & 3));
      ks = g.k_scales[r];
      vs = g.v_scales[r];
    }
  }
};

template <int SCHEME, int D, int NQ>
constexpr int stream_waves() {   // per SIMD, by the registers that a wave's rows and one step's keys and values take
  constexpr int regs = D / 4 * NQ + D / 8 * NQ + D / 4 * (SCHEME == kKvBf16 ? 2 : 1) + 72;
  return regs <= 128 ? 4 : regs <= 168 ? 3 : regs <= 256 ? 2 : 1;
}

template <int SCHEME, int D, int NQ>
__global__ __launch_bounds__(256, (stream_waves<SCHEME, D, NQ>())) void k_attend_stream(AttendArgs g) {
  constexpr int BM = 16 * NQ, JD = D / 16, VW = StreamTile<SCHEME, D>::VW;
  __shared__ float so[4][16][D + 4];
  __shared__ float sm[4][16], sl[4][16], se[4][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q4 = lane >> 4;
  const int hk = (int)(blockIdx.x % (uint32_t)g.Hk);
  Work w;
  if (!find_work<BM, false>(g, blockIdx.x / (uint32_t)g.Hk, w)) return;
  const Sight v = sight_of<BM>(g, w.s, w.tile);
  const int mine = splits_of(v.kt1 - v.kt0, w.chunk);
  if (w.split >= mine) return;
  const int kt_first = v.kt0 + w.split * w.chunk;   // split 0 where chunk is unbounded
  const int kt_last = mine > 1 ? std::min(v.kt1, kt_first + w.chunk) : v.kt1;
  const int key_last = std::min(kt_last * kKeyTile, (v.end + 31) & ~31);
  int key = kt_first * kKeyTile + 32 * wave;
  StreamTile<SCHEME, D> x;
  if (key < key_last) {
    x.find(g, w.b, hk, key);
    x.load_k(g, lane);
    x.load_scales(g, lane);
    x.load_v(g, lane);
  }

  // this lane's rows and what they see
  const int G = g.H / g.Hk;
  const int rows = w.s.n * G;
  uint4 qf[NQ][D / 32];
  int row_end[NQ], row_begin[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = w.tile * BM + 16 * n + c;
    const bool live = r < rows;
    const int i = live ? r / G : 0, h = live ? hk * G + (r - i * G) : 0;
    const uint16_t* p = g.q + (int64_t)(w.s.first + i) * g.ldqt + (int64_t)h * g.ldqh + q4 * (D / 4);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) qf[n][j] = ldg16(p + 8 * j);
    const int pos = w.s.len - w.s.n + i;
    row_end[n] = !live ? 0 : g.causal ? std::min(v.end, pos + 1) : v.end;
    row_begin[n] = window_begin(g, pos);
  }

  const float ks0 = score_scale<SCHEME>(g);
  v4f o[NQ][JD];
  float m[NQ], l[NQ], le[NQ];   // le: bf16 caches, weights before their rounding
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = -INFINITY;
    l[n] = le[n] = 0.0f;
#pragma unroll
    for (int j = 0; j < JD; ++j) o[n][j] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  for (; key < key_last; key += 128) {
    const bool more = key + 128 < key_last;
#pragma unroll
    for (int t = 0; t < 2; ++t) x.held[t] = x.next_held[t];
    if (more) x.find(g, w.b, hk, key + 128);
    // scores of 32 keys: lane (c, q4) has row c's keys 16 t + 4 q4 + i
    float s[NQ][8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      v4f acc[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) acc[n] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        uint4 kf;
        if constexpr (SCHEME == kKvBf16) kf = x.k[t][j];
        else kf = bf16x8_of((j & 1) ? make_uint2(x.k[t][j >> 1].z, x.k[t][j >> 1].w)
                                    : make_uint2(x.k[t][j >> 1].x, x.k[t][j >> 1].y));
#pragma unroll
        for (int n = 0; n < NQ; ++n)
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, kf), __builtin_bit_cast(v8bf, qf[n][j]),
                                                           acc[n], 0, 0, 0);
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][4 * t + i] = acc[n][i];
    }
    float rv[8];
    bool slight = false;   // any such key
    if constexpr (SCHEME == kKvRow) {
      // every lane prepares one of the eight keys that its row of 16 lanes has, and they read each other's
      const float k1 = x.ks * ks0;
      float l1, r1;
      value_scale(x.vs, l1, r1);
      float kk[8], lv[8];
      row_lanes8(k1, kk);
      row_lanes8(l1, lv);
      row_lanes8(r1, rv);
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[n][i] = __builtin_fmaf(s[n][i], kk[i], lv[i]);
      slight = __any(x.vs == 1.0f || x.vs < kSmallestValueScale);
      if (slight) {
        asm volatile("");   // a branch
        row_lanes8(x.vs < kSmallestValueScale ? share_log(x.vs) : r1, rv);
        uint32_t some = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < VW; ++j) some |= magnitude(x.v[i][j]) ? 1u << i : 0u;
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) some |= __shfl_xor(some, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool zero = rv[i] == 1.0f && !(some >> i & 1);
          if (zero) rv[i] = kNoShare;
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[n][i] += zero ? kSmallestLog : 0.0f;
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[n][i] *= ks0;
    }
    // the next step's keys come into the registers of this one's, which are done with
    if (more) {
      x.load_k(g, lane);
      x.load_scales(g, lane);
    }
    // Keys that some rows do not see: their scores go, and values that are not finite are taken out of the
    // product (0 times them is not 0) and make the scores of rows that do see them NaN.
    const bool edge = key < v.all_begin || key + 32 > v.all_end || !x.held[0] || !x.held[1];
    if (edge) {
      asm volatile("");   // a branch: without it much of this is done for every step
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bool b = false;
#pragma unroll
        for (int j = 0; j < VW; ++j) b |= bad_word<SCHEME>(x.v[i][j]);
        bad |= (uint32_t)b << i;
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) bad |= __shfl_xor(bad, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool is_bad = (bad >> i) & 1;
#pragma unroll
        for (int j = 0; j < VW; ++j) x.v[i][j] = is_bad ? 0u : x.v[i][j];
        const int at = key + 16 * (i >> 2) + 4 * q4 + (i & 3);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const bool seen = x.held[i >> 2] && at < row_end[n] && at >= row_begin[n];
          s[n][i] = !seen ? -INFINITY : is_bad ? NAN : s[n][i];
        }
        if constexpr (SCHEME == kKvRow) rv[i] = rv[i] == rv[i] ? rv[i] : 1.0f;   // such a scale's score is NaN where seen
      }
    }
    uint4 wf[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = s[n][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, s[n][i]);
      top = max32(max16(top));
      if (__any(top > m[n] + kRise)) {
        const float next = top > m[n] + kRise ? top : m[n];
        const Factor f = next == m[n] ? Factor{1.0f, 1.0f} : factor_of<SCHEME>(m[n] - next);
        const float a = f.whole();
        m[n] = next;
        l[n] = l[n] * f.a * f.b;
        le[n] *= a;
#pragma unroll
        for (int j = 0; j < JD; ++j) o[n][j] *= a;
      }
      const float base = m[n] == -INFINITY ? 0.0f : m[n] - weight_shift<SCHEME>();
      if constexpr (SCHEME == kKvRow) {
        if (slight) {
          asm volatile("");   // a branch
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (rv[i] < 0.0f) {
              l[n] += __builtin_amdgcn_exp2f(s[n][i] - kSmallestLog - base);
              s[n][i] += rv[i];
            }
        }
      }
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f(s[n][i] - base);
      if (SCHEME == kKvBf16 && g.lse)
        le[n] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      wf[n] = make_uint4(pack_weights<SCHEME>(e[0], e[1]), pack_weights<SCHEME>(e[2], e[3]),
                         pack_weights<SCHEME>(e[4], e[5]), pack_weights<SCHEME>(e[6], e[7]));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (SCHEME == kKvRow) l[n] = __builtin_fmaf(e[i], rv[i], l[n]);
        else l[n] += e[i];
      }
    }
    // values: eight keys of D / 16 values each, transposed four by four
#pragma unroll
    for (int u = 0; u < JD / 4; ++u) {
      uint4 vf[4];
      if constexpr (SCHEME == kKvBf16) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 2 * u + e;
          vf[2 * e] = make_uint4(low16s(x.v[0][j], x.v[1][j]), low16s(x.v[2][j], x.v[3][j]),
                                 low16s(x.v[4][j], x.v[5][j]), low16s(x.v[6][j], x.v[7][j]));
          vf[2 * e + 1] = make_uint4(high16s(x.v[0][j], x.v[1][j]), high16s(x.v[2][j], x.v[3][j]),
                                     high16s(x.v[4][j], x.v[5][j]), high16s(x.v[6][j], x.v[7][j]));
        }
      } else {
        const uint32_t a[4] = {x.v[0][u], x.v[1][u], x.v[2][u], x.v[3][u]};
        const uint32_t b[4] = {x.v[4][u], x.v[5][u], x.v[6][u], x.v[7][u]};
        uint32_t ta[4], tb[4];
        transpose4(a, ta);
        transpose4(b, tb);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vf[e] = make_uint4(f16x2_of(ta[e], false), f16x2_of(ta[e], true), f16x2_of(tb[e], false), f16x2_of(tb[e], true));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int n = 0; n < NQ; ++n) o[n][4 * u + e] = mfma16_pv<SCHEME>(vf[e], wf[n], o[n][4 * u + e]);
    }
    if (more) x.load_v(g, lane);
  }

  // join the four waves, 16 rows at a time: lane (c, q4) holds row c's values (4 q4 + i) D / 16 + j
  constexpr int TR = D / 8, RP = 256 / TR;   // threads per row, rows at a time
  const int tr = threadIdx.x % TR, r0 = threadIdx.x / TR;
  const float fin = final_scale<SCHEME>(g);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (n > 0) __syncthreads();
    l[n] = add32(add16(l[n]));
    le[n] = add32(add16(le[n]));
    if (q4 == 0) {
      sm[wave][c] = m[n];
      sl[wave][c] = l[n];
      se[wave][c] = le[n];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < JD; j += 4)
        *reinterpret_cast<float4*>(&so[wave][c][(4 * q4 + i) * JD + j]) =
            make_float4(o[n][j][i], o[n][j + 1][i], o[n][j + 2][i], o[n][j + 3][i]);
    __syncthreads();
    for (int r = r0; r < 16 && r0 < RP; r += RP) {
      const int row = w.tile * BM + 16 * n + r;
      if (row >= rows) break;
      const float top = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.0f, exact = 0.0f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const Factor by = join_factor<SCHEME>(sm[x][r], sl[x][r], top);
        const float f = by.whole();
        sum = __builtin_fmaf(sl[x][r] * by.b, by.a, sum);
        exact = __builtin_fmaf(f, se[x][r], exact);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(f, so[x][r][8 * tr + e], acc[e]);
      }
      if (mine == 1) {
        store_row<SCHEME>(g, w.s, row, hk, 8 * tr, acc, top, sum, exact, fin);
      } else if (w.part < (uint32_t)g.parts) {
        float* p = part_sums(g, BM, D, hk, w.part, 16 * n + r) + 8 * tr;
        *reinterpret_cast<float4*>(p) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (tr == 0) *part_ml(g, BM, D, hk, w.part, 16 * n + r) = make_float4(top, sum, exact, 0.0f);
      }
    }
  }
}

// ---------------------------------------------------------------- many rows: key tiles through LDS
// Four waves of 32 rows, 32 x 32 x 16 matrix instructions.  A tile of 64 keys (32 where a head has more than 128
// values) is read into registers one tile ahead, turned into 16-bit operands once for all four waves on its
// way to LDS (values transposed, so that a fragment of either operand is one 16-byte read), and
// double-buffered: one barrier per tile.
//
// Bound by what lies between the products: 8192 new tokens over 32768, 32 heads of 128, run at 800 to 850 TFLOP/s
// (4.53 to 4.82 ms from card to card), three quarters of a large bf16 library product.
// Vector instructions issue 53 % of the time, LDS is busy 50 % (bank conflicts 9 %), the matrix cores 36 %; copies that
// leave a step out are faster by 22 % (staging; its stores to LDS alone 11), 18 (the second product) and 6 (the
// exponentials).  32 rows per wave, because O, q and a tile's
// scores for 64 do not fit in registers beside the loads (spills: slower), and four waves, because eight on a tile of
// 256 rows leave one workgroup per CU (five chunks of 300: 103 -> 121 us).
template <int SCHEME, int D>
struct KeyTile {
  static constexpr int NT = 256;                              // threads
  static constexpr int KT = D <= 128 ? 64 : 32;
  static constexpr int EB = SCHEME == kKvBf16 ? 2 : 1;
  static constexpr int PK = D * EB / 16;                      // 16-byte pieces of a key
  static constexpr int NK = (KT * PK + NT - 1) / NT;            // pieces per thread
  static constexpr int UV = KT / 4 * (D / 4);                 // units of 4 keys x 4 values
  static constexpr int NV = (UV + NT - 1) / NT;
  static constexpr int kBytes = KT * D * 2;                   // of one operand in LDS

  uint4 k[NK];
  uint2 v[NV][4];                                             // FP8: .x alone
  float ks, vs;                                               // of key threadIdx.x, in `row` of the cache
  int64_t row;

  static __device__ __forceinline__ int v_dq(int e) { return e % (D / 4); }
  // Units 2 apart in a group of four keys' order lie in the two halves of a 16-byte chunk: lanes of a wave
  // write both.
  static __device__ __forceinline__ int v_kg(int e) {
    const int i = e / (D / 4);
    return (i & ~3) | ((i & 1) << 1) | ((i >> 1) & 1);
  }

  // Lane i's page of the tile's keys 16 i .. 16 i + 15 (page 0, and a bit off in `held`, where the cache has none).
  int page;
  uint32_t held;
  __device__ __forceinline__ void find(const AttendArgs& g, int b, int key) {
    const int i = threadIdx.x & (KT / 16 - 1);
    const int p = (key + 16 * i) >> g.page_shift, last_page = (int)g.width - 1;
    const int at = g.pages[b * g.ldp + std::min(p, last_page)];
    const bool there = at >= 0 && at < g.n_pages && p <= last_page;
    page = there ? at : 0;
    held = (uint32_t)__ballot(there) & ((1u << (KT / 16)) - 1);
  }
  // Bytes from the head's first value in page 0 to the tile's key 16 i, i the group of 16 keys that r lies in.  A
  // wave's piece or unit falls into one such group for all of its lanes, at every head size, so this is a
  // scalar.  A page of all heads is below 2^31 bytes.
  __device__ __forceinline__ uint64_t at(const AttendArgs& g, int key, int r) const {
    const int i = __builtin_amdgcn_readfirstlane(r >> 4);
    const uint32_t p = (uint32_t)__builtin_amdgcn_readlane(page, i);
    const uint32_t page_bytes = ((uint32_t)g.Hk << g.page_shift) * (uint32_t)(D * EB);
    return (uint64_t)p * page_bytes + (uint32_t)((key + 16 * i) & ((1 << g.page_shift) - 1)) * (uint32_t)(D * EB);
  }
  // Codes of one byte at 64 or 128 values: a thread's pieces of keys and units of values are of the same 16 keys.
  static constexpr bool kSameGroup = EB == 1 && D <= 128;

  __device__ __forceinline__ void load(const AttendArgs& g, int hk, int key) {
    const int t = threadIdx.x;
    const uint64_t head = ((uint64_t)hk << g.page_shift) * (D * EB);
    const uint8_t* kp = static_cast<const uint8_t*>(g.k_codes) + head;
    const uint8_t* vp = static_cast<const uint8_t*>(g.v_codes) + head;
    uint64_t from[NK];
#pragma unroll
    for (int u = 0; u < NK; ++u) {
      const int e = t + NT * u;
      if (KT * PK % NT == 0 || e < KT * PK) {
        from[u] = at(g, key, e / PK);
        k[u] = ldg16(kp + from[u] + (uint32_t)((e / PK & 15) * (D * EB) + (e % PK) * 16));
      }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int e = t + NT * u;
      if (UV % NT == 0 || e < UV) {
        const int r = 4 * v_kg(e);
        const uint8_t* q = vp + (kSameGroup ? from[u] : at(g, key, r)) + (uint32_t)((r & 15) * (D * EB) + v_dq(e) * (4 * EB));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (SCHEME == kKvBf16) v[u][i] = *reinterpret_cast<const uint2*>(q + i * (D * EB));
          else v[u][i].x = *reinterpret_cast<const uint32_t*>(q + i * (D * EB));
        }
      }
    }
    if constexpr (SCHEME == kKvRow) {
      if (t < KT) {
        row = (((int64_t)__shfl(page, t >> 4) * g.Hk + hk) << g.page_shift) + ((key + t) & ((1 << g.page_shift) - 1));
        ks = g.k_scales[row];
        vs = g.v_scales[row];
      }
    }
  }

  // Where 16-byte chunk c (8 values) of key r lies, and 4 keys x 1 value of the transposed values: chosen so that
  // 16 lanes that read one chunk of consecutive rows meet all 64 banks.
  static __device__ __forceinline__ int k_at(int r, int c) {
    return r * (D * 2) + ((D % 128 == 0 ? c ^ (r & 15) : c ^ ((r >> 1) & 7)) << 4);
  }
  static __device__ __forceinline__ int v_row(int d) { return d * (KT * 2); }
  static __device__ __forceinline__ int v_swizzle(int d) {
    return KT == 64 ? ((d >> 1) & 7) ^ ((d >> 4) & 1) : (d >> 2) & 3;
  }
  static __device__ __forceinline__ int v_at(int d, int kg) {
    return v_row(d) + (((2 * (kg >> 2) + (kg & 1)) ^ v_swizzle(d)) << 4) + ((kg >> 1) & 1) * 8;
  }

  // A thread's places in LDS: k0 of its first piece, v0 of its first unit.  Up to 128 values the others follow
  // from these: the next piece is whole periods of the swizzle of rows further, the second half of a piece, the
  // next two values of a unit and the next unit differ in one bit of the chunk.
  static constexpr bool kNear = D <= 128;
  static __device__ __forceinline__ int k_first() { return k_at(threadIdx.x / PK, (threadIdx.x % PK) * (2 / EB)); }
  static __device__ __forceinline__ int v_first() { return v_at(4 * v_dq(threadIdx.x), v_kg(threadIdx.x)); }
  __device__ __forceinline__ void store_k(uint8_t* kl, int k0) const {
    const int t = threadIdx.x;
#pragma unroll
    for (int u = 0; u < NK; ++u) {
      const int e = t + NT * u;
      if (KT * PK % NT == 0 || e < KT * PK) {
        const int r = e / PK, c = (e % PK) * (2 / EB);
        const int at = kNear ? k0 + u * (NT / PK) * (D * 2) : k_at(r, c);
        if constexpr (SCHEME == kKvBf16) {
          stg16(kl + at, k[u]);
        } else {
          stg16(kl + at, bf16x8_of(make_uint2(k[u].x, k[u].y)));
          stg16(kl + (kNear ? (k0 ^ 16) + u * (NT / PK) * (D * 2) : k_at(r, c + 1)), bf16x8_of(make_uint2(k[u].z, k[u].w)));
        }
      }
    }
  }
  // Values that are not finite are taken out, and their key is marked with the tile's number (a tile of which
  // some row does not see every key: 0 times such a value is not 0).
  __device__ __forceinline__ void clean_v(int* marks, int number) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int e = threadIdx.x + NT * u;
      if (UV % NT == 0 || e < UV) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bool bad = bad_word<SCHEME>(v[u][i].x);
          if constexpr (SCHEME == kKvBf16) bad |= bad_word<SCHEME>(v[u][i].y);
          if (bad) {
            v[u][i] = make_uint2(0u, 0u);
            marks[4 * v_kg(e) + i] = number;
          }
        }
      }
    }
  }
  __device__ __forceinline__ void store_v(const AttendArgs& g, uint8_t* vl, int v0, float* params, float ks0, int* slight,
                                          int number) const {
    const int t = threadIdx.x;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int e = t + NT * u;
      if (UV % NT == 0 || e < UV) {
        const int d0 = 4 * v_dq(e), kg = v_kg(e);
        uint2 out[4];
        if constexpr (SCHEME == kKvBf16) {
          out[0] = make_uint2(low16s(v[u][0].x, v[u][1].x), low16s(v[u][2].x, v[u][3].x));
          out[1] = make_uint2(high16s(v[u][0].x, v[u][1].x), high16s(v[u][2].x, v[u][3].x));
          out[2] = make_uint2(low16s(v[u][0].y, v[u][1].y), low16s(v[u][2].y, v[u][3].y));
          out[3] = make_uint2(high16s(v[u][0].y, v[u][1].y), high16s(v[u][2].y, v[u][3].y));
        } else {
          const uint32_t a[4] = {v[u][0].x, v[u][1].x, v[u][2].x, v[u][3].x};
          uint32_t ta[4];
          transpose4(a, ta);
#pragma unroll
          for (int i = 0; i < 4; ++i) out[i] = make_uint2(f16x2_of(ta[i], false), f16x2_of(ta[i], true));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)   // at 128 values the next unit is 8 groups of keys on: 4 chunks
          stg8(vl + (kNear ? (v0 ^ ((i >> 1) << 4 | u << 6)) + i * (KT * 2) : v_at(d0 + i, kg)), out[i]);
      }
    }
    if constexpr (SCHEME == kKvRow) {
      if (t < KT) {
        float lv, rv;
        value_scale(vs, lv, rv);
        if (vs < kSmallestValueScale) {
          rv = share_log(vs);
          *slight = number;
        }
        if (vs == 1.0f) {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(g.v_codes) + row * D);
          uint32_t some = 0;
          for (int i = 0; i < D / 16; ++i) some |= magnitude(p[i].x | p[i].y | p[i].z | p[i].w);
          if (!some) {
            lv = kSmallestLog;
            rv = kNoShare;
            *slight = number;
          }
        }
        params[t] = ks * ks0;
        params[KT + t] = lv;
        params[2 * KT + t] = rv == rv ? rv : 1.0f;   // such a scale's score is NaN where seen
      }
    }
  }
};

// Workgroups per CU.  192 values with a scale per token spill 12 registers at two, and one is slower still (4096 new
// tokens over 8192, 16 heads: 763 | 871 us; 512 over 16384: 223 | 313).  64 values of FP8 left alone take one register too many for three.
template <int SCHEME, int D>
constexpr int tile_waves() { return D == 64 && SCHEME != kKvBf16 ? 3 : D <= 192 ? 2 : 1; }

template <int SCHEME, int D>
__global__ __launch_bounds__(256, (tile_waves<SCHEME, D>())) void k_attend_tile(AttendArgs g) {
  typedef KeyTile<SCHEME, D> Tile;
  constexpr int BM = 128, KT = Tile::KT, NB = KT / 32, ND = D / 32;
  __shared__ __align__(16) uint8_t lds_k[2][Tile::kBytes];
  __shared__ __align__(16) uint8_t lds_v[2][Tile::kBytes];
  __shared__ __align__(16) float params[2][SCHEME == kKvRow ? 3 * KT : 4];
  __shared__ __align__(16) int marks[2][KT + 4];   // tile numbers: of a key with values that are not finite; [KT], of any slight key
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, h2 = lane >> 5;
  const int hk = (int)(blockIdx.x % (uint32_t)g.Hk);
  Work w;
  if (!find_work<BM, false>(g, blockIdx.x / (uint32_t)g.Hk, w)) return;
  const Sight v = sight_of<BM>(g, w.s, w.tile);
  const int mine = splits_of(v.kt1 - v.kt0, w.chunk);
  if (w.split >= mine) return;
  const int kt_first = v.kt0 + w.split * w.chunk;
  const int kt_last = mine > 1 ? std::min(v.kt1, kt_first + w.chunk) : v.kt1;
  const int G = g.H / g.Hk;
  const int rows = w.s.n * G;

  const int row = w.tile * BM + 32 * wave + c;
  const bool live = row < rows;
  const bool wave_live = w.tile * BM + 32 * wave < rows;
  const int i = live ? row / G : 0, h = live ? hk * G + (row - i * G) : 0;
  uint4 qf[D / 16];
  {
    const uint16_t* p = g.q + (int64_t)(w.s.first + i) * g.ldqt + (int64_t)h * g.ldqh + 8 * h2;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) qf[j] = ldg16(p + 16 * j);
  }
  const int pos = w.s.len - w.s.n + i;
  const int row_end = !live ? 0 : g.causal ? std::min(v.end, pos + 1) : v.end;
  const int row_begin = window_begin(g, pos);
  // the last key that any row of this wave sees, and the first
  const int last = std::min(rows, w.tile * BM + 32 * wave + 32) - 1;
  const int wave_end = g.causal ? std::min(v.end, w.s.len - w.s.n + last / G + 1) : v.end;
  const int wave_begin = window_begin(g, w.s.len - w.s.n + (w.tile * BM + 32 * wave) / G);

  const float ks0 = score_scale<SCHEME>(g);
  v16f o[ND];
#pragma unroll
  for (int j = 0; j < ND; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[j][r] = 0.0f;
  float m = -INFINITY, l = 0.0f, le = 0.0f;   // le: bf16 caches, weights before their rounding

  const int key_first = kt_first * kKeyTile;
  const int key_last = std::min(kt_last * kKeyTile, (v.end + KT - 1) / KT * KT);
  const int tiles = key_last > key_first ? (key_last - key_first) / KT : 0;
  auto is_edge = [&](int key, uint32_t held) {
    return key < v.all_begin || key + KT > v.all_end || held != (1u << (KT / 16)) - 1;
  };
  if (threadIdx.x <= KT) marks[0][threadIdx.x] = marks[1][threadIdx.x] = -1;
  __syncthreads();
  Tile next;
  uint32_t held = 0, held_next = 0;
  const int k0 = Tile::k_first(), v0 = Tile::v_first();
  auto put = [&](int x, int key) {   // the registers' tile x to LDS
    if (is_edge(key, held_next)) next.clean_v(marks[x & 1], x);
    next.store_k(lds_k[x & 1], k0);
    next.store_v(g, lds_v[x & 1], v0, params[x & 1], ks0, &marks[x & 1][KT], x);
  };
  auto get = [&](int key) {          // the tile at `key` to the registers, and the pages of the one behind it
    next.load(g, hk, key);
    held_next = next.held;
    next.find(g, w.b, std::min(key + KT, key_last - KT));
  };
  if (tiles > 0) {
    next.find(g, w.b, key_first);
    get(key_first);
    held = held_next;
    put(0, key_first);
    if (tiles > 1) get(key_first + KT);
  }
  const int k_lane = Tile::k_at(c, h2);            // key c's chunk h2; chunk 2 j + h2 is an exclusive or away
  constexpr int kGroup = D % 128 == 0 ? 8 : 4;     // fragments whose chunks the swizzle permutes among themselves
  for (int x = 0; x < tiles; ++x) {
    __syncthreads();
    const int buf = x & 1;
    const int key = key_first + x * KT;
    const bool edge = is_edge(key, held);
    const uint32_t held_now = held;
    if (x + 1 < tiles) {
      held = held_next;
      put(x + 1, key + KT);
      if (x + 2 < tiles) get(key + 2 * KT);
    }
    if (!wave_live || key >= wave_end || key + KT <= wave_begin) continue;
    const uint8_t* kl = lds_k[buf];
    const uint8_t* vl = lds_v[buf];
    v16f s[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[b][r] = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 kf = ldg16(kl + b * 32 * (D * 2) + j / kGroup * (32 * kGroup) + (k_lane ^ (j % kGroup << 5)));
        s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, kf), __builtin_bit_cast(v8bf, qf[j]), s[b],
                                                       0, 0, 0);
      }
    // lane (c, h2) has row c's keys 32 b + 8 (r / 4) + 4 h2 + r % 4
    const float* pr = params[buf];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if constexpr (SCHEME == kKvRow) {
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const float4 k4 = *reinterpret_cast<const float4*>(pr + 32 * b + 2 * r + 4 * h2);
          const float4 l4 = *reinterpret_cast<const float4*>(pr + KT + 32 * b + 2 * r + 4 * h2);
          s[b][r] = __builtin_fmaf(s[b][r], k4.x, l4.x);
          s[b][r + 1] = __builtin_fmaf(s[b][r + 1], k4.y, l4.y);
          s[b][r + 2] = __builtin_fmaf(s[b][r + 2], k4.z, l4.z);
          s[b][r + 3] = __builtin_fmaf(s[b][r + 3], k4.w, l4.w);
        }
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[b][r] *= ks0;
      }
    }
    if (edge) {
      asm volatile("");   // a branch
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int kk = 32 * b + 8 * (r >> 2) + 4 * h2 + (r & 3);
          const bool seen = ((held_now >> (2 * b + (r >> 3))) & 1) && key + kk < row_end && key + kk >= row_begin;
          s[b][r] = !seen ? -INFINITY : marks[buf][kk] == x ? NAN : s[b][r];
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
    top = max32(top);
    if (__any(top > m + kRise)) {
      const float nm = top > m + kRise ? top : m;
      const Factor f = nm == m ? Factor{1.0f, 1.0f} : factor_of<SCHEME>(m - nm);
      const float a = f.whole();
      m = nm;
      l = l * f.a * f.b;
      le *= a;
#pragma unroll
      for (int j = 0; j < ND; ++j) o[j] *= a;
    }
    const float base = m == -INFINITY ? 0.0f : m - weight_shift<SCHEME>();
    uint4 wf[2 * NB];
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (SCHEME == kKvRow && marks[buf][KT] == x) {
      asm volatile("");   // a branch
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (const float log = pr[2 * KT + 32 * b + 8 * (r >> 2) + 4 * h2 + (r & 3)]; log < 0.0f) {
            sum[r & 3] += __builtin_amdgcn_exp2f(s[b][r] - kSmallestLog - base);
            s[b][r] += log;
          }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[b][r] = __builtin_amdgcn_exp2f(s[b][r] - base);
      if (SCHEME == kKvBf16 && g.lse) {
        float e = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) e += s[b][r];
        le += e;
      }
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a0 = s[b][8 * f + 2 * e], a1 = s[b][8 * f + 2 * e + 1];
          p[e] = pack_weights<SCHEME>(a0, a1);
          if constexpr (SCHEME == kKvBf16) {
            s[b][8 * f + 2 * e] = a0;
            s[b][8 * f + 2 * e + 1] = a1;
          }
        }
        wf[2 * b + f] = make_uint4(p[0], p[1], p[2], p[3]);
      }
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        if constexpr (SCHEME == kKvRow) {
          const float4 r4 = *reinterpret_cast<const float4*>(pr + 2 * KT + 32 * b + 2 * r + 4 * h2);
          sum[0] = __builtin_fmaf(s[b][r], r4.x, sum[0]);
          sum[1] = __builtin_fmaf(s[b][r + 1], r4.y, sum[1]);
          sum[2] = __builtin_fmaf(s[b][r + 2], r4.z, sum[2]);
          sum[3] = __builtin_fmaf(s[b][r + 3], r4.w, sum[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] += s[b][r + e];
        }
      }
    }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
    for (int f = 0; f < 2 * NB; ++f)
#pragma unroll
      for (int j = 0; j < ND; ++j) {
        const int d = 32 * j + c;
        const uint4 vf = ldg16(vl + Tile::v_row(d) + (((2 * f + h2) ^ Tile::v_swizzle(d)) << 4));
        o[j] = mfma32_pv<SCHEME>(vf, wf[f], o[j]);
      }
  }

  // lane (c, h2) has row c's values 32 j + 8 (r / 4) + 4 h2 + r % 4
  l = add32(l);
  le = add32(le);
  if (mine > 1) {
    if (!live || w.part >= (uint32_t)g.parts) return;
    const int r_in = 32 * wave + c;
    float* p = part_sums(g, BM, D, hk, w.part, r_in);
#pragma unroll
    for (int j = 0; j < ND; ++j)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4*>(p + 32 * j + 2 * r + 4 * h2) = make_float4(o[j][r], o[j][r + 1], o[j][r + 2], o[j][r + 3]);
    if (h2 == 0) *part_ml(g, BM, D, hk, w.part, r_in) = make_float4(m, l, le, 0.0f);
    return;
  }
  const float f = l == 0.0f ? 0.0f : final_scale<SCHEME>(g) / l;
  const int64_t t = w.s.first + i;
  uint16_t* out = g.out + t * g.ldot + (int64_t)h * g.ldoh;
#pragma unroll
  for (int j = 0; j < ND; ++j)
#pragma unroll
    for (int r = 0; r < 16; r += 8) {
      // lanes c and c + 32 exchange, so that each has 8 consecutive values
      const auto lo = __builtin_amdgcn_permlane32_swap(gemm::pack_bf16x2(o[j][r] * f, o[j][r + 1] * f),
                                                       gemm::pack_bf16x2(o[j][r + 4] * f, o[j][r + 5] * f), false, false);
      const auto hi = __builtin_amdgcn_permlane32_swap(gemm::pack_bf16x2(o[j][r + 2] * f, o[j][r + 3] * f),
                                                       gemm::pack_bf16x2(o[j][r + 6] * f, o[j][r + 7] * f), false, false);
      if (live) stg16(out + 32 * j + 2 * r + 8 * h2, make_uint4(lo[0], hi[0], lo[1], hi[1]));
    }
  if (g.lse && live && h2 == 0) g.lse[t * g.H + h] = lse_of<SCHEME>(m, SCHEME == kKvBf16 ? le : l);
}

// ---------------------------------------------------------------- join
// The rows of a tile whose keys were cut into several ranges: the ranges' sums, each at its own maximum.  RW
// rows per workgroup; the threads of a row, D / 8 across, share its ranges out among them and meet in LDS, four
// ranges in flight each.  Bound by latency: 4.5 us for one token's heads, 7.5 for 64 sequences, 9 for five chunks of 300.
template <int SCHEME, int BM, int D, int RW>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs g) {
  constexpr int TR = D / 8, NG = 256 / TR / RW;   // groups of threads per row
  constexpr int U = 4;                                                    // ranges in flight
  __shared__ float so[RW][NG][D + 4];
  __shared__ float sm[RW][NG], sl[RW][NG], se[RW][NG];
  const int hk = (int)(blockIdx.x % (uint32_t)g.Hk);
  Work w;
  if (!find_work<BM, true>(g, blockIdx.x / (uint32_t)g.Hk, w)) return;
  const int rows = w.s.n * (g.H / g.Hk), r_first = (int)blockIdx.y * RW;
  if (w.tile * BM + r_first >= rows) return;
  const Sight v = sight_of<BM>(g, w.s, w.tile);
  const int mine = splits_of(v.kt1 - v.kt0, w.chunk);
  if (mine < 2 || (uint64_t)w.part + (uint64_t)mine > (uint64_t)g.parts) return;
  const int tr = (int)(threadIdx.x % TR), group = (int)(threadIdx.x / TR) % NG, ri = (int)(threadIdx.x / (TR * NG));
  const int r = r_first + ri, row = w.tile * BM + r;
  const bool live = ri < RW && row < rows;
  if (live) {
    const float4* ml = part_ml(g, BM, D, hk, w.part, r);
    const float* sums = part_sums(g, BM, D, hk, w.part, r) + 8 * tr;
    float top = -INFINITY;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.0f, exact = 0.0f;
    for (int x0 = group; x0 < mine; x0 += NG * U) {
      float4 p[U], a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = (int64_t)std::min(x0 + u * NG, mine - 1) * BM;
        p[u] = ml[at];
        a[u] = *reinterpret_cast<const float4*>(sums + at * D);
        b[u] = *reinterpret_cast<const float4*>(sums + at * D + 4);
      }
      float next = top;
#pragma unroll
      for (int u = 0; u < U; ++u) next = fmaxf(next, x0 + u * NG < mine ? p[u].x : -INFINITY);
      const Factor by = join_factor<SCHEME>(top, sum, next);
      const float old = by.whole();
      top = next;
      sum = sum * by.b * by.a;
      exact *= old;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= old;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (x0 + u * NG >= mine) break;
        const Factor by = join_factor<SCHEME>(p[u].x, p[u].y, top);
        const float f = by.whole();
        sum = __builtin_fmaf(p[u].y * by.b, by.a, sum);
        exact = __builtin_fmaf(f, p[u].z, exact);
        acc[0] = __builtin_fmaf(f, a[u].x, acc[0]);
        acc[1] = __builtin_fmaf(f, a[u].y, acc[1]);
        acc[2] = __builtin_fmaf(f, a[u].z, acc[2]);
        acc[3] = __builtin_fmaf(f, a[u].w, acc[3]);
        acc[4] = __builtin_fmaf(f, b[u].x, acc[4]);
        acc[5] = __builtin_fmaf(f, b[u].y, acc[5]);
        acc[6] = __builtin_fmaf(f, b[u].z, acc[6]);
        acc[7] = __builtin_fmaf(f, b[u].w, acc[7]);
      }
    }
    if (tr == 0) {
      sm[ri][group] = top;
      sl[ri][group] = sum;
      se[ri][group] = exact;
    }
    *reinterpret_cast<float4*>(&so[ri][group][8 * tr]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    *reinterpret_cast<float4*>(&so[ri][group][8 * tr + 4]) = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  __syncthreads();
  if (!live || group != 0) return;
  float top = -INFINITY;
  for (int x = 0; x < NG; ++x) top = fmaxf(top, sm[ri][x]);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.0f, exact = 0.0f;
  for (int x = 0; x < NG; ++x) {
    const Factor by = join_factor<SCHEME>(sm[ri][x], sl[ri][x], top);
    const float f = by.whole();
    sum = __builtin_fmaf(sl[ri][x] * by.b, by.a, sum);
    exact = __builtin_fmaf(f, se[ri][x], exact);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(f, so[ri][x][8 * tr + e], acc[e]);
  }
  store_row<SCHEME>(g, w.s, row, hk, 8 * tr, acc, top, sum, exact, final_scale<SCHEME>(g));
}

// ---------------------------------------------------------------- choice and launch
// The choices, by what the host knows (sizes, not lengths).  us, codes with a scale per token, G = 4, Hk = 8.
//
// Rows per tile by the mean rows of a sequence's head.  The three kernels at 128 head values
// (16 | 32 | 128 rows per tile):
//   32 sequences over 8192, rows 16: 79 | 86 | 125, 32: 90 | 90 | 127, 48: 99 | 100 | 138, 64: 114 | 114 | 138,
//   128: 175 | 149 | 147;   8 sequences, 64: 44 | 35 | 46, 128: 71 | 65 | 51, 256: 110 | 99 | 64;
//   1 over 16384, 64: 29 | 26 | 41, 128: 40 | 35 | 44, 256: 63 | 49 | 48.
// 64 values are alike (8 sequences, 64: 29 | 29 | 36, 128: 53 | 44 | 40).  At 192 and 256 values the many-row
// kernel has half the waves or half the key tile (256 values, 8 sequences, 64 rows: 78 | 81 | 141, 128:
// 124 | 113 | 149, 256: 203 | 174 | 199), so that few rows reach further there; up to 128 rows, because many
// short contexts, which the host can not tell, want tiles of 128 earlier (32 of 600 tokens, bf16, 128 rows: 86 |
// 81 | 62).  The mean serves a batch of like sequences: a chunk of 2048 beside 60 single tokens over 8192 takes tiles of 128
// for all, 642 us where two calls take 210 + 337, one of 256 beside them tiles of 16 for all, 305 for 210 + 63.
struct Plan {
  int bm;
  int target, min_chunk;
  int64_t tiles, parts;   // bounds, per head of the cache
};

template <int NQ>
int stream_waves_of(const AttendArgs& g) {
  const bool bf16 = g.scheme == kKvBf16;
  switch (g.D) {
    case 64: return bf16 ? stream_waves<kKvBf16, 64, NQ>() : stream_waves<kKvRow, 64, NQ>();
    case 128: return bf16 ? stream_waves<kKvBf16, 128, NQ>() : stream_waves<kKvRow, 128, NQ>();
    case 192: return bf16 ? stream_waves<kKvBf16, 192, NQ>() : stream_waves<kKvRow, 192, NQ>();
    default: return bf16 ? stream_waves<kKvBf16, 256, NQ>() : stream_waves<kKvRow, 256, NQ>();
  }
}

Plan plan_of(const AttendArgs& g) {
  const int64_t rows = g.T * (g.H / g.Hk), seqs = std::max<int64_t>(1, std::min<int64_t>(g.B, g.T));
  const int64_t mean = (rows + seqs - 1) / seqs;
  Plan p;
  p.bm = mean <= (g.D <= 128 ? 32 : 64) ? 16 : mean <= (g.D <= 128 ? 64 : 128) ? 32 : 128;
  p.tiles = rows / p.bm + seqs;
  // Ranges in rounds of the workgroups that fit on the card: each row tile's last range is half a range short
  // on average, so that `target` full ones make target + tiles / 2.  Many rows: as few rounds as leave half of
  // the last one's ranges full (five chunks of 300: 96 -> 76 us), of 512 at every head size, though one workgroup per CU
  // fits at 256 values and three of FP8 at 64.  Rounds of 256 and 768 there: 256 values, 512 over 16384: 344 -> 327, 8 x 64
  // over 8192: 210 -> 196, uncut contexts level; 64 values, 5 x 300 over 12000: 170 -> 140, but 3 x 700 over 9000: 190 ->
  // 198, 32 x 128 over 2000: 84 -> 88.  Few rows: one round where few row tiles share
  // the card (one token over 131000, in ranges: 512: 64, 768: 63, 1024: 75), three where ranges of many
  // sequences have to even out (64 sequences up to 16384, 768: 157, 1536: 134, 2304: 129).
  //
  // The shortest range, in key tiles: few rows 4 (one token over 6007 in 2: 13.0, 4: 12.5, 8: 14.6).  Many rows 16,
  // or 8 where row tiles leave three quarters of the card idle (1 sequence over 16384, 128 rows of 64 values: 42 ->
  // 30; 32 of 600 tokens, 256 rows, not cut at 16: 34, cut at 8: 47; at 256 values 8 is no better).
  const int64_t all = std::max((rows + p.bm - 1) / p.bm, seqs) * g.Hk;   // row tiles, at least
  if (p.bm == 128) {
    constexpr int fit = 512;
    const int64_t rounds = (all / 2 + fit / 2 + fit - 1) / fit;
    p.target = (int)(rounds * fit - all / 2);
    p.min_chunk = 4 * all <= fit && g.D <= 192 ? 8 : 16;
  } else {
    const int fit = 256 * (p.bm == 16 ? stream_waves_of<1>(g) : stream_waves_of<2>(g));
    p.target = all * 4 <= fit ? fit - (int)all / 2 : (int)std::max<int64_t>(fit, 3 * fit - all / 2);
    p.min_chunk = 4;
  }
  const int64_t key_tiles = ((g.width << g.page_shift) + kKeyTile - 1) / kKeyTile;
  p.parts = 0;
  if (key_tiles <= p.min_chunk) p.target = 0;
  else
    // A tile of kt > chunk key tiles has fewer than kt / chunk + 1 < 2 kt / chunk ranges, and chunk >= total Hk / target:
    // all tiles together fewer than 2 target / Hk.
    p.parts = std::min<int64_t>(2 * ((int64_t)p.target / g.Hk + 1), p.tiles * ((key_tiles + p.min_chunk - 1) / p.min_chunk));
  return p;
}

template <int SCHEME, int D>
hipError_t attend_with(AttendArgs& g, const Plan& p, hipStream_t st) {
  const dim3 grid((unsigned)((p.tiles + p.parts) * g.Hk));
  if (p.bm == 16) hipLaunchKernelGGL((k_attend_stream<SCHEME, D, 1>), grid, dim3(256), 0, st, g);
  else if (p.bm == 32) hipLaunchKernelGGL((k_attend_stream<SCHEME, D, 2>), grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL((k_attend_tile<SCHEME, D>), grid, dim3(256), 0, st, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.target == 0) return e;
  // Rows per workgroup of the join: 1 where there are few, for the most threads per row (one token over 60000, one
  // head: 33 -> 19 us), else 4 (256 sequences over 4096: 277 -> 241 with 4).
  const unsigned joins = (unsigned)(std::min(p.tiles, p.parts / 2 + 1) * g.Hk);
  constexpr int kRows = D <= 128 ? 16 : 8;
  if (p.bm == 128) hipLaunchKernelGGL((k_attend_join<SCHEME, 128, D, kRows>), dim3(joins, 128 / kRows), dim3(256), 0, st, g);
  else if (joins < 64 && p.bm == 16) hipLaunchKernelGGL((k_attend_join<SCHEME, 16, D, 1>), dim3(joins, 16), dim3(256), 0, st, g);
  else if (p.bm == 16) hipLaunchKernelGGL((k_attend_join<SCHEME, 16, D, 4>), dim3(joins, 4), dim3(256), 0, st, g);
  else if (joins < 64) hipLaunchKernelGGL((k_attend_join<SCHEME, 32, D, 1>), dim3(joins, 32), dim3(256), 0, st, g);
  else hipLaunchKernelGGL((k_attend_join<SCHEME, 32, D, 4>), dim3(joins, 8), dim3(256), 0, st, g);
  return hipGetLastError();
}

template <int SCHEME>
hipError_t attend_as(AttendArgs& g, const Plan& p, hipStream_t st) {
  if (g.D == 64) return attend_with<SCHEME, 64>(g, p, st);
  if (g.D == 128) return attend_with<SCHEME, 128>(g, p, st);
  return g.D == 192 ? attend_with<SCHEME, 192>(g, p, st) : attend_with<SCHEME, 256>(g, p, st);
}

}  // namespace

bool kv_attention_fits(const AttendArgs& g) {
  const Plan p = plan_of(g);
  return (p.tiles + p.parts) * g.Hk < (int64_t(1) << 24);   // a launch has at most 2^32 - 1 threads
}

size_t kv_attention_ws_bytes(const AttendArgs& g) {
  const Plan p = plan_of(g);
  return (size_t)p.parts * g.Hk * p.bm * (g.D + 4) * 4;
}

hipError_t launch_kv_attention(AttendArgs g, hipStream_t st) {
  const Plan p = plan_of(g);
  g.target = p.target;
  g.min_chunk = p.min_chunk;
  g.parts = (int)p.parts;
  if (g.scheme == kKvBf16) return attend_as<kKvBf16>(g, p, st);
  return g.scheme == kKvTensor ? attend_as<kKvTensor>(g, p, st) : attend_as<kKvRow>(g, p, st);
}

const char* kv_attention_kernel_name(const AttendArgs& g) {
  const Plan p = plan_of(g);
  if (p.target) return p.bm == 16 ? "k_attend_stream<16>+k_attend_join" : p.bm == 32 ? "k_attend_stream<32>+k_attend_join" : "k_attend_tile+k_attend_join";
  return p.bm == 16 ? "k_attend_stream<16>" : p.bm == 32 ? "k_attend_stream<32>" : "k_attend_tile";
}

}  // namespace pql
