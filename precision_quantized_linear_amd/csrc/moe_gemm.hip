// Grouped FP8 products of a mixture-of-experts layer, gfx950.
//
// C[p, n] = sum_k a_hat[row(p), k] w_hat[e(p), n, k] for the assignments p in expert order:
// offsets[e] .. offsets[e + 1] - 1 are expert e's, row(p) is the token of assignment order[p]
// (gather) or p itself.  FP8_BLOCK128: partial products of each 128-wide K-group promoted with
// s_a[row, g] s_w[e, n / 128, g] in fp32; FP8_ROW: one fp32 sum scaled by s_a[row] s_w[e, n].
//
// k_moe_stream: a workgroup owns 32 columns of one expert and walks the expert's rows (or every
// z-th pass over them) up to 64 at a time; the weight is streamed past them, as in the few-token qlinear kernels: 8 waves take the
// K-chunks (128 bytes) round-robin, feed 16x16x128 MFMAs straight from registers, and add
// their sums in LDS.  Bound by the weight stream.  With fewer assignments than experts the grid has one row of
// workgroups per assignment, and a workgroup finds the experts that have any by ballots over
// the offsets (a workgroup per expert would be mostly empty ones: 8 of 128 for one token).
// The first weight loads go out before the rows are looked up: they depend on the expert alone.
#include <algorithm>
#include <type_traits>

#include "gemm_common.hpp"
#include "moe_gemm.hpp"
#include "pql_device.hpp"
#include "pql_internal.hpp"

namespace pql {

namespace {

using namespace gemm;

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kCols = 32;

typedef float v4f_t __attribute__((ext_vector_type(4)));

// The expert of grid row `slot`: the slot-th with any assignment, or -1.
__device__ __forceinline__ int active_expert(const MoeGemmArgs& g, int slot, int lane) {
  int before = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int lo = 0, hi = 0;
    if (e0 + lane < g.E) expert_range(g, e0 + lane, lo, hi);
    const uint64_t any = __ballot(hi > lo);
    const int n = __popcll(any);
    if (slot < before + n) {   // the (slot - before)-th set bit
      const uint64_t rank_hit = __ballot((any >> lane & 1) && __popcll(any & ((uint64_t(1) << lane) - 1)) == slot - before);
      return e0 + __ffsll((unsigned long long)rank_hit) - 1;
    }
    before += n;
  }
  return -1;
}

// MAXB: row blocks of 16 a pass may take; EU: waves per SIMD the registers are kept to.  A wave has
// one K-chunk in flight at a time and many waves run instead: with two or three chunks per wave
// and half the waves the one-token case (8 experts, N = 2048, K = 4096) takes 14.4 and 15.9 us
// instead of 13.6, 37 tokens x 6 of 64 experts (N = 2816, K = 2048) 58 and 80 instead of 56.
template <bool ROW, int MAXB, int EU>
__global__ __launch_bounds__(kThreads, EU) void k_moe_stream(MoeGemmArgs g) {
  __shared__ float part[kWaves][MAXB * 16][kCols + 1];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int e = __builtin_amdgcn_readfirstlane((int)gridDim.y < g.E ? active_expert(g, blockIdx.y, lane) : (int)blockIdx.y);
  if (e < 0) return;
  int lo, hi;
  expert_range(g, e, lo, hi);
  if (lo == hi) return;
  const int64_t n0 = (int64_t)blockIdx.x * kCols;
  const int nk = (int)(g.K / 128);
  const uint8_t* wrow[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    wrow[j] = g.w + ((int64_t)e * g.N + std::min<int64_t>(n0 + 16 * j + r16, g.N - 1)) * g.K + 16 * q4;
  const float* swb = g.w_scales + (ROW ? (int64_t)e * g.N : ((int64_t)e * (g.N / 128) + n0 / 128) * nk);

  // Up to 16 MB rows from m0 on.
  auto pass = [&](auto blocks, int m0) __attribute__((always_inline)) {
    constexpr int MB = decltype(blocks)::value;
    uint4 wv[2][2];
    float sw = 0.0f;
    auto fetch_w = [&](int ck) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        wv[j][0] = ldg16(wrow[j] + (int64_t)ck * 128);
        wv[j][1] = ldg16(wrow[j] + (int64_t)ck * 128 + 64);
      }
      if constexpr (!ROW) sw = swb[ck];
    };
    fetch_w(std::min(wave, nk - 1));   // a wave without a chunk: unused
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* arow[MB];
    const float* sarow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int64_t row = a_row(g, std::min(m0 + 16 * b + r16, hi - 1));
      arow[b] = g.a + row * g.K + 16 * q4;
      sarow[b] = g.a_scales + row * (ROW ? 1 : nk);
    }
    v4f_t acc[MB][2];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[b][j] = v4f_t{0.f, 0.f, 0.f, 0.f};
    for (int ck = wave; ck < nk; ck += kWaves) {
      uint4 x[MB][2];
      float sa[MB];
      if (ck != wave) fetch_w(ck);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        x[b][0] = ldg16(arow[b] + (int64_t)ck * 128);
        x[b][1] = ldg16(arow[b] + (int64_t)ck * 128 + 64);
        if constexpr (!ROW) sa[b] = sarow[b][ck];
      }
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const v8i qa = cat(x[b][0], x[b][1]);
        if constexpr (ROW) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[b][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(qa, cat(wv[j][0], wv[j][1]), acc[b][j], 0, 0, 0,
                                                                        127, 0, 127);
        } else {
          float sr[4];   // the lane's outputs are rows 4 q4 + r, whose scales sit in lanes 4 q4 + r
#pragma unroll
          for (int r = 0; r < 4; ++r) sr[r] = __shfl(sa[b], 4 * q4 + r);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const v4f_t P = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                qa, cat(wv[j][0], wv[j][1]), v4f_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, 127);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[b][j][r] = __builtin_fmaf(P[r], sr[r] * sw, acc[b][j][r]);
          }
        }
      }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][16 * b + 4 * q4 + r][16 * j + r16] = acc[b][j][r];
    __syncthreads();
#pragma unroll
    for (int b = 0; b < MB; ++b) {   // 512 threads, 16 x 32 outputs of a row block
      const int m = 16 * b + t / kCols, col = t % kCols;
      const int64_t n = n0 + col;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += part[w][m][col];
      if (m0 + m < hi && n < g.N) {
        if constexpr (ROW) v = v * g.a_scales[a_row(g, m0 + m)] * swb[n];
        g.c[(int64_t)(m0 + m) * g.ldc + n] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
      }
    }
  };
  constexpr int kStep = MAXB >= 4 ? 64 : 16;   // rows of a pass; the grid's z splits an expert's passes
  for (int m0 = lo + kStep * blockIdx.z; m0 < hi; m0 += kStep * gridDim.z) {
    if (m0 != lo + kStep * (int)blockIdx.z) __syncthreads();   // the last pass's sums are read
    if constexpr (MAXB >= 4) {
      const int left = hi - m0;
      if (left > 32) pass(std::integral_constant<int, 4>{}, m0);
      else if (left > 16) pass(std::integral_constant<int, 2>{}, m0);
      else pass(std::integral_constant<int, 1>{}, m0);
    } else {
      pass(std::integral_constant<int, 1>{}, m0);
    }
  }
}

}  // namespace

// Which kernel, from the sizes alone (the groups' sizes stay on the device): rows per tile, or
// minus the row blocks of a streaming pass.  Times in us with block-128 scales, the same number of
// rows for every expert, three weights in turn (none is left in a cache):
//   rows per expert          2      4      8     16     32     64    128    256   1024
//   E = 64, N = 4096, K = 2048 (1024 tiles and more)
//     stream, 1 block       87     88     94    114    199
//     tiles of 128         101    101    102    105    109     --    142     --    776
//     tiles of 256         107    107    108    110    113     --    142     --    644
//   E = 16, N = 2816, K = 2048 (176 tiles and more)
//     stream, 1 / 4 blocks  19     --     20     23     40     59    108    207
//     tiles of 128          25     --     25     25     26     28     31     54
//     tiles of 256          26     --     26     26     27     28     31     41
//   E = 8, N = 1024, K = 2048 (32 tiles and more)
//     stream, 4 blocks                            7      9     12     22     40
//     tiles of 128                               17     17     20     24     25
//   E = 4, N = 4096, K = 2048 (64 tiles and more)
//     stream, 4 blocks                           12     15     22     39     72
//     tiles of 128                               17     17     21     25     26
// A tile reads a weight once for 128 rows; the stream reads it once per pass (16 or 64 rows), but
// spreads an expert over N / 32 workgroups and more, so it holds on longer where tiles leave CUs
// idle: up to 2^19 outputs at 32 rows per expert and more, whatever K (512, 2048 and 8192
// measured: at worst 9 % over the better there), and below 2048 rows over tiles.  The border at 6
// rows costs up to 11 % (16 experts of 16 rows).
// Tiles of 256 rows read the weight half as often (64 experts of 1024 rows with row scales: 582
// against 665).  With fewer than 512 of them a last round is nearly empty: 16 experts of 64 rows, N =
// 2816, row scales take 29 against 23, though block scales and 256 rows 41 against 54.
// Only the mean is known here: an expert far above it is walked by the same N / 32 workgroups of the
// stream, and its weight read again for every 16 rows (512 x 2 assignments of 256 experts, N = 1024, K =
// 2048: 91 us evenly routed, 158 with half of them on one expert; N = 2048, K = 4096: 354 and 401).
static int kernel_choice(int64_t P, int64_t E, bool gather, int64_t a_rows, int64_t N, int64_t K) {
  const int64_t active = std::min(P, E), per = P / active, tiles_n = (N + 255) / 256;
  const int64_t tiles = (P / 128 + active) * tiles_n;
  if (per < 6) return -1;
  // gathered rows of a tile are addressed with 32-bit offsets from the activation's start
  const bool few = per < 2048 / tiles || (per >= 32 && P * N <= (1 << 19));
  if (few || (gather && a_rows * K > int64_t(0xFFFF0000))) return per <= 8 ? -1 : -4;
  return per >= 32 && (P / 256 + active) * tiles_n >= 512 ? 256 : 128;
}

template <bool ROW>
static hipError_t launch_stream(int blocks, const MoeGemmArgs& g, hipStream_t st) {
  // The passes of an expert (of twice the mean rows) are split over up to 1024 workgroups in all: 4
  // experts of 128 rows, N = 128, K = 2048 take 9.8 us, not split 24.5; 8 of 64 rows, N = 512, 10.9
  // and 17.1.  512 are too few (16 experts of 64 rows, N = 1024: 32 against 25), 2048 no better.
  const int64_t cols = (g.N + kCols - 1) / kCols, slots = std::min(g.E, g.P), passes = 2 * (g.P / slots) / 64;
  const int64_t split = std::max<int64_t>(1, std::min(passes, 1024 / (cols * slots)));
  const dim3 grid((unsigned)cols, (unsigned)slots, (unsigned)split);
  if (blocks == 1) hipLaunchKernelGGL((k_moe_stream<ROW, 1, 6>), grid, dim3(kThreads), 0, st, g);
  else hipLaunchKernelGGL((k_moe_stream<ROW, 4, 3>), grid, dim3(kThreads), 0, st, g);
  return hipGetLastError();
}

hipError_t launch_moe_gemm(bool row_scales, const MoeGemmArgs& g, hipStream_t st) {
  const int c = kernel_choice(g.P, g.E, g.gather, g.a_rows, g.N, g.K);
  if (c > 0) return launch_moe_tile(row_scales, c, g, st);
  return row_scales ? launch_stream<true>(-c, g, st) : launch_stream<false>(-c, g, st);
}

const char* moe_gemm_kernel_name(bool row_scales, bool gather, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K) {
  switch (kernel_choice(T * k, E, gather, gather ? T : T * k, N, K)) {
    case -1: return row_scales ? "k_moe_stream<1, fp8_row>" : "k_moe_stream<1, fp8_block128>";
    case -4: return row_scales ? "k_moe_stream<4, fp8_row>" : "k_moe_stream<4, fp8_block128>";
    case 128: return row_scales ? "k_moe_tile<128, fp8_row>" : "k_moe_tile<128, fp8_block128>";
  }
  return row_scales ? "k_moe_tile<256, fp8_row>" : "k_moe_tile<256, fp8_block128>";
}

}  // namespace pql
