// Grouped FP8 products of a mixture-of-experts layer, gfx950.
//
// C[p, n] = sum_k a_hat[row(p), k] w_hat[e(p), n, k] for the assignments p in expert order:
// offsets[e] .. offsets[e + 1] - 1 are expert e's, row(p) is the token of assignment order[p]
// (gather) or p itself.  FP8_BLOCK128: partial products of each 128-wide K-group promoted with
// s_a[row, g] s_w[e, n / 128, g] in fp32; FP8_ROW: one fp32 sum scaled by s_a[row] s_w[e, n].
//
// k_moe_stream: a workgroup owns 32 columns of one expert and walks the expert's rows 16 at a
// time; the weight is streamed past them, as in the few-token qlinear kernels: 8 waves take the
// K-chunks (128 bytes) round-robin, feed 16x16x128 MFMAs straight from registers, and add
// their sums in LDS.
#include <algorithm>

#include "gemm_common.hpp"
#include "moe_gemm.hpp"
#include "pql_device.hpp"
#include "pql_internal.hpp"

namespace pql {

namespace {

using namespace gemm;

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kBatch = 3;
constexpr int kCols = 32;

typedef float v4f_t __attribute__((ext_vector_type(4)));

template <bool ROW>
__global__ __launch_bounds__(kThreads) void k_moe_stream(MoeGemmArgs g) {
  __shared__ float part[kWaves][16][kCols + 1];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int e = blockIdx.y;
  int lo, hi;
  expert_range(g, e, lo, hi);
  if (lo == hi) return;
  const int64_t n0 = (int64_t)blockIdx.x * kCols;
  const int nk = (int)(g.K / 128);
  const uint8_t* wrow[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    wrow[j] = g.w + ((int64_t)e * g.N + std::min<int64_t>(n0 + 16 * j + r16, g.N - 1)) * g.K;
  const float* swb = g.w_scales + (ROW ? (int64_t)e * g.N : ((int64_t)e * (g.N / 128) + n0 / 128) * nk);

  for (int m0 = lo; m0 < hi; m0 += 16) {
    const int64_t row = a_row(g, std::min(m0 + r16, hi - 1));
    const uint8_t* arow = g.a + row * g.K;
    const float* sarow = g.a_scales + row * (ROW ? 1 : nk);
    v4f_t acc[2] = {v4f_t{0.f, 0.f, 0.f, 0.f}, v4f_t{0.f, 0.f, 0.f, 0.f}};
    for (int ck0 = wave; ck0 < nk; ck0 += kWaves * kBatch) {
      uint4 x[kBatch][2], wv[kBatch][2][2];
      float sa[kBatch], sw[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int ck = ck0 + u * kWaves;
        if (ck < nk) {   // wave-uniform
          const int64_t k0 = (int64_t)ck * 128 + 16 * q4;
          x[u][0] = ldg16(arow + k0);
          x[u][1] = ldg16(arow + k0 + 64);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            wv[u][j][0] = ldg16(wrow[j] + k0);
            wv[u][j][1] = ldg16(wrow[j] + k0 + 64);
          }
          if constexpr (!ROW) {
            sa[u] = sarow[ck];
            sw[u] = swb[ck];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (ck0 + u * kWaves >= nk) continue;
        const v8i qa = cat(x[u][0], x[u][1]);
        if constexpr (ROW) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(qa, cat(wv[u][j][0], wv[u][j][1]), acc[j], 0, 0,
                                                                      0, 127, 0, 127);
        } else {
          float sr[4];   // the lane's outputs are rows 4 q4 + r, whose scales sit in lanes 4 q4 + r
#pragma unroll
          for (int r = 0; r < 4; ++r) sr[r] = __shfl(sa[u], 4 * q4 + r);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const v4f_t P = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                qa, cat(wv[u][j][0], wv[u][j][1]), v4f_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, 127);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[j][r] = __builtin_fmaf(P[r], sr[r] * sw[u], acc[j][r]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][4 * q4 + r][16 * j + r16] = acc[j][r];
    __syncthreads();
    {
      const int m = t / kCols, col = t % kCols;   // 512 threads, 16 x 32 outputs
      const int64_t n = n0 + col;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += part[w][m][col];
      if (m0 + m < hi && n < g.N) {
        if constexpr (ROW) v = v * g.a_scales[a_row(g, m0 + m)] * swb[n];
        g.c[(int64_t)(m0 + m) * g.ldc + n] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
      }
    }
    __syncthreads();
  }
}

}  // namespace

// Rows per tile, or 0 for the streaming kernel.
static int tile_rows(int64_t P, int64_t E, bool gather, int64_t a_rows, int64_t K) {
  // gathered rows are addressed with 32-bit offsets from the activation's start
  if (gather && a_rows * K > int64_t(0xFFFF0000)) return 0;
  const int64_t per = P / E;   // rows per expert, were they spread evenly
  if (per < 24) return 0;
  return per < 96 ? 64 : per < 384 ? 128 : 256;
}

hipError_t launch_moe_gemm(bool row_scales, const MoeGemmArgs& g, hipStream_t st) {
  const int bm = tile_rows(g.P, g.E, g.gather, g.a_rows, g.K);
  if (bm) return launch_moe_tile(row_scales, bm, g, st);
  const dim3 grid((unsigned)((g.N + kCols - 1) / kCols), (unsigned)g.E);
  if (row_scales) hipLaunchKernelGGL(k_moe_stream<true>, grid, dim3(kThreads), 0, st, g);
  else hipLaunchKernelGGL(k_moe_stream<false>, grid, dim3(kThreads), 0, st, g);
  return hipGetLastError();
}

const char* moe_gemm_kernel_name(bool row_scales, bool gather, int64_t T, int64_t k, int64_t E, int64_t K) {
  switch (tile_rows(T * k, E, gather, gather ? T : T * k, K)) {
    case 64: return row_scales ? "k_moe_tile<64, fp8_row>" : "k_moe_tile<64, fp8_block128>";
    case 128: return row_scales ? "k_moe_tile<128, fp8_row>" : "k_moe_tile<128, fp8_block128>";
    case 256: return row_scales ? "k_moe_tile<256, fp8_row>" : "k_moe_tile<256, fp8_block128>";
  }
  return row_scales ? "k_moe_stream<fp8_row>" : "k_moe_stream<fp8_block128>";
}

}  // namespace pql
