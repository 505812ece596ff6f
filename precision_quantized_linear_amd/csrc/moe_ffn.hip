// The memory-bound steps around the experts' products, gfx950: the gated activation that
// quantizes its own result, and the weighted sum of the experts' rows back to tokens.
#include <algorithm>

#include "gemm_common.hpp"
#include "pql_device.hpp"
#include "pql_internal.hpp"
#include "quant_common.hpp"

namespace pql {

namespace {

// ---------------------------------------------------------------- swiglu + quantize
// h = g / (1 + exp(-g)) * u in fp32 from a row's bf16 gate and up halves, then the scheme's
// activation rule on h (never rounded to bf16 in between).  exp(-g) is 2^(-g log2 e).  Far below
// zero 1 + exp(-g) nears the end of fp32 (its reciprocal is subnormal from g = -87.3 on, which the
// instruction flushes, and it overflows at -88.7), but a large u brings h back well inside:
// silu(-90) 1e6 = -7e-32, silu(-190) 3e38 = -2e-42.  There 1 + exp(-g) is exp(-g) to all 24
// bits, and h = g 2^(g log2 e) u takes its power of two last, in one rounding.  A chunk without such
// a gate pays for their minimum alone.
//
// Bound by memory (4 bytes read, 1 written per element): 65536 rows of F = 2048 with block
// scales take 124 us, 5.4 TB/s, of F = 1408 with row scales 83, 5.5 TB/s; 222 rows of those 2.7.  A lane holds 8 columns
// of both halves, so every load and store is whole lines and nothing is staged.
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
  return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

constexpr float kFarGate = -80.0f;
// For g < kFarGate.  2^-10 keeps the product with u finite; gates below -300 give 0 for any finite u.
__device__ __forceinline__ float far_silu_mul(float g, float u) {
  g = fmaxf(g, -300.0f);
  const float y = g * 1.44269504f, n = __builtin_rintf(y);
  return ldexpf(__builtin_amdgcn_exp2f(y - n) * 0x1p-10f * g * u, (int)n + 10);
}

__device__ __forceinline__ void swiglu_chunk(uint4 gc, uint4 uc, float (&h)[8]) {
  float g[8], u[8];
  chunk_to_f32(gc, g);
  chunk_to_f32(uc, u);
  float least = g[0];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h[j] = silu_mul(g[j], u[j]);
    least = fminf(least, g[j]);
  }
  if (least < kFarGate) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (g[j] < kFarGate) h[j] = far_silu_mul(g[j], u[j]);
  }
}

__device__ __forceinline__ float absmax8(const float (&h)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(h[j]));
  return m;
}

__device__ __forceinline__ uint2 fp8_codes8(const float (&h)[8], float s) {
  float q[8];
  if (s >= kSmallestFastScale) {
    const float rcp = __fdiv_rn(1.0f, s);
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = quot<true>(h[j], s, rcp);
  } else {
    // The statement keeps this a branch: without it both quotients are formed for every element
    // (65536 rows of 1408 with row scales: 114 us instead of 83).
    asm volatile("");
    // A subnormal scale is the nearest of few steps, and a quotient can pass 464, which the convert
    // makes a NaN (h of 656 2^-149: scale 2^-149).  A NaN h stays one.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = quot<false>(h[j], s, 0.0f);
      q[j] = fabsf(v) > 448.0f ? __builtin_copysignf(448.0f, v) : v;
    }
  }
  return make_uint2(fp8x4(q[0], q[1], q[2], q[3]), fp8x4(q[4], q[5], q[6], q[7]));
}

__device__ __forceinline__ int64_t live_rows(const int32_t* count, int64_t rows) {
  return count ? std::min<int64_t>(rows, std::max(0, *count)) : rows;
}

// Block-128: a 128-wide group is 16 consecutive lanes; four rows per workgroup, one per wave.
constexpr int kSwU = 2;   // 64-chunk segments per wave
__global__ __launch_bounds__(256) void k_swiglu_block(const uint16_t* __restrict__ x, int64_t rows, int64_t F,
                                                      int64_t ldx, const int32_t* __restrict__ count,
                                                      uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= live_rows(count, rows)) return;
  const int64_t cpr = F >> 3;
  const uint16_t* xr = x + row * ldx;
#pragma unroll
  for (int u = 0; u < kSwU; ++u) {
    const int64_t c = (int64_t)blockIdx.y * 64 * kSwU + 64 * u + lane;
    if (c >= cpr) break;   // whole groups: F % 128 == 0
    float h[8];
    swiglu_chunk(ldg16_nt(xr + c * 8), ldg16_nt(xr + F + c * 8), h);
    const float s = fp8_scale(group16_max(absmax8(h)));
    stg8(codes + row * F + c * 8, fp8_codes8(h, s));
    if ((lane & 15) == 0) scales[row * (F / 128) + (c >> 4)] = s;
  }
}

// Per row: a workgroup per row, the row's h held in registers between the maximum and the
// cast (CH chunks of 8 per thread), or formed twice where it is longer than that (CH == 0).
template <int CH>
__global__ __launch_bounds__(256) void k_swiglu_row(const uint16_t* __restrict__ x, int64_t rows, int64_t F,
                                                    int64_t ldx, const int32_t* __restrict__ count,
                                                    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ float red[4];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  if (row >= live_rows(count, rows)) return;
  const int64_t cpr = F >> 3;
  const uint16_t* xr = x + row * ldx;
  float h[CH > 0 ? CH : 1][8];
  float m = 0.0f;
  if constexpr (CH > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int64_t c = t + 256 * i;
      if (c < cpr) {
        swiglu_chunk(ldg16_nt(xr + c * 8), ldg16_nt(xr + F + c * 8), h[i]);
        m = fmaxf(m, absmax8(h[i]));
      }
    }
  } else {
    for (int64_t c = t; c < cpr; c += 256) {
      swiglu_chunk(ldg16(xr + c * 8), ldg16(xr + F + c * 8), h[0]);
      m = fmaxf(m, absmax8(h[0]));
    }
  }
  m = wave_max(m);
  if ((t & 63) == 0) red[t >> 6] = m;
  __syncthreads();
  const float s = fp8_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
  if (t == 0) scales[row] = s;
  uint8_t* cr = codes + row * F;
  if constexpr (CH > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int64_t c = t + 256 * i;
      if (c < cpr) stg8(cr + c * 8, fp8_codes8(h[i], s));
    }
  } else {
    for (int64_t c = t; c < cpr; c += 256) {
      swiglu_chunk(ldg16(xr + c * 8), ldg16(xr + F + c * 8), h[0]);
      stg8(cr + c * 8, fp8_codes8(h[0], s));
    }
  }
}

// ---------------------------------------------------------------- combine
// out[t] = add[t] + sum_j w[t, j] y[slot[t, j]], summed in fp32 in the order of j, one
// rounding to bf16.  A slot outside 0 .. P - 1 (an expert held elsewhere) adds w * 0: nothing,
// unless the weight is NaN (a broken row of logits), which then shows in the output.
//
// Bound by memory: the rows of a token are whole lines at random places, a workgroup covers 2048
// columns of one token (8192 tokens of 8 rows, N = 4096, a quarter of them elsewhere: 94 us,
// 5.0 TB/s, a copy's rate; 3 tokens: 3.7 us).  Rows that do not all start on 16 bytes go by single
// columns: N = 4095 takes 287 us.
template <int W>   // columns per thread: 8 (16-byte accesses) or 1
__global__ __launch_bounds__(256) void k_moe_combine(CombineArgs g) {
  const int64_t t = blockIdx.x;
  const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * W;
  if (c >= g.N) return;
  float acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) acc[i] = 0.0f;
  for (int j = 0; j < g.k; ++j) {
    const int64_t slot = g.slots[t * g.k + j];
    const float w = g.weights[t * g.k + j];
    float y[W];
#pragma unroll
    for (int i = 0; i < W; ++i) y[i] = 0.0f;
    if (slot >= 0 && slot < g.P) {
      const uint16_t* p = g.y + slot * g.ldy + c;
      if constexpr (W == 8) chunk_to_f32(ldg16(p), y);
      else y[0] = __uint_as_float((uint32_t)p[0] << 16);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = __builtin_fmaf(w, y[i], acc[i]);
  }
  if (g.add) {
    const uint16_t* p = g.add + t * g.ldadd + c;
    float a[W];
    if constexpr (W == 8) chunk_to_f32(ldg16(p), a);
    else a[0] = __uint_as_float((uint32_t)p[0] << 16);
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] += a[i];
  }
  uint16_t* o = g.out + t * g.ldo + c;
  if constexpr (W == 8)
    stg16(o, make_uint4(gemm::pack_bf16x2(acc[0], acc[1]), gemm::pack_bf16x2(acc[2], acc[3]),
                        gemm::pack_bf16x2(acc[4], acc[5]), gemm::pack_bf16x2(acc[6], acc[7])));
  else
    o[0] = (uint16_t)(gemm::pack_bf16x2(acc[0], 0.0f) & 0xFFFFu);
}

}  // namespace

hipError_t launch_swiglu_quantize(bool per_row, const uint16_t* x, int64_t rows, int64_t F, int64_t ldx,
                                  const int32_t* count, uint8_t* codes, float* scales, hipStream_t st) {
  if (!per_row) {
    const dim3 grid((unsigned)((rows + 3) / 4), (unsigned)((F / 8 + 64 * kSwU - 1) / (64 * kSwU)));
    hipLaunchKernelGGL(k_swiglu_block, grid, dim3(256), 0, st, x, rows, F, ldx, count, codes, scales);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)rows);
  if (F <= 2048) hipLaunchKernelGGL(k_swiglu_row<1>, grid, dim3(256), 0, st, x, rows, F, ldx, count, codes, scales);
  else if (F <= 8192) hipLaunchKernelGGL(k_swiglu_row<4>, grid, dim3(256), 0, st, x, rows, F, ldx, count, codes, scales);
  else hipLaunchKernelGGL(k_swiglu_row<0>, grid, dim3(256), 0, st, x, rows, F, ldx, count, codes, scales);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const CombineArgs& g, bool vec, hipStream_t st) {
  const int per = 256 * (vec ? 8 : 1);
  const dim3 grid((unsigned)g.T, (unsigned)((g.N + per - 1) / per));
  if (vec) hipLaunchKernelGGL(k_moe_combine<8>, grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL(k_moe_combine<1>, grid, dim3(256), 0, st, g);
  return hipGetLastError();
}

}  // namespace pql
