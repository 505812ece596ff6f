// Attention of a batch's new tokens over the paged cache of keys and values, gfx950.
#include <algorithm>
#include <cmath>

#include "gemm_common.hpp"
#include "kv_common.hpp"
#include "pql_device.hpp"
#include "pql_internal.hpp"

namespace pql {

namespace {

template <int SCHEME>
__device__ __forceinline__ void row8(const void* codes, int64_t row, int D, int c, float s, float (&f)[8]) {
  if constexpr (SCHEME == kKvBf16) {
    chunk_to_f32(ldg16(static_cast<const uint16_t*>(codes) + row * D + c), f);
  } else {
    fp8x8_to_f32(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(codes) + row * D + c), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= s;
  }
}

// A wave per query row: a key per lane for the scores, D / 64 values per lane for the sums.
template <int SCHEME, int D>
__global__ __launch_bounds__(64) void k_attend_row(AttendArgs g) {
  __shared__ float qs[D];
  __shared__ float ps[64];
  __shared__ int64_t rows[64];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, hk = h / (g.H / g.Hk);
  int b = -1;
  for (int i = lane; i - lane < g.B && b < 0; i += 64) {
    bool mine = false;
    if (i < g.B) {
      const Seq s = sequence(g.starts, g.lens, i, g.T);
      mine = t >= s.first && t < s.first + s.n;
    }
    const uint64_t m = __ballot(mine);
    if (m) b = i - lane + __builtin_ctzll(m);
  }
  if (b < 0) return;
  const Seq s = sequence(g.starts, g.lens, b, g.T);
  const int pos = s.len - s.n + (int)(t - s.first);
  const int64_t cap = g.width << g.page_shift;
  const int64_t end = std::min<int64_t>(cap, g.causal ? std::max(0, std::min(s.len, pos + 1)) : s.len);
  const int64_t begin = g.window ? std::max<int64_t>(0, (int64_t)pos - g.window + 1) : 0;
  for (int d = lane; d < D; d += 64)
    qs[d] = __uint_as_float((uint32_t)g.q[t * g.ldqt + h * g.ldqh + d] << 16);
  __syncthreads();
  float m = -INFINITY, l = 0.0f, o[D / 64];
  for (int i = 0; i < D / 64; ++i) o[i] = 0.0f;
  for (int64_t k0 = begin; k0 < end; k0 += 64) {
    const int64_t j = k0 + lane;
    float sc = -INFINITY;
    int64_t row = -1;
    if (j < end) {
      const int page = g.pages[b * g.ldp + (j >> g.page_shift)];
      if (page >= 0 && page < g.n_pages) {
        row = (((int64_t)page * g.Hk + hk) << g.page_shift) + (j & ((1 << g.page_shift) - 1));
        const float ks = SCHEME == kKvBf16 ? 1.0f : g.k_scales[SCHEME == kKvRow ? row : 0];
        sc = 0.0f;
        for (int c = 0; c < D; c += 8) {
          float f[8];
          row8<SCHEME>(g.k_codes, row, D, c, ks, f);
          for (int e = 0; e < 8; ++e) sc += f[e] * qs[c + e];
        }
        sc *= g.scale;
      }
    }
    const float mx = fmaxf(m, wave_max(sc));
    const float safe = mx == -INFINITY ? 0.0f : mx;
    const float p = row < 0 ? 0.0f : expf(sc - safe), alpha = expf(m - safe);
    m = mx;
    float sum = p;
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    l = l * alpha + sum;
    ps[lane] = p;
    rows[lane] = row;
    __syncthreads();
    for (int i = 0; i < D / 64; ++i) o[i] *= alpha;
    for (int e = 0; e < 64; ++e) {
      if (rows[e] < 0) continue;
      const float vs = SCHEME == kKvBf16 ? 1.0f : g.v_scales[SCHEME == kKvRow ? rows[e] : 0];
      for (int i = 0; i < D / 64; ++i) {
        const int64_t at = rows[e] * D + 64 * i + lane;
        float v;
        if constexpr (SCHEME == kKvBf16) v = __uint_as_float((uint32_t)static_cast<const uint16_t*>(g.v_codes)[at] << 16);
        else v = __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(g.v_codes)[at], 0) * vs;
        o[i] += ps[e] * v;
      }
    }
    __syncthreads();
  }
  for (int i = 0; i < D / 64; ++i) {
    const float y = l == 0.0f ? 0.0f : o[i] / l;
    g.out[t * g.ldot + h * g.ldoh + 64 * i + lane] = (uint16_t)(gemm::pack_bf16x2(y, 0.0f) & 0xFFFFu);
  }
  if (g.lse && lane == 0) g.lse[t * g.H + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <int SCHEME>
hipError_t attend_as(const AttendArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)g.T, (unsigned)g.H);
  if (g.D == 64) hipLaunchKernelGGL((k_attend_row<SCHEME, 64>), grid, dim3(64), 0, st, g);
  else if (g.D == 128) hipLaunchKernelGGL((k_attend_row<SCHEME, 128>), grid, dim3(64), 0, st, g);
  else if (g.D == 192) hipLaunchKernelGGL((k_attend_row<SCHEME, 192>), grid, dim3(64), 0, st, g);
  else hipLaunchKernelGGL((k_attend_row<SCHEME, 256>), grid, dim3(64), 0, st, g);
  return hipGetLastError();
}

}  // namespace

bool kv_attention_fits(const AttendArgs& g) { return g.T < (int64_t(1) << 25) && g.T * g.H < (int64_t(1) << 24); }   // threads

size_t kv_attention_ws_bytes(const AttendArgs&) { return 0; }

hipError_t launch_kv_attention(int scheme, AttendArgs g, hipStream_t st) {
  if (scheme == kKvBf16) return attend_as<kKvBf16>(g, st);
  return scheme == kKvTensor ? attend_as<kKvTensor>(g, st) : attend_as<kKvRow>(g, st);
}

const char* kv_attention_kernel_name(const AttendArgs&) { return "k_attend_row"; }

}  // namespace pql
