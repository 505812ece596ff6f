// Around the cache of keys and values, gfx950: rotary positions, the slots of a batch's new
// tokens, quantizing keys and values as they are written, and reading them back.
#include <algorithm>

#include "gemm_common.hpp"
#include "kv_common.hpp"
#include "pql_device.hpp"
#include "pql_internal.hpp"
#include "quant_common.hpp"

namespace pql {

namespace {

// ---------------------------------------------------------------- angles
// cos and sin (times the table's scale) of 8 consecutive pairs of one position.  The angle is
// counted in turns: position * freq / 2 pi in fp64, less its nearest whole number, is exact to
// 2^-52 of the angle, so a position of 10^6 still has 30 bits behind the point; the rest is fp32.
struct Turn8 {
  float c[8], s[8];
  __device__ __forceinline__ void set(const double* __restrict__ freqs, int first, int step, int count, int pos,
                                      float scale) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= count) break;
      const double t = (double)pos * (freqs[first + j * step] * 0.15915494309189535);
      const float r = (float)(t - __builtin_rint(t));
      float si, co;
      sincospif(2.0f * r, &si, &co);
      c[j] = co * scale;
      s[j] = si * scale;
    }
  }
};

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  return make_uint4(gemm::pack_bf16x2(y[0], y[1]), gemm::pack_bf16x2(y[2], y[3]), gemm::pack_bf16x2(y[4], y[5]),
                    gemm::pack_bf16x2(y[6], y[7]));
}

// ---------------------------------------------------------------- rope
// A unit is 8 pairs (16 values) of a head, or 8 values behind the turned ones that are copied.  A
// thread takes one unit of `per` consecutive heads of one token: the angles are formed once and used
// for all of them.  Both values of a pair are read before either is written, by the same thread, so
// x and out may be the same.
// Bound by memory once tokens are many: 8192 x 40 heads of 128, half of each turned, in 34.5 us, 4.9 TB/s (a large
// copy 4.7 to 5.1); with angles for each head 60 us, the fp64 products and the sines being the bound.  7 tokens: 3 us.
template <bool HALF>
__global__ __launch_bounds__(256) void k_rope(RopeArgs g) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= g.T * g.groups * g.units) return;
  const int u = (int)(i % g.units);
  const int64_t r = i / g.units;
  const int h0 = (int)(r % g.groups) * g.per;
  const int64_t t = r / g.groups;
  const int h1 = std::min(h0 + g.per, g.H);
  const uint16_t* x = g.x + t * g.ldxt;
  uint16_t* o = g.out + t * g.ldot;
  const int turned = g.rotary >> 4;
  if (u >= turned) {
    const int c = g.rotary + (u - turned) * 8;
    for (int h = h0; h < h1; ++h) stg16(o + h * g.ldoh + c, ldg16(x + h * g.ldxh + c));
    return;
  }
  Turn8 a;
  a.set(g.freqs, u * 8, 1, 8, g.positions[t], g.scale);
  const int c1 = HALF ? u * 8 : u * 16, c2 = HALF ? c1 + g.rotary / 2 : c1 + 8;
  for (int h = h0; h < h1; ++h) {
    float p[8], q[8], y[8], z[8];
    chunk_to_f32(ldg16(x + h * g.ldxh + c1), p);
    chunk_to_f32(ldg16(x + h * g.ldxh + c2), q);
    if constexpr (HALF) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = p[j] * a.c[j] - q[j] * a.s[j];
        z[j] = q[j] * a.c[j] + p[j] * a.s[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = p[2 * j] * a.c[j] - p[2 * j + 1] * a.s[j];
        y[2 * j + 1] = p[2 * j + 1] * a.c[j] + p[2 * j] * a.s[j];
        z[2 * j] = q[2 * j] * a.c[4 + j] - q[2 * j + 1] * a.s[4 + j];
        z[2 * j + 1] = q[2 * j + 1] * a.c[4 + j] + q[2 * j] * a.s[4 + j];
      }
    }
    stg16(o + h * g.ldoh + c1, pack8(y));
    stg16(o + h * g.ldoh + c2, pack8(z));
  }
}

// ---------------------------------------------------------------- slots
// Row t belongs to the sequence b with starts[b] <= t < starts[b + 1]: a binary search for the last
// start at or below t, then both ends checked, so that any starts give an answer inside the batch.  A chain
// of log2 B reads from the cache bounds it: 24 sequences of a token 2.3 us, 150 of up to 200 tokens 3.0.
__global__ __launch_bounds__(256) void k_kv_slots(const int32_t* __restrict__ starts, const int32_t* __restrict__ lens,
                                                  const int32_t* __restrict__ pages, int B, int64_t width, int64_t ldp,
                                                  int page_shift, int64_t T, int32_t* __restrict__ slots,
                                                  int32_t* __restrict__ positions) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= T) return;
  if (B == 0) {   // there are no lens to read
    slots[t] = -1;
    positions[t] = 0;
    return;
  }
  int lo = 0, hi = B;   // starts[lo] <= t < starts[hi] where the ends allow it
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t) lo = mid;
    else hi = mid;
  }
  const Seq q = sequence(starts, lens, lo, T);
  int slot = -1;
  int64_t pos = -1;
  if (t >= q.first && t < q.first + q.n) pos = (int64_t)q.len - q.n + (t - q.first);
  if (pos >= 0) {
    const int64_t p = pos >> page_shift;
    if (p < width) {
      const int64_t page = pages[lo * ldp + p];
      const int64_t s = (page << page_shift) + (pos & ((1 << page_shift) - 1));
      if (page >= 0 && s <= INT32_MAX) slot = (int)s;
    }
  }
  slots[t] = slot;
  positions[t] = pos < 0 ? 0 : (int)pos;
}

// ---------------------------------------------------------------- append
// A head of one token is D / 8 lanes of 8 values (a group of 8, 16 or 32 lanes); blockIdx.y picks keys
// or values.  A thread walks `per` heads of its token, so that the keys' angles are formed once.  In the
// half layout a lane reads its partner's 8 values itself (they are in the cache line its neighbour
// reads).  The maximum of a head is an exchange within the group.
// Bound by memory: 16384 x 8 heads of 128, a scale per token and head, an eighth of the rows padding, in 20.6 us,
// 4.3 TB/s; its writes are pieces of 128 bytes.  24 tokens: 3.6 us.
template <int SCHEME, int LANES>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs g) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int l = (int)(i % LANES);
  const int64_t r = i / LANES;
  const int64_t t = r / g.groups;
  if (t >= g.T) return;
  const int64_t slot = g.slots[t];
  if (slot < 0 || slot >= ((int64_t)g.n_pages << g.page_shift)) return;   // a group's lanes share t
  const bool value = blockIdx.y != 0;
  const int h0 = (int)(r % g.groups) * g.per, h1 = std::min(h0 + g.per, g.Hk);
  const uint16_t* x = value ? g.v + t * g.ldvt : g.k + t * g.ldkt;
  const int64_t ldh = value ? g.ldvh : g.ldkh;
  const int64_t page = slot >> g.page_shift, off = slot & ((1 << g.page_shift) - 1);
  const int c = l * 8;
  const bool live = LANES * 8 == g.D || c < g.D;   // D = 192 has 24 of 32 lanes
  const bool turn = !value && g.positions && c < g.rotary;
  const bool half = g.layout == 0;
  Turn8 a;
  int partner = 0;
  float sign = 1.0f;
  if (turn) {
    if (half) {
      const int h = g.rotary / 2;
      const bool second = c >= h;
      partner = second ? c - h : c + h;
      sign = second ? 1.0f : -1.0f;
      a.set(g.freqs, second ? c - h : c, 1, 8, g.positions[t], g.rope_scale);
    } else {
      a.set(g.freqs, c / 2, 1, 4, g.positions[t], g.rope_scale);
    }
  }
  uint8_t* codes = static_cast<uint8_t*>(value ? g.v_codes : g.k_codes);
  float* scales = value ? g.v_scales : g.k_scales;
  for (int h = h0; h < h1; ++h) {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) chunk_to_f32(ldg16(x + h * ldh + c), f);
    if (turn) {
      if (half) {
        float p[8];
        chunk_to_f32(ldg16(x + h * ldh + partner), p);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * a.c[j] + sign * (p[j] * a.s[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = f[2 * j], q = f[2 * j + 1];
          f[2 * j] = p * a.c[j] - q * a.s[j];
          f[2 * j + 1] = q * a.c[j] + p * a.s[j];
        }
      }
    }
    const int64_t row = ((page * g.Hk + h) << g.page_shift) + off;
    if constexpr (SCHEME == kKvBf16) {
      if (live) stg16(codes + (row * g.D + c) * 2, pack8(f));
    } else {
      float s;
      if constexpr (SCHEME == kKvRow) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
        s = fp8_scale(m);
        if (l == 0) scales[row] = s;
      } else {
        s = scales[0];
      }
      if (live) stg8(codes + row * g.D + c, fp8_codes8<SCHEME == kKvTensor>(f, s));
    }
  }
}

// ---------------------------------------------------------------- read
// 8 values of one slot's head per thread, keys or values by blockIdx.y.  Bound by memory: a context of 60000
// tokens, 8 heads of 128 with a scale each, 87 us, 4.3 TB/s.
template <int SCHEME>
__global__ __launch_bounds__(256) void k_kv_read(ReadArgs g) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int units = g.D >> 3;
  const int c = (int)(i % units) * 8;
  const int64_t r = i / units;
  const int h = (int)(r % g.Hk);
  const int64_t t = r / g.Hk;
  if (t >= g.n) return;
  const bool value = blockIdx.y != 0;
  const int64_t slot = g.slots[t];
  uint4 y = make_uint4(0u, 0u, 0u, 0u);
  if (slot >= 0 && slot < ((int64_t)g.n_pages << g.page_shift)) {
    const int64_t page = slot >> g.page_shift, off = slot & ((1 << g.page_shift) - 1);
    const int64_t row = ((page * g.Hk + h) << g.page_shift) + off;
    const uint8_t* codes = static_cast<const uint8_t*>(value ? g.v_codes : g.k_codes);
    if constexpr (SCHEME == kKvBf16) {
      y = ldg16(codes + (row * g.D + c) * 2);
    } else {
      const float* scales = value ? g.v_scales : g.k_scales;
      const float s = scales[SCHEME == kKvRow ? row : 0];
      const uint2 q = *reinterpret_cast<const uint2*>(codes + row * g.D + c);
      float f[8];
      fp8x8_to_f32(q, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= s;
      y = pack8(f);
    }
  }
  uint16_t* o = value ? g.v_out + t * g.ldvt + h * g.ldvh : g.k_out + t * g.ldkt + h * g.ldkh;
  stg16(o + c, y);
}

// Heads per thread: as many as leave the card 2^16 threads, at most 8 (1 | 4 | 8: rope of 8192 x 40 heads 60 | 35 | 35 us,
// append of 16384 x 8 heads 28 | 22 | 21; 7 and 24 tokens are level).
int heads_per_thread(int64_t threads_per_head, int heads) {
  int per = 1;
  while (per < 8 && per < heads && threads_per_head * ((heads + 2 * per - 1) / (2 * per)) >= (1 << 16)) per *= 2;
  return per;
}

template <int SCHEME>
hipError_t append_as(AppendArgs& g, hipStream_t st) {
  const int lanes = g.D <= 64 ? 8 : g.D <= 128 ? 16 : 32;
  g.per = heads_per_thread(g.T * lanes, g.Hk);
  g.groups = (g.Hk + g.per - 1) / g.per;
  const dim3 grid((unsigned)((g.T * g.groups * lanes + 255) / 256), 2);
  if (lanes == 8) hipLaunchKernelGGL((k_kv_append<SCHEME, 8>), grid, dim3(256), 0, st, g);
  else if (lanes == 16) hipLaunchKernelGGL((k_kv_append<SCHEME, 16>), grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL((k_kv_append<SCHEME, 32>), grid, dim3(256), 0, st, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(int layout, RopeArgs g, hipStream_t st) {
  g.units = g.rotary / 16 + (g.out == g.x ? 0 : (g.D - g.rotary) / 8);   // in place nothing needs copying
  g.per = heads_per_thread(g.T * g.units, g.H);
  g.groups = (g.H + g.per - 1) / g.per;
  const dim3 grid((unsigned)((g.T * g.groups * g.units + 255) / 256));
  if (layout == 0) hipLaunchKernelGGL(k_rope<true>, grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL(k_rope<false>, grid, dim3(256), 0, st, g);
  return hipGetLastError();
}

hipError_t launch_kv_slots(const int32_t* starts, const int32_t* lens, const int32_t* pages, int B, int64_t width,
                           int64_t ldp, int page_shift, int64_t T, int32_t* slots, int32_t* positions, hipStream_t st) {
  hipLaunchKernelGGL(k_kv_slots, dim3((unsigned)((T + 255) / 256)), dim3(256), 0, st, starts, lens, pages, B, width, ldp,
                     page_shift, T, slots, positions);
  return hipGetLastError();
}

hipError_t launch_kv_append(int scheme, AppendArgs g, hipStream_t st) {
  if (scheme == kKvBf16) return append_as<kKvBf16>(g, st);
  return scheme == kKvTensor ? append_as<kKvTensor>(g, st) : append_as<kKvRow>(g, st);
}

hipError_t launch_kv_read(int scheme, const ReadArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)((g.n * g.Hk * (g.D / 8) + 255) / 256), 2);
  if (scheme == kKvBf16) hipLaunchKernelGGL(k_kv_read<kKvBf16>, grid, dim3(256), 0, st, g);
  else if (scheme == kKvTensor) hipLaunchKernelGGL(k_kv_read<kKvTensor>, grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL(k_kv_read<kKvRow>, grid, dim3(256), 0, st, g);
  return hipGetLastError();
}

}  // namespace pql
