// Shared by the kernels of the cache of keys and values (internal to the library): a batch's
// sequences, read so that no value in them leads out of a buffer, and the codes' decoding.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pql {

constexpr int kKvBf16 = 0, kKvTensor = 1, kKvRow = 2;   // pql_kv_scheme

// A sequence's new tokens, rows first .. first + n - 1, and its tokens in the cache.
struct Seq {
  int first, n, len;
};

// starts are cut to 0 .. T and an end below its start is none; a length below 0 is 0.
__device__ __forceinline__ Seq sequence(const int32_t* __restrict__ starts, const int32_t* __restrict__ lens, int b,
                                        int64_t T) {
  const int64_t s0 = starts[b], s1 = starts[b + 1], l = lens[b];
  const int64_t first = s0 < 0 ? 0 : s0 > T ? T : s0;
  const int64_t end = s1 < first ? first : s1 > T ? T : s1;
  return Seq{(int)first, (int)(end - first), (int)(l < 0 ? 0 : l)};
}

// 8 e4m3fn codes -> fp32.
__device__ __forceinline__ void fp8x8_to_f32(uint2 q, float (&f)[8]) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true);
  const v2f c = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}

}  // namespace pql
