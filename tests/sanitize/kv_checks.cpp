// Argument validation of the entry points around the cache of keys and values under AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code of abi.cpp (test infrastructure): every call must be
// refused, or accepted as an empty no-op, before a device is touched.  Fake pointers are never
// dereferenced.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "pql.h"

static int failures = 0;

static void expect(const char* what, pql_status got, pql_status want) {
  if (got != want) {
    std::printf("FAIL %s: status %d, expected %d (%s)\n", what, (int)got, (int)want, pql_last_error());
    ++failures;
  }
}

template <class T = void>
static T* P(uintptr_t off = 0) { return reinterpret_cast<T*>((uintptr_t)1 << 20 | off); }

int main() {
  const pql_status bad = PQL_ERR_INVALID_ARGUMENT;
  const int64_t extremes[] = {INT64_MIN, INT64_MIN + 1, -1, 0, INT64_MAX - 1, INT64_MAX};
  int32_t* i32 = P<int32_t>();
  float* f32 = P<float>();
  double* f64 = P<double>();

  auto rope = [&](int64_t T, int64_t H, int64_t D, int64_t lt, int64_t lh, int64_t rotary) {
    return pql_rope(0, P(), T, H, D, lt, lh, i32, f64, rotary, 1.f, P(0x1000), lt, lh, nullptr);
  };
  for (int64_t v : extremes) {
    if (v != 0) expect("rope T", rope(v, 2, 128, 256, 128, 128), bad);
    expect("rope H", rope(4, v, 128, 256, 128, 128), bad);
    expect("rope D", rope(4, 2, v, 256, 128, 128), bad);
    expect("rope token stride", rope(4, 2, 128, v, 128, 128), bad);
    expect("rope head stride", rope(4, 2, 128, 256, v, 128), bad);
    expect("rope rotary", rope(4, 2, 128, 256, 128, v), bad);
  }
  expect("rope empty", pql_rope(0, nullptr, 0, 2, 128, 256, 128, nullptr, nullptr, 128, 1.f, nullptr, 256, 128, nullptr), PQL_OK);

  size_t codes = 0, scales = 0;
  for (int64_t v : extremes) {
    expect("sizes pages", pql_kv_sizes(2, v, 16, 8, 128, &codes, &scales), bad);
    expect("sizes page", pql_kv_sizes(2, 4, v, 8, 128, &codes, &scales), bad);
    expect("sizes heads", pql_kv_sizes(2, 4, 16, v, 128, &codes, &scales), bad);
    expect("sizes head", pql_kv_sizes(2, 4, 16, 8, v, &codes, &scales), bad);
  }
  expect("sizes", pql_kv_sizes(2, 4, 16, 8, 128, nullptr, nullptr), PQL_OK);
  expect("sizes scheme", pql_kv_sizes(7, 4, 16, 8, 128, &codes, &scales), PQL_ERR_UNSUPPORTED);

  auto slots = [&](int64_t B, int64_t width, int64_t ldp, int64_t ps, int64_t T) {
    return pql_kv_slots(i32, i32, i32, B, width, ldp, ps, T, i32, i32, nullptr);
  };
  for (int64_t v : extremes) {
    if (v != 0) expect("slots B", slots(v, 2, 2, 16, 4), bad);
    if (v != 0) expect("slots width", slots(2, v, v, 16, 4), bad);
    expect("slots ldp", slots(2, 2, v == INT64_MAX || v == INT64_MAX - 1 ? v : v, 16, 4), bad);
    expect("slots page", slots(2, 2, 2, v, 4), bad);
    if (v != 0) expect("slots T", slots(2, 2, 2, 16, v), bad);
  }

  for (int scheme : {(int)PQL_KV_BF16, (int)PQL_KV_FP8_TENSOR, (int)PQL_KV_FP8_ROW}) {
    auto append = [&](int64_t T, int64_t lt, int64_t lh, int64_t rotary, int64_t pages, int64_t ps, int64_t Hk, int64_t D) {
      return pql_kv_append(scheme, P(), lt, lh, P(), lt, lh, T, i32, 0, i32, f64, rotary, 1.f, P(), P(), f32, f32, pages,
                           ps, Hk, D, nullptr);
    };
    auto read = [&](int64_t n, int64_t lt, int64_t lh, int64_t pages, int64_t ps, int64_t Hk, int64_t D) {
      return pql_kv_read(scheme, P(), P(), f32, f32, pages, ps, Hk, D, i32, n, P(), lt, lh, P(), lt, lh, nullptr);
    };
    auto attend = [&](int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t B, int64_t width, int64_t ps, int64_t window,
                      int64_t lt) {
      return pql_kv_attention(scheme, P(), lt, 128, T, H, P(), P(), f32, f32, 4, ps, Hk, D, i32, i32, i32, B, width, width,
                              1, window, 0.1f, P(), lt, 128, nullptr, P(), SIZE_MAX, nullptr);
    };
    for (int64_t v : extremes) {
      if (v != 0) expect("append T", append(v, 256, 128, 128, 4, 16, 2, 128), bad);
      if (v != 0) expect("append token stride", append(4, v, 128, 128, 4, 16, 2, 128), bad);
      if (v != 0) expect("append head stride", append(4, 256, v, 128, 4, 16, 2, 128), bad);
      expect("append rotary", append(4, 256, 128, v, 4, 16, 2, 128), bad);
      expect("append pages", append(4, 256, 128, 128, v, 16, 2, 128), bad);
      expect("append page", append(4, 256, 128, 128, 4, v, 2, 128), bad);
      expect("append heads", append(4, 256, 128, 128, 4, 16, v, 128), bad);
      expect("append head", append(4, 256, 128, 128, 4, 16, 2, v), bad);
      if (v != 0) expect("read n", read(v, 256, 128, 4, 16, 2, 128), bad);
      expect("read token stride", read(4, v, 128, 4, 16, 2, 128), bad);
      expect("read heads", read(4, 256, 128, 4, 16, v, 128), bad);
      if (v != 0) expect("attend T", attend(v, 4, 2, 128, 2, 2, 16, 0, 512), bad);
      expect("attend H", attend(4, v, 2, 128, 2, 2, 16, 0, 512), bad);
      expect("attend Hk", attend(4, 4, v, 128, 2, 2, 16, 0, 512), bad);
      expect("attend D", attend(4, 4, 2, v, 2, 2, 16, 0, 512), bad);
      if (v != 0) expect("attend B", attend(4, 4, 2, 128, v, 2, 16, 0, 512), bad);
      if (v != 0) expect("attend width", attend(4, 4, 2, 128, 2, v, 16, 0, 512), bad);
      expect("attend page", attend(4, 4, 2, 128, 2, 2, v, 0, 512), bad);
      if (v < 0) expect("attend window", attend(4, 4, 2, 128, 2, 2, 16, v, 512), bad);
      expect("attend stride", attend(4, 4, 2, 128, 2, 2, 16, 0, v), bad);
    }
    expect("attend empty", attend(0, 4, 2, 128, 2, 2, 16, INT64_MAX, 512), PQL_OK);
    // every size that is accepted has a workspace and a kernel's name
    for (int64_t T : {int64_t(-1), int64_t(0), int64_t(1), int64_t(300), int64_t(1) << 20, int64_t(1) << 28, INT64_MAX})
      for (int64_t H : {int64_t(1), int64_t(8), int64_t(128), INT64_MAX})
        for (int64_t B : {int64_t(0), int64_t(1), int64_t(1) << 20, INT64_MAX})
          for (int64_t width : {int64_t(0), int64_t(1), int64_t(1) << 26, INT64_MAX}) {
            size_t bytes = 1;
            const pql_status st = pql_kv_attention_workspace(scheme, T, H, 1, 64, B, width, 16, &bytes);
            const char* n = pql_kv_kernel_name(scheme, T, H, 1, 64, B, width, 16);
            if (!n || (st == PQL_OK && T > 0 && B > 0) != (*n != 0) || (st != PQL_OK && bytes != 0)) {
              std::printf("FAIL workspace or name: T %lld H %lld B %lld width %lld\n", (long long)T, (long long)H,
                          (long long)B, (long long)width);
              ++failures;
            }
          }
  }
  std::printf("%s: %d failures\n", failures ? "FAILED" : "ok", failures);
  return failures ? 1 : 0;
}
