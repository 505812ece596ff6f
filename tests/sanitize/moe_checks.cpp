// Argument validation of the mixture-of-experts entry points under AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code of abi.cpp (test infrastructure): every call must
// be refused, or accepted as an empty no-op, before a device is touched.  Fake pointers are never
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
  auto route = [&](int64_t T, int64_t E, int64_t ldl, int64_t k, int64_t groups, int64_t top, float scale) {
    return pql_moe_route(0, 0, P(), T, E, ldl, nullptr, k, groups, top, 0, 1, scale, i32, f32, nullptr);
  };
  for (int64_t v : extremes) {
    if (v != 0) expect("route T", route(v, 16, 16, 2, 1, 1, 1.f), bad);
    expect("route E", route(4, v, v, 2, 1, 1, 1.f), bad);
    expect("route k", route(4, 16, 16, v, 1, 1, 1.f), bad);
    expect("route groups", route(4, 16, 16, 2, v, 1, 1.f), bad);
    expect("route top_groups", route(4, 16, 16, 2, 4, v, 1.f), bad);
    if (v <= 0 || v >= INT64_MAX - 1) expect("route ldl", route(4, 16, v, 2, 1, 1, 1.f), bad);
  }
  expect("route scale", route(4, 16, 16, 2, 1, 1, std::nanf("")), bad);
  expect("route empty", route(0, 16, 16, 2, 1, 1, 1.f), PQL_OK);

  size_t bytes = 0;
  for (int64_t v : extremes) {
    if (v != 0) expect("plan workspace T", pql_moe_plan_workspace(v, 2, 16, &bytes), bad);
    expect("plan workspace k", pql_moe_plan_workspace(4, v, 16, &bytes), bad);
    expect("plan workspace E", pql_moe_plan_workspace(4, 2, v, &bytes), bad);
    expect("plan E", pql_moe_plan(i32, 4, 2, v, i32, i32, i32, nullptr, 0, nullptr), bad);
  }
  expect("plan workspace", pql_moe_plan_workspace(1 << 20, 8, 1024, &bytes), PQL_OK);
  expect("plan short workspace", pql_moe_plan(i32, 1 << 20, 8, 1024, i32, i32, i32, P(), bytes - 1, nullptr),
         PQL_ERR_WORKSPACE);
  expect("plan workspace NULL", pql_moe_plan_workspace(4, 2, 16, nullptr), bad);

  auto gemm = [&](int scheme, int64_t rows, int gather, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K,
                  int64_t ldc) {
    return pql_moe_qgemm(scheme, P(), P(), rows, gather, P(), P(), i32, i32, T, k, E, N, K, P(), ldc, nullptr);
  };
  for (int scheme : {(int)PQL_FP8_ROW, (int)PQL_FP8_BLOCK128})
    for (int64_t v : extremes) {
      if (v != 0) expect("gemm T", gemm(scheme, v, 1, v, 2, 8, 256, 256, 256), bad);
      expect("gemm k", gemm(scheme, 8, 0, 4, v, 8, 256, 256, 256), bad);
      expect("gemm E", gemm(scheme, 8, 0, 4, 2, v, 256, 256, 256), bad);
      expect("gemm N", gemm(scheme, 8, 0, 4, 2, 8, v, 256, 256), bad);
      expect("gemm K", gemm(scheme, 8, 0, 4, 2, 8, 256, v, 256), bad);
      expect("gemm ldc", gemm(scheme, 8, 0, 4, 2, 8, 256, 256, v), bad);
      expect("gemm rows", gemm(scheme, v, 0, 4, 2, 8, 256, 256, 256), bad);
    }
  expect("gemm scheme", gemm(PQL_INT8_ROW, 8, 0, 4, 2, 8, 256, 256, 256), PQL_ERR_UNSUPPORTED);
  expect("gemm weight too large", gemm(PQL_FP8_ROW, 8, 0, 4, 2, 1024, 1 << 20, 1 << 20, 1 << 20), bad);
  expect("gemm empty", gemm(PQL_FP8_ROW, 0, 1, 0, 2, 8, 256, 256, 256), PQL_OK);

  for (int64_t v : extremes) {
    if (v != 0)
      expect("swiglu rows", pql_swiglu_quantize(PQL_FP8_ROW, P(), v, 256, 512, nullptr, P(), P(), nullptr), bad);
    expect("swiglu cols", pql_swiglu_quantize(PQL_FP8_ROW, P(), 4, v, 512, nullptr, P(), P(), nullptr), bad);
    expect("swiglu ldx", pql_swiglu_quantize(PQL_FP8_ROW, P(), 4, 256, v, nullptr, P(), P(), nullptr), bad);
    expect("combine N", pql_moe_combine(P(), 8, 64, i32, f32, 4, 2, v, nullptr, 0, P(), 64, nullptr), bad);
    if (v != 0) expect("combine T", pql_moe_combine(P(), 8, 64, i32, f32, v, 2, 64, nullptr, 0, P(), 64, nullptr), bad);
    expect("combine ldy", pql_moe_combine(P(), 8, v, i32, f32, 4, 2, 64, nullptr, 0, P(), 64, nullptr), bad);
    expect("combine ldo", pql_moe_combine(P(), 8, 64, i32, f32, 4, 2, 64, nullptr, 0, P(), v, nullptr), bad);
    expect("combine ldadd", pql_moe_combine(P(), 8, 64, i32, f32, 4, 2, 64, P(), v, P(), 64, nullptr), bad);
    if (v != 0) expect("combine rows", pql_moe_combine(P(), v, 64, i32, f32, 4, 2, 64, nullptr, 0, P(), 64, nullptr), bad);
  }

  for (int scheme = -1; scheme <= 9; ++scheme)
    for (int gather : {0, 1})
      for (int64_t T : {int64_t(-1), int64_t(0), int64_t(1), int64_t(37), int64_t(8192), int64_t(1) << 24, INT64_MAX})
        for (int64_t N : {int64_t(0), int64_t(1), int64_t(4096), int64_t(1) << 20, INT64_MAX}) {
          const char* n = pql_moe_kernel_name(scheme, gather, T, 8, 64, N, 1 << 20);
          if (!n) { std::printf("FAIL kernel name NULL\n"); ++failures; }
          else (void)std::strlen(n);
        }
  std::printf("%s: %d failures\n", failures ? "FAILED" : "ok", failures);
  return failures ? 1 : 0;
}
