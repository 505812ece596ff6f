// Expert routing and the grouping of assignments by expert, gfx950.
//
// Route: for each token the k experts of highest choice score, and their weights.
//   s_e = softmax(x)_e or sigmoid(x_e);  choice c_e = s_e + b_e (b: a bias that balances the
//   experts, in the choice only);  without a bias the choice is the logits' own order, which
//   is the scores' order;  optionally only the best groups of experts take part (a group's
//   score is its best choice, or the sum of its two best);  ties go to the lowest index;
//   weight = s (without the bias), divided by the sum over the k where asked, times a factor.
// With a bias two experts' choices can be closer than fp32 resolves them, and then the order
// itself would depend on rounding, so scores and choices are formed in fp64 there; without
// one the keys are the logits, compared exactly.
#include <algorithm>
#include <type_traits>

#include "pql_device.hpp"
#include "pql_internal.hpp"

namespace pql {

namespace {

constexpr int kRouteThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr double kNegInfD = -__builtin_huge_val();

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (DT == 0) return static_cast<const float*>(p)[i];
  else if constexpr (DT == 1) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  else return (float)static_cast<const _Float16*>(p)[i];
}

// L lanes per token, V logits per lane: lane i of the token's L holds experts i, i + L, ...
template <int DT, int L, int V, bool WIDE>
__global__ __launch_bounds__(kRouteThreads) void k_moe_route(RouteArgs r) {
  using Key = std::conditional_t<WIDE, double, float>;
  constexpr Key kOut = WIDE ? (Key)kNegInfD : (Key)kNegInf;
  constexpr int kTokens = kRouteThreads / L;
  __shared__ double choice_lds[kTokens][L * V];   // groups only: the choices by expert
  __shared__ double group_lds[kTokens][64];
  const int lane = threadIdx.x % L, sub = threadIdx.x / L;
  const int64_t token = (int64_t)blockIdx.x * kTokens + sub;
  const int64_t t = std::min<int64_t>(token, r.T - 1);   // lanes past the last token repeat it, and store nothing
  const int E = r.E;

  float x[V];
  bool broken = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + lane;
    x[v] = e < E ? load_logit<DT>(r.logits, t * r.ldl + e) : kNegInf;
    broken |= !(x[v] < -kNegInf);   // NaN or +inf
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) broken |= (bool)__shfl_xor((int)broken, o, L);
  float top = kNegInf;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (broken) x[v] = kNegInf;
    top = fmaxf(top, x[v]);
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, L));
  const double dtop = top > kNegInf ? (double)top : 0.0;
  const bool softmax = r.score == 0;

  // the softmax's denominator (every expert takes part, masked ones with 0)
  double denom = 1.0;
  if (softmax) {
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += x[v] > kNegInf ? exp((double)x[v] - dtop) : 0.0;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) sum += __shfl_xor(sum, o, L);
    denom = sum;
  }
  auto score = [&](float xv) -> double {
    if (!(xv > kNegInf)) return 0.0;
    return softmax ? exp((double)xv - dtop) / denom : 1.0 / (1.0 + exp(-(double)xv));
  };

  Key key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + lane;
    key[v] = kOut;
    if (x[v] > kNegInf) {
      if constexpr (WIDE) {
        const double c = score(x[v]) + (double)r.bias[e];
        if (c > kNegInfD) key[v] = c;
      } else {
        key[v] = x[v];
      }
    }
  }

  if (r.groups > 1) {
    const int per = E / r.groups;
    const bool top2 = r.group_score == 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + lane;
      double c = kNegInfD;
      if (key[v] > kOut) {
        if constexpr (WIDE) c = key[v];
        else c = top2 ? score(x[v]) : (double)x[v];
      }
      if (e < E) choice_lds[sub][e] = c;
    }
    __syncthreads();
    for (int g = lane; g < r.groups; g += L) {
      double a = kNegInfD, b = kNegInfD;   // the two best
      for (int i = 0; i < per; ++i) {
        const double c = choice_lds[sub][g * per + i];
        b = fmax(b, fmin(a, c));
        a = fmax(a, c);
      }
      group_lds[sub][g] = top2 && b > kNegInfD ? a + b : a;
    }
    __syncthreads();
    uint64_t kept = 0;
    for (int g = 0; g < r.groups; ++g) {
      const double s = group_lds[sub][g];
      int rank = 0;
      for (int h = lane; h < r.groups; h += L) {
        const double q = group_lds[sub][h];
        rank += q > s || (q == s && h < g);
      }
#pragma unroll
      for (int o = 1; o < L; o <<= 1) rank += __shfl_xor(rank, o, L);
      if (rank < r.top_groups) kept |= uint64_t(1) << g;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!((kept >> std::min((v * L + lane) / per, 63)) & 1)) key[v] = kOut;
  }

  // k rounds: the best key of the token's lanes, lowest index first among equals
  constexpr int kSlots = L >= 32 ? 1 : 32 / L;   // results a lane keeps (k <= 32)
  int my_id[kSlots];
  float my_x[kSlots];
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    my_id[q] = -1;
    my_x[q] = kNegInf;
  }
  for (int j = 0; j < r.k; ++j) {
    Key best = kOut;
    int at = 0x7fffffff;
    float bx = kNegInf;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v * L + lane;
        bx = x[v];
      }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      const Key ob = __shfl_xor(best, o, L);
      const int oa = __shfl_xor(at, o, L);
      const float ox = __shfl_xor(bx, o, L);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
        bx = ox;
      }
    }
    const bool found = best > kOut;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (found && at == v * L + lane) key[v] = kOut;
#pragma unroll
    for (int q = 0; q < kSlots; ++q)
      if (found && j == q * L + lane) {
        my_id[q] = at;
        my_x[q] = bx;
      }
  }

  double w[kSlots], sum = 0.0;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    w[q] = score(my_x[q]);
    sum += w[q];
  }
  if (r.renormalize) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) sum += __shfl_xor(sum, o, L);
#pragma unroll
    for (int q = 0; q < kSlots; ++q) w[q] = sum > 0.0 ? w[q] / sum : 0.0;
  }
  if (token >= r.T) return;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const int j = q * L + lane;
    if (j >= r.k) continue;
    r.ids[t * r.k + j] = my_id[q];
    r.weights[t * r.k + j] = broken ? __builtin_nanf("") : (float)(w[q] * (double)r.scale);
  }
}

template <int DT, int L, int V>
hipError_t launch_route_shape(const RouteArgs& r, hipStream_t st) {
  const dim3 grid((unsigned)((r.T + kRouteThreads / L - 1) / (kRouteThreads / L)));
  if (r.bias) hipLaunchKernelGGL((k_moe_route<DT, L, V, true>), grid, dim3(kRouteThreads), 0, st, r);
  else hipLaunchKernelGGL((k_moe_route<DT, L, V, false>), grid, dim3(kRouteThreads), 0, st, r);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_route_type(const RouteArgs& r, hipStream_t st) {
  if (r.E <= 64) return launch_route_shape<DT, 16, 4>(r, st);
  if (r.E <= 128) return launch_route_shape<DT, 16, 8>(r, st);
  if (r.E <= 256) return launch_route_shape<DT, 16, 16>(r, st);
  if (r.E <= 512) return launch_route_shape<DT, 32, 16>(r, st);
  return launch_route_shape<DT, 64, 16>(r, st);
}

// ---------------------------------------------------------------- grouping
// A stable counting sort by expert.  One workgroup walks the assignments in rounds of 512:
// a wave ranks its 64 ids among themselves with one ballot per bit of the id, the waves'
// counts per expert are summed in wave order, and every round starts where the last ended.
constexpr int kPlanThreads = 512, kPlanWaves = kPlanThreads / 64;

__global__ __launch_bounds__(kPlanThreads) void k_moe_plan(const int32_t* __restrict__ ids, int P, int E,
                                                           int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                           int32_t* __restrict__ slots) {
  extern __shared__ int plan_lds[];
  int* next = plan_lds;              // [E]: where an expert's next assignment goes
  int* count = plan_lds + E;         // [kPlanWaves][E]
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int bits = 32 - __builtin_clz(E);   // ids 0 .. E (E: not held here)
  for (int e = t; e < E; e += kPlanThreads) next[e] = 0;
  __syncthreads();
  for (int i = t; i < P; i += kPlanThreads) {
    const int id = ids[i];
    if ((unsigned)id < (unsigned)E) atomicAdd(&next[id], 1);   // integer counts: any order gives the same
  }
  __syncthreads();
  if (wave == 0) {   // exclusive prefix over the experts
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int n = e0 + lane < E ? next[e0 + lane] : 0;
      int s = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o);
        if (lane >= o) s += u;
      }
      if (e0 + lane < E) {
        next[e0 + lane] = carry + s - n;
        offsets[e0 + lane] = carry + s - n;
      }
      carry += __shfl(s, 63);
    }
    if (lane == 0) offsets[E] = carry;
    if (lane == 0) count[0] = carry;
  }
  __syncthreads();
  const int total = count[0];
  __syncthreads();
  for (int i = total + t; i < P; i += kPlanThreads) order[i] = -1;
  for (int base = 0; base < P; base += kPlanThreads) {
    const int i = base + t;
    int id = i < P ? ids[i] : E;
    if ((unsigned)id >= (unsigned)E) id = E;
    for (int q = t; q < kPlanWaves * E; q += kPlanThreads) count[q] = 0;
    __syncthreads();
    uint64_t same = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (id < E && rank == 0) count[wave * E + id] = __popcll(same);
    __syncthreads();
    for (int e = t; e < E; e += kPlanThreads) {
      int at = next[e];
      for (int w = 0; w < kPlanWaves; ++w) {
        const int n = count[w * E + e];
        count[w * E + e] = at;
        at += n;
      }
      next[e] = at;
    }
    __syncthreads();
    if (i < P) {
      const int place = id < E ? count[wave * E + id] + rank : -1;
      slots[i] = place;
      if (place >= 0) order[place] = i;
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_moe_route(int dtype, const RouteArgs& r, hipStream_t st) {
  switch (dtype) {
    case 0: return launch_route_type<0>(r, st);
    case 1: return launch_route_type<1>(r, st);
    default: return launch_route_type<2>(r, st);
  }
}

size_t moe_plan_ws_bytes(int64_t, int) { return 0; }
const char* moe_plan_kernel_name(int64_t, int) { return "k_moe_plan"; }

hipError_t launch_moe_plan(const int32_t* ids, int64_t P, int E, int32_t* offsets, int32_t* order, int32_t* slots,
                           int32_t*, hipStream_t st) {
  const size_t lds = sizeof(int) * (size_t)E * (kPlanWaves + 1);   // 36,864 bytes at most (E = 1024)
  hipLaunchKernelGGL(k_moe_plan, dim3(1), dim3(kPlanThreads), lds, st, ids, (int)P, E, offsets, order, slots);
  return hipGetLastError();
}

}  // namespace pql
