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
// A stable counting sort by expert.  A workgroup owns a contiguous chunk of the assignments and
// a wave a contiguous part of the chunk, walked 64 ids at a time: a wave ranks its 64 ids among
// themselves with one ballot per bit of the id, and adds what it has counted before (a counter
// per wave and expert in LDS that only this wave touches, so no atomics and no order to lose).
// Up to kPlanChunk assignments take one launch of one workgroup; more take two: k_moe_count
// writes each chunk's counts, and every workgroup of k_moe_place sums those of all chunks and
// of the chunks before its own.
constexpr int kPlanThreads = 512, kPlanWaves = kPlanThreads / 64;
constexpr int kPlanChunk = 2048;
constexpr int kPlanMaxBlocks = 256;   // beyond 2^19 assignments the chunks grow instead

int64_t plan_chunk(int64_t P) {
  const int64_t per = (P + kPlanMaxBlocks - 1) / kPlanMaxBlocks;
  return std::max<int64_t>(kPlanChunk, (per + kPlanThreads - 1) / kPlanThreads * kPlanThreads);
}
int plan_blocks(int64_t P) { return (int)std::max<int64_t>(1, (P + plan_chunk(P) - 1) / plan_chunk(P)); }

__global__ __launch_bounds__(kPlanThreads) void k_moe_count(const int32_t* __restrict__ ids, int P, int E, int chunk,
                                                            int32_t* __restrict__ counts) {
  __shared__ int n[kMoeMaxExperts];
  for (int e = threadIdx.x; e < E; e += kPlanThreads) n[e] = 0;
  __syncthreads();
  const int end = (int)std::min<int64_t>(P, (int64_t)(blockIdx.x + 1) * chunk);
  for (int i = blockIdx.x * chunk + threadIdx.x; i < end; i += kPlanThreads) {
    const int id = ids[i];
    if ((unsigned)id < (unsigned)E) atomicAdd(&n[id], 1);   // whole numbers: any order gives the same
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kPlanThreads) counts[(int64_t)blockIdx.x * E + e] = n[e];
}

// counts: [gridDim.x][E] from k_moe_count; unused by a single workgroup.
__global__ __launch_bounds__(kPlanThreads) void k_moe_place(const int32_t* __restrict__ ids, int P, int E, int chunk,
                                                            const int32_t* __restrict__ counts,
                                                            int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                            int32_t* __restrict__ slots) {
  __shared__ int seen[kPlanWaves][kMoeMaxExperts];   // per wave: assignments of an expert so far
  __shared__ int start[kMoeMaxExperts];
  __shared__ int part[kMoeMaxExperts / 64 + 1];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int bits = 32 - __builtin_clz(E);            // ids 0 .. E (E: takes no part)
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int share = chunk / kPlanWaves;              // a multiple of 64
  const int begin = (int)std::min<int64_t>(P, (int64_t)blockIdx.x * chunk + (int64_t)wave * share);
  const int end = std::min(P, begin + share);
  for (int e = lane; e < E; e += 64) seen[wave][e] = 0;
  auto id_at = [&](int i) __attribute__((always_inline)) {
    const int id = i < end ? ids[i] : E;
    return (unsigned)id < (unsigned)E ? id : E;
  };
  auto lanes_with = [&](int id) __attribute__((always_inline)) {
    uint64_t same = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? set : ~set;
    }
    return same;
  };
  // Only this wave touches seen[wave], and LDS runs a wave's accesses in order; the fences
  // keep the compiler from reordering or merging them across lanes.
  for (int i0 = begin; i0 < end; i0 += 64) {
    const int id = id_at(i0 + lane);
    const uint64_t same = lanes_with(id);
    if (id < E && !(same & below)) seen[wave][id] += __popcll(same);
    asm volatile("" ::: "memory");
  }
  __syncthreads();

  // per expert: all of its assignments, those of earlier chunks, and the waves' starts
  for (int e = t; e < E; e += kPlanThreads) {
    int all = 0, before = 0;
    if (gridDim.x == 1) {
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) all += seen[w][e];
    } else {
#pragma unroll 8
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const int n = counts[(int64_t)b * E + e];
        all += n;
        before += b < (int)blockIdx.x ? n : 0;
      }
    }
    start[e] = all;
    int at = before;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const int n = seen[w][e];
      seen[w][e] = at;
      at += n;
    }
  }
  __syncthreads();
  // exclusive prefix of start[] over the experts: 64 at a time, then the sums before them
  for (int e0 = wave * 64; e0 < E; e0 += kPlanThreads) {
    const int n = e0 + lane < E ? start[e0 + lane] : 0;
    int s = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(s, o);
      if (lane >= o) s += u;
    }
    if (e0 + lane < E) start[e0 + lane] = s - n;
    if (lane == 63) part[e0 / 64] = s;
  }
  __syncthreads();
  int total = 0;
  for (int q = 0; q < (E + 63) / 64; ++q) total += part[q];
  for (int e = t; e < E; e += kPlanThreads) {
    int base = start[e];
    for (int q = 0; q < e / 64; ++q) base += part[q];
    start[e] = base;
    if (blockIdx.x == 0) offsets[e] = base;
  }
  if (blockIdx.x == 0 && t == 0) offsets[E] = total;
  __syncthreads();

  for (int i0 = begin; i0 < end; i0 += 64) {
    const int i = i0 + lane;
    const int id = id_at(i);
    const uint64_t same = lanes_with(id);
    int place = -1;
    if (id < E) place = start[id] + seen[wave][id] + __popcll(same & below);
    asm volatile("" ::: "memory");
    if (id < E && !(same & below)) seen[wave][id] += __popcll(same);
    asm volatile("" ::: "memory");
    if (i < end) slots[i] = place;
    if (place >= 0) order[place] = i;
  }
  for (int64_t i = total + (int64_t)blockIdx.x * kPlanThreads + t; i < P; i += (int64_t)gridDim.x * kPlanThreads)
    order[i] = -1;
}

}  // namespace

hipError_t launch_moe_route(int dtype, const RouteArgs& r, hipStream_t st) {
  switch (dtype) {
    case 0: return launch_route_type<0>(r, st);
    case 1: return launch_route_type<1>(r, st);
    default: return launch_route_type<2>(r, st);
  }
}

size_t moe_plan_ws_bytes(int64_t P, int E) {
  const int blocks = plan_blocks(P);
  return blocks > 1 ? sizeof(int32_t) * (size_t)blocks * (size_t)E : 0;
}

const char* moe_plan_kernel_name(int64_t P) { return plan_blocks(P) > 1 ? "k_moe_count+k_moe_place" : "k_moe_place"; }

hipError_t launch_moe_plan(const int32_t* ids, int64_t P, int E, int32_t* offsets, int32_t* order, int32_t* slots,
                           int32_t* ws, hipStream_t st) {
  const int blocks = plan_blocks(P), chunk = (int)plan_chunk(P);
  if (blocks > 1) hipLaunchKernelGGL(k_moe_count, dim3(blocks), dim3(kPlanThreads), 0, st, ids, (int)P, E, chunk, ws);
  hipLaunchKernelGGL(k_moe_place, dim3(blocks), dim3(kPlanThreads), 0, st, ids, (int)P, E, chunk, ws, offsets, order,
                     slots);
  return hipGetLastError();
}

}  // namespace pql
