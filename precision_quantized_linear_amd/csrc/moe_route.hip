// Expert routing and the grouping of assignments by expert, gfx950.
//
// Route: for each token the k experts of highest choice score, and their weights.
//   s_e = softmax(x)_e or sigmoid(x_e);  choice c_e = s_e + b_e (b: a bias that balances the
//   experts, in the choice only);  without a bias the choice is the logits' own order, which
//   is the scores' order;  optionally only the best groups of experts take part (a group's
//   score is its best choice, or the sum of its two best);  ties go to the lowest index;
//   weight = s (without the bias), divided by the sum over the k where asked, times a factor.
// With a bias two experts' choices can be closer than fp32 resolves them, and then the order
// itself would depend on rounding, so the order is that of the fp64 choices.  Forming E of them
// per token in fp64 costs more than everything else, so the choices are formed in fp32 with a
// bound on their error (delta), the k best and whatever lies within 2 delta of the k-th become
// candidates, one per lane, and only those are evaluated in fp64 and ranked.  Where the fp32
// choices cannot settle it (more candidates than lanes, group scores within the bound of each
// other) the wave takes the fp64 path for all E.  Without a bias the keys are the logits,
// compared exactly.
#include <algorithm>
#include <type_traits>

#include "pql_device.hpp"
#include "pql_internal.hpp"

namespace pql {

namespace {

constexpr int kRouteThreads = 256;
// Up to this many tokens a wave takes one token (E = 256 with bias and groups: 2048 tokens 7.7 us
// a launch against 8.1 with two tokens a wave, 4096 tokens 10.0 against 9.3).
constexpr int64_t kRouteWide = 2048;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr double kNegInfD = -__builtin_huge_val();

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (DT == 0) return static_cast<const float*>(p)[i];
  else if constexpr (DT == 1) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  else return (float)static_cast<const _Float16*>(p)[i];
}

// Reductions over a token's L lanes, the result in every lane: DPP inside rows of 16, lane
// swaps between rows (no LDS permutes: k rounds of two reductions each are one long chain).
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL, class T>
__device__ __forceinline__ T dpp_of(T v) {
  if constexpr (sizeof(T) == 8) {
    const v2i w = __builtin_bit_cast(v2i, v);
    return __builtin_bit_cast(T, v2i{dpp<CTRL>(w.x), dpp<CTRL>(w.y)});
  } else {
    return __builtin_bit_cast(T, dpp<CTRL>(__builtin_bit_cast(int, v)));
  }
}
template <int L, class F, class T>
__device__ __forceinline__ T reduce(T v, F f) {
  static_assert(L == 16 || L == 32 || L == 64);
  auto step = [&](auto ctrl) __attribute__((always_inline)) {
    v = f(v, dpp_of<decltype(ctrl)::value>(v));
  };
  step(std::integral_constant<int, 0xB1>{});    // lane ^ 1
  step(std::integral_constant<int, 0x4E>{});    // lane ^ 2
  step(std::integral_constant<int, 0x141>{});   // the other quad of 8
  step(std::integral_constant<int, 0x140>{});   // the other 8 of 16
  auto swap = [&](auto rows) __attribute__((always_inline)) {   // both sides' values, in every lane
    constexpr int n = sizeof(T) / 4;
    uint32_t w[2], a[2], b[2];
    __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if constexpr (decltype(rows)::value == 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(w[i], w[i], false, false);
        a[i] = p[0];
        b[i] = p[1];
      } else {
        const auto p = __builtin_amdgcn_permlane32_swap(w[i], w[i], false, false);
        a[i] = p[0];
        b[i] = p[1];
      }
    }
    T va, vb;
    __builtin_memcpy(&va, a, sizeof(T));
    __builtin_memcpy(&vb, b, sizeof(T));
    v = f(va, vb);
  };
  if constexpr (L >= 32) swap(std::integral_constant<int, 16>{});
  if constexpr (L >= 64) swap(std::integral_constant<int, 32>{});
  return v;
}
template <int L> __device__ __forceinline__ float lanes_max(float v) { return reduce<L>(v, [](float a, float b) { return fmaxf(a, b); }); }
template <int L> __device__ __forceinline__ int lanes_min(int v) { return reduce<L>(v, [](int a, int b) { return std::min(a, b); }); }
template <int L> __device__ __forceinline__ float lanes_sum(float v) { return reduce<L>(v, [](float a, float b) { return a + b; }); }
template <int L> __device__ __forceinline__ double lanes_max(double v) { return reduce<L>(v, [](double a, double b) { return fmax(a, b); }); }
template <int L> __device__ __forceinline__ double lanes_sum(double v) { return reduce<L>(v, [](double a, double b) { return a + b; }); }

// 1 / (1 + exp(-x)) and exp(x - top): fp64 for the order and for weights too small for fp32.
__device__ __forceinline__ double score64(bool softmax, float x, double top, double denom) {
  if (!(x > kNegInf)) return 0.0;
  return softmax ? exp((double)x - top) / denom : 1.0 / (1.0 + exp(-(double)x));
}

// The best key of a lane and its place among the lane's V.
template <int V, class Key>
__device__ __forceinline__ void lane_best(const Key (&key)[V], Key out, Key& best, int& at) {
  best = out;
  at = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (key[v] > best) {
      best = key[v];
      at = v;
    }
}

// One round: the best key over the token's lanes, taken out of its lane; its expert (the lowest
// among equals) or -1.
template <int L, int V, class Key>
__device__ __forceinline__ int take_best(Key (&key)[V], Key out, Key& best, int& at, int lane, Key& value) {
  value = lanes_max<L>(best);
  const bool found = value > out;
  const int id = lanes_min<L>(found && best == value ? at * L + lane : 0x7fffffff);
  if (id == at * L + lane) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v == at) key[v] = out;
    lane_best<V>(key, out, best, at);
  }
  return found ? id : -1;
}

// i / n for 0 <= i < 1024, 1 <= n <= 1024: (i + 1/2) / n is at least 1 / (2 n) away from a whole
// number, far more than the fp32 error, so rounding down is exact (an integer division is ~30
// instructions, and a lane needs one per logit).
__device__ __forceinline__ int small_div(int i, float inverse_n) { return (int)(((float)i + 0.5f) * inverse_n); }

// Groups of experts: the mask of the kept ones.  `choice` (LDS, the token's own) holds the
// choices by expert, `score` room for the groups'.  Scores within `slack` of each other are not told apart: then
// `unsure` is set (slack 0: equal scores go to the lowest group).
template <int L, class Key>
__device__ __forceinline__ uint64_t kept_groups(const RouteArgs& r, int per, const Key* choice, Key* score, int lane,
                                                Key slack, bool& unsure) {
  const float inverse_per = 1.0f / (float)per;
  const Key out = (Key)kNegInfD;
  // share lanes (1, 2, 4 or 8) read a group together
  const int share = r.groups * 8 <= L ? 8 : r.groups * 4 <= L ? 4 : r.groups * 2 <= L ? 2 : 1;
  for (int g0 = 0; g0 < r.groups; g0 += L) {
    const int g = g0 + lane / share, part = lane & (share - 1);
    Key a = out, b = out;   // the two best
    if (g < r.groups) {
      int at = (threadIdx.x & 63) - part;   // groups start apart: they and the tokens would share LDS banks
      if (at >= per) at -= small_div(at, inverse_per) * per;
#pragma unroll 4
      for (int i = part; i < per; i += share) {
        const int place = at + i >= per ? at + i - per : at + i;
        const Key c = choice[g * per + place];
        b = c > a ? a : (c > b ? c : b);
        a = c > a ? c : a;
      }
    }
    auto merge = [&](auto ctrl) __attribute__((always_inline)) {
      const Key oa = dpp_of<decltype(ctrl)::value>(a), ob = dpp_of<decltype(ctrl)::value>(b);
      const Key low = oa < a ? oa : a, high = ob > b ? ob : b;
      a = oa > a ? oa : a;
      b = low > high ? low : high;
    };
    if (share > 1) merge(std::integral_constant<int, 0xB1>{});
    if (share > 2) merge(std::integral_constant<int, 0x4E>{});
    if (share > 4) merge(std::integral_constant<int, 0x141>{});
    if (g < r.groups && part == 0) score[g] = r.group_score == 1 && b > out ? a + b : a;
  }
  asm volatile("" ::: "memory");   // a token's lanes share a wave, whose LDS accesses run in order
  uint64_t kept = 0;
  bool open = false;
  for (int g0 = 0; g0 < r.groups; g0 += L) {
    const int g = std::min(g0 + lane, r.groups - 1);
    const Key s = score[g];
    int above = 0, near = 0;   // certainly above; above or too close to tell
#pragma unroll 4
    for (int h = 0; h < r.groups; ++h) {
      const Key q = score[h];
      above += q > s + slack || (slack == 0 && q == s && h < g);
      near += h != g && q > s - slack;
    }
    const bool mine = above < r.top_groups && g0 + lane < r.groups;
    open |= slack > 0 && mine && near >= r.top_groups;
    const uint64_t bits = __ballot(mine) >> (threadIdx.x & 63 & ~(L - 1));
    kept |= (L == 64 ? bits : bits & ((uint64_t(1) << (L & 63)) - 1)) << g0;
  }
  const uint64_t any = __ballot(open) >> (threadIdx.x & 63 & ~(L - 1));
  unsure |= (L == 64 ? any : any & ((uint64_t(1) << (L & 63)) - 1)) != 0;
  return kept;
}

// L lanes per token, V logits per lane: lane i of the token's L holds experts i, i + L, ...
template <int DT, int L, int V, bool BIASED>
__global__ __launch_bounds__(kRouteThreads) void k_moe_route(RouteArgs r) {
  constexpr int kTokens = kRouteThreads / L;
  __shared__ double choice_lds[kTokens][L * V + 8];   // groups only: the choices by expert (padded: tokens on other banks)
  __shared__ double group_lds[kTokens][kMoeMaxGroups];
  const int lane = threadIdx.x % L, sub = threadIdx.x / L;
  const int64_t token = (int64_t)blockIdx.x * kTokens + sub;
  const int64_t t = std::min<int64_t>(token, r.T - 1);   // lanes past the last token repeat it, and store nothing
  const int E = r.E;
  const bool softmax = r.score == 0;
  const int per = r.per_group;
  const float inverse_per = 1.0f / (float)per;

  float x[V], bias[V];
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + lane;
    x[v] = e < E ? load_logit<DT>(r.logits, t * r.ldl + e) : kNegInf;
    if constexpr (BIASED) bias[v] = e < E ? r.bias[e] : kNegInf;
  }
  float top = kNegInf;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bad |= !(x[v] < -kNegInf);   // NaN or +inf
    top = fmaxf(top, x[v]);
  }
  const bool broken = lanes_min<L>(bad ? 0 : 1) == 0;
  if (broken) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = kNegInf;
    top = kNegInf;
  }
  top = lanes_max<L>(top);
  if (!(top > kNegInf)) top = 0.0f;
  auto score32 = [&](float xv, float denom) __attribute__((always_inline)) {   // 0 for an unavailable expert
    return softmax ? expf(xv - top) / denom : 1.0f / (1.0f + expf(-xv));
  };
  auto rough = [&](float xv, float inverse) __attribute__((always_inline)) {   // the same within the bound below
    constexpr float kLog2e = 1.44269504f;
    return softmax ? __builtin_amdgcn_exp2f((xv - top) * kLog2e) * inverse
                   : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(xv * -kLog2e));
  };
  float denom = 1.0f;   // the softmax's (unavailable experts add 0)
  if (softmax && (BIASED || !r.renormalize || r.groups > 1)) {
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += __builtin_amdgcn_exp2f((x[v] - top) * 1.44269504f);
    denom = lanes_sum<L>(sum);
  }
  const float inverse = BIASED || r.groups > 1 ? __builtin_amdgcn_rcpf(denom) : 1.0f;
  auto denom64 = [&]() __attribute__((always_inline)) {   // rare: reads the logits again
    double sum = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += L) {
      const float xv = load_logit<DT>(r.logits, t * r.ldl + e);
      sum += !broken && xv > kNegInf ? exp((double)xv - (double)top) : 0.0;
    }
    return lanes_sum<L>(sum);
  };

  // ---- fp32 keys, and the bound of their error, in units of u = 2^-24 (half an ulp of 1).  In
  // rough() the exponential of an argument y is off by (a |y| + 2) u relative: log2 e is rounded
  // (0.23), its product with y (1) and the softmax's y = x - top (1), and the instruction is within
  // one ulp (2): a = 1.23 and 2.23.
  //   sigmoid: that enters as s (1 - s) (1.23 |y| + 2) <= 0.7, the sum and the reciprocal of a
  //   value below 1 add 3: below 4 u.
  //   softmax: it enters as s (2.23 |y| + 2) <= 2.1 (s <= exp(y), y <= 0); the denominator's relative
  //   error, the terms' (their mean |y| is below ln E = 7) and at most 22 roundings, is below 40, its
  //   reciprocal and the product add 3: below 46 u.
  // Adding the bias rounds once more, |c| u.  Two choices are told apart by 2 delta, delta = (6 or
  // 50, and 2 |c|) u: two errors, and |c| u for the rounding of their difference or of c - 2 delta,
  // 2 (46 + |c|) + |c|.  A group's sum of two choices rounds by 2 |c| u, as does a sum plus or
  // minus the slack that tells two of them apart: 2 (2 (4 or 46, and |c|) + 2 |c|) + 2 |c| =
  // 16 or 184, and 10 |c|; 18 and 192 leave room for the slack's own part in the last rounding (it
  // is below 1: see `unsure`).
  float key[V];
  float biggest = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    key[v] = kNegInf;
    if (x[v] > kNegInf) {
      if constexpr (BIASED) {
        const float c = rough(x[v], inverse) + bias[v];
        if (c > kNegInf) {
          key[v] = c;
          biggest = fmaxf(biggest, fabsf(c));
        }
      } else {
        key[v] = x[v];
      }
    }
  }
  bool unsure = false;
  float delta = 0.0f;
  biggest = BIASED ? lanes_max<L>(biggest) : 1.0f;   // scores are at most 1
  if constexpr (BIASED) {
    delta = ((softmax ? 50.0f : 6.0f) + 2.0f * biggest) * 0x1p-24f;
    unsure = !(delta < 0.125f) || r.k > L - 2;   // biases of 2^20 and more; no lane left for a further candidate
  }
  if (r.groups > 1) {
    const bool exact = !BIASED && r.group_score == 0;   // the logits themselves
    float* choice = reinterpret_cast<float*>(choice_lds[sub]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float c = key[v];
      if constexpr (!BIASED) {
        if (r.group_score == 1 && c > kNegInf) c = rough(c, inverse);
      }
      choice[v * L + lane] = c;
    }
    asm volatile("" ::: "memory");
    const float slack = exact ? 0.0f : ((softmax ? 192.0f : 18.0f) + 10.0f * biggest) * 0x1p-24f;
    bool level = false;   // group scores too close for fp32
    uint64_t kept = kept_groups<L, float>(r, per, choice, reinterpret_cast<float*>(group_lds[sub]), lane, slack, level);
    if (__ballot(level)) {   // their choices in fp64, one token at a time on all 64 lanes
      asm volatile("" ::: "memory");
      const int wl = threadIdx.x & 63;
#pragma unroll 1
      for (int q = 0; q < 64 / L; ++q) {
        if (!__shfl((int)level, q * L)) continue;
        const int row = sub - wl / L + q;   // the token's place in the workgroup
        const int64_t tq = std::min<int64_t>((int64_t)blockIdx.x * kTokens + row, r.T - 1);
        const double tops = (double)__shfl(top, q * L);
        double z = 0.0;
#pragma unroll 1
        for (int e = wl; softmax && e < E; e += 64) z += score64(true, load_logit<DT>(r.logits, tq * r.ldl + e), tops, 1.0);
        z = softmax ? lanes_sum<64>(z) : 1.0;
#pragma unroll 1
        for (int e = wl; e < E; e += 64) {
          const float xv = load_logit<DT>(r.logits, tq * r.ldl + e);
          double c = kNegInfD;
          if (xv > kNegInf) {
            c = score64(softmax, xv, tops, z);
            if constexpr (BIASED) c = c + (double)r.bias[e] > kNegInfD ? c + (double)r.bias[e] : kNegInfD;
          }
          choice_lds[row][e] = c;
        }
      }
      asm volatile("" ::: "memory");
      bool never = false;
      const uint64_t kept64 = kept_groups<L, double>(r, per, choice_lds[sub], group_lds[sub], lane, 0.0, never);
      if (level) kept = kept64;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!((kept >> std::min(small_div(v * L + lane, inverse_per), 63)) & 1)) key[v] = kNegInf;
  }

  // ---- k rounds.  Lane j % L keeps the j-th (k <= 32).
  constexpr int kSlots = L >= 32 ? 1 : 32 / L;
  int my_id[kSlots];
  double my_w[kSlots];   // scores, then weights
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    my_id[q] = -1;
    my_w[q] = 0.0;
  }
  int rank0 = lane;      // the slot that lane's first result goes to
  if (!__ballot(unsure)) {
    float best, value = 0.0f, last = -kNegInf;
    int at;
    lane_best<V>(key, kNegInf, best, at);
    bool close = false;   // two neighbours in the order within the error bound of each other
    int j = 0;
    for (; j < r.k; ++j) {
      const int id = take_best<L, V>(key, kNegInf, best, at, lane, value);
      if constexpr (BIASED) {
        close |= value > kNegInf && last - value <= 2.0f * delta;
        last = value;
      }
#pragma unroll
      for (int q = 0; q < kSlots; ++q)
        if (j == q * L + lane) my_id[q] = id;
    }
    if constexpr (BIASED) {
      // whatever lies within 2 delta of the k-th may belong before it
      const float least = value - 2.0f * delta;
      bool more = value > kNegInf && lanes_max<L>(best) >= least;
      close |= more;
      for (; j < L && __ballot(more); ++j) {
        const int id = take_best<L, V>(key, kNegInf, best, at, lane, value);
        if (j == lane) my_id[0] = id;
        more = more && value > kNegInf && lanes_max<L>(best) >= least;
      }
      unsure = more;   // more candidates than lanes
    }
    if (__ballot(close)) {   // rank the candidates by their fp64 choices
      const double z = softmax ? denom64() : 1.0;
      const int id = my_id[0];
      const float xi = id >= 0 ? load_logit<DT>(r.logits, t * r.ldl + id) : kNegInf;
      my_w[0] = score64(softmax, xi, (double)top, z);
      const double c = id >= 0 ? my_w[0] + (double)r.bias[id] : kNegInfD;
      rank0 = 0;
      for (int q = 0; q < j; ++q) {
        const double oc = __shfl(c, q, L);
        const int oid = __shfl(id, q, L);
        rank0 += oid >= 0 && (id < 0 || oc > c || (oc == c && oid < id));
      }
      if (id < 0) rank0 = std::max(rank0, lane);   // empty slots after all candidates
    } else {
      bool tiny = false;
#pragma unroll
      for (int q = 0; q < kSlots; ++q)
        if (my_id[q] >= 0) {
          const float xi = load_logit<DT>(r.logits, t * r.ldl + my_id[q]);
          const float s = score32(xi, !BIASED && r.renormalize ? 1.0f : denom);
          my_w[q] = (double)s;
          tiny |= s < 0x1p-100f;
        }
      if (__ballot(tiny)) {   // weights near or below the end of fp32's range: in fp64
        const double z = softmax ? denom64() : 1.0;
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
          if (my_id[q] >= 0)
            my_w[q] = score64(softmax, load_logit<DT>(r.logits, t * r.ldl + my_id[q]), (double)top, z);
      }
    }
  }

  // ---- all of it in fp64, where fp32 did not settle the order of biased choices (wave-uniform)
  if constexpr (BIASED) {
    if (__ballot(unsure)) {
      const double z = softmax ? denom64() : 1.0;
      double wide[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        wide[v] = kNegInfD;
        if (x[v] > kNegInf) {
          const double c = score64(softmax, x[v], (double)top, z) + (double)r.bias[v * L + lane];
          if (c > kNegInfD) wide[v] = c;
        }
      }
      if (r.groups > 1) {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int v = 0; v < V; ++v) choice_lds[sub][v * L + lane] = wide[v];
        asm volatile("" ::: "memory");
        bool never = false;
        const uint64_t kept = kept_groups<L, double>(r, per, choice_lds[sub], group_lds[sub], lane, 0.0, never);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (!((kept >> std::min(small_div(v * L + lane, inverse_per), 63)) & 1)) wide[v] = kNegInfD;
      }
      double best, value;
      int at;
      lane_best<V>(wide, kNegInfD, best, at);
#pragma unroll
      for (int q = 0; q < kSlots; ++q) my_id[q] = -1;
      for (int j = 0; j < r.k; ++j) {
        const int id = take_best<L, V>(wide, kNegInfD, best, at, lane, value);
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
          if (j == q * L + lane) my_id[q] = id;
      }
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        const float xi = my_id[q] >= 0 ? load_logit<DT>(r.logits, t * r.ldl + my_id[q]) : kNegInf;
        my_w[q] = score64(softmax, xi, (double)top, z);
      }
      rank0 = lane;
    }
  }

  // ---- weights: over their sum where asked (0 where that is 0), times the factor
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const int j = q == 0 ? rank0 : q * L + lane;
    if (j >= r.k) my_w[q] = 0.0;   // a candidate that lost
    sum += my_w[q];
  }
  double factor = (double)r.scale;
  if (r.renormalize) {
    sum = lanes_sum<L>(sum);
    factor = sum > 0.0 ? factor / sum : 0.0;
  }
  if (token >= r.T) return;
#pragma unroll
  for (int q = 0; q < kSlots; ++q) {
    const int j = q == 0 ? rank0 : q * L + lane;
    if (j >= r.k) continue;
    r.ids[t * r.k + j] = my_id[q];
    r.weights[t * r.k + j] = broken ? __builtin_nanf("") : (float)(my_w[q] * factor);
  }
}

template <int DT, int L, int V, bool BIASED>
hipError_t launch_route_shape(const RouteArgs& r, hipStream_t st) {
  const dim3 grid((unsigned)((r.T + kRouteThreads / L - 1) / (kRouteThreads / L)));
  hipLaunchKernelGGL((k_moe_route<DT, L, V, BIASED>), grid, dim3(kRouteThreads), 0, st, r);
  return hipGetLastError();
}

// 16 lanes per token while a lane then holds at most 16 logits: a round's reductions serve four
// tokens of a wave at once (32 lanes for 129 - 256 experts with a bias, whose fp64 tail is then
// shorter: 4096 tokens 9.3 us against 10.7, 8192 tokens 12.4 against 11.9).  Few tokens take a wave each: shorter chains.
template <int DT, bool BIASED>
hipError_t launch_route_type(const RouteArgs& r, hipStream_t st) {
  if (r.T <= kRouteWide) {
    if (r.E <= 64) return launch_route_shape<DT, 64, 1, BIASED>(r, st);
    if (r.E <= 128) return launch_route_shape<DT, 64, 2, BIASED>(r, st);
    if (r.E <= 256) return launch_route_shape<DT, 64, 4, BIASED>(r, st);
    if (r.E <= 512) return launch_route_shape<DT, 64, 8, BIASED>(r, st);
  } else {
    if (r.E <= 64) return launch_route_shape<DT, 16, 4, BIASED>(r, st);
    if (r.E <= 128) return launch_route_shape<DT, 16, 8, BIASED>(r, st);
    if (r.E <= 256) return launch_route_shape<DT, BIASED ? 32 : 16, BIASED ? 8 : 16, BIASED>(r, st);
    if (r.E <= 512) return launch_route_shape<DT, 32, 16, BIASED>(r, st);
  }
  return launch_route_shape<DT, 64, 16, BIASED>(r, st);
}

// ---------------------------------------------------------------- grouping
// A stable counting sort by expert.  A workgroup owns a contiguous chunk of the assignments and
// a wave a contiguous part of the chunk, walked 64 ids at a time: a wave ranks its 64 ids among
// themselves with one ballot per bit of the id, and adds what it has counted before (a counter
// per wave and expert in LDS that only this wave touches, so no atomics and no order to lose).
// Up to kPlanChunk assignments take one launch of one workgroup; more take two: k_moe_count
// writes each chunk's counts, and every workgroup of k_moe_place sums those of all chunks and
// of the chunks before its own.  Latency throughout: 144 assignments 3.2 us, 65536 of 256
// experts 9.2.
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

// counts: [gridDim.x][E] from k_moe_count; unused by a single workgroup.  ROUNDS > 0: a wave's
// part is at most 64 ROUNDS ids, held in registers with their ranks (their loads are then one
// latency, not two per round); 0: any length, read and ranked twice.
template <int ROUNDS>
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
  // keep the compiler from reordering or merging them across lanes.  Returns the rank among the
  // wave's ids so far.
  auto count_in = [&](int id) __attribute__((always_inline)) {
    const uint64_t same = lanes_with(id);
    int rank = 0;
    if (id < E) rank = seen[wave][id] + __popcll(same & below);
    asm volatile("" ::: "memory");
    if (id < E && !(same & below)) seen[wave][id] += __popcll(same);
    asm volatile("" ::: "memory");
    return rank;
  };
  constexpr int kHeld = ROUNDS > 0 ? ROUNDS : 1;
  int held[kHeld], rank[kHeld];
  if constexpr (ROUNDS > 0) {
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) held[q] = id_at(begin + 64 * q + lane);
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) rank[q] = count_in(held[q]);
  } else {
    for (int i0 = begin; i0 < end; i0 += 64) count_in(id_at(i0 + lane));
  }
  __syncthreads();

  // per expert: all of its assignments, those of earlier chunks, and the waves' starts
  for (int e = t; e < E; e += kPlanThreads) {
    int all = 0, before = 0;
    if (gridDim.x == 1) {
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) all += seen[w][e];
    } else {
#pragma unroll 16
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

  // seen[wave][e] is now where the wave's first assignment of e goes, from the expert's start on
  auto put = [&](int i, int id, int place) __attribute__((always_inline)) {
    if (i < end) slots[i] = id < E ? place : -1;
    if (id < E) order[place] = i;
  };
  if constexpr (ROUNDS > 0) {
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) {
      const int id = held[q];
      put(begin + 64 * q + lane, id, id < E ? start[id] + seen[wave][id] + rank[q] : -1);
    }
  } else {
    for (int i0 = begin; i0 < end; i0 += 64) {
      const int id = id_at(i0 + lane);
      const int r = count_in(id);
      put(i0 + lane, id, id < E ? start[id] + r : -1);
    }
  }
  for (int64_t i = total + (int64_t)blockIdx.x * kPlanThreads + t; i < P; i += (int64_t)gridDim.x * kPlanThreads)
    order[i] = -1;
}

}  // namespace

hipError_t launch_moe_route(int dtype, const RouteArgs& r, hipStream_t st) {
  switch (dtype) {
    case 0: return r.bias ? launch_route_type<0, true>(r, st) : launch_route_type<0, false>(r, st);
    case 1: return r.bias ? launch_route_type<1, true>(r, st) : launch_route_type<1, false>(r, st);
    default: return r.bias ? launch_route_type<2, true>(r, st) : launch_route_type<2, false>(r, st);
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
  constexpr int kRounds = kPlanChunk / kPlanThreads;
  if (P <= kPlanThreads)
    hipLaunchKernelGGL(k_moe_place<1>, dim3(1), dim3(kPlanThreads), 0, st, ids, (int)P, E, kPlanThreads, ws, offsets,
                       order, slots);
  else if (chunk == kPlanChunk)
    hipLaunchKernelGGL(k_moe_place<kRounds>, dim3(blocks), dim3(kPlanThreads), 0, st, ids, (int)P, E, chunk, ws,
                       offsets, order, slots);
  else
    hipLaunchKernelGGL(k_moe_place<0>, dim3(blocks), dim3(kPlanThreads), 0, st, ids, (int)P, E, chunk, ws, offsets,
                       order, slots);
  return hipGetLastError();
}

}  // namespace pql
