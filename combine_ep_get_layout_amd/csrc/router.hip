// The router on gfx950: top-k experts and their weights from a token's logits, and the
// gradient of the logits from that of the weights.
//
// With l a token's logits and s their scores (softmax, or sigmoid of each):
//   choice_e = s_e + bias_e (without a bias the logits themselves, which are in the same order)
//   a group of experts counts the sum of its group_top largest choices; of the groups the
//   groups_kept largest stay, and of their experts the K largest, ties to the lowest index
//   w_k = scale * s_k / sum_j s_j  (normalised)  or  scale * s_k.
// Gradients, with D = sum_k dw_k w_k / scale, over the experts that were chosen:
//   normalised:  dl_e = w_e (dw_e - D),  for sigmoid times (1 - s_e);  0 elsewhere
//   sigmoid:     dl_e = scale dw_e s_e (1 - s_e)
//   softmax:     dl_e = scale s_e (dw_e - sum_k dw_k s_k), for every expert.
//
// LPT lanes take a token, PER consecutive experts each, so that the first lane with the
// largest value also has its lowest index.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "experts_choice.hpp"
#include "router.hpp"

namespace ep {

constexpr int kRouteThreads = 256;

// ---- lanes of a token ----------------------------------------------------------

__device__ __forceinline__ float low_inf() { return -__builtin_inff(); }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}

// The two values that step STEP of a butterfly joins, the same pair in both lanes: of
// lanes 1, 2, 4 and 8 apart (the latter two mirrored, which is the same once the smaller
// steps are done), of rows of 16 lanes and of halves of the wave.
template <int STEP>
__device__ __forceinline__ void exchange(uint32_t v, uint32_t& a, uint32_t& b) {
  if constexpr (STEP < 4) {
    a = v;
    b = dpp<STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140>(v);
  } else if constexpr (STEP == 4) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  }
}

template <int STEP>
__device__ __forceinline__ void exchange(float v, float& a, float& b) {
  uint32_t x, y;
  exchange<STEP>(__float_as_uint(v), x, y);
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}

template <int STEP>
__device__ __forceinline__ void exchange(double v, double& a, double& b) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, v);
  uint32_t x0, y0, x1, y1;
  exchange<STEP>((uint32_t)bits, x0, y0);
  exchange<STEP>((uint32_t)(bits >> 32), x1, y1);
  a = __builtin_bit_cast(double, (uint64_t)x1 << 32 | x0);
  b = __builtin_bit_cast(double, (uint64_t)y1 << 32 | y0);
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }

template <int LPT, int STEP = 0, class V>
__device__ __forceinline__ V all_max(V v) {
  if constexpr ((1 << STEP) < LPT) {
    V a, b;
    exchange<STEP>(v, a, b);
    return all_max<LPT, STEP + 1>(larger(a, b));
  } else {
    return v;
  }
}

template <int LPT, int STEP = 0, class V>
__device__ __forceinline__ V all_sum(V v) {
  if constexpr ((1 << STEP) < LPT) {
    V a, b;
    exchange<STEP>(v, a, b);
    return all_sum<LPT, STEP + 1>(a + b);
  } else {
    return v;
  }
}

// The two largest values of several lanes.
template <class V>
struct Top2 {
  V first, second;
  __device__ __forceinline__ void add(V v) {
    second = larger(second, smaller(first, v));
    first = larger(first, v);
  }
  // joins lanes 2^STEP apart while that is below `lanes`
  template <int LPT, int STEP = 0>
  __device__ __forceinline__ void join(int lanes) {
    if constexpr ((1 << STEP) < LPT) {
      if ((1 << STEP) < lanes) {
        V a1, b1, a2, b2;
        exchange<STEP>(first, a1, b1);
        exchange<STEP>(second, a2, b2);
        first = larger(a1, b1);
        second = larger(smaller(a1, b1), larger(a2, b2));
        join<LPT, STEP + 1>(lanes);
      }
    }
  }
  // the sum of the `top` largest that there are
  __device__ __forceinline__ V sum(int top) const {
    return top == 2 && second > (V)low_inf() ? first + second : first;
  }
};

// The token's lanes of a ballot, and their first.
template <int LPT>
__device__ __forceinline__ uint64_t token_bits(uint64_t mask) {
  return LPT == 64 ? mask : mask >> (lane_id() & ~(LPT - 1)) & ((1ull << (LPT % 64)) - 1);
}

template <int LPT>
__device__ __forceinline__ int first_lane(uint64_t bits) {
  const int lane = __builtin_ctzll(bits | 1ull << (LPT - 1));
  return LPT == 64 ? uniform(lane) : lane;
}

// v of the token's lane `from`
template <int LPT>
__device__ __forceinline__ int of_lane(int v, int from) {
  if (LPT == 64) return __builtin_amdgcn_readlane(v, from);
  return __builtin_amdgcn_ds_bpermute(((lane_id() & ~(LPT - 1)) | from) << 2, v);
}
template <int LPT>
__device__ __forceinline__ float of_lane(float v, int from) {
  return __int_as_float(of_lane<LPT>(__float_as_int(v), from));
}
template <int LPT>
__device__ __forceinline__ double of_lane(double v, int from) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)of_lane<LPT>((int)(uint32_t)bits, from);
  const uint32_t hi = (uint32_t)of_lane<LPT>((int)(uint32_t)(bits >> 32), from);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// ---- values ---------------------------------------------------------------------

// PER consecutive logits as fp32, `fill` past the last expert; -0 becomes 0, which it equals.
template <int PER, bool BF16>
__device__ __forceinline__ void load_logits(const char* row, int first, int E, float fill,
                                            float (&l)[PER]) {
  constexpr int kBytes = PER * (BF16 ? 2 : 4);
  if (PER > 1 && E % PER == 0) {  // whole and aligned in every lane that has any
    union {
      uint32_t w[kBytes / 4];
      uint16_t b[kBytes / 2];
    } u;
    const char* from = row + (int64_t)(first < E ? first : 0) * (BF16 ? 2 : 4);
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = ((const uint4*)from)[i];
        u.w[4 * i] = v.x;
        u.w[4 * i + 1] = v.y;
        u.w[4 * i + 2] = v.z;
        u.w[4 * i + 3] = v.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 v = *(const uint2*)from;
      u.w[0] = v.x;
      u.w[1] = v.y;
    } else {
      u.w[0] = *(const uint32_t*)from;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      l[i] = first >= E ? fill
             : 0.0f + (BF16 ? (i % 2 ? bf16_hi(u.w[i / 2]) : bf16_lo(u.w[i / 2]))
                            : __uint_as_float(u.w[i]));
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = first + i < E ? first + i : 0;
      const float v = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)row)[e] << 16)
                           : ((const float*)row)[e];
      l[i] = first + i < E ? 0.0f + v : fill;
    }
  }
}

__device__ __forceinline__ float exponential(float v) { return expf(v); }
__device__ __forceinline__ double exponential(double v) { return exp(v); }

// 1 / (1 + exp(-v)), relatively exact for large negative v too
template <class V>
__device__ __forceinline__ V sigmoid_of(V v) {
  const V z = exponential(v < (V)0 ? v : -v);
  return (v < (V)0 ? z : (V)1) / ((V)1 + z);
}

// ---- the choice -------------------------------------------------------------------

// One token's experts in LPT lanes.  V: the type that choices are compared in.
template <int LPT, int PER, class V>
struct Choice {
  const RouteArgs& a;
  const int at, first;     // lane of the token, and its first expert
  V c[PER];
  V most = 0, total = 1;   // softmax: the largest logit and the sum of exp(l - most)

  __device__ __forceinline__ explicit Choice(const RouteArgs& a_)
      : a(a_), at(lane_id() & (LPT - 1)), first(at * PER) {}

  __device__ __forceinline__ V score(float l) const {
    if (a.sigmoid) return sigmoid_of((V)l);
    return exponential((V)l - most) / total;
  }

  __device__ __forceinline__ void softmax_sums(const float (&l)[PER]) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, l[i]);
    m = all_max<LPT>(m);
    most = (V)(m > low_inf() ? m : 0.0f);
    V sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += exponential((V)l[i] - most);
    total = all_sum<LPT>(sum);
  }

  // c of every expert; whether some is not a number
  __device__ __forceinline__ bool fill(const float (&l)[PER], const float (&bias)[PER]) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (a.scored) {
        c[i] = l[i] > low_inf() ? score(l[i]) + (V)bias[i] : (V)low_inf();
        bad |= c[i] != c[i];
      } else {
        c[i] = (V)l[i];
      }
    }
    return bad;
  }

  // Experts outside the kept groups to -inf.  Returns by how much the last kept group is
  // ahead of the first one left.
  __device__ __forceinline__ V keep_groups() {
    const int size = a.group_size, lanes = size / PER;
    V mine;       // the score of group at / lanes, or of group `at`
    bool stays[PER];
    V lowest = (V)__builtin_inff(), highest = (V)low_inf();
    if (size % PER == 0 && (lanes & (lanes - 1)) == 0 && lanes <= LPT) {
      // a group is a power of two of lanes
      Top2<V> top{c[0], (V)low_inf()};
#pragma unroll
      for (int i = 1; i < PER; ++i) top.add(c[i]);
      top.template join<LPT>(lanes);
      mine = top.sum(a.group_top);
      const int own = at / lanes;
      int rank = 0;
      for (int g = 0; g < a.groups; ++g) {
        const V other = of_lane<LPT>(mine, g * lanes);
        rank += other > mine || (other == mine && g < own);
      }
      const bool in = own < a.groups, stay = in && rank < a.groups_kept;
#pragma unroll
      for (int i = 0; i < PER; ++i) stays[i] = stay;
      if (stay) lowest = mine;
      else if (in) highest = mine;
    } else {
      mine = (V)low_inf();
      for (int g = 0; g < a.groups; ++g) {
        Top2<V> top{(V)low_inf(), (V)low_inf()};
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = first + i - g * size;
          top.add(e >= 0 && e < size ? c[i] : (V)low_inf());
        }
        top.template join<LPT>(LPT);
        if (g == at) mine = top.sum(a.group_top);
      }
      int rank = 0;
      for (int g = 0; g < a.groups; ++g) {
        const V other = of_lane<LPT>(mine, g);
        rank += other > mine || (other == mine && g < at);
      }
      const bool in = at < a.groups, stay = in && rank < a.groups_kept;
      const uint64_t kept = token_bits<LPT>(__ballot(stay));
      int group = first / size, rest = first - group * size;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        stays[i] = group < a.groups && (kept >> group & 1) != 0;
        if (++rest == size) rest = 0, ++group;
      }
      if (stay) lowest = mine;
      else if (in) highest = mine;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!stays[i]) c[i] = (V)low_inf();
    return -all_max<LPT>(-lowest) - all_max<LPT>(highest);
  }

  // The n largest, one a lane: id -1 where there are no more.
  __device__ __forceinline__ void largest(int n, V& value, int& id) {
    value = (V)low_inf();
    id = -1;
    for (int k = 0; k < n; ++k) {
      V best = c[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) best = larger(best, c[i]);
      const V top = all_max<LPT>(best);
      const bool any = top > (V)low_inf();
      if (__ballot(any) == 0) return;
      const int from = first_lane<LPT>(token_bits<LPT>(__ballot(any && best == top)));
      // the lane's first expert of that value, taken out
      int which = PER;
      bool open = at == from && any;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const bool hit = open && c[i] == top;
        if (hit) c[i] = (V)low_inf(), which = i;
        open = open && !hit;
      }
      const int e = of_lane<LPT>(first + which, from);
      if (at == k && any) value = top, id = e;
    }
  }
};

template <int LPT, int PER, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void route(RouteArgs a) {
  constexpr int kTokens = kRouteThreads / LPT;
  typedef Choice<LPT, PER, double> Exact;
  const int at = lane_id() & (LPT - 1), first = at * PER;
  float bias[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    bias[i] = a.bias && first + i < a.E ? a.bias[first + i] : 0.0f;
  for (int64_t base = (int64_t)blockIdx.x * kTokens; base < a.tokens;
       base += (int64_t)gridDim.x * kTokens) {
    const int64_t t = base + threadIdx.x / LPT;
    const bool in = t < a.tokens;  // lanes without a token repeat the last one
    const int64_t token = in ? t : a.tokens - 1;
    const char* row = (const char*)a.logits + token * a.E * (BF16 ? 2 : 4);
    float l[PER];
    load_logits<PER, BF16>(row, first, a.E, low_inf(), l);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      bad |= l[i] != l[i] || (!a.sigmoid && l[i] == __builtin_inff());

    Exact exact(a);
    if (!a.sigmoid && (a.scored || !a.normalize)) exact.softmax_sums(l);
    bad |= exact.fill(l, bias);
    bad = token_bits<LPT>(__ballot(bad)) != 0;
    if (a.groups_kept < a.groups) exact.keep_groups();
    if (a.scored && !a.bias)  // the logits are in the scores' order, and told apart where those are 1
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (exact.c[i] > (double)low_inf()) exact.c[i] = l[i];
    double value;
    int id;
    exact.largest(a.K, value, id);
    if (bad) id = -1;

    // weights: lane k has entry k
    const bool has = id >= 0;
    float mine = low_inf();
    if (has)
      mine = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)row)[id] << 16)
                  : ((const float*)row)[id];
    const float top = all_max<LPT>(mine);
    float w = 0.0f;
    if (has) {
      // sigmoids so small that they might vanish are exponentials
      if (a.sigmoid && !(a.normalize && top < -30.0f)) w = sigmoid_of(mine);
      else if (a.normalize) w = expf(mine - top);
      else w = expf(mine - (float)exact.most) / (float)exact.total;
    }
    if (a.normalize) {
      const float sum = all_sum<LPT>(w);
      if (has) w = w / sum;
    }
    if (in && at < a.K) {
      a.idx[t * a.K + at] = id;
      a.weights[t * a.K + at] = w * a.scale;
    }
    if (bad && in && at == 0) set_err(a.err, EP_DEVERR_LOGITS);
  }
}

// ---- gradient -----------------------------------------------------------------------

template <int PER, bool BF16>
__device__ __forceinline__ void store_logits(char* row, int first, int E, const float (&g)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (first + i < E) {
      if (BF16) ((__bf16*)row)[first + i] = (__bf16)g[i];
      else ((float*)row)[first + i] = g[i];
    }
  }
}

template <int LPT, int PER, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void route_grad(RouteGradArgs a) {
  constexpr int kTokens = kRouteThreads / LPT;
  const int at = lane_id() & (LPT - 1), first = at * PER;
  for (int64_t base = (int64_t)blockIdx.x * kTokens; base < a.tokens;
       base += (int64_t)gridDim.x * kTokens) {
    const int64_t t = base + threadIdx.x / LPT;
    const bool in = t < a.tokens;
    const int64_t token = in ? t : a.tokens - 1;
    const int64_t size = BF16 ? 2 : 4;
    float l[PER];
    load_logits<PER, BF16>((const char*)a.logits + token * a.E * size, first, a.E, low_inf(), l);
    int id = at < a.K ? a.idx[token * a.K + at] : -1;
    float dw = at < a.K ? a.dweights[token * a.K + at] : 0.0f;
    if (id < -1 || id >= a.E) {
      if (in) set_err(a.err, EP_DEVERR_TOPK_RANGE);
      id = -1;
    }
    // an expert's part of the entries: how many name it, and the sum of their gradients
    float count[PER], d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) count[i] = d[i] = 0.0f;
    bool any = false;
    for (int k = 0; k < a.K; ++k) {
      const int e = of_lane<LPT>(id, k);
      const float g = of_lane<LPT>(dw, k);
      any |= e >= 0;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e == first + i) count[i] += 1.0f, d[i] += g;
    }
    float g[PER];
    // softmax over the chosen experts where it is normalised, over all otherwise
    float most = low_inf();
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!a.normalize || count[i] > 0.0f) most = fmaxf(most, l[i]);
    most = all_max<LPT>(most);
    if (!(most > low_inf())) most = 0.0f;
    const bool small = a.sigmoid && a.normalize && most < -30.0f;
    float s[PER], rest[PER], sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (a.sigmoid) {
        const float z = expf(l[i] < 0.0f ? l[i] : -l[i]), r = 1.0f / (1.0f + z);
        s[i] = l[i] < 0.0f ? z * r : r;
        rest[i] = l[i] < 0.0f ? r : z * r;  // 1 - s
        if (small) s[i] = expf(l[i] - most);
      } else {
        s[i] = expf(l[i] - most);
        rest[i] = 1.0f;
      }
      if (a.normalize) {
        s[i] = count[i] > 0.0f ? s[i] : 0.0f;
        sum += count[i] * s[i];
      } else if (!a.sigmoid) {
        sum += s[i];
      }
      dot += d[i] * s[i];
    }
    float part = 1.0f, mean = 0.0f;
    if (a.normalize || !a.sigmoid) {
      sum = all_sum<LPT>(sum);
      part = sum > 0.0f ? 1.0f / sum : 0.0f;
      mean = all_sum<LPT>(dot) * part;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float less = a.normalize ? count[i] * mean : a.sigmoid ? 0.0f : mean;
      g[i] = a.scale * (s[i] * part) * (d[i] - less) * rest[i];
      // without a chosen expert there is no gradient, whatever the logits hold
      if (!any || ((a.normalize || a.sigmoid) && count[i] == 0.0f)) g[i] = 0.0f;
    }
    if (in)
      store_logits<PER, BF16>((char*)a.dlogits + token * a.E * size, first, a.E, g);
  }
}

// ---- launches -------------------------------------------------------------------------

constexpr int64_t kRouteBlocks = 8 * kCus;

#define EP_ROUTE_FORMS(KERNEL)                                                                \
  do {                                                                                        \
    if (a.bf16) EP_ROUTE_TYPE(KERNEL, true);                                                  \
    else EP_ROUTE_TYPE(KERNEL, false);                                                        \
  } while (0)
#define EP_ROUTE_TYPE(KERNEL, BF16)                                                           \
  do {                                                                                        \
    if (narrow && a.E <= 64) EP_ROUTE_LAUNCH(KERNEL, 16, 4, BF16);                            \
    else if (narrow && a.E <= 128) EP_ROUTE_LAUNCH(KERNEL, 16, 8, BF16);                      \
    else if (narrow && a.E <= 256) EP_ROUTE_LAUNCH(KERNEL, 16, 16, BF16);                     \
    else if (a.E <= 128) EP_ROUTE_LAUNCH(KERNEL, 64, 2, BF16);                                \
    else if (a.E <= 512) EP_ROUTE_LAUNCH(KERNEL, 64, 8, BF16);                                \
    else EP_ROUTE_LAUNCH(KERNEL, 64, 32, BF16);                                               \
  } while (0)
#define EP_ROUTE_LAUNCH(KERNEL, LPT, PER, BF16)                                               \
  hipLaunchKernelGGL((KERNEL<LPT, PER, BF16>),                                                \
                     dim3((unsigned)std::min((a.tokens * LPT + kRouteThreads - 1) /           \
                                                 kRouteThreads, kRouteBlocks)),               \
                     dim3(kRouteThreads), 0, st, a)

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const bool narrow = a.K < 16 && (a.groups_kept == a.groups || a.groups <= 16);
  EP_ROUTE_FORMS(route);
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const bool narrow = a.K <= 16;
  EP_ROUTE_FORMS(route_grad);
  return hipGetLastError();
}

}  // namespace ep
