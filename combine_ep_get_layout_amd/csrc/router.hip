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
// largest value also has its lowest index.  Choices are compared in fp32, and where two that
// decide are nearer to each other than that tells, again in 64 bits, a token at a time: all
// in 64 bits took 61 us for 32,768 tokens over 256 experts (8 groups, bias).  These take 28
// to 31 us now, 1.2 TB/s, bound by vector instructions (82% of what the busy compute units can
// issue); one token over 64 experts 4.4 us, latency.  The gradient, softmax over 128 experts,
// 131,072 tokens in bf16: 16 to 18 us, 4.3 to 4.6 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "experts.hpp"
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
  __device__ __forceinline__ V magnitude() const {
    return (first > (V)low_inf() ? fabs(first) : (V)0) + (second > (V)low_inf() ? fabs(second) : (V)0);
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

// v of the token's lane `from`, which is the same in all lanes of the token
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

// v of the lane after this one; of the token's last lane whatever
__device__ __forceinline__ float of_next(float v) {
  return __int_as_float(
      __builtin_amdgcn_ds_bpermute(((lane_id() + 1) & (kWave - 1)) << 2, __float_as_int(v)));
}

// ---- values ---------------------------------------------------------------------

// The same value, of which the compiler knows nothing: what rare branches compute from it
// stays in them instead of being computed and kept in registers for all tokens.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// `per` consecutive logits as fp32, `fill` behind them and past the last expert; -0 becomes 0,
// which it equals.
template <int PER, bool BF16>
__device__ __forceinline__ void load_logits(const char* row, int first, int E, float fill,
                                            float (&l)[PER], int per = PER) {
  constexpr int kBytes = PER * (BF16 ? 2 : 4);
  if (PER > 1 && E % PER == 0 && per == PER) {  // whole and aligned in every lane that has any
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
    // one lane's address, not one for each expert: that many registers would halve the waves
    const int f = here(first);
    const char* from = row + (int64_t)f * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      l[i] = fill;
      if (i < per && f + i < E)
        l[i] = 0.0f + (BF16 ? __uint_as_float((uint32_t)((const uint16_t*)from)[i] << 16)
                            : ((const float*)from)[i]);
    }
  }
}

// In fp32 the hardware's exponential and reciprocal, for choices, gradients and the sum that
// softmax weights which are not normalised are divided by: the exponential's argument times
// log2 e is rounded to 2^-24 of itself, results below 2^-126 are 0.
__device__ __forceinline__ float exponential(float v) {
  return __builtin_amdgcn_exp2f(v * 1.4426950408889634f);
}
__device__ __forceinline__ float inverse(float v) { return __builtin_amdgcn_rcpf(v); }

// 1 / (1 + exp(-v)), relatively exact for large negative v too
__device__ __forceinline__ float sigmoid_of(float v) {
  const float z = exponential(-fabsf(v));
  return (v < 0.0f ? z : 1.0f) * inverse(1.0f + z);
}

// for weights, as expf and their quotients are: each step rounded correctly, or to a unit in the
// last place
__device__ __forceinline__ float sigmoid_exact(float v) {
  const float z = expf(v < 0.0f ? v : -v);
  return (v < 0.0f ? z : 1.0f) / (1.0f + z);
}

// ---- the choice -------------------------------------------------------------------

// One token's experts in LPT lanes, in fp32.
template <int LPT, int PER>
struct Choice {
  const RouteArgs& a;
  const int at, first;     // lane of the token, and its first expert
  float c[PER];
  float most = 0, total = 1, part = 1;  // softmax: the largest logit, the sum of exp(l - most), its inverse

  __device__ __forceinline__ explicit Choice(const RouteArgs& a_)
      : a(a_), at(lane_id() & (LPT - 1)), first(at * a_.per) {}

  __device__ __forceinline__ void softmax_sums(const float (&l)[PER]) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, l[i]);
    m = all_max<LPT>(m);
    most = m > low_inf() ? m : 0.0f;
    float sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += exponential(l[i] - most);
    total = all_sum<LPT>(sum);
    part = inverse(total);
  }

  // c of every expert; whether some is not a number.  One branch for all values.
  __device__ __forceinline__ bool fill(const float (&l)[PER], const float* bias_row) {
    if (!a.scored) {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = l[i];
    } else {
      float bias[PER];
      if (bias_row) {
        load_logits<PER, false>((const char*)bias_row, first, a.E, 0.0f, bias, a.per);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) bias[i] = 0.0f;
      }
      if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; ++i) c[i] = sigmoid_of(l[i]) + bias[i];
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) c[i] = __builtin_fmaf(exponential(l[i] - most), part, bias[i]);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = l[i] == low_inf() ? low_inf() : c[i];
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) bad |= c[i] != c[i];
    if (!a.sigmoid)
#pragma unroll
      for (int i = 0; i < PER; ++i) bad |= l[i] == __builtin_inff();
    return bad;
  }

  // Experts outside the kept groups to -inf.  Whether the last kept group is no more than
  // `sure` and 2^-22 of the choices in a sum (its additions) ahead of the first one left.
  __device__ __forceinline__ bool keep_groups(float sure) {
    const int size = a.group_size, lanes = size / a.per;
    float mine;       // the score of group at / lanes, or of group `at`
    bool stays[PER];
    float lowest = __builtin_inff(), highest = low_inf(), size_of = 0.0f;
    if (size % a.per == 0 && (lanes & (lanes - 1)) == 0 && lanes <= LPT) {
      // a group is a power of two of lanes
      Top2<float> top{c[0], low_inf()};
#pragma unroll
      for (int i = 1; i < PER; ++i) top.add(c[i]);
      top.template join<LPT>(lanes);
      mine = top.sum(a.group_top);
      size_of = top.magnitude();
      const int own = at / lanes;
      int rank = 0;
      for (int g = 0; g < a.groups; ++g) {
        const float other = of_lane<LPT>(mine, g * lanes);
        rank += other > mine || (other == mine && g < own);
      }
      const bool in = own < a.groups, stay = in && rank < a.groups_kept;
#pragma unroll
      for (int i = 0; i < PER; ++i) stays[i] = stay;
      if (stay) lowest = mine;
      else if (in) highest = mine;
    } else {
      mine = low_inf();
      for (int g = 0; g < a.groups; ++g) {
        Top2<float> top{low_inf(), low_inf()};
        const int f = here(first) - g * size;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = f + i;
          top.add(e >= 0 && e < size ? c[i] : low_inf());
        }
        top.template join<LPT>(LPT);
        if (g == at) mine = top.sum(a.group_top);
        size_of = fmaxf(size_of, top.magnitude());
      }
      int rank = 0;
      for (int g = 0; g < a.groups; ++g) {
        const float other = of_lane<LPT>(mine, g);
        rank += other > mine || (other == mine && g < at);
      }
      const bool in = at < a.groups, stay = in && rank < a.groups_kept;
      const uint64_t kept = token_bits<LPT>(__ballot(stay));
      const int f = here(first);
      int group = f / size, rest = f - group * size;
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
      if (!stays[i]) c[i] = low_inf();
    lowest = -all_max<LPT>(-lowest);
    highest = all_max<LPT>(highest);
    return highest > low_inf() && !(lowest - highest > sure + 0x1p-22f * all_max<LPT>(size_of));
  }

  // The n largest, one a lane: id -1 where there are no more.
  __device__ __forceinline__ void largest(int n, float& value, int& id) {
    value = low_inf();
    id = -1;
    for (int k = 0; k < n; ++k) {
      float best = c[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) best = larger(best, c[i]);
      const float top = all_max<LPT>(best);
      const bool any = top > low_inf();
      if (__ballot(any) == 0) return;
      const int from = first_lane<LPT>(token_bits<LPT>(__ballot(any && best == top)));
      // the lane's first expert of that value, taken out
      int which = PER;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i) which = c[i] == top ? i : which;
      const int e = of_lane<LPT>(first + which, from);
      which = at == from && any ? which : PER;
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = i == which ? low_inf() : c[i];
      if (at == k && any) value = top, id = e;
    }
  }
};

template <bool BF16>
__device__ __forceinline__ float logit_at(const char* row, int e) {
  return 0.0f + (BF16 ? __uint_as_float((uint32_t)((const uint16_t*)row)[e] << 16)
                      : ((const float*)row)[e]);
}

// Writes a token's entries, entry k's expert (or -1) in its lane k.  most, total: softmax, as
// softmax_sums has them, so that weights go by the logits alone and not by how the token was
// chosen.  The sum is within 2^-18 of itself (score_error), which is as large an error of weights
// that are not normalised; all others are within a few units in the last place, and half of one
// for each unit that the logit is below the largest (its difference is rounded).
template <int LPT, bool BF16>
__device__ __forceinline__ void store_entries(const RouteArgs& a, const char* row, int64_t t, int id,
                                              float most, float total) {
  const int at = lane_id() & (LPT - 1);
  const bool has = id >= 0;
  const float mine = has ? logit_at<BF16>(row, id) : low_inf();
  const float top = all_max<LPT>(mine);
  float w = 0.0f;
  if (has) {
    // sigmoids so small that they might vanish are exponentials
    if (a.sigmoid && !(a.normalize && top < -30.0f)) w = sigmoid_exact(mine);
    else if (a.normalize) w = expf(mine - top);
    else w = expf(mine - most) / total;
  }
  if (a.normalize) {
    const float sum = all_sum<LPT>(w);
    if (has) w = w / sum;
  }
  if (t < a.tokens && at < a.K) {
    a.idx[t * a.K + at] = id;
    a.weights[t * a.K + at] = w * a.scale;
  }
}

// A token chosen in 64 bits, by the whole wave; c: its choices in LDS, total32: its sum in
// fp32.  Lane l has experts per l .. as above.  Few tokens come here (of 32,768 tens), but the
// last of them ends the kernel: what counts is one token's latency.  More do where equal choices
// stand at the border of a choice in 64 lanes (32,768 tokens over 1,024 experts in bf16, softmax:
// 194 us under a random bias, 328 under one of zeros).
template <bool BF16>
__device__ __forceinline__ void route_exactly(const RouteArgs& a, int64_t t, float total32,
                                              double* c) {
  const char* row = (const char*)a.logits + t * a.E * (BF16 ? 2 : 4);
  const int lane = lane_id(), per = (a.E + kWave - 1) / kWave;
  const int first = min(lane * per, a.E), end = min(first + per, a.E);
  double most = 0.0, total = 1.0;
  if (!a.sigmoid) {
    float m = low_inf();
#pragma unroll 4
    for (int e = first; e < end; ++e) m = fmaxf(m, logit_at<BF16>(row, e));
    m = all_max<64>(m);
    if (m > low_inf()) most = m;
    total = 0.0;
#pragma unroll 4
    for (int e = first; e < end; ++e) total += exp((double)logit_at<BF16>(row, e) - most);
    total = all_sum<64>(total);
  }
#pragma unroll 4
  for (int e = first; e < end; ++e) {
    const float l = logit_at<BF16>(row, e);
    const double x = a.sigmoid ? (l < 0.0f ? (double)l : -(double)l) : (double)l - most;
    const double z = exp(x);
    const double score = a.sigmoid ? (l < 0.0f ? z : 1.0) / (1.0 + z) : z / total;
    c[e] = l > low_inf() ? score + (a.bias ? (double)a.bias[e] : 0.0) : (double)low_inf();
  }
  wave_lds_sync();
  if (a.groups_kept < a.groups) {
    Top2<double> top{(double)low_inf(), (double)low_inf()};
    if (lane < a.groups)
#pragma unroll 8
      for (int i = 0; i < a.group_size; ++i) top.add(c[lane * a.group_size + i]);
    const double mine = top.sum(a.group_top);
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
      const double other = of_lane<64>(mine, g);
      rank += other > mine || (other == mine && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.groups_kept);
    wave_lds_sync();
#pragma unroll 4
    for (int e = first; e < end; ++e) {
      if (!(kept >> e / a.group_size & 1)) c[e] = (double)low_inf();
      else if (!a.bias) c[e] = (double)logit_at<BF16>(row, e);
    }
    wave_lds_sync();
  }
  int id = -1;
#pragma unroll 1
  for (int k = 0; k < a.K; ++k) {
    double best = (double)low_inf();
    int at = first;
#pragma unroll 4
    for (int e = first; e < end; ++e)
      if (c[e] > best) best = c[e], at = e;
    const double top = all_max<64>(best);
    if (!(top > (double)low_inf())) break;
    const int e = __builtin_amdgcn_readlane(at, __builtin_ctzll(__ballot(best == top)));
    if (lane == k) id = e;
    if (lane == 0) c[e] = (double)low_inf();
    wave_lds_sync();
  }
  store_entries<64, BF16>(a, row, t, id, (float)most, total32);
}

// A token's candidates, one in each of its 16 lanes: value (-inf: none) and expert.
struct Candidate {
  float value;
  int id;
};

// v of the token's lane `by` places on, in turn
template <int BY>
__device__ __forceinline__ float rotated(float v) {
  return __uint_as_float(dpp<0x120 + BY>(__float_as_uint(v)));
}
template <int BY>
__device__ __forceinline__ int rotated(int v) {
  return (int)dpp<0x120 + BY>((uint32_t)v);
}
template <int BY>
__device__ __forceinline__ double rotated(double v) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<0x120 + BY>((uint32_t)(bits >> 32)) << 32 |
                                        dpp<0x120 + BY>((uint32_t)bits));
}

// Calls f with 1 .. 15, as constants.
template <int BY = 1, class F>
__device__ __forceinline__ void each_rotation(F f) {
  if constexpr (BY < 16) {
    f(std::integral_constant<int, BY>());
    each_rotation<BY + 1>(f);
  }
}

// How many of the token's candidates come before this lane's.
template <class V>
__device__ __forceinline__ int rank_of(V value, int id) {
  int rank = 0;
  each_rotation([&](auto by) {
    const V v = rotated<decltype(by)::value>(value);
    const int e = rotated<decltype(by)::value>(id);
    rank += v > value || (v == value && e < id);
  });
  return rank;
}

// The candidates of 16 lanes with PER choices each: the n largest (n <= 16), or all that there
// are, and, with sure > 0, all that are no more than sure and 2^-23 of both below the n-th.
// False where they are more than 16.  Of the lanes' two largest the n-th is found by counting;
// it is no larger than the n-th of all.  (With a round over all lanes for each of the n largest
// 32,768 tokens over 256 experts took 40 us instead of 30.)
template <int PER>
__device__ __forceinline__ bool candidates(const float (&c)[PER], int first, int n, float sure,
                                           Candidate* slots, Candidate& mine) {
  const int at = lane_id() & 15;
  Top2<float> top{c[0], low_inf()};
#pragma unroll
  for (int i = 1; i < PER; ++i) top.add(c[i]);
  int above_first = 0, above_second = 1;
  each_rotation([&](auto by) {
    const float a = rotated<decltype(by)::value>(top.first);
    const float b = rotated<decltype(by)::value>(top.second);
    above_first += a > top.first;
    above_first += b > top.first;
    above_second += a > top.second;
    above_second += b > top.second;
  });
  // the smallest of those with fewer than n above them
  const float least = above_second < n ? top.second : above_first < n ? top.first : __builtin_inff();
  float from = -all_max<16>(-least);
  // the n-th of all lies between this and the largest
  if (sure > 0.0f) from -= sure + 0x1p-21f * (fabsf(from) + fabsf(all_max<16>(top.first)));
  if (!(from > low_inf())) from = -__FLT_MAX__;  // every number
  int count = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) count += c[i] >= from;
  int upto = count;
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const int v = __shfl_up(upto, d, 16);
    if (at >= d) upto += v;
  }
  const int total = of_lane<16>(upto, 15);
  Candidate* to = slots + upto - count;
  if (total <= 16)
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (c[i] >= from) *to++ = Candidate{c[i], first + i};
  wave_lds_sync();
  mine = at < total && total <= 16 ? slots[at] : Candidate{low_inf(), -1};
  wave_lds_sync();
  return total <= 16;
}

// How far off a score in fp32 may be.  Sigmoid: z = exp(-|l|) is off by 2^-23 of itself and
// by |l| z 2^-24 <= 0.37 2^-24 for its rounded argument, one plus it by 2^-24, the reciprocal
// by 2^-23: together less than 1.6 2^-23.  Softmax: the exponential likewise, and their sum, of
// 32 values a lane one after another and in six steps between lanes, by 38 2^-24 of itself
// beside, so less than 2^-18 of the largest score.
__device__ __forceinline__ float score_error(const RouteArgs& a, float largest) {
  return a.sigmoid ? 0x1p-22f : 0x1p-18f * largest;
}

// The first part of a wave's tokens in fp32; false for a token that has to be chosen again.
// total: softmax, the sum that its weights are divided by
template <int LPT, int PER, bool BF16>
__device__ __forceinline__ bool route_fast(const RouteArgs& a, int64_t t, Candidate* slots,
                                           float& total) {
  const int at = lane_id() & (LPT - 1), first = at * a.per;
  const bool in = t < a.tokens;  // lanes without a token repeat the last one
  const int64_t token = in ? t : a.tokens - 1;
  const char* row = (const char*)a.logits + token * a.E * (BF16 ? 2 : 4);
  float l[PER];
  load_logits<PER, BF16>(row, first, a.E, low_inf(), l, a.per);
  Choice<LPT, PER> choice(a);
  if (!a.sigmoid && (a.scored || !a.normalize)) choice.softmax_sums(l);
  total = choice.total;
  const bool bad = token_bits<LPT>(__ballot(choice.fill(l, a.bias))) != 0;
  // two choices have to be this far apart, four (a group's sum of two) twice as far
  const float sure = a.scored ? 2.0f * score_error(a, choice.part) : 0.0f;
  bool close = false;
  if (a.groups_kept < a.groups) close = choice.keep_groups(2.0f * sure) && a.scored;
  if (a.scored && !a.bias)  // the logits are in the scores' order, and told apart where those are 1
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (choice.c[i] > low_inf()) choice.c[i] = l[i];
  const bool check = a.bias != nullptr;
  float value;
  int id;
  bool chosen = false;
  if constexpr (LPT == 16) {
    // n candidates and those that might be as large as the last of them
    Candidate mine;
    chosen = __ballot(!candidates<PER>(choice.c, first, a.K, check ? sure : 0.0f, slots, mine)) == 0;
    if (chosen) {
      int rank = rank_of(mine.value, mine.id);
      if (check) {
        // two that are nearer to each other than fp32 tells, one of them among the first K
        bool near = false;
        each_rotation([&](auto by) {
          const float other = rotated<decltype(by)::value>(mine.value);
          near |= other > low_inf() && !(fabsf(mine.value - other) >
                                         sure + 0x1p-23f * (fabsf(mine.value) + fabsf(other)));
        });
        near = near && mine.id >= 0 && rank < a.K && !bad;
        if (__ballot(near) != 0) {
          const float logit = mine.id >= 0 ? logit_at<BF16>(row, mine.id) : 0.0f;
          const float bias = mine.id >= 0 ? a.bias[mine.id] : 0.0f;
          if (a.sigmoid) {
            const double l = logit, z = exp(l < 0.0 ? l : -l);
            const double by = mine.id >= 0 ? (l < 0.0 ? z : 1.0) / (1.0 + z) + (double)bias
                                           : (double)low_inf();
            rank = rank_of(by, mine.id);
          } else {
            // The sum of all in 64 bits, but not for equal logits and biases: they make equal
            // choices in any number of bits, and are in their order.  32,768 tokens over 256
            // experts in bf16 under a bias of zeros, where four in ten have such a pair, took 88
            // us with it and take 26.
            bool differ = false;
            each_rotation([&](auto by) {
              const float other = rotated<decltype(by)::value>(mine.value);
              const float l = rotated<decltype(by)::value>(logit);
              const float b = rotated<decltype(by)::value>(bias);
              differ |= other > low_inf() && !(l == logit && b == bias) &&
                        !(fabsf(mine.value - other) >
                          sure + 0x1p-23f * (fabsf(mine.value) + fabsf(other)));
            });
            close |= near && differ;
          }
        }
      }
      // lanes without a candidate come after all that have one, each at a rank of its own
      if (mine.id < 0) rank = at;
      slots[at].id = -1;
      wave_lds_sync();
      if (mine.id >= 0) slots[rank].id = mine.id;
      wave_lds_sync();
      id = slots[at].id;
      wave_lds_sync();
    }
  }
  if (!chosen) {
    // one more than asked for: the last one's distance counts too
    const bool fits = a.K < LPT;
    choice.largest(check && fits ? a.K + 1 : a.K, value, id);
    if (check) {
      // Equal logits and biases make equal choices, in any number of bits; of the last one
      // and the first that is left out that says nothing of the others left out.
      const float mine = id >= 0 ? logit_at<BF16>(row, id) : low_inf();
      const float own = id >= 0 ? a.bias[id] : 0.0f;
      const float below = of_next(value), l_below = of_next(mine), b_below = of_next(own);
      close |= at < a.K && at + 1 < LPT && id >= 0 && below > low_inf() &&
               !(value - below > sure + 0x1p-23f * (fabsf(value) + fabsf(below))) &&
               !(at + 1 < a.K && mine == l_below && own == b_below);
      close |= !fits;
    }
  }
  if (bad || at >= a.K) id = -1;
  store_entries<LPT, BF16>(a, row, t, id, choice.most, choice.total);
  if (bad && in && at == 0) set_err(a.err, EP_DEVERR_LOGITS);
  return !in || bad || token_bits<LPT>(__ballot(close)) == 0;
}

template <int LPT, int PER, bool BF16>
__global__ __launch_bounds__(kRouteThreads, PER <= 16 ? 3 : 1) void route(RouteArgs a) {
  constexpr int kTokens = kRouteThreads / LPT, kWaveTokens = kWave / LPT;
  __shared__ Candidate slots[LPT == 16 ? kTokens : 1][16];
  __shared__ float totals[kRouteThreads / kWave][kWave];  // of tokens that are chosen again
  extern __shared__ double choices[];  // where choices are scores: [waves][E]
  const int wave = uniform(threadIdx.x / kWave);
  const int64_t step = (int64_t)gridDim.x * kTokens;
  const int64_t mine = (int64_t)blockIdx.x * kTokens + wave * kWaveTokens;
  for (int64_t base = mine; base < a.tokens;) {
    // as many rounds as a word has bits for their tokens, then those that have to be chosen
    // again: their code keeps its registers out of the loop that all tokens take
    uint64_t again = 0;
    const int64_t start = base;
    for (int r = 0; r < LPT && base < a.tokens; ++r, base += step) {
      float total;
      const bool sure = route_fast<LPT, PER, BF16>(
          a, base + lane_id() / LPT, slots[LPT == 16 ? threadIdx.x / LPT : 0], total);
      const bool redo = !sure && (lane_id() & (LPT - 1)) == 0;
      if (redo) totals[wave][r * kWaveTokens + lane_id() / LPT] = total;
      uint64_t at = __ballot(redo);
      for (; at; at &= at - 1)
        again |= 1ull << (r * kWaveTokens + __builtin_ctzll(at) / LPT);
    }
    wave_lds_sync();
    for (; again; again &= again - 1) {  // rarely
      const int bit = __builtin_ctzll(again);
      route_exactly<BF16>(a, start + (bit / kWaveTokens) * step + bit % kWaveTokens,
                          totals[wave][bit], choices + wave * a.E);
    }
  }
}

// ---- gradient -----------------------------------------------------------------------

// PER consecutive values of a row, as one vector where all lanes' are whole
template <int PER, bool BF16>
__device__ __forceinline__ void store_logits(char* row, int first, int E, const float (&g)[PER]) {
  constexpr int kBytes = PER * (BF16 ? 2 : 4);
  if (PER > 1 && E % PER == 0) {
    if (first >= E) return;
    uint32_t w[kBytes / 4];
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i)
      w[i] = BF16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(
                                                     (f32x2){g[2 * i], g[2 * i + 1]}, bf16x2))
                  : __float_as_uint(g[i]);
    char* to = row + (int64_t)first * (BF16 ? 2 : 4);
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        ((uint4*)to)[i] = uint4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    } else if constexpr (kBytes == 8) {
      *(uint2*)to = uint2{w[0], w[1]};
    } else {
      *(uint32_t*)to = w[0];
    }
  } else {
    const int f = here(first);
    char* to = row + (int64_t)f * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (f + i < E) {
        if (BF16) ((__bf16*)to)[i] = (__bf16)g[i];
        else ((float*)to)[i] = g[i];
      }
    }
  }
}

// Entry k's terms are computed in the token's lane k and spread over the row in LDS.
template <int LPT, int PER, bool BF16>
__global__ __launch_bounds__(kRouteThreads) void route_grad(RouteGradArgs a) {
  constexpr int kTokens = kRouteThreads / LPT;
  __shared__ __align__(16) float rows[kTokens][LPT * PER];
  const int at = lane_id() & (LPT - 1), first = at * PER;
  float* const spread = rows[threadIdx.x / LPT];
  const bool dense = !a.sigmoid && !a.normalize;  // every expert has a gradient
#pragma unroll
  for (int i = 0; i < PER; ++i) spread[first + i] = 0.0f;
  wave_lds_sync();
  for (int64_t base = (int64_t)blockIdx.x * kTokens; base < a.tokens;
       base += (int64_t)gridDim.x * kTokens) {
    const int64_t t = base + threadIdx.x / LPT;
    const bool in = t < a.tokens;
    const int64_t token = in ? t : a.tokens - 1;
    const int64_t size = BF16 ? 2 : 4;
    const char* row = (const char*)a.logits + token * a.E * size;
    int id = at < a.K ? a.idx[token * a.K + at] : -1;
    float dw = at < a.K ? a.dweights[token * a.K + at] : 0.0f;
    float l[PER];
    if (dense) load_logits<PER, BF16>(row, first, a.E, low_inf(), l);
    if (id < -1 || id >= a.E) {
      if (in) set_err(a.err, EP_DEVERR_TOPK_RANGE);
      id = -1;
    }
    const bool has = id >= 0;
    if (!has) dw = 0.0f;
    const bool any = token_bits<LPT>(__ballot(has)) != 0;
    float g = dw;
    if (!dense) {
      const float mine = has ? logit_at<BF16>(row, id) : low_inf();
      float s = 0.0f, rest = 1.0f, part = 1.0f, mean = 0.0f;
      float top = all_max<LPT>(mine);
      if (a.sigmoid) {
        const float z = exponential(mine < 0.0f ? mine : -mine), r = inverse(1.0f + z);
        s = mine < 0.0f ? z * r : r;
        rest = mine < 0.0f ? r : z * r;  // 1 - s
      }
      if (a.normalize) {
        // softmax over the chosen; sigmoids so small that they might vanish are exponentials
        if (!(top > low_inf())) top = 0.0f;
        if (!a.sigmoid || top < -30.0f) s = exponential(mine - top);
        if (!has) s = 0.0f;
        const float sum = all_sum<LPT>(s);
        part = sum > 0.0f ? 1.0f / sum : 0.0f;
        mean = all_sum<LPT>(dw * s) * part;
      }
      g = has ? a.scale * (s * part) * (dw - mean) * rest : 0.0f;
    }
    // an expert that several entries name gets their sum, from the first of them
    float all = 0.0f;
    bool again = false;
    for (int k = 0; k < a.K; ++k) {
      const bool same = of_lane<LPT>(id, k) == id;
      const float other = of_lane<LPT>(g, k);
      all += same ? other : 0.0f;
      again |= same && k < at;
    }
    const bool writes = has && !again;
    if (writes) spread[id] = all;
    wave_lds_sync();
    float d[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i] = spread[first + i];
    wave_lds_sync();
    if (writes) spread[id] = 0.0f;
    wave_lds_sync();
    if (dense) {
      float most = l[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) most = fmaxf(most, l[i]);
      most = all_max<LPT>(most);
      if (!(most > low_inf())) most = 0.0f;
      float sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        l[i] = exponential(l[i] - most);
        sum += l[i];
        dot = __builtin_fmaf(d[i], l[i], dot);
      }
      sum = all_sum<LPT>(sum);
      dot = all_sum<LPT>(dot);
      const float part = sum > 0.0f ? 1.0f / sum : 0.0f, mean = dot * part;
      const float factor = any ? a.scale * part : 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) d[i] = any ? (l[i] * factor) * (d[i] - mean) : 0.0f;
    }
    if (in) store_logits<PER, BF16>((char*)a.dlogits + token * a.E * size, first, a.E, d);
  }
}

// ---- launches -------------------------------------------------------------------------

// Up to 512 experts 16 lanes take a token's choice, so that a wave has four of them in a
// butterfly's steps; they hold 16 candidates (32,768 tokens over 256 / 384 / 512 experts: 64
// lanes 79 / 65 / 84 us, 16 lanes 30 / 42 / 55).  The gradient's 64 from 257 on (384: 18 us,
// with 16 lanes 24).
constexpr int64_t kRouteBlocks = 8 * kCus;

// A lane has fewer than `most` experts where a power of two of lanes then has a group each
// (32,768 tokens over 160 experts in 8 groups: 47 us with 16 a lane, 38 with 10).
static RouteArgs with_lanes(RouteArgs a, int lanes, int most) {
  a.per = most;
  if (a.groups_kept < a.groups)
    for (int of = 1; of * a.groups <= lanes; of *= 2)
      if (a.group_size % of == 0 && a.group_size / of <= most) {
        a.per = a.group_size / of;
        break;
      }
  return a;
}
static const RouteGradArgs& with_lanes(const RouteGradArgs& a, int, int) { return a; }

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
                     dim3(kRouteThreads), lds, st, with_lanes(a, LPT, PER))

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const bool narrow = a.K < 16 && (a.groups_kept == a.groups || a.groups <= 16);
  const size_t lds = a.scored ? kRouteThreads / kWave * a.E * sizeof(double) : 0;
  if (narrow && a.E > 256 && a.E <= 512) {
    if (a.bf16) EP_ROUTE_LAUNCH(route, 16, 32, true);
    else EP_ROUTE_LAUNCH(route, 16, 32, false);
  } else {
    EP_ROUTE_FORMS(route);
  }
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const bool narrow = a.K <= 16;
  const size_t lds = 0;
  EP_ROUTE_FORMS(route_grad);
  return hipGetLastError();
}

}  // namespace ep
