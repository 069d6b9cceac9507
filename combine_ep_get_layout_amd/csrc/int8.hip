// 8-bit integer rows on gfx950: dispatch with a scale per token, and the rows of a
// layout's segments quantised in the receive layout.  For a row x
//   scale = max(amax |x|, 2^-100) / 127,  code = rint(x / scale),
// both divisions correctly rounded, ties of rint to even; the floor keeps the scale a
// normal number and an all-zero row finite.  |code| <= 127: amax / scale is at most
// 127 (1 + 2^-23).  A row with a NaN or infinity has no codes that stand for it: it gets
// zeros and the scale NaN, so that every product of it is NaN.
//
// Bound by memory: a row is read once, kept in registers, and its codes are written.  16,384
// tokens of 7168 channels to 131,072 rows take 206 us (5.7 TB/s), 131,072 rows of 2048 channels
// in place of a layout 163 to 172 us (4.7 to 4.9 TB/s, 86 to 90% of a large copy).
#include <algorithm>

#include "experts.hpp"
#include "quant.hpp"

namespace ep {

constexpr int kInt8Threads = 256;

// A row's codes: GROUP threads (a wave, or the workgroup) hold a pair of 16-byte vectors,
// 16 channels, in each of NP places.
template <int NP, int GROUP>
struct Int8Row {
  u32x4 codes[NP];
  float scale;
  int place;  // of this thread among the group

  __device__ __forceinline__ Int8Row() : place(threadIdx.x % GROUP) {}

  __device__ __forceinline__ void load(const uint16_t* row, int pairs, u32x4 (&lo)[NP],
                                       u32x4 (&hi)[NP]) const {
    const u32x4* src = (const u32x4*)row;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int j = min(place + i * GROUP, pairs - 1);  // past the end: the last pair again
      lo[i] = __builtin_nontemporal_load(src + 2 * j);
      hi[i] = __builtin_nontemporal_load(src + 2 * j + 1);
    }
  }

  // parts: LDS for a word per wave, where the group is the workgroup
  __device__ __forceinline__ void quantise(const u32x4 (&lo)[NP], const u32x4 (&hi)[NP],
                                           uint32_t* parts) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) most = max(most, absmax16(lo[i], hi[i]));
    most = max8_lanes(most);
    most = max(most, (uint32_t)__shfl_xor((int)most, 8));
    most = max(most, (uint32_t)__shfl_xor((int)most, 16));
    most = max(most, (uint32_t)__shfl_xor((int)most, 32));
    if (GROUP > kWave) {
      if (lane_id() == 0) parts[threadIdx.x / kWave] = most;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < GROUP / kWave; ++w) most = max(most, parts[w]);
      __syncthreads();
    }
    most = (uint32_t)uniform((int)most);
    if (most >= 0x7F80u) {
      scale = __uint_as_float(0x7FC00000u);
#pragma unroll
      for (int i = 0; i < NP; ++i) codes[i] = u32x4{0u, 0u, 0u, 0u};
      return;
    }
    scale = __fdiv_rn(fmaxf(__uint_as_float(most << 16), 0x1p-100f), 127.0f);
#pragma unroll
    for (int i = 0; i < NP; ++i) codes[i] = u32x4{four(lo[i], 0), four(lo[i], 2), four(hi[i], 0), four(hi[i], 2)};
  }

  // codes of the four bf16 in words q and q + 1
  __device__ __forceinline__ uint32_t four(const u32x4& v, int q) const {
    return one(bf16_lo(v[q])) | one(bf16_hi(v[q])) << 8 | one(bf16_lo(v[q + 1])) << 16 |
           one(bf16_hi(v[q + 1])) << 24;
  }
  // 1.5 * 2^23 + t has t's nearest integer, ties to even, in its low bits
  __device__ __forceinline__ uint32_t one(float x) const {
    return __float_as_uint(__fdiv_rn(x, scale) + 0x1.8p23f) & 0xFFu;
  }

  __device__ __forceinline__ void store(int8_t* row, float* to, int pairs) const {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (place + i * GROUP < pairs) *((u32x4*)row + place + i * GROUP) = codes[i];
    if (place == 0) *to = scale;
  }
};

// One token a group: read once, written to each of its rows.
template <int NP, int GROUP>
__global__ __launch_bounds__(kInt8Threads) void dispatch_int8(DispatchArgs a) {
  __shared__ uint32_t parts[kInt8Threads / kWave];
  constexpr int kGroups = kInt8Threads / GROUP;
  const int pairs = a.g.H / 16, K = a.g.K;
  const int64_t tokens = (int64_t)a.g.R * a.g.T;
  const int lane = lane_id();
  for (int64_t t = (int64_t)blockIdx.x * kGroups + uniform(threadIdx.x / GROUP); t < tokens;
       t += (int64_t)gridDim.x * kGroups) {
    Int8Row<NP, GROUP> row;
    u32x4 lo[NP], hi[NP];
    const int at = lane < K ? a.send_pos[t * K + lane] : -1;
    row.load(a.x + t * a.g.H, pairs, lo, hi);
    row.quantise(lo, hi, parts);
    if (__ballot(at >= a.cap) != 0 && row.place == 0) set_err(a.err, EP_DEVERR_CAPACITY);
    for (uint64_t has = __ballot(at >= 0 && at < a.cap); has; has &= has - 1) {
      const int64_t r = __builtin_amdgcn_readlane(at, __ffsll((unsigned long long)has) - 1);
      row.store((int8_t*)a.recv_x + r * a.g.H, (float*)a.recv_scales + r, pairs);
    }
  }
}

// The rows of the segments, a group a row.
template <int NP, int GROUP>
__global__ __launch_bounds__(kInt8Threads) void rows_int8(Int8Args a) {
  __shared__ TilePlan plan;
  __shared__ uint32_t parts[kInt8Threads / kWave];
  constexpr int kGroups = kInt8Threads / GROUP;
  plan_tiles<kInt8Threads>(a.seg, kGroups, plan, (int*)parts);
  const int pairs = a.C / 16, tiles = plan.upto[a.seg.E - 1];
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int e = expert_of(plan, a.seg.E, (int)t);
    int64_t start;
    int count;
    segment_of(a.seg, e, start, count);
    const int in = ((int)t - plan.first(e)) * kGroups + uniform(threadIdx.x / GROUP);
    if (in >= count) continue;  // a whole wave; with one group a workgroup never
    Int8Row<NP, GROUP> row;
    u32x4 lo[NP], hi[NP];
    row.load(a.x + (start + in) * a.C, pairs, lo, hi);
    row.quantise(lo, hi, parts);
    row.store(a.codes + (start + in) * a.C, a.scales + start + in, pairs);
  }
}

// The fewest registers that hold a row: a wave up to 8192 channels, then the workgroup.
#define EP_INT8_FORMS(channels, LAUNCH)                    \
  do {                                                     \
    if ((channels) <= 1024) LAUNCH(1, kWave);              \
    else if ((channels) <= 2048) LAUNCH(2, kWave);         \
    else if ((channels) <= 4096) LAUNCH(4, kWave);         \
    else if ((channels) <= 8192) LAUNCH(2, kInt8Threads);  \
    else if ((channels) <= 16384) LAUNCH(4, kInt8Threads); \
    else LAUNCH(8, kInt8Threads);                          \
  } while (0)

constexpr int64_t kInt8Blocks = 8 * kCus;

hipError_t launch_dispatch_int8(const DispatchArgs& a, hipStream_t st) {
  const int64_t tokens = (int64_t)a.g.R * a.g.T;
  if (tokens == 0) return hipSuccess;
#define EP_LAUNCH(NP, GROUP)                                                                  \
  hipLaunchKernelGGL((dispatch_int8<NP, GROUP>),                                              \
                     dim3((unsigned)std::min((tokens * (GROUP) + kInt8Threads - 1) / kInt8Threads, \
                                             kInt8Blocks)),                                   \
                     dim3(kInt8Threads), 0, st, a)
  EP_INT8_FORMS(a.g.H, EP_LAUNCH);
#undef EP_LAUNCH
  return hipGetLastError();
}

hipError_t launch_rows_int8(const Int8Args& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
#define EP_LAUNCH(NP, GROUP)                                                                \
  hipLaunchKernelGGL((rows_int8<NP, GROUP>),                                                \
                     dim3((unsigned)std::min(a.rows * (GROUP) / kInt8Threads + a.seg.E,     \
                                             kInt8Blocks)),                                 \
                     dim3(kInt8Threads), 0, st, a)
  EP_INT8_FORMS(a.C, EP_LAUNCH);
#undef EP_LAUNCH
  return hipGetLastError();
}

}  // namespace ep
