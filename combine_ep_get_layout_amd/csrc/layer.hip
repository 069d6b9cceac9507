// A whole MoE layer for a few tokens on gfx950, in two launches and without layout or
// dispatch: for every token t and its entries (e, w),
//   h = act(x Wg_e^T) * (x Wu_e^T),  rounded to bf16,        (layer_gated)
//   out_t = sum_k w_k h W2_e^T,      in fp32, in k order.    (layer_down)
//
// With few tokens the time is that of reading the weights of the experts that are hit, so
// each is read once, straight into the registers of the matrix instructions (16 rows of
// weights x 64 bytes a load), while the tokens' rows come from the cache.  Rows stay bf16
// whatever the weights' type: e4m3 and 8-bit codes are converted (both fit bf16 exactly),
// and their scales are applied to the fp32 sums.
#include <algorithm>

#include "experts.hpp"
#include "layer.hpp"

namespace ep {

constexpr int kUpWaves = 4;    // of a workgroup of layer_gated, which share a contraction
constexpr int kDownWaves = 8;  // of a workgroup of layer_down, an expert each
constexpr int kTileRows = 64;  // entries of an expert that are multiplied at once

// ---- who is hit ------------------------------------------------------------------

// The ids in LDS, and a bit for each expert with an entry: lane l's word has experts 32 l ...
struct Routing {
  int ids[kLayerEntries];
  uint32_t hit[kMaxExperts / 32];
};

template <int THREADS>
__device__ __forceinline__ void read_routing(const LayerArgs& a, Routing& r) {
  for (int i = threadIdx.x; i < kMaxExperts / 32; i += THREADS) r.hit[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < kLayerEntries; i += THREADS) {
    int id = i < a.entries ? a.idx[i] : -1;
    if (id < -1 || id >= a.E) {
      if (blockIdx.x == 0) set_err(a.err, EP_DEVERR_TOPK_RANGE);
      id = -1;
    }
    r.ids[i] = id;
    if (id >= 0) atomicOr(&r.hit[id / 32], 1u << (id % 32));
  }
  __syncthreads();
}

// The experts hit, in the order of their index, from a wave's lanes.
struct Hits {
  uint32_t word;
  int upto, total;
  __device__ __forceinline__ explicit Hits(const Routing& r) {
    const int lane = lane_id();
    word = r.hit[lane];
    upto = __popc(word);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    total = __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  // the i-th of them, i < total
  __device__ __forceinline__ int expert(int i) const {
    const int lane = __builtin_ctzll(__ballot(upto > i));
    const uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)word, lane);
    const int nth = i - (__builtin_amdgcn_readlane(upto, lane) - __popc(w));
    const int b = lane_id() & 31;
    const bool is = (w >> b & 1u) && __popc(w & ((1u << b) - 1u)) == nth;
    return uniform(lane * 32 + __builtin_ctzll(__ballot(is)));
  }
};

// Expert e's entries (t * K + k) in their order; a wave's own list.
__device__ __forceinline__ int entries_of(const LayerArgs& a, const Routing& r, int e,
                                          uint16_t* list) {
  const int lane = lane_id();
  int n = 0;
  for (int c = 0; c < a.entries; c += kWave) {
    const bool is = r.ids[c + lane] == e;
    const uint64_t mask = __ballot(is);
    if (is) list[n + rank_below(mask)] = (uint16_t)(c + lane);
    n += __popcll(mask);
  }
  wave_lds_sync();
  return n;
}

// ---- 16 rows of weights times up to 64 rows --------------------------------------------

// A line is 128 bytes of a row of weights: two loads of 16 bytes a lane, lane l taking row
// l % 16 and bytes 16 (l / 16) of either half.  The products follow from that: in bf16 a load
// is one step of 32 channels, in 8 bits two, of each lane's first and last eight codes.
template <int KIND, int TT>
struct Strip {
  static constexpr bool kBytes = KIND != EP_WEIGHTS_BF16;
  // lines in flight: as many as leave the registers for 16 waves on a compute unit
  static constexpr int U = TT == 1 ? (kBytes ? 2 : 4) : TT == 2 ? (kBytes ? 1 : 2) : 1;
  static constexpr int kRowLoads = kBytes ? 4 : 2;  // of a line, for a lane's row

  const char* w;           // the lane's row of weights, at its 16 bytes
  const char* x[TT];       // the lane's rows, likewise
  const float* scale;      // FP8: the lane's row's blocks along the contraction
  f32x4 acc[TT];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  static __device__ __forceinline__ bf16x8 codes(uint32_t lo, uint32_t hi) {
    union {
      bf16x2 p[4];
      bf16x8 v;
    } u;
    if constexpr (KIND == EP_WEIGHTS_FP8) {
      u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
      u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
      u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
      u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t from = i < 2 ? lo : hi;
        const f32x2 f = {(float)(int8_t)(from >> (16 * (i & 1))),
                         (float)(int8_t)(from >> (16 * (i & 1) + 8))};
        u.p[i] = __builtin_convertvector(f, bf16x2);
      }
    }
    return u.v;
  }

  struct Weights {
    u32x4 v[2];
    float s;
  };
  struct Rows {
    u32x4 v[TT][kRowLoads];
  };

  __device__ __forceinline__ void load(int line, Weights& to) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      to.v[i] = __builtin_nontemporal_load((const u32x4*)(w + (int64_t)line * 128 + 64 * i));
    if (KIND == EP_WEIGHTS_FP8) to.s = scale[line];
  }
  __device__ __forceinline__ void load(int line, Rows& to) const {
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
      for (int i = 0; i < kRowLoads; ++i)
        to.v[j][i] = *(const u32x4*)(x[j] + (int64_t)line * (kBytes ? 256 : 128) +
                                     (kBytes ? 128 * (i / 2) + 16 * (i % 2) : 64 * i));
  }
  __device__ __forceinline__ void multiply(const Weights& a, const Rows& b) {
    bf16x8 f[kRowLoads];
#pragma unroll
    for (int i = 0; i < kRowLoads; ++i) {
      if constexpr (kBytes) f[i] = codes(a.v[i / 2][2 * (i % 2)], a.v[i / 2][2 * (i % 2) + 1]);
      else f[i] = __builtin_bit_cast(bf16x8, a.v[i]);
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      f32x4 sum = KIND == EP_WEIGHTS_FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[j];
#pragma unroll
      for (int i = 0; i < kRowLoads; ++i)
        sum = Mfma<16>::bf16(f[i], __builtin_bit_cast(bf16x8, b.v[j][i]), sum);
      if (KIND == EP_WEIGHTS_FP8) {
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][q] = __builtin_fmaf(sum[q], a.s, acc[j][q]);
      } else {
        acc[j] = sum;
      }
    }
  }

  // Lines first, first + step, .. of a row of `bytes` bytes.  The next U lines of weights are
  // on their way while these are multiplied; the rows' loads come out of the cache, and are
  // issued before those so that waiting for them waits for nothing else.
  __device__ __forceinline__ void run(int bytes, int first, int step) {
    const int lines = bytes / 128;
    const int n = first < lines ? (lines - first + step - 1) / step : 0;
    const int last = first + (n - 1) * step;
    if (n > 0) {
      Weights now[U];
      Rows rows[U];
#pragma unroll
      for (int i = 0; i < U; ++i) load(min(first + i * step, last), now[i]);
      int at = first;
      for (int done = U; done < n; done += U, at += U * step) {
        Weights next[U];
#pragma unroll
        for (int i = 0; i < U; ++i) load(at + i * step, rows[i]);
#pragma unroll
        for (int i = 0; i < U; ++i) load(min(at + (U + i) * step, last), next[i]);
#pragma unroll
        for (int i = 0; i < U; ++i) multiply(now[i], rows[i]);
#pragma unroll
        for (int i = 0; i < U; ++i) now[i] = next[i];
      }
#pragma unroll
      for (int i = 0; i < U; ++i) load(min(at + i * step, last), rows[i]);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (at + i * step <= last) multiply(now[i], rows[i]);
    }
    // less than a line is left (never in FP8): chunks past the end are zeros on both sides
    if (KIND != EP_WEIGHTS_FP8 && bytes % 128 != 0 && lines % step == first % step) {
      Weights a;
      Rows b;
      const u32x4 zero = {0u, 0u, 0u, 0u};
      const int left = bytes % 128 - 16 * (lane_id() / 16);
      a.s = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a.v[i] = 64 * i < left ? *(const u32x4*)(w + (int64_t)lines * 128 + 64 * i) : zero;
#pragma unroll
      for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int i = 0; i < kRowLoads; ++i)
          b.v[j][i] = 64 * (kBytes ? i / 2 : i) < left
                          ? *(const u32x4*)(x[j] + (int64_t)lines * (kBytes ? 256 : 128) +
                                            (kBytes ? 128 * (i / 2) + 16 * (i % 2) : 64 * i))
                          : zero;
      multiply(a, b);
    }
  }
};

// ---- gated block -------------------------------------------------------------------

// A workgroup's unit: eight channels of one expert, their gates and ups the 16 rows of
// weights, the contraction's lines dealt to its four waves in turn.
constexpr int kUpStride = 20;  // floats of a column of partial sums, 16 and a gap

template <int KIND, int TT>
__device__ __forceinline__ void up_tile(const LayerArgs& a, int e, int n0, const uint16_t* list,
                                        int rows, float* parts) {
  const int lane = lane_id(), wave = uniform(threadIdx.x / kWave), row = lane % 16;
  constexpr int kSize = KIND == EP_WEIGHTS_BF16 ? 2 : 1;
  Strip<KIND, TT> s;
  const int channel = row < 8 ? n0 + row : a.I + n0 + row - 8;
  s.w = a.w13 + ((int64_t)e * 2 * a.I + channel) * a.H * kSize + 16 * (lane / 16);
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int token = list[min(16 * j + row, rows - 1)] / a.K;
    s.x[j] = (const char*)(a.x + (int64_t)token * a.H) + (kSize == 2 ? 16 : 32) * (lane / 16);
  }
  // sums are of rows 4 (lane / 16) ..: the first half of the lanes has the gates
  if (KIND == EP_WEIGHTS_FP8)
    s.scale = a.s13 + ((int64_t)e * (2 * a.I / 128) + ((lane < 32 ? 0 : a.I) + n0) / 128) * (a.H / 128);
  s.clear();
  s.run(a.H * kSize, wave, kUpWaves);
#pragma unroll
  for (int j = 0; j < TT; ++j)
    *(f32x4*)(parts + (wave * kTileRows + 16 * j + row) * kUpStride + 4 * (lane / 16)) = s.acc[j];
  __syncthreads();
  for (int o = threadIdx.x; o < TT * 16 * 8; o += kUpWaves * kWave) {
    const int col = o / 8, ch = o % 8;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kUpWaves; ++w) {
      g += parts[(w * kTileRows + col) * kUpStride + ch];
      u += parts[(w * kTileRows + col) * kUpStride + 8 + ch];
    }
    if (KIND == EP_WEIGHTS_INT8) {
      const float* scale = a.s13 + (int64_t)e * 2 * a.I + n0 + ch;
      g *= scale[0];
      u *= scale[a.I];
    }
    float value, slope;
    act_both(a.act, g, value, slope);
    if (col < rows) ((__bf16*)a.h)[(int64_t)list[col] * a.I + n0 + ch] = (__bf16)(value * u);
  }
  __syncthreads();
}

template <int KIND>
__global__ __launch_bounds__(kUpWaves* kWave, 4) void layer_gated(LayerArgs a) {
  __shared__ Routing routing;
  __shared__ uint16_t lists[kUpWaves][kLayerEntries];
  __shared__ __align__(16) float parts[kUpWaves * kTileRows * kUpStride];
  read_routing<kUpWaves * kWave>(a, routing);
  const Hits hits(routing);
  const int tiles = a.I / 8, units = hits.total * tiles;
  uint16_t* list = lists[uniform(threadIdx.x / kWave)];
  int held = -1, n = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int e = hits.expert(u / tiles), n0 = u % tiles * 8;
    if (e != held) n = entries_of(a, routing, e, list);
    held = e;
    for (int at = 0; at < n; at += kTileRows) {
      const int rows = min(n - at, kTileRows);
      if (rows <= 16) up_tile<KIND, 1>(a, e, n0, list + at, rows, parts);
      else if (rows <= 32) up_tile<KIND, 2>(a, e, n0, list + at, rows, parts);
      else up_tile<KIND, 4>(a, e, n0, list + at, rows, parts);
    }
  }
}

// ---- down projection and the weighted sum ---------------------------------------------

template <int KIND, int TT>
__device__ __forceinline__ void down_tile(const LayerArgs& a, int e, int n0, const uint16_t* list,
                                          int rows, int part, int parts, float* y) {
  const int lane = lane_id(), row = lane % 16;
  constexpr int kSize = KIND == EP_WEIGHTS_BF16 ? 2 : 1;
  Strip<KIND, TT> s;
  const int channel = min(n0 + row, a.H - 1);  // past the last one: not stored
  s.w = a.w2 + ((int64_t)e * a.H + channel) * a.I * kSize + 16 * (lane / 16);
#pragma unroll
  for (int j = 0; j < TT; ++j)
    s.x[j] = (const char*)(a.h + (int64_t)list[min(16 * j + row, rows - 1)] * a.I) +
             (kSize == 2 ? 16 : 32) * (lane / 16);
  if (KIND == EP_WEIGHTS_FP8) s.scale = a.s2 + ((int64_t)e * (a.H / 128) + n0 / 128) * (a.I / 128);
  s.clear();
  s.run(a.I * kSize, part, parts);
  f32x4 scale = {1.0f, 1.0f, 1.0f, 1.0f};
  if (KIND == EP_WEIGHTS_INT8)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      scale[q] = a.s2[(int64_t)e * a.H + min(n0 + 4 * (lane / 16) + q, a.H - 1)];
#pragma unroll
  for (int j = 0; j < TT; ++j)
    if (16 * j + row < rows)
      *(f32x4*)(y + list[16 * j + row] * 16 + 4 * (lane / 16)) = s.acc[j] * scale;
}

// A workgroup has 16 channels of every token: its waves take an expert each in turn (or parts
// of its contraction, where there are fewer experts than waves) and put every entry's
// result into its own place in LDS; then they are summed in k order.
template <int KIND>
__global__ __launch_bounds__(kDownWaves* kWave, 4) void layer_down(LayerArgs a) {
  extern __shared__ __align__(16) float y[];  // [parts][entries][16]
  __shared__ Routing routing;
  __shared__ uint16_t lists[kDownWaves][kLayerEntries];
  read_routing<kDownWaves * kWave>(a, routing);
  const Hits hits(routing);
  const int n0 = blockIdx.x * 16, wave = uniform(threadIdx.x / kWave);
  uint16_t* list = lists[wave];
  // parts that every expert's contraction is cut into
  int parts = 1;
  while (2 * parts * hits.total <= kDownWaves && 2 * parts * a.entries <= a.slots) parts *= 2;
  for (int u = wave; u < hits.total * parts; u += kDownWaves) {
    const int e = hits.expert(u / parts), part = u % parts;
    const int n = entries_of(a, routing, e, list);
    float* to = y + part * a.entries * 16;
    for (int at = 0; at < n; at += kTileRows) {
      const int rows = min(n - at, kTileRows);
      if (rows <= 16) down_tile<KIND, 1>(a, e, n0, list + at, rows, part, parts, to);
      else if (rows <= 32) down_tile<KIND, 2>(a, e, n0, list + at, rows, part, parts, to);
      else down_tile<KIND, 4>(a, e, n0, list + at, rows, part, parts, to);
    }
  }
  __syncthreads();
  for (int o = threadIdx.x; o < a.tokens * 16; o += kDownWaves * kWave) {
    const int t = o / 16, ch = o % 16;
    float sum = 0.0f;
    for (int k = 0; k < a.K; ++k) {
      const int i = t * a.K + k;
      if (routing.ids[i] < 0) continue;
      float v = 0.0f;
      for (int p = 0; p < parts; ++p) v += y[(p * a.entries + i) * 16 + ch];
      sum = __builtin_fmaf(a.weights[i], v, sum);
    }
    if (n0 + ch < a.H) ((__bf16*)a.out)[(int64_t)t * a.H + n0 + ch] = (__bf16)sum;
  }
}

template <int KIND>
static void launch(const LayerArgs& a, hipStream_t st) {
  const int64_t units = (int64_t)std::min(a.E, a.entries) * (a.I / 8);
  hipLaunchKernelGGL((layer_gated<KIND>), dim3((unsigned)std::min<int64_t>(units, 4 * kCus)),
                     dim3(kUpWaves * kWave), 0, st, a);
  hipLaunchKernelGGL((layer_down<KIND>), dim3((a.H + 15) / 16), dim3(kDownWaves * kWave),
                     (size_t)a.slots * 16 * sizeof(float), st, a);
}

hipError_t launch_layer(LayerArgs a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  a.slots = std::max(a.entries, std::min(kDownWaves * a.entries, 256));
  switch (a.kind) {
    case EP_WEIGHTS_BF16: launch<EP_WEIGHTS_BF16>(a, st); break;
    case EP_WEIGHTS_FP8: launch<EP_WEIGHTS_FP8>(a, st); break;
    default: launch<EP_WEIGHTS_INT8>(a, st); break;
  }
  return hipGetLastError();
}

}  // namespace ep
