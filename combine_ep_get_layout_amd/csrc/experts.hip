// The experts' forward products on gfx950: the gated feed-forward block
//   h = act(x Wg^T) * (x Wu^T)
// and the product with bias, activation and residual
//   y = act(x W^T + b) + r
// over the rows of each expert's segment, one launch each.
//
// With many rows an expert the products are bound by the matrix cores and their
// power: 64 experts x 2,048 rows, 7168 -> 2 x 2048, take 6.31 ms (1,220 TFLOP/s), the
// cores busy 77% of the time at 1.6 GHz.  2048 -> 7168 with a residual takes 3.65
// ms (1,050 TFLOP/s): a quarter of it starts and ends tiles.  In FP8 the same two take
// 5.48 and 3.32 ms (1,400 and 1,160): a stage's reads, products and scaling wait for each
// other (RingEngine8).  With few rows they are
// bound by reading the weights: 256 experts x 32 rows in FP8, 7168 -> 2 x 2048, 1.29
// ms (5.9 TB/s); 2048 -> 7168, 0.74 ms (5.2 TB/s, 16 stages a tile).  Eight rows
// of eight experts, 2048 -> 2 x 768, take 14 us, half of it latency.
#include <algorithm>
#include <type_traits>

#include "experts.hpp"
#include "quant.hpp"

namespace ep {

// Replaces the NaNs and infinities of eight bf16 by zeros; their halves come back as
// 0xFFFF.
__device__ __forceinline__ u32x4 take_not_finite(u32x4& v) {
  u32x4 at;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    at[q] = ((v[q] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) |
            ((v[q] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
    v[q] &= ~at[q];
  }
  return at;
}

// e4m3 NaN codes where the halves of two words are set
__device__ __forceinline__ uint32_t nan_codes(uint32_t a, uint32_t b) {
  return (a & 0x7Fu) | (a >> 16 & 0x7Fu) << 8 | (b & 0x7Fu) << 16 | (b >> 16 & 0x7Fu) << 24;
}

// Nothing to load for a row's result.
struct NoRow {};

// What a tile's epilogue needs of it.
struct Tile {
  int64_t row;     // first row in the row buffers
  int64_t block;   // that row within its low-latency block
  int e, rows, n0;
};

// One workgroup's state: where its loads read, and the epilogue.  Q: EP_QUANT_*
template <class S, bool GATED, int Q>
struct Forward {
  static constexpr bool FP8 = Q != EP_QUANT_NONE;
  static constexpr int MF = S::MF, CT = S::CT;
  // gated: a wave's channel tiles are half gates and half ups of the same channels
  static constexpr int CH = GATED ? CT / 2 : CT;         // channel tiles of the output per wave
  static constexpr int ON = GATED ? S::BN / 2 : S::BN;   // output channels per workgroup tile
  static constexpr int GS = S::GS;                       // FP8 scale groups of a wave's stage
  static constexpr int kPeriod = GATED ? CT * MF : 1 << 20;
  typedef RowTile<S::BN, S::KB> Chan;
  typedef RowTile<S::BM, S::KB> Row;
  static constexpr int kSlot = Chan::kBytes + Row::kBytes;
  static constexpr int kPasses = Chan::kPasses + Row::kPasses;
  static constexpr int kLoads = kPasses + (FP8 ? GS * S::SLOADS + 1 : 0);
  static constexpr int kScales = S::kScaleFloats;
  static constexpr int kScaleBytes = Q == EP_QUANT_FP8_F32 ? 4 : 1;
  static constexpr int kTurn = S::kTurnBytes;
  static constexpr int kRow = ON * 2 + 16;  // FP8 output: a row of the tile in bf16

  const ExpertArgs& a;
  const TilePlan& plan;
  lds_char* lds;
  lds_float* scales;
  S place;
  int nk, nfull, wave, wc, wr, turn;
  int mt, nt;
  int64_t row_bytes;
  Chan w_tile;
  Row x_tile;
  const char *gate_base, *up_base, *x_base;
  // FP8: scales of this wave's rows (column-major: a contraction group's side
  // by side) and of the weights' 128 x 128 blocks
  const char *xs, *ws;
  int64_t xs_stride;
  uint32_t xs_off[S::SLOADS], ws_off;
  typename S::acc_t (*acc)[S::TT];

  __device__ __forceinline__ Forward(const ExpertArgs& a_, const TilePlan& p,
                                     lds_char* l, lds_float* s)
      : a(a_), plan(p), lds(l), scales(s) {
    wave = uniform(threadIdx.x >> 6);
    wc = place.wc;
    wr = place.wr;
    row_bytes = (int64_t)a.C * (FP8 ? 1 : 2);
    nk = (int)((row_bytes + S::KB - 1) / S::KB);
    nfull = (int)(row_bytes / S::KB);
    mt = uniform(plan.upto[a.seg.E - 1]);
    nt = (a.N + ON - 1) / ON;
  }

  __device__ __forceinline__ Tile setup(int64_t t) {
    const int lane = lane_id();
    int m, n;
    tile_at(t, mt, nt, m, n);
    const int e = expert_of(plan, a.seg.E, m);
    int64_t start;
    int count;
    segment_at(a.seg, e, start, count);
    const int row0 = (m - uniform(plan.first(e))) * S::BM;  // within the segment
    const int rows = min(count - row0, S::BM);
    const int n0 = n * ON;
    // Few rows an expert: the weights are read once, by workgroups that would
    // all be at the same channel of their rows at the same time, and where a
    // row's length is a power of two those addresses share few memory
    // channels.  So every tile begins somewhere else (64 experts x 64 rows,
    // 4096 x 4096: 520 -> 403 us; 3584 channels: 344 -> 350 us).  Large tiles
    // share their operands in the die's cache and stay in step.
    turn = S::STAGES > 2 && nk == nfull ? (n * 11 + e * 7) % nk : 0;
    // rows and channels past the end repeat the last one; they are not stored
    gate_base = a.w + ((int64_t)e * (GATED ? 2 : 1) * a.N + n0) * row_bytes;
    up_base = gate_base + (GATED ? (int64_t)a.N * row_bytes : 0);
    x_base = a.x + (start + row0) * row_bytes;
    w_tile.init([&](int r) -> uint32_t {
      const int in = r % (CT * MF);
      const int ch = (r / (CT * MF)) * (CH * MF) + in % (CH * MF);
      return (uint32_t)min(ch, a.N - 1 - n0) * (uint32_t)row_bytes;
    });
    x_tile.init([&](int r) -> uint32_t { return (uint32_t)min(r, rows - 1) * (uint32_t)row_bytes; });
    if (FP8) {
      const int G = a.C / 128;
      const int64_t group = a.seg.start ? a.x_cap : a.seg.block_rows;
      const int64_t first = a.seg.start ? start + row0 : (int64_t)e * G * group + row0;
      xs = (const char*)a.x_scales + first * kScaleBytes;
      xs_stride = group * kScaleBytes;
#pragma unroll
      for (int l = 0; l < S::SLOADS; ++l)
        xs_off[l] = min(wr * S::WROWS + l * kWave + lane, rows - 1) * kScaleBytes;
      const int blocks = (GATED ? 2 : 1) * a.N / 128;
      const int ch = min(n0 + wc * CH * MF, a.N - 1) / 128;
      ws = (const char*)(a.w_scales + ((int64_t)e * blocks + ch) * G);
      ws_off = GATED && lane % 2 ? (uint32_t)(a.N / 128) * G * 4 : 0;  // odd lanes: the ups'
    }
    return Tile{start + row0, row0, e, rows, n0};
  }

  // the stage of the rows that is multiplied k-th
  __device__ __forceinline__ int turned(int k) const {
    return S::STAGES == 2 ? k : k + turn >= nk ? k + turn - nk : k + turn;
  }
  __device__ __forceinline__ void load_scales(int k, int slot) {
    // a short last stage repeats the last group's; its products are zero
    const int last = a.C / 128 - 1, first = turned(k) * (S::KB / 128) + place.wk * GS;
    lds_float* to = scales + (slot * 4 + wave) * kScales;
#pragma unroll
    for (int g = 0; g < GS; ++g)
#pragma unroll
      for (int l = 0; l < S::SLOADS; ++l)
        load_lds4<Q == EP_QUANT_FP8_UE8M0>(xs + min(first + g, last) * xs_stride, xs_off[l],
                                           (const lds_char*)(to + (g * S::SLOADS + l) * kWave));
    load_lds4<false>(ws, ws_off + 4 * min(first + lane_id() / 2 % GS, last),
                     (const lds_char*)(to + GS * S::SLOADS * kWave));
  }
  __device__ __forceinline__ void load_at(int k, lds_char* buf, int p) {
    const int64_t at = (int64_t)turned(k) * S::KB;
    if (p < Chan::kPasses)
      w_tile.template load<kPeriod>(p, gate_base + at, up_base + at, buf);
    else
      x_tile.template load<1 << 20>(p - Chan::kPasses, x_base + at, nullptr, buf + Chan::kBytes);
  }
  __device__ __forceinline__ void tail_at(int k, lds_char* buf) {
    const int64_t at = (int64_t)k * S::KB;
    const int left = (int)(row_bytes - at);
    w_tile.template load_tail<kPeriod>(gate_base + at, up_base + at, left, buf);
    x_tile.template load_tail<1 << 20>(x_base + at, nullptr, left, buf + Chan::kBytes);
  }
  __device__ __forceinline__ void load(int k, int slot, int p) {
    load_at(k, lds + slot * kSlot, p);
    if (FP8 && p == kPasses - 1) load_scales(k, slot);
  }
  __device__ __forceinline__ void tail(int k, int slot) {
    tail_at(k, lds + slot * kSlot);
    if (FP8) load_scales(k, slot);
  }

  // Offsets within a tile's rows fit 32 bits.
  __device__ __forceinline__ void epilogue(const Tile& t, lds_char* base) {
    typedef TurnLane<S, CH> Lane;
    constexpr int B = Lane::kBatch, kStep = Lane::kRows;
    // With two stages the residual is loaded ahead of its use (turn_out).  In the
    // ring it is loaded and used in one branch: a load that some path leaves
    // unused is waited for where its registers are next written, in the main loop,
    // and with it every load of the stages in flight (1 expert, 4096 x 8192, 64
    // rows of Medium: 35 -> 55 us).
    constexpr bool kAhead = S::STAGES == 2 && !GATED;
    typedef typename std::conditional<kAhead, u32x4, NoRow>::type Row8;
    const bool codes = FP8 && ON >= 128 && a.y_quant != EP_QUANT_NONE;
    const Lane lane;
    const int ch = lane.wc * CH * MF + lane.channel;  // within the tile
    const bool in = t.n0 + ch < a.N;
    const int64_t first = t.row * a.N + t.n0;
    uint16_t* const y = (uint16_t*)a.y + first;
    uint16_t* const pre = a.pre ? a.pre + (GATED ? t.row * 2 * a.N + t.n0 : first) : nullptr;
    const float* const bias = a.bias + ((int64_t)t.e * a.N + t.n0 + (in ? ch : 0));
    turn_out<S, CH>(
        base, *(typename S::acc_t(*)[S::CT][S::TT])acc,
        [&](int r) {
          Row8 row = {};
          if constexpr (kAhead)
            if (a.residual && r < t.rows && in)
              row = *(const u32x4*)(a.residual + first + (uint32_t)r * (uint32_t)a.N + ch);
          return row;
        },
        [&](int r, const Turned<S>(&turned)[B], const Row8(&add)[B]) {
          float v[B][8];
#pragma unroll
          for (int b = 0; b < B; ++b) turned[b].get(0, v[b]);
          if constexpr (GATED) {
            float u[B][8];
#pragma unroll
            for (int b = 0; b < B; ++b) turned[b].get(CH * MF, u[b]);
            if (pre)
#pragma unroll
              for (int b = 0; b < B; ++b)
                if (r + b * kStep < t.rows && in) {
                  uint16_t* to = pre + ((uint32_t)(r + b * kStep) * 2u * (uint32_t)a.N + ch);
                  *(u32x4*)to = pack8(v[b]);
                  *(u32x4*)(to + a.N) = pack8(u[b]);
                }
            act_each(a.act, v);
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
              for (int c = 0; c < 8; ++c) v[b][c] *= u[b][c];
          } else {
            if (a.bias) {
              const f32x4 b0 = *(const f32x4*)bias, b1 = *(const f32x4*)(bias + 4);
#pragma unroll
              for (int b = 0; b < B; ++b)
#pragma unroll
                for (int c = 0; c < 8; ++c) v[b][c] += c < 4 ? b0[c] : b1[c - 4];
            }
            if (pre)
#pragma unroll
              for (int b = 0; b < B; ++b)
                if (r + b * kStep < t.rows && in)
                  *(u32x4*)(pre + ((uint32_t)(r + b * kStep) * (uint32_t)a.N + ch)) = pack8(v[b]);
            act_each(a.act, v);
            if (a.residual) {
              u32x4 row[B];
#pragma unroll
              for (int b = 0; b < B; ++b) {
                if constexpr (kAhead)
                  row[b] = add[b];
                else  // past the tile's end: its first row
                  row[b] = *(const u32x4*)(
                      a.residual + first +
                      (r + b * kStep < t.rows && in
                           ? (uint32_t)(r + b * kStep) * (uint32_t)a.N + ch : 0u));
              }
#pragma unroll
              for (int b = 0; b < B; ++b) {
                float more[8];
                unpack8(row[b], more);
#pragma unroll
                for (int c = 0; c < 8; ++c) v[b][c] += more[c];
              }
            }
          }
#pragma unroll
          for (int b = 0; b < B; ++b)
            if (r + b * kStep < t.rows && in) {
              if (codes)
                *(EP_LDS u32x4*)(base + kTurn + (r + b * kStep) * kRow + ch * 2) = pack8(v[b]);
              else
                *(u32x4*)(y + ((uint32_t)(r + b * kStep) * (uint32_t)a.N + ch)) = pack8(v[b]);
            }
        });
    if (codes) store_codes(t, base);
  }

  // FP8 output: eight lanes take 128 channels of a row, quantised as dispatch
  // does a bf16 row.  That takes a group's maximum by bit patterns and saturates, so a
  // NaN or infinity would turn the group into plausible finite values: each is
  // quantised as a zero here and gets the NaN code (e4m3 has no infinity).
  __device__ __forceinline__ void store_codes(const Tile& t, lds_char* base) {
    barrier();
    constexpr int kGroups = ON >= 128 ? ON / 128 : 1;
    for (int at = threadIdx.x / 8; at < S::BM * kGroups; at += kGemmThreads / 8) {
      const int r = at / kGroups, g = at % kGroups, l = threadIdx.x % 8;
      const EP_LDS u32x4* from = (const EP_LDS u32x4*)(base + kTurn + r * kRow + g * 256 + l * 32);
      u32x4 lo = from[0], hi = from[1];
      const bool bad = absmax16(lo, hi) >= 0x7F80u;
      u32x4 bad_lo = {}, bad_hi = {};
      if (bad) {
        bad_lo = take_not_finite(lo);
        bad_hi = take_not_finite(hi);
      }
      u32x4 out;
      float scale;
      uint32_t exponent;
      if (a.y_quant == EP_QUANT_FP8_F32)
        quantise_pair<EP_QUANT_FP8_F32>(lo, hi, out, scale, exponent);
      else
        quantise_pair<EP_QUANT_FP8_UE8M0>(lo, hi, out, scale, exponent);
      if (bad) {  // their codes are zero
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          out[q] |= nan_codes(bad_lo[2 * q], bad_lo[2 * q + 1]);
          out[2 + q] |= nan_codes(bad_hi[2 * q], bad_hi[2 * q + 1]);
        }
      }
      const int ch = t.n0 + g * 128;
      if (r < t.rows && ch < a.N) {
        *(u32x4*)((char*)a.y + (t.row + r) * a.N + ch + l * 16) = out;
        const int64_t at_scale =
            a.seg.start ? (int64_t)(ch / 128) * a.y_cap + t.row + r
                        : ((int64_t)t.e * (a.N / 128) + ch / 128) * a.seg.block_rows + t.block + r;
        if (l == 0) {
          if (a.y_quant == EP_QUANT_FP8_F32) ((float*)a.y_scales)[at_scale] = scale;
          else ((uint8_t*)a.y_scales)[at_scale] = (uint8_t)exponent;
        }
      }
    }
  }
};

template <class S, bool GATED, int Q>
__global__ __launch_bounds__(kGemmThreads, 1) void expert_forward(ExpertArgs a) {
  typedef Forward<S, GATED, Q> F;
  __shared__ __align__(16) char lds[S::STAGES][F::kSlot];
  // FP8: every wave's own copy of its rows' scales and, behind them, of its two
  // weight blocks'.  They come by the same asynchronous loads as the tiles: a
  // load into a register would have to be waited for, and with it every
  // load issued before it.
  __shared__ float scales[F::FP8 ? S::STAGES * 4 * F::kScales : 1];
  __shared__ TilePlan plan;
  static_assert(F::kTurn + (F::FP8 && F::ON >= 128 ? S::BM * F::kRow : 0) <= sizeof(lds),
                "the epilogue fits the tile buffers");
  plan_tiles<kGemmThreads>(a.seg, S::BM, plan, (int*)lds);
  lds_char* base = (lds_char*)&lds[0][0];
  F f(a, plan, base, (lds_float*)scales);
  const int64_t tiles = (int64_t)f.mt * f.nt;
  if constexpr (S::STAGES == 2) {
    typename S::acc_t acc[S::CT][S::TT];
    f.acc = acc;
    for (int64_t t = block_place(); t < tiles; t += gridDim.x) {
      const Tile tile = f.setup(t);
      clear<S>(acc);
      products_deep<S>(
          f.w_tile, f.x_tile, base, f.nk, f.nfull,
          [&](int k, lds_char* buf, int p) { f.load_at(k, buf, p); },
          [&](int k, lds_char* buf) { f.tail_at(k, buf); }, acc);
      f.epilogue(tile, base);
    }
  } else if constexpr (F::FP8) {
    RingEngine8<S, typename F::Chan, typename F::Row, GATED, Q> engine(base, (lds_float*)scales);
    f.acc = engine.acc;
    run_ring<S, S::kChains>(f, engine, base, block_place(), tiles,
                                      a.y_quant == EP_QUANT_NONE);
  } else {
    RingEngine<S, typename F::Chan, typename F::Row> engine(base);
    f.acc = engine.acc;
    run_ring<S, S::kChains>(f, engine, base, block_place(), tiles, true);
  }
}

typedef Shape<BigDims> Big;
typedef Shape<Big8Dims> Big8;
typedef Shape<MediumDims> Medium;
typedef Shape<NarrowDims> Narrow;
typedef Shape<SmallDims> Small;
typedef Shape<TinyDims> Tiny;

template <class S, bool GATED, int Q>
static void launch(const ExpertArgs& a, hipStream_t st) {
  const int on = GATED ? S::BN / 2 : S::BN;
  const int64_t tiles = ((a.rows + S::BM - 1) / S::BM + a.seg.E) * ((a.N + on - 1) / on);
  constexpr int64_t kSlots = forward_slots<S, Q != EP_QUANT_NONE>();
  hipLaunchKernelGGL((expert_forward<S, GATED, Q>), dim3((unsigned)std::min(tiles, kSlots)),
                     dim3(kGemmThreads), 0, st, a);
}

template <bool GATED, int Q>
static void choose(const ExpertArgs& a, hipStream_t st) {
  constexpr bool FP8 = Q != EP_QUANT_NONE;
  typedef typename std::conditional<FP8, Big8, Big>::type Large;
  switch (choose_forward<FP8>(a.seg.E, a.rows, a.C, (int64_t)a.N * (GATED ? 2 : 1),
                              a.y_quant != EP_QUANT_NONE)) {
    case kTinyTile: return launch<Tiny, GATED, Q>(a, st);
    case kSmallTile: return launch<Small, GATED, Q>(a, st);
    case kNarrowTile: return launch<Narrow, GATED, Q>(a, st);
    case kMediumTile: return launch<Medium, GATED, Q>(a, st);
    case kLargeTile: return launch<Large, GATED, Q>(a, st);
  }
}

template <bool GATED>
static void choose(const ExpertArgs& a, hipStream_t st) {
  switch (a.quant) {
    case EP_QUANT_NONE: return choose<GATED, EP_QUANT_NONE>(a, st);
    case EP_QUANT_FP8_F32: return choose<GATED, EP_QUANT_FP8_F32>(a, st);
    default: return choose<GATED, EP_QUANT_FP8_UE8M0>(a, st);
  }
}

hipError_t launch_expert_forward(const ExpertArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (a.gated) choose<true>(a, st);
  else choose<false>(a, st);
  return hipGetLastError();
}

}  // namespace ep
