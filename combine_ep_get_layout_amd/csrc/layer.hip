// A whole MoE layer for a few tokens on gfx950, in two or three launches and without layout
// or dispatch: for every token t and its entries (e, w),
//   h = act(x Wg_e^T) * (x Wu_e^T),                       (layer_gated, many_gated)
//   out_t = sum_k w_k h W2_e^T,   in fp32, in k order.    (layer_down, many_down + many_sum)
// h is kept as two bf16, its value rounded and what that leaves, 16 bits together: in one,
// its rounding alone would be as large an error of the result as the result's own.  They are
// two rows of the second product, whose sums are added.
//
// With few tokens the time is that of reading the weights of the experts that are hit: 64
// tokens over 256 experts (FP8, 7168 -> 2048) take 1.45 to 1.48 ms, 6.7 TB/s, in 8-bit integers
// 1.44; 32 over 16 experts (bf16, 4096 -> 1408) 97 us, 5.6 TB/s; one token over 8 (bf16, 2048 ->
// 768) 21.9 us, of which two launches' start and end are 7.8 and the second product 10 to 11: a
// workgroup has 16 channels of the result there, so with fewer than 4096 some units are idle.
// A wave multiplies strips of 16 rows of weights with up to 64 rows of one expert's entries.  It
// streams both through a ring in LDS (of its own, or with the rows in common to four waves), by
// asynchronous loads that never stop: towards the end of a strip they are the next one's.  Weights come as whole 128-byte lines of eight rows a load:
// straight into the registers of the matrix instructions, which take 16 rows x 64 bytes, they
// came at 4.1 TB/s instead.  Rows stay bf16 whatever the weights' type: e4m3 and 8-bit codes
// are converted (both fit bf16 exactly), and their scales are applied to the fp32 sums.
// Weights that are read once are not kept in the caches, which the rows come from (the first
// layer's gated part, each wave with its own rows: 1176 -> 1056 us).
#include <algorithm>

#include "experts.hpp"
#include "layer.hpp"

namespace ep {

constexpr int kMost = 64;  // entries of an expert that are multiplied at once, at most

// ---- who is hit ------------------------------------------------------------------

// The ids in LDS, and a bit for each expert with an entry: lane l's word has experts 32 l ...
struct Routing {
  int16_t ids[kLayerEntries];  // -1 or below kMaxExperts
  uint32_t hit[kMaxExperts / 32];
};

// weights: room for them in LDS, or NULL
template <int THREADS>
__device__ __forceinline__ void read_routing(const LayerArgs& a, Routing& r, float* weights) {
  for (int i = threadIdx.x; i < kMaxExperts / 32; i += THREADS) r.hit[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < kLayerEntries; i += THREADS) {
    int id = i < a.entries ? a.idx[i] : -1;
    if (weights && i < a.entries) weights[i] = a.weights[i];
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

// Expert e's entries (t * K + k), in their order: how many, and from the at-th on up to `room`
// of them to `list`, the wave's own.
__device__ __forceinline__ int entries_of(const LayerArgs& a, const Routing& r, int e, int at,
                                          int room, uint16_t* list) {
  const int lane = lane_id();
  int n = 0;
  for (int c = 0; c < a.entries; c += kWave) {
    const bool is = r.ids[c + lane] == e;
    const uint64_t mask = __ballot(is);
    const int place = n + rank_below(mask) - at;
    if (is && place >= 0 && place < room) list[place] = (uint16_t)(c + lane);
    n += __popcll(mask);
  }
  wave_lds_sync();
  return n;
}

// ---- a stream of lines -----------------------------------------------------------------

// What a wave multiplies next: up to a slot's room of an expert's entries, from the at-th
// on, with one strip.
struct Unit {
  int e, strip, at, rows, n;  // n: the expert's entries in all
  int start;                  // the line that it begins with, of the wave's
  uint16_t* list;             // the unit's
};

// A line is 128 bytes of each of 16 CT rows of weights and the channels that these
// multiply of the rows, which is 128 bytes of each in bf16 and 256 where the weights have 8
// bits.  A slot of the ring holds one: two loads (2 KiB) of weights a strip and NB of rows.  In
// LDS chunk c (16 bytes) of row r stands at c ^ turn(r), so that 16 lanes' reads of one chunk
// of 16 rows fall into different banks.
// SHARE waves of a workgroup may have the rows in common: then each loads a part of them, and
// they meet at every line.  ONCE: weights are not kept in the caches.
template <int KIND, int CT, int NB, int D, int SHARE = 1, bool ONCE = true>
struct Stream {
  static constexpr bool kBytes = KIND != EP_WEIGHTS_BF16;
  static constexpr int kSize = kBytes ? 1 : 2;
  static constexpr int kChunks = kBytes ? 16 : 8;           // of a row in a line
  static constexpr int kRows = NB * kWave / kChunks;        // that a slot has room for
  static constexpr int TT = (kRows + 15) / 16;              // in matrix-core tiles
  static constexpr int kWSlot = CT * 2048, kXSlot = NB * 1024;
  static constexpr int kMine = NB / SHARE;                  // loads of rows, a wave's
  static constexpr int kLoads = 2 * CT + kMine;
  static constexpr int kSteps = kBytes ? 4 : 2;             // matrix steps of a line
  static_assert(kRows <= kMost && (kRows < 16 || kRows % 16 == 0) && NB % SHARE == 0, "");

  lds_char *w_ring, *x_ring;
  int member;              // of those that share rows
  int lines, left;         // of a row of weights, and the last one's bytes
  bool turns;              // strips start at different lines
  const char *w, *x;       // of the unit that is loaded: uniform, with the lanes' offsets
  uint32_t w_off[2 * CT], x_off[kMine];
  f32x4 acc[CT][TT];

  __device__ __forceinline__ Stream(lds_char* w_r, lds_char* x_r, int m, int channels)
      : w_ring(w_r), x_ring(x_r), member(m), lines((channels * kSize + 127) / 128),
        left(channels * kSize - (lines - 1) * 128),
        turns(channels * kSize % 4096 == 0) {}

  static __device__ __forceinline__ int w_turn(int r) { return r / 2 & 7; }
  static __device__ __forceinline__ int x_turn(int r) { return kBytes ? r & 15 : r / 2 & 7; }

  // the row that the lane loads in the wave's i-th load of rows
  __device__ __forceinline__ int x_row(int i) const {
    return (i * SHARE + member) * (kWave / kChunks) + lane_id() / kChunks;
  }
  // row(r): byte offset from w of weight row r; entry(r): from x of the unit's row r
  template <class Row, class Entry>
  __device__ __forceinline__ void point(const char* w_, const char* x_, Row row, Entry entry) {
    const int lane = lane_id();
    w = w_;
    x = x_;
#pragma unroll
    for (int i = 0; i < 2 * CT; ++i) {
      const int r = 8 * i + lane / 8;
      w_off[i] = row(r) + ((lane % 8 ^ w_turn(r)) << 4);
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int r = x_row(i);
      x_off[i] = entry(r) + ((lane % kChunks ^ x_turn(r)) << 4);
    }
  }
  __device__ __forceinline__ void load(int line, int slot) const {
    lds_char* to = w_ring + slot * kWSlot;
    lds_char* x_to = x_ring + slot * kXSlot + 1024 * member;
    const char* wl = w + (int64_t)line * 128;
    const char* xl = x + (int64_t)line * (16 * kChunks);
    if (KIND == EP_WEIGHTS_FP8 || line < lines - 1 || left == 128) {
#pragma unroll
      for (int i = 0; i < 2 * CT; ++i) {
        if (ONCE) stream_lds16(wl, w_off[i], to + 1024 * i);
        else load_lds16(wl, w_off[i], to + 1024 * i);
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) load_lds16(xl, x_off[i], x_to + 1024 * SHARE * i);
    } else {  // chunks past the end are zeros on both sides
      const int lane = lane_id(), chunks = left / 16 * (kBytes ? 2 : 1);
#pragma unroll
      for (int i = 0; i < 2 * CT; ++i) {
        const bool in = (lane % 8 ^ w_turn(8 * i + lane / 8)) * 16 < left;
        load_lds16(in ? wl + w_off[i] : (const char*)k_zeros, to + 1024 * i);
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const bool in = (lane % kChunks ^ x_turn(x_row(i))) < chunks;
        load_lds16(in ? xl + x_off[i] : (const char*)k_zeros, x_to + 1024 * SHARE * i);
      }
    }
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

  // Lane l holds row l % 16 of both operands.  In bf16 a step is 32 channels, in 8 bits a
  // lane's 16 codes are two steps, the first eight of every lane and the last.
  // scale: FP8, of this line's 128 channels
  __device__ __forceinline__ void multiply(int slot, float scale) {
    const lds_char *from = w_ring + slot * kWSlot, *x_from = x_ring + slot * kXSlot;
    const int lane = lane_id(), r = lane % 16, q = lane / 16;
    i32x4 wv[CT][2];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        wv[c][i] = *(const EP_LDS i32x4*)(from + (16 * c + r) * 128 + ((q + 4 * i ^ w_turn(r)) << 4));
    bf16x8 f[CT][kSteps];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if constexpr (kBytes)
          f[c][i] = codes((uint32_t)wv[c][i / 2][2 * (i % 2)], (uint32_t)wv[c][i / 2][2 * (i % 2) + 1]);
        else
          f[c][i] = __builtin_bit_cast(bf16x8, wv[c][i]);
      }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      // rows past the slot's room repeat its last one; their columns are not used
      const int xr = kRows < 16 ? min(r, kRows - 1) : 16 * j + r;
      bf16x8 xv[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int c = kBytes ? 8 * (i / 2) + 2 * q + i % 2 : q + 4 * i;
        xv[i] = __builtin_bit_cast(bf16x8, *(const EP_LDS i32x4*)(x_from + xr * 16 * kChunks +
                                                                  ((c ^ x_turn(xr)) << 4)));
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        f32x4 sum = KIND == EP_WEIGHTS_FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[c][j];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) sum = Mfma<16>::bf16(f[c][i], xv[i], sum);
        if (KIND == EP_WEIGHTS_FP8) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) acc[c][j][q4] = __builtin_fmaf(sum[q4], scale, acc[c][j][q4]);
        } else {
          acc[c][j] = sum;
        }
      }
    }
  }

  // Unit after unit; of each the lines part, part + parts, ..
  //   next(unit): the wave's next unit, false after the last
  //   aim(unit): calls point()
  //   scales(unit, line): FP8, the line's scale
  //   done(unit): takes acc
  template <class Next, class Aim, class Scales, class Done>
  __device__ __forceinline__ void run(int part, int parts, Next next, Aim aim, Scales scales,
                                      Done done) {
    const int n = part < lines ? (lines - part + parts - 1) / parts : 0;
    // The waves are at the same channels of their rows at the same time, and where a row's
    // length is a multiple of 4 KiB those share few memory channels: there every strip begins
    // somewhere else (rows of 8 KiB, 32 tokens over 16 experts: 67 -> 63 us; of 2 and 7 KiB
    // 2% slower).
    auto begin = [&](Unit& unit) {
      unit.start = turns ? uniform((uint32_t)(unit.strip / SHARE * 11 + unit.e * 7) % (uint32_t)n) : 0;
      aim(unit);
    };
    auto line_of = [&](const Unit& unit, int i) {
      i += unit.start;
      return part + (i >= n ? i - n : i) * parts;
    };
    Unit now, then;
    if (!next(now)) return;
    begin(now);
    const bool chain = n >= D - 1;
    int slot = 0;
    auto after = [](int s) { return s + 1 == D ? 0 : s + 1; };
    bool fresh = true;
    for (;;) {
      if (fresh) {
#pragma unroll
        for (int i = 0; i < D - 1; ++i)
          if (i < n) load(line_of(now, i), i);
        slot = 0;
      }
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[c][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      bool more = false;
      float scale = n > 0 ? scales(now, line_of(now, 0)) : 0.0f;
      for (int i = 0; i < n; ++i) {
        const int ahead = i + D - 1, into = slot == 0 ? D - 1 : slot - 1;
        // the line before has been read out of the slot that is loaded
        if (SHARE > 1) {  // by all, and all have their part of this one
          if (ahead - 1 < n || more) wait_loads<kLoads*(D - 2)>();
          else wait_loads<0>();
          barrier();
        } else {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        if (ahead < n) {
          load(line_of(now, ahead), into);
          if (SHARE == 1) wait_loads<kLoads*(D - 1)>();
        } else {
          if (ahead == n && chain) {
            more = next(then);
            if (more) begin(then);
          }
          if (more) {
            load(line_of(then, ahead - n), into);
            if (SHARE == 1) wait_loads<kLoads*(D - 1)>();
          } else if (SHARE == 1) {
            wait_loads<0>();
          }
        }
        const float own = scale;  // the next line's is on its way during this one's products
        scale = scales(now, line_of(now, i + 1 < n ? i + 1 : 0));
        multiply(slot, own);
        slot = after(slot);
      }
      done(now);
      if (!chain) {
        if (SHARE > 1) barrier();
        else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        more = next(then);
        if (more) begin(then);
      }
      if (!more) return;
      now = then;
      fresh = !chain;
    }
  }
};

// FP8 scales are the same for the whole wave and do not change: scalar loads, since a vector
// load would be waited for together with every asynchronous load before it.
__device__ __forceinline__ float fixed_float(const float* p) {
  return *(const __attribute__((address_space(4))) float*)p;
}

// a: v in the lower half of the wave, b: in the upper one, in all lanes
__device__ __forceinline__ void halves(float v, float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}

// What rounding leaves of h; nothing of a NaN or infinity, which is its rounded value alone.
__device__ __forceinline__ float rest_of(float h, float rounded) {
  return fabsf(rounded) < __builtin_inff() ? h - rounded : 0.0f;
}

// ---- gated block -------------------------------------------------------------------

constexpr int kUpStride = 20;  // floats of a column of partial sums, 16 and a gap

// The stream's next loads: strips of 8 gates and ups from channel n0 on, and the unit's rows
template <class S>
__device__ __forceinline__ void aim_gated(const LayerArgs& a, S& stream, const Unit& unit, int n0,
                                          int64_t w_row) {
  stream.point(
      a.w13 + ((int64_t)unit.e * 2 * a.I + n0) * w_row, (const char*)a.x,
      [&](int r) {  // past the last channel: that one again, not stored
        const int ch = min(r / 16 * 8 + r % 8, a.I - 1 - n0);
        return (uint32_t)((r % 16 < 8 ? ch : a.I + ch) * w_row);
      },
      [&](int r) {
        return (uint32_t)(unit.list[min(r, unit.rows - 1)] / a.K) * (uint32_t)(a.H * 2);
      });
}

// FP8: the scale of expert e's channels n0 .. in a line, of its gates in the lower half of the
// wave and of its ups in the upper one
template <int KIND>
__device__ __forceinline__ float gated_scale(const LayerArgs& a, int e, int n0, int line) {
  if (KIND != EP_WEIGHTS_FP8) return 1.0f;
  const int64_t groups = a.H / 128;
  const float* s = a.s13 + ((int64_t)e * (2 * a.I / 128) + n0 / 128) * groups + line;
  const float gate = fixed_float(s), up = fixed_float(s + a.I / 128 * groups);
  return lane_id() < 32 ? gate : up;
}

// h of the unit's r-th row: channels n0 + ch (0 or 4) and three more, of the sums of their
// gates and ups
template <int KIND>
__device__ __forceinline__ void store_h(const LayerArgs& a, const Unit& unit, int r, int n0,
                                        int ch, float (&g)[4], float (&up)[4]) {
  const float* scale = a.s13 + (int64_t)unit.e * 2 * a.I + n0;
  bf16x2 high[2], low[2];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (KIND == EP_WEIGHTS_INT8) {
      const float g0 = fixed_float(scale + q), g1 = fixed_float(scale + 4 + q);
      const float u0 = fixed_float(scale + a.I + q), u1 = fixed_float(scale + a.I + 4 + q);
      g[q] *= ch == 0 ? g0 : g1;
      up[q] *= ch == 0 ? u0 : u1;
    }
    float value, slope;
    act_both(a.act, g[q], value, slope);
    const float h = value * up[q];
    high[q / 2][q % 2] = (__bf16)h;
    low[q / 2][q % 2] = (__bf16)rest_of(h, (float)high[q / 2][q % 2]);
  }
  if (r < unit.rows) {
    uint16_t* to = a.h + (int64_t)unit.list[r] * 2 * a.I + n0 + ch;
    *(uint2*)to = __builtin_bit_cast(uint2, high);
    *(uint2*)(to + a.I) = __builtin_bit_cast(uint2, low);
  }
}

// A strip is eight channels of one expert, their gates and ups.  WK waves share CT strips,
// the lines dealt to them in turn; a wave's sums of rows 4 (lane / 16) .. are gates in the
// lower half of its lanes and ups in the upper one.
template <int KIND, int CT, int NB, int D, int WK>
__global__ __launch_bounds__(kUpWaves* kWave) void layer_gated(LayerArgs a) {
  typedef Stream<KIND, CT, NB, D> S;
  static_assert(WK == 1 || WK == kUpWaves, "a workgroup's barriers");
  constexpr int kCols = 16 * S::TT;
  __shared__ Routing routing;
  __shared__ uint16_t lists[kUpWaves][2][S::kRows];
  __shared__ __align__(16) char rings[kUpWaves][D * (S::kWSlot + S::kXSlot)];
  __shared__ __align__(16) float parts[WK > 1 ? WK * kCols * kUpStride : 1];
  read_routing<kUpWaves * kWave>(a, routing, nullptr);
  const Hits hits(routing);
  const int wave = uniform(threadIdx.x / kWave), lane = lane_id(), row = lane % 16;
  const int strips = (a.I + 8 * CT - 1) / (8 * CT), units = hits.total * strips;
  const int64_t w_row = (int64_t)a.H * S::kSize;
  constexpr int kTeams = kUpWaves / WK;
  int u = blockIdx.x * kTeams + wave / WK - gridDim.x * kTeams, turn = 0;
  Unit last;
  last.n = 0;
  last.at = last.e = -1;
  S stream((lds_char*)rings[wave], (lds_char*)rings[wave] + D * S::kWSlot, 0, a.H);
  stream.run(
      WK > 1 ? wave % WK : 0, WK,
      [&](Unit& unit) {
        const int e = last.e, at = last.at;
        last.at += S::kRows;  // more entries of the same expert
        if (e < 0 || last.at >= last.n) {
          u += gridDim.x * kTeams;
          if (u >= units) return false;
          last.e = hits.expert(u / strips);
          last.strip = u % strips;
          last.at = 0;
        }
        if (last.e != e || last.at != at) {
          last.list = lists[wave][turn ^= 1];
          last.n = entries_of(a, routing, last.e, last.at, S::kRows, last.list);
        }
        last.rows = min(last.n - last.at, S::kRows);
        unit = last;
        return true;
      },
      [&](const Unit& unit) {
        aim_gated(a, stream, unit, unit.strip * 8 * CT, w_row);
      },
      [&](const Unit& unit, int line) { return gated_scale<KIND>(a, unit.e, unit.strip * 8 * CT, line); },
      [&](const Unit& unit) {
        const int ch = 4 * (lane / 16 % 2);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const int n0 = (unit.strip * CT + c) * 8;
          if (WK > 1) {
#pragma unroll
            for (int j = 0; j < S::TT; ++j)
              *(f32x4*)(parts + (wave % WK * kCols + 16 * j + row) * kUpStride + 4 * (lane / 16)) =
                  stream.acc[c][j];
            barrier();
          }
          if (n0 < a.I) {
#pragma unroll
            for (int j = 0; j < S::TT; ++j) {
              if (WK > 1 && j % WK != wave) continue;  // a tile each
              float g[4], up[4];
              if (WK > 1) {
#pragma unroll
                for (int q = 0; q < 4; ++q) g[q] = up[q] = 0.0f;
#pragma unroll
                for (int w = 0; w < WK; ++w) {
                  const float* from = parts + (w * kCols + 16 * j + row) * kUpStride + ch;
#pragma unroll
                  for (int q = 0; q < 4; ++q) g[q] += from[q], up[q] += from[8 + q];
                }
              } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) halves(stream.acc[c][j][q], g[q], up[q]);
              }
              if (lane < 32) store_h<KIND>(a, unit, 16 * j + row, n0, ch, g, up);
            }
          }
          if (WK > 1) barrier();
        }
      });
}

// v of the lane beside: even and odd ones in pairs
__device__ __forceinline__ float neighbour(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
}

// ---- down projection and the weighted sum ---------------------------------------------

template <int KIND>
__device__ __forceinline__ float down_scale(const LayerArgs& a, int e, int n0, int line) {
  if (KIND != EP_WEIGHTS_FP8) return 1.0f;
  return fixed_float(a.s2 + ((int64_t)e * (a.H / 128) + n0 / 128) * (a.I / 128) + line);
}

// The stream's next loads: strips of 16 channels from n0 on, and the unit's rows of h
template <class S>
__device__ __forceinline__ void aim_down(const LayerArgs& a, S& stream, const Unit& unit, int n0,
                                         int64_t w_row) {
  stream.point(
      a.w2 + ((int64_t)unit.e * a.H + n0) * w_row, (const char*)a.h,
      // past the last channel: that one again, not stored
      [&](int r) { return (uint32_t)(min(r, a.H - 1 - n0) * w_row); },
      [&](int r) {
        return (unit.list[min(r / 2, unit.rows - 1)] * 2u + r % 2) * (uint32_t)(a.I * 2);
      });
}

// The results of a unit's entries in one strip, from the sums of their two rows
template <int TT>
__device__ __forceinline__ void store_y(float* y, int64_t y_row, const Unit& unit,
                                        const f32x4 (&acc)[TT]) {
  const int row = lane_id() % 16, ch = 4 * (lane_id() / 16);
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    f32x4 sum = acc[j];
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[q] += neighbour(sum[q]);
    const int r = (16 * j + row) / 2;
    if (row % 2 == 0 && r < unit.rows) *(f32x4*)(y + unit.list[r] * y_row + ch) = sum;
  }
}

// A workgroup has a strip of 16 channels of every token.  Its waves take an expert each in turn
// (or parts of the contraction, where there are fewer experts than waves) and put every
// entry's result into a place of its own; then they are summed in k order.
template <int KIND, int NB, int D, int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void layer_down(LayerArgs a) {
  typedef Stream<KIND, 1, NB, D> S;
  __shared__ Routing routing;
  constexpr int kEntries = S::kRows / 2;  // a slot's, two rows each
  __shared__ uint16_t lists[WAVES][2][kEntries];
  __shared__ __align__(16) char rings[WAVES][D * (S::kWSlot + S::kXSlot)];
  __shared__ float weights[kLayerPlaces];
  __shared__ __align__(16) float places[kLayerPlaces * 16];
  read_routing<WAVES * kWave>(a, routing, weights);
  const Hits hits(routing);
  const int wave = uniform(threadIdx.x / kWave), n0 = blockIdx.x * 16;
  const int64_t w_row = (int64_t)a.I * S::kSize;
  // parts that every expert's contraction is cut into
  int parts = 1;
  while (2 * parts * hits.total <= WAVES && 2 * parts * a.entries <= kLayerPlaces) parts *= 2;
  const int part = wave % parts;
  float* const y = places + part * a.entries * 16;
  int u = wave / parts - WAVES / parts, turn = 0;
  Unit last;
  last.n = 0;
  last.at = last.e = -1;
  last.strip = blockIdx.x;
  S stream((lds_char*)rings[wave], (lds_char*)rings[wave] + D * S::kWSlot, 0, a.I);
  stream.run(
      part, parts,
      [&](Unit& unit) {
        last.at += kEntries;
        if (last.e < 0 || last.at >= last.n) {
          u += WAVES / parts;
          if (u >= hits.total) return false;
          last.e = hits.expert(u);
          last.at = 0;
        }
        last.list = lists[wave][turn ^= 1];
        last.n = entries_of(a, routing, last.e, last.at, kEntries, last.list);
        last.rows = min(last.n - last.at, kEntries);
        unit = last;
        return true;
      },
      [&](const Unit& unit) { aim_down(a, stream, unit, n0, w_row); },
      [&](const Unit& unit, int line) { return down_scale<KIND>(a, unit.e, n0, line); },
      [&](const Unit& unit) { store_y(y, 16, unit, stream.acc[0]); });
  __syncthreads();
  for (int o = threadIdx.x; o < a.tokens * 16; o += WAVES * kWave) {
    const int t = o / 16, ch = o % 16;
    if (n0 + ch >= a.H) continue;
    float sum = 0.0f;
    for (int k = 0; k < a.K; ++k) {
      const int i = t * a.K + k, e = routing.ids[i];
      if (e < 0) continue;
      float v = 0.0f;
      for (int p = 0; p < parts; ++p) v += places[(p * a.entries + i) * 16 + ch];
      if (KIND == EP_WEIGHTS_INT8) v *= a.s2[(int64_t)e * a.H + n0 + ch];
      sum = __builtin_fmaf(weights[i], v, sum);
    }
    ((__bf16*)a.out)[(int64_t)t * a.H + n0 + ch] = (__bf16)sum;
  }
}

// ---- many entries an expert ------------------------------------------------------------

// kTeam waves share the rows of up to a slot's room of one expert's entries (a chunk), each with
// CT strips of its own; entries' results go to the workspace, and a third launch sums them.
// A wave alone would read the rows for one or two strips: 16 experts with 16 / 32 / 64 entries
// (bf16 4096 -> 1408) take 118 / 131 / 174 us, waves alone 162 / 207 / 339; 256 with 2 in FP8
// (7168 -> 2048) 1480 and 1770 us.  Layout, dispatch, the experts' products and combine take 136
// / 152 / 150 us for those 16.
constexpr int kTeam = 4;

template <int ROWS>
struct Chunks {
  uint16_t expert[kLayerEntries], at[kLayerEntries];  // every one has an entry
  int sums[kTeam], total;
  // count: room for kMaxExperts
  __device__ __forceinline__ void find(const LayerArgs& a, const Routing& r, int* count) {
    constexpr int kEach = kMaxExperts / (kTeam * kWave);
    const int first = threadIdx.x * kEach, lane = lane_id(), wave = threadIdx.x / kWave;
    for (int i = threadIdx.x; i < kMaxExperts; i += kTeam * kWave) count[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.entries; i += kTeam * kWave)
      if (r.ids[i] >= 0) atomicAdd(&count[r.ids[i]], 1);
    __syncthreads();
    int own = 0;
    for (int e = first; e < first + kEach; ++e) own += (count[e] + ROWS - 1) / ROWS;
    int place = own;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int v = __shfl_up(place, d);
      if (lane >= d) place += v;
    }
    if (lane == kWave - 1) sums[wave] = place;
    __syncthreads();
    place -= own;
    for (int w = 0; w < wave; ++w) place += sums[w];
    for (int e = first; e < first + kEach; ++e)
      for (int n = 0; n < count[e]; n += ROWS, ++place) expert[place] = e, at[place] = n;
    if (threadIdx.x == kTeam * kWave - 1) total = place;
    __syncthreads();
  }
};

// A workgroup's next unit of `groups` groups of strips by all chunks, of it the part of this
// wave; false after the last.  A die takes a run of units, chunks of the same weights one after
// the other.
template <int ROWS>
__device__ __forceinline__ bool team_next(const LayerArgs& a, const Routing& routing,
                                          const Chunks<ROWS>& chunks, int groups, int& u,
                                          uint16_t* list, Unit& unit) {
  const int total = uniform(chunks.total), units = total * groups;
  int v;
  do {
    u += gridDim.x;
    if (u >= xcd_blocks(units)) return false;
    v = uniform(xcd_run(u, units));
  } while (v >= units);
  const int group = uniform(v / total), c = v - group * total;
  unit.e = uniform(chunks.expert[c]);
  unit.at = uniform(chunks.at[c]);
  unit.strip = group * kTeam + uniform(threadIdx.x / kWave);
  unit.list = list;
  unit.n = entries_of(a, routing, unit.e, unit.at, ROWS, list);
  unit.rows = min(unit.n - unit.at, ROWS);
  return true;
}

template <int KIND, int CT, int NB, int D, bool ONCE>
__global__ __launch_bounds__(kTeam* kWave) void many_gated(LayerArgs a) {
  typedef Stream<KIND, CT, NB, D, kTeam, ONCE> S;
  __shared__ Routing routing;
  __shared__ Chunks<S::kRows> chunks;
  __shared__ uint16_t lists[kTeam][2][S::kRows];
  __shared__ __align__(16) char w_rings[kTeam][D * S::kWSlot], x_ring[D * S::kXSlot];
  read_routing<kTeam * kWave>(a, routing, nullptr);
  chunks.find(a, routing, (int*)w_rings);
  const int wave = uniform(threadIdx.x / kWave), lane = lane_id(), row = lane % 16;
  const int64_t w_row = (int64_t)a.H * S::kSize;
  int u = blockIdx.x - gridDim.x, turn = 0;
  S stream((lds_char*)w_rings[wave], (lds_char*)x_ring, wave, a.H);
  stream.run(
      0, 1,
      [&](Unit& unit) {
        return team_next(a, routing, chunks, (a.I + 8 * CT * kTeam - 1) / (8 * CT * kTeam), u,
                         lists[wave][turn ^= 1], unit);
      },
      [&](const Unit& unit) {
        aim_gated(a, stream, unit, min(unit.strip * 8 * CT, a.I - 1), w_row);
      },
      [&](const Unit& unit, int line) { return gated_scale<KIND>(a, unit.e, unit.strip * 8 * CT, line); },
      [&](const Unit& unit) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const int n0 = (unit.strip * CT + c) * 8;
          if (n0 >= a.I) continue;
#pragma unroll
          for (int j = 0; j < S::TT; ++j) {
            float g[4], up[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) halves(stream.acc[c][j][q], g[q], up[q]);
            if (lane < 32) store_h<KIND>(a, unit, 16 * j + row, n0, 4 * (lane / 16 % 2), g, up);
          }
        }
      });
}

template <int KIND, int CT, int NB, int D, bool ONCE>
__global__ __launch_bounds__(kTeam* kWave) void many_down(LayerArgs a) {
  typedef Stream<KIND, CT, NB, D, kTeam, ONCE> S;
  constexpr int kEntries = S::kRows / 2;
  __shared__ Routing routing;
  __shared__ Chunks<kEntries> chunks;
  __shared__ uint16_t lists[kTeam][2][kEntries];
  __shared__ __align__(16) char w_rings[kTeam][D * S::kWSlot], x_ring[D * S::kXSlot];
  read_routing<kTeam * kWave>(a, routing, nullptr);
  chunks.find(a, routing, (int*)w_rings);
  const int wave = uniform(threadIdx.x / kWave);
  const int64_t w_row = (int64_t)a.I * S::kSize, y_row = (a.H + 15) / 16 * 16;
  int u = blockIdx.x - gridDim.x, turn = 0;
  S stream((lds_char*)w_rings[wave], (lds_char*)x_ring, wave, a.I);
  stream.run(
      0, 1,
      [&](Unit& unit) {
        return team_next(a, routing, chunks, (a.H + 16 * CT * kTeam - 1) / (16 * CT * kTeam), u,
                         lists[wave][turn ^= 1], unit);
      },
      [&](const Unit& unit) {
        aim_down(a, stream, unit, min(unit.strip * 16 * CT, a.H - 1), w_row);
      },
      [&](const Unit& unit, int line) { return down_scale<KIND>(a, unit.e, unit.strip * 16 * CT, line); },
      [&](const Unit& unit) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const int n0 = (unit.strip * CT + c) * 16;
          if (n0 < a.H) store_y(a.y + n0, y_row, unit, stream.acc[c]);
        }
      });
}

// Four channels of a token a thread
template <int KIND>
__global__ __launch_bounds__(kWave * 4) void many_sum(LayerArgs a) {
  const int t = blockIdx.x, ch = (blockIdx.y * kWave * 4 + threadIdx.x) * 4;
  if (ch >= a.H) return;
  const int64_t y_row = (a.H + 15) / 16 * 16;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int k = 0; k < a.K; ++k) {
    const int i = t * a.K + k, e = a.idx[i];
    if (e < 0 || e >= a.E) continue;
    f32x4 v = *(const f32x4*)(a.y + i * y_row + ch);
    if (KIND == EP_WEIGHTS_INT8) {
      const f32x4 scale = *(const f32x4*)(a.s2 + (int64_t)e * a.H + ch);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] *= scale[q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[q] = __builtin_fmaf(a.weights[i], v[q], sum[q]);
  }
  bf16x2 out[2];
#pragma unroll
  for (int q = 0; q < 4; ++q) out[q / 2][q % 2] = (__bf16)sum[q];
  *(uint2*)(a.out + (int64_t)t * a.H + ch) = __builtin_bit_cast(uint2, out);
}

// ---- launches ------------------------------------------------------------------------

// WK: waves that a strip's lines are dealt to
template <int KIND, int CT, int NB, int D, int WK>
static void launch_gated(const LayerArgs& a, hipStream_t st) {
  const int64_t strips = (int64_t)std::min(a.E, a.entries) * ((a.I + 8 * CT - 1) / (8 * CT));
  const int64_t blocks = WK == 1 ? kUpRoom : std::min<int64_t>(strips, 4 * kCus);
  hipLaunchKernelGGL((layer_gated<KIND, CT, NB, D, WK>), dim3((unsigned)blocks),
                     dim3(kUpWaves * kWave), 0, st, a);
}

template <int KIND, int NB, int D, int WAVES>
static void launch_down(const LayerArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((layer_down<KIND, NB, D, WAVES>), dim3((a.H + 15) / 16), dim3(WAVES * kWave),
                     0, st, a);
}

// In 8 bits a slot's rows are as many bytes as its weights, or more, so two strips share them.
template <int KIND>
static void choose_gated(const LayerArgs& a, hipStream_t st) {
  constexpr bool kBytes = KIND != EP_WEIGHTS_BF16;
  switch (choose_layer_gated(kBytes, a.entries, a.E, a.I)) {
    case kGatedFew: return launch_gated<KIND, 1, 1, 3, 1>(a, st);
    case kGatedFewSplit: return launch_gated<KIND, 1, 1, 3, kUpWaves>(a, st);
    case kGatedSome:
      return launch_gated<KIND, kBytes ? 2 : 1, kBytes ? 4 : 2, kBytes ? 2 : 3, kUpWaves>(a, st);
    case kGatedMost: return launch_gated<KIND, 2, 8, 2, kUpWaves>(a, st);
  }
}

// An entry has two rows here, a workgroup as many waves as the LDS has rings for, up to 8.
template <int KIND>
static void choose_down(const LayerArgs& a, hipStream_t st) {
  constexpr bool kBytes = KIND != EP_WEIGHTS_BF16;
  switch (choose_layer_down(kBytes, a.entries, a.E)) {
    case kDown4: return launch_down<KIND, kBytes ? 2 : 1, 3, 8>(a, st);
    case kDown8: return launch_down<KIND, kBytes ? 4 : 2, kBytes ? 2 : 3, 8>(a, st);
    case kDown16: return launch_down<KIND, kBytes ? 8 : 4, kBytes ? 2 : 3, 6>(a, st);
    case kDown32:
      if constexpr (!kBytes) return launch_down<KIND, 8, 2, 6>(a, st);
  }
}

template <int KIND, bool GATED, int CT, int NB, int D, bool ONCE>
static void launch_many(const LayerArgs& a, hipStream_t st) {
  constexpr int kEntries = NB * (KIND == EP_WEIGHTS_BF16 ? 8 : 4) / (GATED ? 1 : 2);
  constexpr int kGroup = (GATED ? 8 : 16) * CT * kTeam;  // channels
  const int64_t chunks = a.entries / kEntries + std::min(a.E, a.entries);
  const int64_t units = chunks * (((GATED ? a.I : a.H) + kGroup - 1) / kGroup);
  const int64_t room = (NB == 4 ? 3 : 2) * kCus;  // workgroups at once
  const dim3 grid((unsigned)std::min<int64_t>(xcd_blocks(units), room)), threads(kTeam * kWave);
  if (GATED) hipLaunchKernelGGL((many_gated<KIND, CT, NB, D, ONCE>), grid, threads, 0, st, a);
  else hipLaunchKernelGGL((many_down<KIND, CT, NB, D, ONCE>), grid, threads, 0, st, a);
}

template <int KIND, bool GATED>
static void choose_many(const LayerArgs& a, hipStream_t st) {
  constexpr bool kBytes = KIND != EP_WEIGHTS_BF16;
  constexpr int NB = kBytes ? 16 : 8;
  switch (choose_layer_many(GATED, a.entries, a.E, GATED ? a.I : a.H)) {
    case kManyFew1: return launch_many<KIND, GATED, 1, 4, 3, true>(a, st);
    case kManyFew2: return launch_many<KIND, GATED, 2, 4, 2, true>(a, st);
    case kManyRows1: return launch_many<KIND, GATED, 1, NB, kBytes ? 3 : 4, false>(a, st);
    case kManyRows2Once: return launch_many<KIND, GATED, 2, NB, kBytes ? 2 : 3, true>(a, st);
    case kManyRows2: return launch_many<KIND, GATED, 2, NB, kBytes ? 2 : 3, false>(a, st);
  }
}

template <int KIND>
static void choose(const LayerArgs& a, hipStream_t st) {
  if (layer_many(a.entries, a.E, a.I)) {
    choose_many<KIND, true>(a, st);
    choose_many<KIND, false>(a, st);
    hipLaunchKernelGGL((many_sum<KIND>),
                       dim3(a.tokens, (a.H + 4 * 4 * kWave - 1) / (4 * 4 * kWave)),
                       dim3(4 * kWave), 0, st, a);
    return;
  }
  choose_gated<KIND>(a, st);
  choose_down<KIND>(a, st);
}

hipError_t launch_layer(const LayerArgs& a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  switch (a.kind) {
    case EP_WEIGHTS_BF16: choose<EP_WEIGHTS_BF16>(a, st); break;
    case EP_WEIGHTS_FP8: choose<EP_WEIGHTS_FP8>(a, st); break;
    default: choose<EP_WEIGHTS_INT8>(a, st); break;
  }
  return hipGetLastError();
}

}  // namespace ep
