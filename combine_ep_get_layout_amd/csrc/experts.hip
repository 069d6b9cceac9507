// The experts' forward products on gfx950: the gated feed-forward block
//   h = act(x Wg^T) * (x Wu^T)
// and the product with bias, activation and residual
//   y = act(x W^T + b) + r
// over the rows of each expert's segment, one launch each.
#include <type_traits>

#include "experts.hpp"
#include "quant.hpp"

namespace ep {

// Where a workgroup's tile starts in the row buffers (row 0, channel 0 of the
// tile) and the bias of its channels; offsets from there fit 32 bits.
struct TileOut {
  uint16_t* y;
  uint16_t* pre;
  const uint16_t* residual;
  const float* bias;
};

// Eight consecutive channels of one row: the epilogue's arithmetic.  at: the
// vector's offset in a buffer of N channels; gated: r, ch its row and channel.
// Returns the result in bf16.
template <bool GATED, class T>
__device__ __forceinline__ u32x4 finish8(const ExpertArgs& a, const TileOut& o, uint32_t at, int r,
                                         int ch, int further, const T& turned) {
  float v[8];
  turned.get(0, v);
  if (GATED) {
    float u[8];
    turned.get(further, u);
    if (o.pre) {
      uint16_t* to = o.pre + ((uint32_t)r * 2u * (uint32_t)a.N + ch);
      *(u32x4*)to = pack8(v);
      *(u32x4*)(to + a.N) = pack8(u);
    }
    act_each(a.act, v);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] *= u[c];
  } else {
    if (o.bias) {
      const f32x4 b0 = *(const f32x4*)(o.bias + ch), b1 = *(const f32x4*)(o.bias + ch + 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] += b0[c], v[4 + c] += b1[c];
    }
    if (o.pre) *(u32x4*)(o.pre + at) = pack8(v);
    act_each(a.act, v);
    if (o.residual) {
      float add[8];
      unpack8(*(const u32x4*)(o.residual + at), add);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] += add[c];
    }
  }
  return pack8(v);
}

// Q: EP_QUANT_*
template <class S, bool GATED, int Q>
__global__ __launch_bounds__(kGemmThreads, 1) void expert_forward(ExpertArgs a) {
  constexpr bool FP8 = Q != EP_QUANT_NONE;
  constexpr int MF = S::MF, CT = S::CT, TT = S::TT;
  // gated: a wave's channel tiles are half gates and half ups of the same channels
  constexpr int CH = GATED ? CT / 2 : CT;      // channel tiles of the output per wave
  constexpr int ON = GATED ? S::BN / 2 : S::BN;  // output channels per workgroup tile
  typedef typename S::acc_t acc_t;
  __shared__ __align__(16) char lds[S::STAGES][(S::BN + S::BM) * S::KB];
  // FP8: every wave's own copy of its rows' scales and, behind them, of its two
  // weight blocks'.  They come by the same asynchronous loads as the tiles: a
  // load into a register would have to be waited for, and with it every
  // load issued before it.
  __shared__ float lds_scales[FP8 ? S::STAGES : 1][4][FP8 ? (S::SLOADS + 1) * kWave : 1];
  __shared__ TilePlan<kGemmThreads> plan;

  const int lane = lane_id(), wave = uniform(threadIdx.x >> 6);
  const int wc = wave % S::WC, wt = wave / S::WC;
  plan_tiles(a.seg, S::BM, plan);
  const int mt = plan.first[a.seg.E];
  const int nt = (a.N + ON - 1) / ON;
  const int64_t tiles = (int64_t)mt * nt;
  const int esize = FP8 ? 1 : 2;
  const int64_t row_bytes = (int64_t)a.C * esize;
  const int nk = (int)((row_bytes + S::KB - 1) / S::KB), nfull = (int)(row_bytes / S::KB);

  for (int64_t t = block_place(); t < tiles; t += gridDim.x) {
    int m, n;
    tile_at(t, mt, nt, m, n);
    const int e = expert_of(plan, a.seg.E, m);
    int64_t start;
    int count;
    segment_of(a.seg, e, start, count);
    const int row0 = (m - plan.first[e]) * S::BM;  // within the segment
    const int rows = min(count - row0, S::BM);
    const int n0 = n * ON;

    RowTile<S::BN, S::KB> wt_tile;
    RowTile<S::BM, S::KB> x_tile;
    const char* w_base = a.w + (int64_t)e * (GATED ? 2 : 1) * a.N * row_bytes;
    const char* x_base = a.x + (start + row0) * row_bytes;
    // rows and channels past the end repeat the last one; they are not stored
    const char* gate_base = w_base + n0 * row_bytes;
    const char* up_base = gate_base + (GATED ? (int64_t)a.N * row_bytes : 0);
    wt_tile.init([&](int r) -> uint32_t {
      const int in = r % (CT * MF);
      const int ch = (r / (CT * MF)) * (CH * MF) + in % (CH * MF);
      return (uint32_t)(min(ch, a.N - 1 - n0) * row_bytes);
    });
    x_tile.init([&](int r) -> uint32_t { return (uint32_t)(min(r, rows - 1) * row_bytes); });

    // FP8: scales of this wave's rows (column-major: a contraction group's
    // side by side) and of the weights' 128 x 128 blocks
    constexpr int kScaleBytes = Q == EP_QUANT_FP8_F32 ? 4 : 1;
    const char* xs = nullptr;
    int64_t xs_stride = 0;
    uint32_t xs_off[S::SLOADS];
    const char* ws = nullptr;
    uint32_t ws_off = 0;
    if (FP8) {
      const int G = a.C / 128;
      const int64_t group = a.seg.start ? a.x_cap : a.seg.block_rows;
      const int64_t first = a.seg.start ? start + row0 : (int64_t)e * G * group + row0;
      xs = (const char*)a.x_scales + first * kScaleBytes;
      xs_stride = group * kScaleBytes;
#pragma unroll
      for (int l = 0; l < S::SLOADS; ++l)
        xs_off[l] = min(wt * S::WROWS + l * kWave + lane, rows - 1) * kScaleBytes;
      const int blocks = (GATED ? 2 : 1) * a.N / 128;
      const int ch = min(n0 + wc * CH * MF, a.N - 1) / 128;
      ws = (const char*)(a.w_scales + ((int64_t)e * blocks + ch) * G);
      ws_off = GATED && lane % 2 ? (uint32_t)(a.N / 128) * G * 4 : 0;  // odd lanes: the ups'
    }

    constexpr int kPeriod = GATED ? CT * MF : 1 << 20;
    constexpr int kWPasses = wt_tile.kPasses, kPasses = kWPasses + x_tile.kPasses;
    auto load = [&](int k, lds_char* buf, int p) {
      const int64_t at = (int64_t)k * S::KB;
      if (p < kWPasses)
        wt_tile.template load<kPeriod>(p, gate_base + at, up_base + at, buf);
      else
        x_tile.template load<1 << 20>(p - kWPasses, x_base + at, nullptr, buf + wt_tile.kBytes);
      if (FP8 && p == kPasses - 1) {
#pragma unroll
        for (int l = 0; l < S::SLOADS; ++l)
          load_lds4<Q == EP_QUANT_FP8_UE8M0>(
              xs + k * xs_stride, xs_off[l],
              (const lds_char*)&lds_scales[k % S::STAGES][wave][l * kWave]);
        load_lds4<false>(ws + (int64_t)k * 4, ws_off,
                         (const lds_char*)&lds_scales[k % S::STAGES][wave][S::SLOADS * kWave]);
      }
    };
    auto tail = [&](int k, lds_char* buf) {
      const int64_t at = (int64_t)k * S::KB;
      const int left = (int)(row_bytes - at);
      wt_tile.template load_tail<kPeriod>(gate_base + at, up_base + at, left, buf);
      x_tile.template load_tail<1 << 20>(x_base + at, nullptr, left, buf + wt_tile.kBytes);
    };

    acc_t acc[CT][TT];
    clear<S>(acc);
    if constexpr (!FP8) {
      products<S>(wt_tile, x_tile, (lds_char*)&lds[0][0], nk, nfull, load, tail, acc);
    } else {
      constexpr int kLoads = wt_tile.kPasses + x_tile.kPasses + S::SLOADS + 1;
      barrier();  // the previous tile's reads
#pragma unroll
      for (int k = 0; k < S::STAGES; ++k)
        if (k < nk) {
#pragma unroll
          for (int p = 0; p < kPasses; ++p) load(k, (lds_char*)lds[k], p);
        }
      wait_stage<S::STAGES, kLoads>(0, nk);
      int buf = 0;
      for (int k = 0; k < nk; ++k) {
        const lds_char* wl = (lds_char*)lds[buf];
        const lds_char* xl = wl + wt_tile.kBytes;
        const float* scales = lds_scales[buf][wave];
        const float w0 = scales[S::SLOADS * kWave], w1 = scales[S::SLOADS * kWave + 1];
        float sx[TT];
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          const float s = scales[j * MF + lane % MF];
          sx[j] = Q == EP_QUANT_FP8_F32 ? s : __builtin_ldexpf(1.0f, __float_as_int(s) - 127);
        }
        i32x8 fb[TT][S::KK8];
#pragma unroll
        for (int j = 0; j < TT; ++j)
#pragma unroll
          for (int kk = 0; kk < S::KK8; ++kk)
            fb[j][kk] = fragment8<MF>(x_tile, xl, (wt * TT + j) * MF, kk);
#pragma unroll
        for (int i = 0; i < CT; ++i) {
          i32x8 fa[S::KK8];
#pragma unroll
          for (int kk = 0; kk < S::KK8; ++kk)
            fa[kk] = fragment8<MF>(wt_tile, wl, (wc * CT + i) * MF, kk);
          const float w = GATED && i >= CH ? w1 : w0;
#pragma unroll
          for (int j = 0; j < TT; ++j) {
            acc_t part;
#pragma unroll
            for (int q = 0; q < S::REGS; ++q) part[q] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < S::KK8; ++kk) part = Mfma<MF>::fp8(fa[kk], fb[j][kk], part);
            const float s = sx[j] * w;
#pragma unroll
            for (int q = 0; q < S::REGS; ++q)
              acc[i][j][q] = __builtin_fmaf(part[q], s, acc[i][j][q]);
          }
        }
        if (k + 1 < nk) {
          wait_stage<S::STAGES, kLoads>(k + 1, nk);
          if (k + S::STAGES < nk) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p) load(k + S::STAGES, (lds_char*)lds[buf], p);
          }
        }
        buf = buf + 1 == S::STAGES ? 0 : buf + 1;
      }
    }

    constexpr int kTurn = 4 * MF * Turned<S>::kRowBytes;
    constexpr int kRow = ON * 2 + 16;  // FP8 output: a row of the tile in bf16
    static_assert(kTurn + (FP8 && ON >= 128 ? S::BM * kRow : 0) <= sizeof(lds),
                  "the epilogue fits the tile buffers");
    lds_char* base = (lds_char*)&lds[0][0];
    const bool codes = FP8 && ON >= 128 && a.y_quant != EP_QUANT_NONE;
    const int64_t first = (start + row0) * a.N + n0;
    TileOut out;
    out.y = (uint16_t*)a.y + first;
    out.pre = a.pre ? a.pre + (GATED ? (start + row0) * 2 * a.N + n0 : first) : nullptr;
    out.residual = a.residual ? a.residual + first : nullptr;
    out.bias = a.bias ? a.bias + (int64_t)e * a.N + n0 : nullptr;
    turn_out<S, CH>(base, acc, [&](int r, int c, const Turned<S>& turned) {
      const int ch = wc * CH * MF + c;
      if (r < rows && n0 + ch < a.N) {
        const uint32_t at = (uint32_t)r * (uint32_t)a.N + ch;
        const u32x4 y = finish8<GATED>(a, out, at, r, ch, CH * MF, turned);
        if (codes)
          *(EP_LDS u32x4*)(base + kTurn + r * kRow + ch * 2) = y;
        else
          *(u32x4*)(out.y + at) = y;
      }
    });
    if (codes) {
      // eight lanes take 128 channels of a row: quantised as dispatch does
      // a bf16 row
      barrier();
      constexpr int kGroups = ON / 128;
      for (int at = threadIdx.x / 8; at < S::BM * kGroups; at += kGemmThreads / 8) {
        const int r = at / kGroups, g = at % kGroups, l = threadIdx.x % 8;
        const EP_LDS u32x4* from =
            (const EP_LDS u32x4*)(base + kTurn + r * kRow + g * 256 + l * 32);
        const u32x4 lo = from[0], hi = from[1];
        u32x4 out;
        float scale;
        uint32_t exponent;
        if (a.y_quant == EP_QUANT_FP8_F32)
          quantise_pair<EP_QUANT_FP8_F32>(lo, hi, out, scale, exponent);
        else
          quantise_pair<EP_QUANT_FP8_UE8M0>(lo, hi, out, scale, exponent);
        const int ch = n0 + g * 128;
        if (r < rows && ch < a.N) {
          const int64_t row = start + row0 + r;
          *(u32x4*)((char*)a.y + row * a.N + ch + l * 16) = out;
          const int64_t at_scale =
              a.seg.start ? (int64_t)(ch / 128) * a.y_cap + row
                          : ((int64_t)e * (a.N / 128) + ch / 128) * a.seg.block_rows + row0 + r;
          if (l == 0) {
            if (a.y_quant == EP_QUANT_FP8_F32) ((float*)a.y_scales)[at_scale] = scale;
            else ((uint8_t*)a.y_scales)[at_scale] = (uint8_t)exponent;
          }
        }
      }
    }
  }
}

template <class S, bool GATED, int Q>
static void launch(const ExpertArgs& a, int64_t rows, hipStream_t st) {
  const int on = GATED ? S::BN / 2 : S::BN;
  const int64_t tiles = ((rows + S::BM - 1) / S::BM + a.seg.E) * ((a.N + on - 1) / on);
  const int per_cu = S::kLds > 70 * 1024 ? 1 : 2;
  const int64_t most = (int64_t)kCus * per_cu;
  hipLaunchKernelGGL((expert_forward<S, GATED, Q>), dim3((unsigned)min(tiles, most)),
                     dim3(kGemmThreads), 0, st, a);
}

typedef Shape<32, 4, 4, 2, 2, 2> Big;     // 256 channels x 256 rows
typedef Shape<32, 4, 2, 2, 2, 3> Big8;    // 256 x 128 (FP8 sums are scaled in vector registers)
typedef Shape<32, 2, 2, 4, 1, 3> Medium;  // 256 x 64
typedef Shape<16, 2, 1, 4, 1, 3> Small;   // 128 x 16

template <bool GATED, int Q>
static void choose(const ExpertArgs& a, hipStream_t st) {
  typedef typename std::conditional<Q == EP_QUANT_NONE, Big, Big8>::type Large;
  const int64_t each = a.rows / a.seg.E;
  if (each > 96) launch<Large, GATED, Q>(a, a.rows, st);
  else if (each > 8 || a.y_quant != EP_QUANT_NONE) launch<Medium, GATED, Q>(a, a.rows, st);
  else launch<Small, GATED, Q>(a, a.rows, st);
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
