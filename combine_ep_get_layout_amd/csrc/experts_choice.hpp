// Which tile shape a call of the experts' products is launched with, from its sizes
// alone.  Host code without HIP, so that a host compiler can build it by itself.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace ep {

constexpr int kMaxExperts = 2048;
constexpr int kCus = 256;        // compute units of an MI355X
constexpr int kGemmThreads = 256;
constexpr int kWavefront = 64;

// A workgroup's tile: WC x WT x WK waves, each CT x TT matrix-core tiles of MF
// channels x MF rows; STAGES buffers of KB bytes along the contraction, of which WK
// waves take a part each.
template <int MF_, int CT_, int TT_, int WC_, int WT_, int STAGES_, int KB_ = 128, int WK_ = 1>
struct Dims {
  static constexpr int KB = KB_, KR = KB / 2;
  static constexpr int MF = MF_, CT = CT_, TT = TT_, WC = WC_, WT = WT_, WK = WK_;
  static constexpr int STAGES = STAGES_;
  static constexpr int BN = WC * CT * MF, BM = WT * TT * MF;
  static constexpr int KK = KR * MF / 512 / WK;     // bf16 matrix-core steps of a wave's stage
  static constexpr int GS = KB / 128 / WK;          // FP8 scale groups of a wave's stage
  static constexpr int KK8 = KB * MF / 2048 / WK;   // FP8 steps
  static constexpr int kSlotBytes = (BN + BM) * KB;  // a stage in LDS
  static constexpr int kLds = STAGES * kSlotBytes;
  static constexpr int REGS = MF * MF / kWavefront;
  static constexpr int WROWS = TT * MF;    // rows of a wave's tile
  static constexpr int SLOADS = (WROWS + kWavefront - 1) / kWavefront;  // FP8 scale loads of a group
  static constexpr int kScaleFloats = (GS * SLOADS + 1) * kWavefront;   // of a wave and stage
  // the epilogue's turn: a row of a wave's channels as two halves, four waves' rows
  static constexpr int kHalfBytes = CT * MF * 2;
  static constexpr int kTurnRowBytes = 2 * kHalfBytes + 16;
  static constexpr int kTurnBytes = 4 * MF * kTurnRowBytes;
  // whether the next tile's loads run through the epilogue: it fits one stage's buffer
  static constexpr bool kChains = STAGES > 2 && kTurnBytes <= kSlotBytes;
  static_assert(WC * WT * WK * kWavefront == kGemmThreads, "four wavefronts");
};

// Row tiles of `step` rows that the segments are expected to make.  The counts
// are on the device: an expert that is hit has the mean number of rows and, unless
// it has all of them, half a tile more.
inline double row_tiles(int experts, int64_t rows, int step) {
  const double hit = (double)std::min<int64_t>(rows, experts);
  if (hit <= 1.0) return (double)((rows + step - 1) / step);
  return hit * std::max(1.0, (double)rows / hit / step + 0.5);
}

// Relative time of tile D: whole rounds of its workgroups (`slots` of them on the
// chip) over a product of `channels` results a row and `bytes` of contraction.
// stage, tile: the time of one of its stages, and of a tile's start and end.
template <class D>
inline double shape_time(int experts, int64_t rows, int64_t channels, int64_t bytes, int slots,
                         double stage, double tile) {
  const double tiles =
      row_tiles(experts, rows, D::BM) * (double)((channels + D::BN - 1) / D::BN);
  return std::ceil(tiles / slots) * ((double)((bytes + D::KB - 1) / D::KB) * stage + tile);
}

// ---- forward products ----------------------------------------------------------

// Large tiles read the LDS least per product; narrow ones waste no products on rows
// that are not there, and with many of them few rows still fill the chip.
typedef Dims<32, 4, 4, 2, 2, 2> BigDims;     // 256 channels x 256 rows
typedef Dims<32, 4, 2, 2, 2, 3> Big8Dims;    // 256 x 128 (FP8 sums are scaled in vector registers)
typedef Dims<32, 2, 2, 4, 1, 3> MediumDims;  // 256 x 64
typedef Dims<32, 2, 1, 2, 2, 3> NarrowDims;  // 128 x 64, in bf16 two workgroups on a compute unit
typedef Dims<16, 2, 1, 4, 1, 3> SmallDims;   // 128 x 16
typedef Dims<16, 2, 1, 1, 1, 3, 512, 4> TinyDims;  // 32 x 16, the waves share the contraction

enum ForwardShape { kLargeTile, kMediumTile, kNarrowTile, kSmallTile, kTinyTile };

// Workgroups of a shape on the chip: by LDS, two a compute unit or one.  Narrow and Tiny
// take exactly 80 KiB with the tile plan; in FP8 their scales take 6 KiB more, so one.
template <class D, bool FP8>
constexpr int forward_slots() {
  const int lds = D::kLds + kMaxExperts * (int)sizeof(int) +
                  (FP8 ? D::STAGES * 4 * D::kScaleFloats * (int)sizeof(float) : 0);
  return lds <= 80 * 1024 ? 2 * kCus : kCus;
}

// The shape with the least expected time, in units of a stage of Medium; the
// stages' times are fitted to measurements of every shape at 1 to 128 experts, 1 to
// 2,048 rows each (random routing), 648 to 8192 channels.  Narrow is for tiles
// that all run at once.  The choice is 3% off the best shape on average and 35% at
// worst (FP8 2% and 48%); by rows per expert alone it was 24% off, and 4.9 times
// at worst (FP8 21%, 4.0 times).  us, bf16, Big / Medium / Narrow / Small / Tiny:
//   1 expert, 2048 x 2048, 8 rows:       42 /  20 /  14 /   12 /    7
//   1 expert, 4096 x 8192, 192 rows:     77 /  38 /  28 /   61 /   60
//   8 experts, 5584 x 1560, 96 rows:    122 /  70 /  48 /  115 /   71
//   64 experts, 4096 x 4096, 64 rows:   554 / 444 / 483 /  829 /  882
//   64 experts, 4096 x 4096, 192 rows:  612 / 762 / 875 / 1900 / 2196
// A result in FP8 needs its groups of 128 channels whole in a tile, which the two largest
// shapes have for gated products and others alike; the smaller ones are not used for it
// (64 experts x 4 tokens, top-8, 2048 x 2048: bf16 result 23 us, FP8 32).
// `wide` channels of C are computed from each row: N, gated 2 N.
template <bool FP8>
ForwardShape choose_forward(int experts, int64_t rows, int C, int64_t wide, bool fp8_result) {
  typedef typename std::conditional<FP8, Big8Dims, BigDims>::type Large;
  const int64_t bytes = (int64_t)C * (FP8 ? 1 : 2);
#define EP_TIME(D, stage, tile) \
  shape_time<D>(experts, rows, wide, bytes, forward_slots<D, FP8>(), stage, tile)
  const double large = EP_TIME(Large, FP8 ? 1.55 : 2.0, FP8 ? 0.0 : 1.0);
  const double medium = EP_TIME(MediumDims, 1.0, FP8 ? 0.3 : 0.0);
  const double small = EP_TIME(SmallDims, FP8 ? 0.9 : 0.95, 0.0);
  const double tiny = EP_TIME(TinyDims, FP8 ? 0.4 : 1.1, FP8 ? 3.5 : 1.5);
  const double tiles = row_tiles(experts, rows, NarrowDims::BM) *
                       (double)((wide + NarrowDims::BN - 1) / NarrowDims::BN);
  const double narrow = tiles > forward_slots<NarrowDims, FP8>()
                            ? HUGE_VAL
                            : EP_TIME(NarrowDims, FP8 ? 0.78 : 0.8, FP8 ? 2.0 : 0.0);
#undef EP_TIME
  if (!fp8_result && tiny < std::min({large, medium, narrow, small})) return kTinyTile;
  if (!fp8_result && small < std::min({large, medium, narrow})) return kSmallTile;
  if (!fp8_result && narrow < std::min(large, medium)) return kNarrowTile;
  return medium < large ? kMediumTile : kLargeTile;
}

// ---- gradients -------------------------------------------------------------------

namespace grad {

typedef Dims<32, 4, 4, 2, 2, 2> Big;     // 256 channels x 256 rows
typedef Dims<32, 2, 2, 4, 1, 3> Medium;  // 256 x 64
typedef Dims<16, 2, 1, 4, 1, 3> Small;   // 128 x 16
typedef Dims<32, 2, 2, 2, 2, 3> Square;  // 128 x 128, one on a compute unit
typedef Dims<32, 2, 2, 2, 2, 4, 64> Pair;  // the same in 64 KiB, two on one

}  // namespace grad

enum DxShape { kDxBig, kDxMedium, kDxSmall };
enum DwShape { kDwBig, kDwSquare, kDwPair };

template <class D>
constexpr int dx_slots() { return D::kLds > 70 * 1024 ? kCus : 2 * kCus; }

// rows of `O` channels to C channels
inline DxShape choose_dx(int experts, int64_t rows, int C, int O) {
  // as in the forward products, in units of a stage of Medium: 1% off the best
  // shape on average over the same sizes, 18% by rows per expert alone.  us, Big
  // / Medium / Small: 1 expert, 2048 x 2048, 512 rows 41 / 20 / 20; 64 experts,
  // 2048 x 2048, 64 rows 139 / 106 / 215, 512 rows 282 / 432 / 1378.
  const auto time = [&](auto dims, double stage, double tile) {
    typedef decltype(dims) D;
    return shape_time<D>(experts, rows, C, (int64_t)O * 2, dx_slots<D>(), stage, tile);
  };
  const double big = time(grad::Big(), 2.0, 1.0), medium = time(grad::Medium(), 1.0, 0.0);
  const double small = time(grad::Small(), 0.95, 0.0);
  if (small < std::min(big, medium)) return kDxSmall;
  return medium < big ? kDxMedium : kDxBig;
}

// C x O channels of every expert
inline DwShape choose_dw(int experts, int C, int O) {
  // The largest tiles that fill the chip; of the smaller ones two on a compute unit
  // where there are more of them than compute units.  us, Square / Pair: 8 experts of
  // 1024 x 1024 (512 tiles), 16 rows 12.1 / 8.4, 512 rows 16.3 / 14.6; 1 expert of
  // 2048 x 2048 (256 tiles), 16 rows 5.7 / 5.4, 8,192 rows 74 / 87.  8 experts of 4096 x
  // 4096, Big / Square: 64 rows 76 / 118, 2,048 rows 470 / 749; 1 of 2048 x 2048 (64 of
  // Big's tiles): 12 / 6 and 60 / 22.
  const auto tiles = [&](int side) {
    return (int64_t)experts * ((C + side - 1) / side) * ((O + side - 1) / side);
  };
  if (tiles(grad::Big::BN) >= kCus) return kDwBig;
  return tiles(grad::Square::BN) <= kCus ? kDwSquare : kDwPair;
}

// Channels of a workgroup of the bias gradient, N channels in all.
inline int choose_dbias(int experts, int64_t rows, int N) {
  // Channels of a workgroup, so that there are enough of them and each has a few
  // rows a thread.  us, 32 / 64 / 256 channels: 1 expert x 8,192 rows x 4096 channels
  // 67 / 123 / 479; 4 x 2,048 x 4096 52 / 38 / 128; 64 x 4 x 4096 48 / 22 / 7.
  const int64_t groups = (int64_t)experts * ((N + 63) / 64);
  if (groups <= kCus / 2) return 32;
  return groups >= 4 * kCus && rows <= (int64_t)experts * 128 ? 256 : 64;
}

}  // namespace ep
