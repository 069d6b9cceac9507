// Which kernels the layer for a few tokens is launched with, from its sizes alone.  Host code
// without HIP, so that a host compiler can build it by itself.
#pragma once

#include "experts_choice.hpp"

namespace ep {

constexpr int kLayerPlaces = 256;  // entries' results that a workgroup of layer_down has in LDS
constexpr int kUpWaves = 4;        // waves of a workgroup of layer_gated
constexpr int kUpRoom = 3 * kCus;  // its workgroups that are on the chip at once

// Workgroups' tiles of 64 rows of an expert by `each` channels that a product has about
inline int64_t layer_tiles(int64_t rows, int experts, int channels, int each) {
  const int64_t chunks = std::max<int64_t>(rows / 64, std::min<int64_t>(experts, rows));
  return chunks * ((channels + each - 1) / each);
}

// Whether workgroups share rows, and entries' results go through the workspace: not with few
// entries, nor with so few tiles that the weights are not read at full speed.  us with shared
// rows / without: 16 entries of one expert (bf16 4096 -> 4096, 64 tiles) 62 / 31, 48 of 4 (FP8
// 3968 -> 1024, 64 tiles) 38 / 21, 128 of 4 (bf16 4096 -> 1408, 88 tiles) 58 / 68; with more
// tiles 16 entries over 32 experts (bf16 3264 -> 1576) 96 / 73, 40 over 143 (FP8 256 -> 2816)
// 39 / 74.
inline bool layer_many(int64_t entries, int experts, int inner) {
  if (entries > kLayerPlaces || entries > 64 * (int64_t)experts) return true;
  const int64_t tiles = layer_tiles(entries, experts, inner, 64);
  return (entries > 64 && tiles >= 48) ||
         (entries > std::min<int64_t>(experts, 24) && tiles >= 128);
}

// ---- waves with their own rows ----------------------------------------------------

// Strips of eight channels that the gated block has about
inline int64_t layer_strips(int64_t entries, int experts, int inner) {
  return std::min<int64_t>(experts, entries) * ((inner + 7) / 8);
}

enum LayerGated {
  kGatedFew,       // slots of 4 entries, in bf16 8, a strip a wave
  kGatedFewSplit,  // the same, but a strip's lines dealt to four waves
  kGatedSome,      // slots of 16, dealt likewise
  kGatedMost,      // of 32, in bf16 64, likewise
};

// How many entries a slot has room for goes by how many an expert has on average: a wave reads
// its weights once for each slot full of them, and multiplies the whole slot.  (bytes: weights
// of 8 bits.)  us of the layer, few / some / most: in bf16 24 entries of 8 experts (4096 -> 896)
// 41 / 41 / 50, 64 of them 53 / 45 / 53, 64 of 4 (4096 -> 1408) 71 / 58 / 58, of 2 60 / 43 / 34;
// in 8-bit integers 16, 24 and 64 of 8 (4096 -> 896) 26 / 26 / 36, 34 / 28 / 38 and 50 / 33 / 41,
// 64 of 4 (4096 -> 1408) 75 / 52 / 49, of 2 81 / 41 / 35; FP8 as the integers, a tenth less.
inline LayerGated choose_layer_gated(bool bytes, int64_t entries, int experts, int inner) {
  const int64_t hit = std::min<int64_t>(experts, entries);
  if (entries <= hit * (bytes ? 2 : 6))
    return layer_strips(entries, experts, inner) < kUpRoom * kUpWaves ? kGatedFewSplit : kGatedFew;
  return entries <= 16 * hit ? kGatedSome : kGatedMost;
}

enum LayerDown { kDown4, kDown8, kDown16, kDown32 };  // entries of a slot

// us of the layer, slots of 4 / 8 / 16 / 32 (4096 -> 896): in bf16 12, 16, 40 and 64 entries of 8
// experts 32 / 32 / 35 / 39, 36 / 34 / 37 / 41, 46 / 41 / 43 / 49 and 53 / 46 / 45 / 50, 64 of 4
// (4096 -> 1408) 72 / 59 / 61 / 58; in 8-bit integers, up to 16, 12, 16, 40 and 64 of 8
// 24 / 24 / 27, 26 / 25 / 28, 32 / 29 / 32 and 37 / 33 / 33, 64 of 2 (4096 -> 1408) 47 / 37 / 35.
inline LayerDown choose_layer_down(bool bytes, int64_t entries, int experts) {
  const int64_t hit = std::min<int64_t>(experts, entries);
  if (entries < 2 * hit) return kDown4;
  if (entries <= 5 * hit) return kDown8;
  return bytes || entries <= 12 * hit ? kDown16 : kDown32;
}

// ---- rows in common ------------------------------------------------------------------

enum LayerMany {
  kManyFew1,       // tiles of 16 rows (32 in bf16), one strip a wave
  kManyFew2,       // two strips a wave
  kManyRows1,      // of 64 rows, one strip, weights through the caches
  kManyRows2Once,  // two strips, weights past the caches
  kManyRows2,      // through them
};

// us of the layer with tiles of 16 rows (32 in bf16) / of 64: 256 experts with 2 entries in
// FP8 (7168 -> 2048) 1480 / 1875, 128 with 4 in bf16 (2048 -> 768) 200 / 227, 32 with 12 in FP8
// (4096 -> 1408) 144 / 132.  One strip a wave / two, where there are few tiles: 256 entries of
// one expert (bf16 4096 -> 1408) 53 / 59, 24 of 8 (bf16 2280 -> 2952) 89 / 124.  Weights past
// the caches / through them: 16 experts with 16 / 64 entries (bf16 4096 -> 1408) 119 / 128 and
// 211 / 200.
// channels: of the result, for the gated block I and 64 a workgroup, else H and 128 (with two
// rows an entry).
inline LayerMany choose_layer_many(bool gated, int64_t entries, int experts, int channels) {
  const int64_t tiles = gated ? layer_tiles(entries, experts, channels, 64)
                              : layer_tiles(2 * entries, experts, channels, 128);
  if (entries <= 8 * (int64_t)experts) return tiles < 2 * kCus ? kManyFew1 : kManyFew2;
  if (tiles < kCus) return kManyRows1;
  return entries <= 32 * (int64_t)experts ? kManyRows2Once : kManyRows2;
}

}  // namespace ep
