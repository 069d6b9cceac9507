// Arguments of the layer for a few tokens.
#pragma once

#include <algorithm>

#include "ep_device.hpp"

namespace ep {

constexpr int kLayerEntries = EP_LAYER_MAX_ENTRIES;
constexpr int kLayerPlaces = 256;  // entries' results that a workgroup of layer_down has in LDS

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

struct LayerArgs {
  int tokens, K, entries, E;
  int H, I;                // channels of x and out; of h
  int kind, act;           // EP_WEIGHTS_*, EP_ACT_*
  const uint16_t* x;       // [tokens][H]
  const int32_t* idx;      // [tokens][K]
  const float* weights;    // [tokens][K]
  const char* w13;         // [E][2 I][H]
  const float* s13;
  const char* w2;          // [E][H][I]
  const float* s2;
  uint16_t* h;             // workspace: [entries][2][I], h rounded and the rest of it
  float* y;                // and where layer_many holds, [entries][H up to 16]
  uint16_t* out;           // [tokens][H]
  int32_t* err;
};

hipError_t launch_layer(const LayerArgs& a, hipStream_t stream);

}  // namespace ep
