// Arguments of the layer for a few tokens.
#pragma once

#include <algorithm>

#include "ep_device.hpp"

namespace ep {

constexpr int kLayerEntries = EP_LAYER_MAX_ENTRIES;
constexpr int kLayerPlaces = 256;  // entries' results that a workgroup of layer_down has in LDS

// Workgroups' tiles of 64 entries of an expert by 64 channels of h that a layer has about
inline int64_t layer_tiles(int64_t entries, int experts, int inner) {
  int64_t chunks = entries / 64 > experts ? entries / 64 : experts;
  if (chunks > entries) chunks = entries;
  return chunks * ((inner + 63) / 64);
}

// Whether workgroups share rows, and entries' results go through the workspace: not with an
// entry an expert or fewer, nor with so few tiles that the weights are not read at full speed
// (16 entries of one expert, bf16 4096 -> 4096: 31 us, with shared rows 62).
inline bool layer_many(int64_t entries, int experts, int inner) {
  if (entries > kLayerPlaces || entries > 64 * (int64_t)experts) return true;
  return entries > experts && layer_tiles(entries, experts, inner) >= 128;
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
