// Arguments of the layer for a few tokens.
#pragma once

#include "ep_device.hpp"
#include "layer_choice.hpp"

namespace ep {

constexpr int kLayerEntries = EP_LAYER_MAX_ENTRIES;

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
