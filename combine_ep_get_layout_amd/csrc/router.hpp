// Arguments of the router's kernels.
#pragma once

#include "ep_device.hpp"

namespace ep {

struct RouteArgs {
  int64_t tokens;
  int E, K;
  bool bf16, sigmoid, normalize;
  bool scored;             // choices are scores (with a bias, or summed over a group)
  int groups, groups_kept, group_top, group_size;
  int per;                 // experts a lane (set by launch_route)
  float scale;
  const void* logits;      // [tokens][E]
  const float* bias;       // [E] or NULL
  int32_t* idx;            // [tokens][K]
  float* weights;          // [tokens][K]
  int32_t* err;
};

hipError_t launch_route(const RouteArgs& a, hipStream_t stream);

struct RouteGradArgs {
  int64_t tokens;
  int E, K;
  bool bf16, sigmoid, normalize;
  float scale;
  const void* logits;      // [tokens][E]
  const int32_t* idx;      // [tokens][K]
  const float* dweights;   // [tokens][K]
  void* dlogits;           // [tokens][E]
  int32_t* err;
};

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t stream);

}  // namespace ep
