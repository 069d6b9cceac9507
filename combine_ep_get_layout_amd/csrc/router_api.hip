// C ABI of the router: argument validation and launches.  Declarations and
// semantics: include/ep.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/ep.h"
#include "ep_internal.hpp"
#include "router.hpp"

using ep::Geometry;

namespace {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int router_ok(const ep_router* r, const Geometry& g) {
  if (!r) return EP_ERR_NULL;
  if (r->reserved != 0) return EP_ERR_SHAPE;
  if (r->score != EP_SCORE_SOFTMAX && r->score != EP_SCORE_SIGMOID) return EP_ERR_MODE;
  if ((r->normalize != 0 && r->normalize != 1) || (r->bf16 != 0 && r->bf16 != 1))
    return EP_ERR_MODE;
  if (!isfinite(r->scale)) return EP_ERR_SHAPE;
  if (r->groups < 1 || r->groups > 64 || g.E % r->groups != 0) return EP_ERR_SHAPE;
  if (r->groups_kept < 1 || r->groups_kept > r->groups) return EP_ERR_SHAPE;
  if (r->group_top < 1 || r->group_top > 2 || r->group_top > g.E / r->groups) return EP_ERR_SHAPE;
  return EP_OK;
}

}  // namespace

extern "C" {

int ep_route(const ep_problem* p, const ep_router* r, const void* logits, const float* bias,
             int32_t* topk_idx, float* topk_weights, int32_t* err, void* stream) {
  Geometry g;
  int st = ep::make_geometry(p, &g);
  if (st == EP_OK) st = router_ok(r, g);
  if (st != EP_OK) return st;
  if ((int64_t)g.R * g.T > 0 && (!logits || !topk_idx || !topk_weights)) return EP_ERR_NULL;
  if (!aligned(logits, 16) || !aligned(bias, 16) || !aligned(topk_idx, 4) ||
      !aligned(topk_weights, 4) || !aligned(err, 4))
    return EP_ERR_ALIGN;
  ep::RouteArgs a;
  memset(&a, 0, sizeof(a));
  a.tokens = (int64_t)g.R * g.T;
  a.E = g.E;
  a.K = g.K;
  a.bf16 = r->bf16;
  a.sigmoid = r->score == EP_SCORE_SIGMOID;
  a.normalize = r->normalize;
  a.groups = r->groups;
  a.groups_kept = r->groups_kept;
  a.group_top = r->group_top;
  a.group_size = g.E / r->groups;
  a.scored = bias || (a.groups_kept < a.groups && a.group_top > 1);
  a.scale = r->scale;
  a.logits = logits;
  a.bias = bias;
  a.idx = topk_idx;
  a.weights = topk_weights;
  a.err = err;
  if (ep::launch_route(a, (hipStream_t)stream) != hipSuccess) return EP_ERR_HIP;
  return EP_OK;
}

int ep_route_backward(const ep_problem* p, const ep_router* r, const void* logits,
                      const int32_t* topk_idx, const float* dweights, void* dlogits,
                      int32_t* err, void* stream) {
  Geometry g;
  int st = ep::make_geometry(p, &g);
  if (st == EP_OK) st = router_ok(r, g);
  if (st != EP_OK) return st;
  if ((int64_t)g.R * g.T > 0 && (!logits || !topk_idx || !dweights || !dlogits))
    return EP_ERR_NULL;
  if (!aligned(logits, 16) || !aligned(dlogits, 16) || !aligned(topk_idx, 4) ||
      !aligned(dweights, 4) || !aligned(err, 4))
    return EP_ERR_ALIGN;
  ep::RouteGradArgs a;
  memset(&a, 0, sizeof(a));
  a.tokens = (int64_t)g.R * g.T;
  a.E = g.E;
  a.K = g.K;
  a.bf16 = r->bf16;
  a.sigmoid = r->score == EP_SCORE_SIGMOID;
  a.normalize = r->normalize;
  a.scale = r->scale;
  a.logits = logits;
  a.idx = topk_idx;
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.err = err;
  if (ep::launch_route_grad(a, (hipStream_t)stream) != hipSuccess) return EP_ERR_HIP;
  return EP_OK;
}

}  // extern "C"
