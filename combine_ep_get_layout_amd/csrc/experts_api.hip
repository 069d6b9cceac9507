// C ABI of the experts' products and of combine's gradient: argument
// validation and launches.  Declarations and semantics: include/ep.h.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/ep.h"
#include "ep_internal.hpp"

using ep::Geometry;
using ep::Segments;

namespace {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline bool channels_ok(int n) { return n >= 8 && n % 8 == 0 && n <= 32768; }

// The segments of a problem's layout, over at most cap rows.
int segments(const ep_problem* p, const Geometry& g, const ep_layout* layout, Segments* s) {
  if (p->mode == EP_MODE_RANK_MAJOR) return EP_ERR_MODE;
  const bool normal = p->mode == EP_MODE_NORMAL;
  // messages are unpacked into the low-latency layout
  const int64_t blocks = (int64_t)g.E * g.R * g.T;
  if (!normal && blocks >= (1ll << 31)) return EP_ERR_SHAPE;
  if (!layout || !layout->err || !layout->recv_tokens_per_expert ||
      (normal && !layout->expert_start))
    return EP_ERR_NULL;
  if (!aligned(layout->err, 4) || !aligned(layout->recv_tokens_per_expert, 4) ||
      (normal && !aligned(layout->expert_start, 4)))
    return EP_ERR_ALIGN;
  s->start = normal ? layout->expert_start : nullptr;
  s->count = layout->recv_tokens_per_expert;
  s->block_rows = (int64_t)g.R * g.T;
  s->cap = (1ll << 31) - 1;
  s->E = g.E;
  s->err = layout->err;
  return EP_OK;
}

// Checks a row buffer of `channels` channels and narrows the segments' cap to it.
int rows_ok(const ep_rows* r, int channels, const Geometry& g, bool fp8_allowed, Segments* s) {
  if (!r) return EP_ERR_NULL;
  if (r->channels != channels) return EP_ERR_SHAPE;
  if (r->quant < EP_QUANT_NONE || r->quant > EP_QUANT_FP8_UE8M0) return EP_ERR_MODE;
  if (r->quant != EP_QUANT_NONE && !fp8_allowed) return EP_ERR_MODE;
  if (r->quant != EP_QUANT_NONE && channels % 128 != 0) return EP_ERR_SHAPE;
  if (r->capacity < 0 || (!s->start && r->capacity < (int64_t)g.E * s->block_rows))
    return EP_ERR_CAPACITY;
  // no rows at all, no buffer needed
  if (r->capacity > 0 && (int64_t)g.R * g.T > 0) {
    if (!r->x || (r->quant != EP_QUANT_NONE && !r->scales)) return EP_ERR_NULL;
  }
  if (!aligned(r->x, 16)) return EP_ERR_ALIGN;
  if (r->quant == EP_QUANT_FP8_F32 && !aligned(r->scales, 4)) return EP_ERR_ALIGN;
  if (r->capacity < s->cap) s->cap = r->capacity;
  return EP_OK;
}

int weights_ok(const ep_weights* w) {
  if (!w) return EP_ERR_NULL;
  if (w->reserved != 0) return EP_ERR_SHAPE;
  if (w->fp8 != 0 && w->fp8 != 1) return EP_ERR_MODE;
  return EP_OK;
}

int act_ok(int act) {
  return act < EP_ACT_NONE || act > EP_ACT_GELU ? EP_ERR_MODE : EP_OK;
}

#define EP_TRY(call)                  \
  do {                                \
    const int st_ = (call);           \
    if (st_ != EP_OK) return st_;     \
  } while (0)

int forward(const ep_problem* p, const ep_layout* layout, const ep_rows* x, const ep_weights* w,
            int32_t act, const ep_rows* residual, const ep_rows* y, const ep_rows* pre,
            bool gated, void* stream) {
  Geometry g;
  EP_TRY(ep::make_geometry(p, &g));
  ep::ExpertArgs a;
  memset(&a, 0, sizeof(a));
  EP_TRY(segments(p, g, layout, &a.seg));
  EP_TRY(act_ok(act));
  EP_TRY(weights_ok(w));
  if (gated && w->out_channels % 2 != 0) return EP_ERR_SHAPE;
  const int C = w->in_channels, O = w->out_channels, N = gated ? O / 2 : O;
  if (!channels_ok(C) || !channels_ok(N)) return EP_ERR_SHAPE;
  if (gated && w->bias) return EP_ERR_MODE;
  EP_TRY(rows_ok(x, C, g, true, &a.seg));
  const bool fp8 = x->quant != EP_QUANT_NONE;
  if (fp8 != (w->fp8 != 0)) return EP_ERR_MODE;
  if (fp8 && (C % 128 != 0 || N % 128 != 0)) return EP_ERR_SHAPE;
  if (!w->w || (fp8 && !w->scales)) return EP_ERR_NULL;
  if (!aligned(w->w, 16) || (fp8 && !aligned(w->scales, 4)) || !aligned(w->bias, 16))
    return EP_ERR_ALIGN;
  EP_TRY(rows_ok(y, N, g, fp8, &a.seg));
  if (residual) EP_TRY(rows_ok(residual, N, g, false, &a.seg));
  if (pre) EP_TRY(rows_ok(pre, O, g, false, &a.seg));
  a.rows = (int64_t)g.R * g.T * g.K;
  a.gated = gated;
  a.quant = x->quant;
  a.act = act;
  a.C = C;
  a.N = N;
  a.x = (const char*)x->x;
  a.x_scales = x->scales;
  a.x_cap = x->capacity;
  a.w = (const char*)w->w;
  a.w_scales = w->scales;
  a.bias = w->bias;
  a.residual = residual ? (const uint16_t*)residual->x : nullptr;
  a.pre = pre ? (uint16_t*)pre->x : nullptr;
  a.y = y->x;
  a.y_scales = y->scales;
  a.y_cap = y->capacity;
  a.y_quant = y->quant;
  if (ep::launch_expert_forward(a, (hipStream_t)stream) != hipSuccess) return EP_ERR_HIP;
  return EP_OK;
}

int backward(const ep_problem* p, const ep_layout* layout, const ep_rows* x, const ep_weights* w,
             int32_t act, const ep_rows* pre, const ep_rows* dy, const ep_rows* dpre,
             const ep_rows* dx, uint16_t* dw, float* dbias, bool gated, void* stream) {
  Geometry g;
  EP_TRY(ep::make_geometry(p, &g));
  ep::GradArgs a;
  memset(&a, 0, sizeof(a));
  EP_TRY(segments(p, g, layout, &a.seg));
  EP_TRY(act_ok(act));
  EP_TRY(weights_ok(w));
  if (w->fp8) return EP_ERR_MODE;  // gradients in bf16
  if (gated && w->out_channels % 2 != 0) return EP_ERR_SHAPE;
  const int C = w->in_channels, O = w->out_channels, N = gated ? O / 2 : O;
  if (!channels_ok(C) || !channels_ok(N)) return EP_ERR_SHAPE;
  EP_TRY(rows_ok(dy, N, g, false, &a.seg));
  const bool same = !gated && act == EP_ACT_NONE;  // dpre is dy
  if (!same) {
    EP_TRY(rows_ok(pre, O, g, false, &a.seg));
    if (dx || dw || dpre || gated) EP_TRY(rows_ok(dpre, O, g, false, &a.seg));
  }
  if (dx) {
    EP_TRY(rows_ok(dx, C, g, false, &a.seg));
    if (!w->w) return EP_ERR_NULL;
    if (!aligned(w->w, 16)) return EP_ERR_ALIGN;
  }
  if (dw) {
    EP_TRY(rows_ok(x, C, g, false, &a.seg));
    if (!aligned(dw, 16)) return EP_ERR_ALIGN;
  }
  if (!aligned(dbias, 4)) return EP_ERR_ALIGN;
  a.rows = (int64_t)g.R * g.T * g.K;
  a.gated = gated;
  a.act = act;
  a.C = C;
  a.N = N;
  a.O = O;
  a.x = dw ? (const uint16_t*)x->x : nullptr;
  a.w = (const uint16_t*)w->w;
  a.pre = same ? nullptr : (const uint16_t*)pre->x;
  a.dy = (const uint16_t*)dy->x;
  a.dz_out = same || !dpre ? nullptr : (uint16_t*)dpre->x;
  a.dz = same ? a.dy : a.dz_out;
  a.dx = dx ? (uint16_t*)dx->x : nullptr;
  a.dw = dw;
  a.dbias = dbias;
  if (ep::launch_expert_grad(a, (hipStream_t)stream) != hipSuccess) return EP_ERR_HIP;
  return EP_OK;
}

}  // namespace

extern "C" {

int ep_expert_gated(const ep_problem* p, const ep_layout* layout, const ep_rows* x,
                    const ep_weights* w, int32_t act, const ep_rows* h, const ep_rows* pre,
                    void* stream) {
  return forward(p, layout, x, w, act, nullptr, h, pre, true, stream);
}

int ep_expert_linear(const ep_problem* p, const ep_layout* layout, const ep_rows* x,
                     const ep_weights* w, int32_t act, const ep_rows* residual,
                     const ep_rows* y, const ep_rows* pre, void* stream) {
  return forward(p, layout, x, w, act, residual, y, pre, false, stream);
}

int ep_expert_gated_backward(const ep_problem* p, const ep_layout* layout, const ep_rows* x,
                             const ep_weights* w, int32_t act, const ep_rows* pre,
                             const ep_rows* dh, const ep_rows* dpre, const ep_rows* dx,
                             uint16_t* dw, void* stream) {
  return backward(p, layout, x, w, act, pre, dh, dpre, dx, dw, nullptr, true, stream);
}

int ep_expert_linear_backward(const ep_problem* p, const ep_layout* layout, const ep_rows* x,
                              const ep_weights* w, int32_t act, const ep_rows* pre,
                              const ep_rows* dy, const ep_rows* dpre, const ep_rows* dx,
                              uint16_t* dw, float* dbias, void* stream) {
  return backward(p, layout, x, w, act, pre, dy, dpre, dx, dw, dbias, false, stream);
}

int ep_combine_backward(const ep_problem* p, const ep_layout* layout, const uint16_t* dout,
                        const float* topk_weights, const uint16_t* y, int64_t y_rows,
                        uint16_t* dy, float* dweights, void* stream) {
  Geometry g;
  EP_TRY(ep::make_geometry(p, &g));
  if (p->mode == EP_MODE_MESSAGES) return EP_ERR_MODE;
  const bool rank_major = p->mode == EP_MODE_RANK_MAJOR;
  if (rank_major && dweights) return EP_ERR_MODE;  // the sum has no weights
  const bool toks = (int64_t)g.R * g.T > 0;
  if (!layout || !layout->err) return EP_ERR_NULL;
  if (toks && (!layout->send_pos || !dout)) return EP_ERR_NULL;
  if (toks && dy && !rank_major && !topk_weights) return EP_ERR_NULL;
  if (toks && dweights && !y && y_rows > 0) return EP_ERR_NULL;
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(topk_weights, 4) ||
      !aligned(dweights, 4) || !aligned(layout->send_pos, 4) || !aligned(layout->err, 4))
    return EP_ERR_ALIGN;
  if (y_rows < 0) return EP_ERR_CAPACITY;
  ep::CombineGradArgs a;
  a.g = g;
  a.rank_major = rank_major;
  a.dout = dout;
  a.y = y;
  a.w = topk_weights;
  a.send_pos = layout->send_pos;
  a.rows = y_rows;
  a.dy = dy;
  a.dw = dweights;
  a.err = layout->err;
  if (ep::launch_combine_grad(a, (hipStream_t)stream) != hipSuccess) return EP_ERR_HIP;
  return EP_OK;
}

}  // extern "C"
