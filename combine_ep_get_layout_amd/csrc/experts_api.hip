// C ABI of the experts' products, of combine's gradient and of the layer for a few
// tokens: argument validation and launches.  Declarations and semantics: include/ep.h.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/ep.h"
#include "ep_internal.hpp"
#include "layer.hpp"

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

inline bool is_fp8(int quant) { return quant == EP_QUANT_FP8_F32 || quant == EP_QUANT_FP8_UE8M0; }

// What a row buffer may hold, beside bf16.
enum { kBf16Rows = 0, kFp8Rows = 1, kInt8Rows = 2 };

// Checks a row buffer of `channels` channels and narrows the segments' cap to it.
int rows_ok(const ep_rows* r, int channels, const Geometry& g, int allowed, Segments* s) {
  if (!r) return EP_ERR_NULL;
  if (r->channels != channels) return EP_ERR_SHAPE;
  if (r->quant < EP_QUANT_NONE || r->quant > EP_QUANT_INT8) return EP_ERR_MODE;
  if (is_fp8(r->quant) && !(allowed & kFp8Rows)) return EP_ERR_MODE;
  if (r->quant == EP_QUANT_INT8 && !(allowed & kInt8Rows)) return EP_ERR_MODE;
  if (is_fp8(r->quant) && channels % 128 != 0) return EP_ERR_SHAPE;
  if (r->quant == EP_QUANT_INT8 && channels % 16 != 0) return EP_ERR_SHAPE;
  if (r->capacity < 0 || (!s->start && r->capacity < (int64_t)g.E * s->block_rows))
    return EP_ERR_CAPACITY;
  // no rows at all, no buffer needed
  if (r->capacity > 0 && (int64_t)g.R * g.T > 0) {
    if (!r->x || (r->quant != EP_QUANT_NONE && !r->scales)) return EP_ERR_NULL;
  }
  if (!aligned(r->x, 16)) return EP_ERR_ALIGN;
  if ((r->quant == EP_QUANT_FP8_F32 || r->quant == EP_QUANT_INT8) && !aligned(r->scales, 4))
    return EP_ERR_ALIGN;
  if (r->capacity < s->cap) s->cap = r->capacity;
  return EP_OK;
}

int weights_ok(const ep_weights* w) {
  if (!w) return EP_ERR_NULL;
  if (w->reserved != 0) return EP_ERR_SHAPE;
  if (w->fp8 < EP_WEIGHTS_BF16 || w->fp8 > EP_WEIGHTS_INT8) return EP_ERR_MODE;
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
  EP_TRY(rows_ok(x, C, g, kFp8Rows | kInt8Rows, &a.seg));
  const bool fp8 = is_fp8(x->quant), int8 = x->quant == EP_QUANT_INT8;
  if (w->fp8 != (fp8 ? EP_WEIGHTS_FP8 : int8 ? EP_WEIGHTS_INT8 : EP_WEIGHTS_BF16))
    return EP_ERR_MODE;
  if (fp8 && (C % 128 != 0 || N % 128 != 0)) return EP_ERR_SHAPE;
  if (!w->w || ((fp8 || int8) && !w->scales)) return EP_ERR_NULL;
  if (!aligned(w->w, 16) || (fp8 && !aligned(w->scales, 4)) || (int8 && !aligned(w->scales, 16)) ||
      !aligned(w->bias, 16))
    return EP_ERR_ALIGN;
  EP_TRY(rows_ok(y, N, g, fp8 ? kFp8Rows : kBf16Rows, &a.seg));
  if (residual) EP_TRY(rows_ok(residual, N, g, kBf16Rows, &a.seg));
  if (pre) EP_TRY(rows_ok(pre, O, g, kBf16Rows, &a.seg));
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
  EP_TRY(rows_ok(dy, N, g, kBf16Rows, &a.seg));
  const bool same = !gated && act == EP_ACT_NONE;  // dpre is dy
  if (!same) {
    EP_TRY(rows_ok(pre, O, g, kBf16Rows, &a.seg));
    if (dx || dw || dpre || gated) EP_TRY(rows_ok(dpre, O, g, kBf16Rows, &a.seg));
  }
  if (dx) {
    EP_TRY(rows_ok(dx, C, g, kBf16Rows, &a.seg));
    if (!w->w) return EP_ERR_NULL;
    if (!aligned(w->w, 16)) return EP_ERR_ALIGN;
  }
  if (dw) {
    EP_TRY(rows_ok(x, C, g, kBf16Rows, &a.seg));
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

// The layer's sizes.
int layer_ok(const Geometry& g, int inner) {
  if (!channels_ok(inner)) return EP_ERR_SHAPE;
  return (int64_t)g.R * g.T * g.K > EP_LAYER_MAX_ENTRIES ? EP_ERR_SHAPE : EP_OK;
}

// The layer's workspace: h, and with many entries their results.
size_t layer_h_bytes(const Geometry& g, int inner) {
  return ((size_t)g.R * g.T * g.K * inner * 4 + 255) & ~(size_t)255;
}

size_t layer_bytes(const Geometry& g, int inner) {
  const size_t entries = (size_t)g.R * g.T * g.K, row = (size_t)(g.H + 15) / 16 * 16;
  const size_t bytes = layer_h_bytes(g, inner) +
                       (ep::layer_many(entries, g.E, inner) ? entries * row * sizeof(float) : 0);
  return bytes < 256 ? 256 : bytes;
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

int ep_quantize_rows(const ep_problem* p, const ep_layout* layout, const ep_rows* x,
                     const ep_rows* q, void* stream) {
  Geometry g;
  EP_TRY(ep::make_geometry(p, &g));
  ep::Int8Args a;
  memset(&a, 0, sizeof(a));
  EP_TRY(segments(p, g, layout, &a.seg));
  if (!x) return EP_ERR_NULL;
  const int C = x->channels;
  if (!channels_ok(C) || C % 16 != 0) return EP_ERR_SHAPE;
  EP_TRY(rows_ok(x, C, g, kBf16Rows, &a.seg));
  EP_TRY(rows_ok(q, C, g, kInt8Rows, &a.seg));
  if (q->quant != EP_QUANT_INT8) return EP_ERR_MODE;
  a.rows = (int64_t)g.R * g.T * g.K;
  a.C = C;
  a.x = (const uint16_t*)x->x;
  a.codes = (int8_t*)q->x;
  a.scales = (float*)q->scales;
  if (ep::launch_rows_int8(a, (hipStream_t)stream) != hipSuccess) return EP_ERR_HIP;
  return EP_OK;
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

size_t ep_expert_layer_workspace_bytes(const ep_problem* p, int32_t inner) {
  Geometry g;
  if (ep::make_geometry(p, &g) != EP_OK || layer_ok(g, inner) != EP_OK) return 0;
  return layer_bytes(g, inner);
}

int ep_expert_layer(const ep_problem* p, const uint16_t* x, const int32_t* topk_idx,
                    const float* topk_weights, const ep_weights* w13, int32_t act,
                    const ep_weights* w2, uint16_t* out, int32_t* err, void* workspace,
                    size_t workspace_bytes, void* stream) {
  Geometry g;
  EP_TRY(ep::make_geometry(p, &g));
  EP_TRY(act_ok(act));
  EP_TRY(weights_ok(w13));
  EP_TRY(weights_ok(w2));
  const int H = g.H, I = w2->in_channels, kind = w13->fp8;
  EP_TRY(layer_ok(g, I));
  if (w13->in_channels != H || w2->out_channels != H || w13->out_channels != 2 * I)
    return EP_ERR_SHAPE;
  if (w2->fp8 != kind || w13->bias || w2->bias) return EP_ERR_MODE;
  const int step = kind == EP_WEIGHTS_FP8 ? 128 : kind == EP_WEIGHTS_INT8 ? 16 : 8;
  if (H % step != 0 || I % step != 0) return EP_ERR_SHAPE;
  const bool toks = (int64_t)g.R * g.T > 0;
  if (!w13->w || !w2->w || (kind != EP_WEIGHTS_BF16 && (!w13->scales || !w2->scales)))
    return EP_ERR_NULL;
  if (toks && (!x || !topk_idx || !topk_weights || !out || !workspace)) return EP_ERR_NULL;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(w13->w, 16) || !aligned(w2->w, 16) ||
      !aligned(workspace, 16) || !aligned(topk_idx, 4) || !aligned(topk_weights, 4) ||
      !aligned(err, 4))
    return EP_ERR_ALIGN;
  const int scales = kind == EP_WEIGHTS_INT8 ? 16 : 4;
  if (kind != EP_WEIGHTS_BF16 && (!aligned(w13->scales, scales) || !aligned(w2->scales, scales)))
    return EP_ERR_ALIGN;
  if (toks && workspace_bytes < layer_bytes(g, I)) return EP_ERR_WORKSPACE;
  ep::LayerArgs a;
  memset(&a, 0, sizeof(a));
  a.tokens = g.R * g.T;
  a.K = g.K;
  a.entries = a.tokens * g.K;
  a.E = g.E;
  a.H = H;
  a.I = I;
  a.kind = kind;
  a.act = act;
  a.x = x;
  a.idx = topk_idx;
  a.weights = topk_weights;
  a.w13 = (const char*)w13->w;
  a.s13 = w13->scales;
  a.w2 = (const char*)w2->w;
  a.s2 = w2->scales;
  a.h = (uint16_t*)workspace;
  a.y = (float*)((char*)workspace + layer_h_bytes(g, I));
  a.out = out;
  a.err = err;
  if (ep::launch_layer(a, (hipStream_t)stream) != hipSuccess) return EP_ERR_HIP;
  return EP_OK;
}

}  // extern "C"
