// libpoetx C ABI of the operators around the layer: argument checks, workspace carving and
// dispatch (declarations and contracts in include/poetx.h).
#include <cmath>
#include <initializer_list>

#include "kernels.h"

using namespace poetx;

namespace {

bool float_dtype(int32_t t) { return t == POETX_F32 || t == POETX_BF16; }

// every pointer is null or 16-byte aligned
bool aligned(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if ((uintptr_t)p & 15) return false;
  return true;
}

// outputs are distinct buffers: none of `outs` equals an input or another output
bool distinct(std::initializer_list<const void *> outs, std::initializer_list<const void *> ins) {
  for (auto i = outs.begin(); i != outs.end(); ++i) {
    if (!*i) continue;
    for (auto j = i + 1; j != outs.end(); ++j)
      if (*i == *j) return false;
    for (const void *p : ins)
      if (*i == p) return false;
  }
  return true;
}

// tiles of 128 x 128 results, the finest tiling of any product
bool tiles_fit(int64_t m, int64_t n) { return cdiv(m, 128) * cdiv(n, 128) <= ((int64_t)1 << 22); }

// The workspace protocol of every call: ws == NULL asks for the size.
int ws_check(const void *ws, size_t *ws_bytes, size_t need, bool *query) {
  *query = !ws;
  if (!ws) {
    *ws_bytes = need;
    return POETX_OK;
  }
  return *ws_bytes < need ? POETX_ERR_WORKSPACE : POETX_OK;
}

int norm_shape(int64_t n, int64_t d, int32_t dtype, int32_t p_dtype) {
  if (n < 0 || !float_dtype(dtype) || !float_dtype(p_dtype)) return POETX_ERR_INVALID_ARG;
  if (d < 1) return POETX_ERR_SHAPE;
  if (d > kNormMaxD) return POETX_ERR_UNSUPPORTED;
  return POETX_OK;
}

}  // namespace

extern "C" int poetx_layernorm_forward(int64_t n_rows, int64_t d, int32_t dtype, const void *x, const void *gamma,
                                       const void *beta, int32_t p_dtype, float eps, void *y, float *mean,
                                       float *rstd, void *stream) {
  POETX_TRY(norm_shape(n_rows, d, dtype, p_dtype));
  if (!(eps >= 0.f) || std::isinf(eps)) return POETX_ERR_INVALID_ARG;
  if (n_rows == 0) return POETX_OK;
  if (!x || !y || !aligned({x, gamma, beta, y, mean, rstd})) return POETX_ERR_INVALID_ARG;
  if (!distinct({y, mean, rstd}, {x, gamma, beta})) return POETX_ERR_INVALID_ARG;
  NormDesc n;
  n.n = n_rows; n.d = d; n.dt = dtype; n.p_bf16 = p_dtype == POETX_BF16;
  n.x = x; n.gamma = gamma; n.beta = beta; n.eps = eps;
  n.out = y; n.mean = mean; n.rstd = rstd;
  return norm_forward(n, (hipStream_t)stream);
}

extern "C" int poetx_layernorm_backward(int64_t n_rows, int64_t d, int32_t dtype, const void *x, const void *dy,
                                        const void *gamma, int32_t p_dtype, const float *mean, const float *rstd,
                                        const void *dres, void *dx, float *dgamma, float *dbeta, void *ws,
                                        size_t *ws_bytes, void *stream) {
  POETX_TRY(norm_shape(n_rows, d, dtype, p_dtype));
  if (!ws_bytes) return POETX_ERR_INVALID_ARG;
  Arena ar(ws);
  float *part = dgamma || dbeta ? (float *)ar.take((size_t)norm_bwd_parts(n_rows, d) * 2 * d * 4) : nullptr;
  bool query;
  POETX_TRY(ws_check(ws, ws_bytes, ar.used, &query));
  if (query) return POETX_OK;
  if (n_rows > 0 && (!x || !dy || !mean || !rstd || !dx)) return POETX_ERR_INVALID_ARG;
  if (!aligned({x, dy, gamma, mean, rstd, dres, dx, dgamma, dbeta, ws})) return POETX_ERR_INVALID_ARG;
  if (!distinct({dx, dgamma, dbeta}, {x, dy, gamma, mean, rstd, dres})) return POETX_ERR_INVALID_ARG;
  NormDesc n;
  n.n = n_rows; n.d = d; n.dt = dtype; n.p_bf16 = p_dtype == POETX_BF16;
  n.x = x; n.dy = dy; n.dres = dres; n.gamma = gamma;
  n.out = dx; n.mean = const_cast<float *>(mean); n.rstd = const_cast<float *>(rstd);
  return norm_backward(n, part, dgamma, dbeta, (hipStream_t)stream);
}

namespace {
int linear_shape(int64_t n, int64_t d_in, int64_t d_out, int32_t dtype, int32_t act) {
  if (n < 0 || !float_dtype(dtype)) return POETX_ERR_INVALID_ARG;
  if (act < POETX_ACT_NONE || act > POETX_ACT_SILU) return POETX_ERR_INVALID_ARG;
  if (d_in < 1 || d_out < 1) return POETX_ERR_SHAPE;
  if (d_in > kMaxWidth || d_out > kMaxWidth) return POETX_ERR_UNSUPPORTED;
  if (n > ((int64_t)1 << 40)) return POETX_ERR_UNSUPPORTED;
  if (!tiles_fit(n, d_out) || !tiles_fit(n, d_in) || !tiles_fit(d_out, d_in)) return POETX_ERR_UNSUPPORTED;
  return POETX_OK;
}
}  // namespace

extern "C" int poetx_linear_forward(int64_t n_tokens, int64_t d_in, int64_t d_out, int32_t dtype, const void *x,
                                    const void *w, const void *bias, int32_t bias_dtype, const void *residual,
                                    int32_t act, void *y, void *saved_pre, void *ws, size_t *ws_bytes, void *stream) {
  POETX_TRY(linear_shape(n_tokens, d_in, d_out, dtype, act));
  if (!float_dtype(bias_dtype) || !ws_bytes) return POETX_ERR_INVALID_ARG;
  LinDesc d;
  d.n = n_tokens; d.d_in = d_in; d.d_out = d_out; d.dt = dtype; d.act = act; d.bias_bf16 = bias_dtype == POETX_BF16;
  d.x = x; d.w = w; d.bias = bias; d.residual = residual; d.y = y; d.pre = saved_pre;
  Arena need(nullptr), ar(ws);
  POETX_TRY(linear_forward(d, need, true, nullptr));
  bool query;
  POETX_TRY(ws_check(ws, ws_bytes, need.used, &query));
  if (query || n_tokens == 0) return POETX_OK;
  if (!x || !w || !y || !aligned({x, w, bias, residual, y, saved_pre, ws})) return POETX_ERR_INVALID_ARG;
  if (!distinct({y, saved_pre}, {x, w, bias, residual})) return POETX_ERR_INVALID_ARG;
  return linear_forward(d, ar, false, (hipStream_t)stream);
}

extern "C" int poetx_linear_backward(int64_t n_tokens, int64_t d_in, int64_t d_out, int32_t dtype, const void *x,
                                     const void *w, const void *dy, const void *saved_pre, int32_t act, void *dx,
                                     void *dw, float *dbias, void *ws, size_t *ws_bytes, void *stream) {
  POETX_TRY(linear_shape(n_tokens, d_in, d_out, dtype, act));
  if (!ws_bytes || (!dx && !dw && !dbias)) return POETX_ERR_INVALID_ARG;
  LinDesc d;
  d.n = n_tokens; d.d_in = d_in; d.d_out = d_out; d.dt = dtype; d.act = act;
  d.x = x; d.w = w; d.dy = dy; d.saved_pre = saved_pre; d.dx = dx; d.dw = dw; d.dbias = dbias;
  Arena need(nullptr), ar(ws);
  POETX_TRY(linear_backward(d, need, true, nullptr));
  bool query;
  POETX_TRY(ws_check(ws, ws_bytes, need.used, &query));
  if (query) return POETX_OK;
  if (n_tokens > 0 && (!dy || (dx && !w) || (dw && !x) || (act != POETX_ACT_NONE && !saved_pre)))
    return POETX_ERR_INVALID_ARG;
  if (!aligned({x, w, dy, saved_pre, dx, dw, dbias, ws})) return POETX_ERR_INVALID_ARG;
  if (!distinct({dx, dw, dbias}, {x, w, dy, saved_pre})) return POETX_ERR_INVALID_ARG;
  return linear_backward(d, ar, false, (hipStream_t)stream);
}

namespace {
int xent_shape(int64_t n, int64_t d, int64_t vocab, int32_t dtype) {
  if (n < 0 || !float_dtype(dtype)) return POETX_ERR_INVALID_ARG;
  if (d < 1 || vocab < 1) return POETX_ERR_SHAPE;
  if (d > kMaxWidth || vocab > 0x7fffffff || n > ((int64_t)1 << 40)) return POETX_ERR_UNSUPPORTED;
  if (!tiles_fit(n, vocab) || !tiles_fit(n, d) || !tiles_fit(vocab, d)) return POETX_ERR_UNSUPPORTED;
  return POETX_OK;
}
}  // namespace

extern "C" int poetx_xent_forward(int64_t n_tokens, int64_t d, int64_t vocab, int32_t dtype, const void *h,
                                  const void *w, const int32_t *target, float *loss, float *lse, void *ws,
                                  size_t *ws_bytes, void *stream) {
  POETX_TRY(xent_shape(n_tokens, d, vocab, dtype));
  if (!ws_bytes) return POETX_ERR_INVALID_ARG;
  XentDesc x;
  x.n = n_tokens; x.d = d; x.v = vocab; x.dt = dtype;
  x.h = h; x.w = w; x.target = target; x.loss = loss; x.lse = lse;
  Arena need(nullptr), ar(ws);
  POETX_TRY(xent_forward(x, need, true, nullptr));
  bool query;
  POETX_TRY(ws_check(ws, ws_bytes, need.used, &query));
  if (query || n_tokens == 0) return POETX_OK;
  if (!h || !w || !target || !loss || !lse || !aligned({h, w, target, loss, lse, ws})) return POETX_ERR_INVALID_ARG;
  if (!distinct({loss, lse}, {h, w, target})) return POETX_ERR_INVALID_ARG;
  return xent_forward(x, ar, false, (hipStream_t)stream);
}

extern "C" int poetx_xent_backward(int64_t n_tokens, int64_t d, int64_t vocab, int32_t dtype, const void *h,
                                   const void *w, const int32_t *target, const float *lse, const float *dloss,
                                   void *dh, void *dw, void *ws, size_t *ws_bytes, void *stream) {
  POETX_TRY(xent_shape(n_tokens, d, vocab, dtype));
  if (!ws_bytes || (!dh && !dw)) return POETX_ERR_INVALID_ARG;
  XentDesc x;
  x.n = n_tokens; x.d = d; x.v = vocab; x.dt = dtype;
  x.h = h; x.w = w; x.target = target; x.lse_in = lse; x.dloss = dloss; x.dh = dh; x.dw = dw;
  Arena need(nullptr), ar(ws);
  POETX_TRY(xent_backward(x, need, true, nullptr));
  bool query;
  POETX_TRY(ws_check(ws, ws_bytes, need.used, &query));
  if (query) return POETX_OK;
  if (n_tokens > 0 && (!h || !w || !target || !lse || !dloss)) return POETX_ERR_INVALID_ARG;
  if (!aligned({h, w, target, lse, dloss, dh, dw, ws})) return POETX_ERR_INVALID_ARG;
  if (!distinct({dh, dw}, {h, w, target, lse, dloss})) return POETX_ERR_INVALID_ARG;
  return xent_backward(x, ar, false, (hipStream_t)stream);
}
