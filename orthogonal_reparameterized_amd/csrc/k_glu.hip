// Gated feed-forward projections:
//   forward   g = x Wg^T,  u = x Wu^T,  h = act(g) u
//   backward  dg = dh u act'(g),  du = dh act(g),
//             dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
#include "act.h"
#include "gemm_core.h"

namespace poetx {

struct GluTag {};

// h = act(g) u from float32 products; g and u kept where wanted.  One thread per 8 columns.
template <typename T>
__global__ __launch_bounds__(256) void k_glu_join(const float *g, const float *u, int act, int64_t n, int64_t f, T *h,
                                                  T *gate, T *up) {
  const int64_t cpr = cdiv(f, 8), total = n * cpr;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / cpr, c = (i - r * cpr) * 8, o = r * f + c;
    const int nv = f - c >= 8 ? 8 : (int)(f - c);
    float a[8], b[8];
    load8(g + o, nv, a);
    load8(u + o, nv, b);
    if (gate) store8(gate + o, nv, a);
    if (up) store8(up + o, nv, b);
    act_values<T>(a, act);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] *= b[e];
    store8(h + o, nv, a);
  }
}

// dg and du in T, rows of ld >= f elements (the rest zero).
template <typename T>
__global__ __launch_bounds__(256) void k_glu_grad(const T *dh, const T *gate, const T *up, int act, int64_t n, int64_t f,
                                                  T *dg, T *du, int64_t ld) {
  const int64_t cpr = cdiv(ld, 8), total = n * cpr;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / cpr, c = (i - r * cpr) * 8, left = f - c;
    const int nv = left >= 8 ? 8 : left > 0 ? (int)left : 0;
    float d[8], a[8], b[8], s[8];
    load8(dh + r * f + c, nv, d);
    load8(gate + r * f + c, nv, a);
    load8(up + r * f + c, nv, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = d[e] * b[e];
    act_slopes<T>(s, a, act);  // past nv: zero times a finite slope
    act_values<T>(a, act);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] *= a[e];
    const int nw = ld - c >= 8 ? 8 : (int)(ld - c);
    store8(dg + r * ld + c, nw, s);
    store8(du + r * ld + c, nw, d);
  }
}

// out = a + b, rounded to T
template <typename T>
__global__ __launch_bounds__(256) void k_glu_add(const float *a, const float *b, int64_t n, T *out) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 2048) {
    const int nv = n - i >= 8 ? 8 : (int)(n - i);
    float v[8], w[8];
    load8(a + i, nv, v);
    load8(b + i, nv, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += w[e];
    store8(out + i, nv, v);
  }
}

namespace {

int64_t round8(int64_t v) { return (v + 7) & ~(int64_t)7; }
dim3 stride_grid(int64_t n) {
  const int64_t g = cdiv(n, 256);
  return dim3((unsigned)(g < 65536 ? g : 65536));
}

// A bf16 operand whose rows are not a multiple of 16 bytes is copied to padded rows.
const void *packed(const void *in, int64_t rows, int64_t cols, int dt, Arena &ar, PackList &l) {
  if (dt == POETX_F32 || cols % 8 == 0) return in;
  void *q = ar.take((size_t)rows * round8(cols) * 2);
  l.add({in, rows, cols, q, round8(cols), nullptr, 0});
  return q;
}

template <typename T, bool AKM, bool BKM, typename C>
int product(const MmDesc &m, int dt, C *out, Arena &ar, bool measure, PackList *l, hipStream_t s) {
  const MmPlan p = mm_plan(m.M, m.N, m.K, dt);
  float *part = p.part_bytes ? (float *)ar.take(p.part_bytes) : nullptr;
  if (measure) return POETX_OK;
  if (l) POETX_TRY(pack_rows(*l, dt, s));
  return mm_run<T, AKM, BKM>(m, p, part, StoreEpi<C, GluTag>{out, m.N, 0}, s);
}

template <typename T>
int fwd_t(const GluDesc &d, Arena &ar, bool measure, hipStream_t s) {
  PackList l;
  const int64_t k = d.dt == POETX_BF16 ? round8(d.d) : d.d;
  float *g = (float *)ar.take((size_t)d.n * d.f * 4), *u = (float *)ar.take((size_t)d.n * d.f * 4);
  MmDesc m;
  m.M = d.n; m.N = d.f; m.K = k; m.lda = m.ldb = k; m.name = "glu_fwd"; m.large = "glu_fwd_large";
  m.A = packed(d.x, d.n, d.d, d.dt, ar, l);
  const void *wg = packed(d.wg, d.f, d.d, d.dt, ar, l), *wu = packed(d.wu, d.f, d.d, d.dt, ar, l);
  m.B = wg;
  POETX_TRY((product<T, false, false>(m, d.dt, g, ar, measure, &l, s)));
  m.B = wu;
  POETX_TRY((product<T, false, false>(m, d.dt, u, ar, measure, nullptr, s)));
  if (measure) return POETX_OK;
  return launch_k("glu_join", s, k_glu_join<T>, stride_grid(d.n * cdiv(d.f, 8)), dim3(256), 0, (const float *)g,
                  (const float *)u, d.act, d.n, d.f, (T *)d.h, (T *)d.gate, (T *)d.up);
}

template <typename T>
int bwd_t(const GluDesc &d, Arena &ar, bool measure, hipStream_t s) {
  if (d.n == 0) {
    if (measure || !d.dwg) return POETX_OK;
    POETX_TRY(fill_zero(d.dwg, d.f * d.d, d.dt, s));
    return fill_zero(d.dwu, d.f * d.d, d.dt, s);
  }
  PackList l;
  const bool b16 = d.dt == POETX_BF16;
  const int64_t lf = b16 ? round8(d.f) : d.f, ld = b16 ? round8(d.d) : d.d;
  T *dg = (T *)ar.take((size_t)d.n * lf * sizeof(T)), *du = (T *)ar.take((size_t)d.n * lf * sizeof(T));
  if (!measure)
    POETX_TRY(launch_k("glu_grad", s, k_glu_grad<T>, stride_grid(d.n * cdiv(lf, 8)), dim3(256), 0, (const T *)d.dh,
                       (const T *)d.gate_in, (const T *)d.up_in, d.act, d.n, d.f, dg, du, lf));
  if (d.dx) {
    float *a = (float *)ar.take((size_t)d.n * d.d * 4), *b = (float *)ar.take((size_t)d.n * d.d * 4);
    MmDesc m;
    m.M = d.n; m.N = d.d; m.K = d.f; m.lda = lf; m.ldb = ld; m.name = "glu_dx"; m.large = "glu_dx_large";
    const void *wg = packed(d.wg, d.f, d.d, d.dt, ar, l), *wu = packed(d.wu, d.f, d.d, d.dt, ar, l);
    m.A = dg; m.B = wg;
    POETX_TRY((product<T, false, true>(m, d.dt, a, ar, measure, &l, s)));
    m.A = du; m.B = wu;
    POETX_TRY((product<T, false, true>(m, d.dt, b, ar, measure, nullptr, s)));
    if (!measure)
      POETX_TRY(launch_k("glu_add", s, k_glu_add<T>, stride_grid(cdiv(d.n * d.d, 8)), dim3(256), 0, (const float *)a,
                         (const float *)b, d.n * d.d, (T *)d.dx));
  }
  if (d.dwg) {
    MmDesc m;
    m.M = d.f; m.N = d.d; m.K = d.n; m.lda = lf; m.ldb = ld; m.name = "glu_dw"; m.large = "glu_dw_large";
    m.B = packed(d.x, d.n, d.d, d.dt, ar, l);
    m.A = dg;
    POETX_TRY((product<T, true, true>(m, d.dt, (T *)d.dwg, ar, measure, &l, s)));
    m.A = du;
    POETX_TRY((product<T, true, true>(m, d.dt, (T *)d.dwu, ar, measure, nullptr, s)));
  }
  return POETX_OK;
}

}  // namespace

int glu_forward(const GluDesc &d, Arena &ar, bool measure, hipStream_t s) {
  if (d.n == 0) return POETX_OK;
  return d.dt == POETX_F32 ? fwd_t<float>(d, ar, measure, s) : fwd_t<bf16_t>(d, ar, measure, s);
}

int glu_backward(const GluDesc &d, Arena &ar, bool measure, hipStream_t s) {
  return d.dt == POETX_F32 ? bwd_t<float>(d, ar, measure, s) : bwd_t<bf16_t>(d, ar, measure, s);
}

}  // namespace poetx
