// Norm of many gradients together, and clipping by it:
//   norm = sqrt(sum_k sum_i g_k[i]^2),  coef = norm <= max ? 1 : max / norm,  out_k = coef g_k
// The squares are taken and added in 64 bits: no value of either type over- or underflows there,
// and the sum of any number of them keeps every digit that a float32 norm shows.  (64-bit
// multiply-adds run at a tenth of their rate beside loads from memory.)
//
// The list of gradients comes with the launch, in its arguments: 120 of them at a time.  Each
// launch deals equal spans of elements to its workgroups; a workgroup's sum goes to one partial,
// and the partials are joined in their order.
#include "kernels.h"
#include "vec.h"

namespace poetx {

namespace {

constexpr int kGradList = 120;
constexpr int64_t kGradBlocks = 2048;  // workgroups over all gradients (and one more per gradient)

struct GradItem {
  const void *g;
  void *out;
  int64_t n;
  uint32_t first;  // its first workgroup in the launch
  uint32_t bf16;
};
struct GradArgs {
  GradItem t[kGradList];
  int count;
  int64_t span;    // elements per workgroup, a multiple of 2048
  double *part;    // this launch's partials
  const float *coef;
};

// the gradient of this workgroup
__device__ inline int item_of(const GradArgs &a) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.t[mid].first <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Elements of [begin, end) from p, 8 at a time from its first 16-byte boundary on:
// visit(index, count) with count <= 8.
template <typename T, class F>
__device__ inline void walk(const T *p, int64_t begin, int64_t end, const F &visit) {
  const int64_t head = ((16 - (int64_t)((uintptr_t)(p + begin) & 15)) & 15) / (int64_t)sizeof(T);
  const int64_t first = begin + head < end ? begin + head : end;
  if ((int64_t)threadIdx.x < first - begin) visit(begin + threadIdx.x, 1);
  for (int64_t i = first + 8 * (int64_t)threadIdx.x; i < end; i += 2048) visit(i, end - i >= 8 ? 8 : (int)(end - i));
}

__device__ inline double block_sum(double v, double *red) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return ((red[0] + red[1]) + red[2]) + red[3];
}

template <typename T>
__device__ inline double squares(const T *p, int64_t begin, int64_t end) {
  double s = 0;
  walk(p, begin, end, [&](int64_t i, int nv) {
    float v[8];
    load8(p + i, nv, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fma((double)v[e], (double)v[e], s);
  });
  return s;
}

template <typename T>
__device__ inline void scale(const T *p, T *out, int64_t begin, int64_t end, float c) {
  walk(p, begin, end, [&](int64_t i, int nv) {
    float v[8];
    load8(p + i, nv, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= c;
    store8(out + i, nv, v);
  });
}

}  // namespace

__global__ __launch_bounds__(256) void k_grad_squares(GradArgs a) {
  __shared__ double red[4];
  const GradItem &t = a.t[item_of(a)];
  const int64_t begin = (int64_t)(blockIdx.x - t.first) * a.span, end = begin + a.span < t.n ? begin + a.span : t.n;
  const double s = block_sum(t.bf16 ? squares((const bf16_t *)t.g, begin, end) : squares((const float *)t.g, begin, end),
                             red);
  if (threadIdx.x == 0) a.part[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void k_grad_join(const double *part, int64_t parts, float max_norm, float *norm,
                                                   float *coef) {
  __shared__ double red[4];
  double s = 0;
  for (int64_t i = threadIdx.x; i < parts; i += 256) s += part[i];
  s = sqrt(block_sum(s, red));
  if (threadIdx.x) return;
  *norm = (float)s;
  *coef = s <= (double)max_norm ? 1.f : (float)((double)max_norm / s);
}

__global__ __launch_bounds__(256) void k_grad_scale(GradArgs a) {
  const GradItem &t = a.t[item_of(a)];
  const float c = *a.coef;
  if (c == 1.f && t.out == t.g) return;
  const int64_t begin = (int64_t)(blockIdx.x - t.first) * a.span, end = begin + a.span < t.n ? begin + a.span : t.n;
  if (t.bf16) scale((const bf16_t *)t.g, (bf16_t *)t.out, begin, end, c);
  else scale((const float *)t.g, (float *)t.out, begin, end, c);
}

int grad_norm(const GradDesc &d, Arena &ar, bool measure, hipStream_t s) {
  int64_t total = 0, blocks = 0;
  for (int64_t k = 0; k < d.n; ++k) total += d.g[k].n;
  int64_t span = cdiv(cdiv(total, kGradBlocks), 2048) * 2048;
  if (span < 8192) span = 8192;
  for (int64_t k = 0; k < d.n; ++k) blocks += cdiv(d.g[k].n, span);
  double *part = (double *)ar.take((size_t)(blocks > 0 ? blocks : 1) * 8);
  if (measure) return POETX_OK;
  for (int pass = 0; pass < (d.clip ? 2 : 1); ++pass) {
    GradArgs a;
    a.span = span; a.part = part; a.coef = d.coef; a.count = 0;
    int64_t grid = 0;
    for (int64_t k = 0; k <= d.n; ++k) {
      if (k < d.n && d.g[k].n > 0) {
        a.t[a.count++] = {d.g[k].g, d.g[k].out, d.g[k].n, (uint32_t)grid, d.g[k].dtype == POETX_BF16 ? 1u : 0u};
        grid += cdiv(d.g[k].n, span);
      }
      if (a.count == kGradList || (k == d.n && a.count)) {
        if (pass == 0) POETX_TRY(launch_k("grad_squares", s, k_grad_squares, dim3((unsigned)grid), dim3(256), 0, a));
        else POETX_TRY(launch_k("grad_scale", s, k_grad_scale, dim3((unsigned)grid), dim3(256), 0, a));
        a.part += grid;
        a.count = 0;
        grid = 0;
      }
    }
    if (pass == 0)
      POETX_TRY(launch_k("grad_join", s, k_grad_join, dim3(1), dim3(256), 0, (const double *)part, blocks, d.max_norm,
                         d.norm, d.coef));
  }
  return POETX_OK;
}

}  // namespace poetx
