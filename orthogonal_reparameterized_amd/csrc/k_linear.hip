// Dense linear layer with its epilogue:
//   forward   p = x W^T + bias,  y = act(p) + residual
//   backward  dp = dy act'(p),  dx = dp W,  dW = dp^T x,  dbias = sum_tokens dp
// The products run on the kernels of gemm_core.h; bias, activation, residual and the kept
// pre-activation are part of the product's epilogue, on the float32 accumulators.
#include "act.h"
#include "gemm_core.h"

namespace poetx {

struct LinTag {};

template <typename T>
struct LinEpi {
  static constexpr bool kStats = false;
  static constexpr int kRows = 0;
  using Tag_ = LinTag;
  struct Cols { float b[8]; };
  T *y, *pre;
  const T *res;
  ParamVec bias;
  int act;
  int64_t ld;
  __device__ const LinEpi &at(int) const { return *this; }
  __device__ Cols cols(int64_t n, int nv, const float *) const {
    Cols c = {};
    if (bias.p && nv) bias.load(n, nv, c.b);
    return c;
  }
  __device__ void put(const Cols &c, int64_t m, int64_t n, float (&v)[8], int nv) const {
    const int64_t o = m * ld + n;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += c.b[e];
    if (pre) store8(pre + o, nv, v);
    act_values<T>(v, act);
    if (res) {
      float r[8];
      load8(res + o, nv, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += r[e];
    }
    store8(y + o, nv, v);
  }
};

// ------------------------------------------------- dp and the bias gradient ----
// dp = dy act'(p) in T, rows of ld_out >= cols elements (the rest zero), and its column
// sums: a workgroup owns 512 columns of a run of rows, a wave one row at a time, 8 columns
// per lane.  The sums take dp before it is rounded to T; the rounding is the precision in which
// the products read it (an operand's half step, independent from element to element).  Bound by
// HBM: 8192 x 4096 bf16 41.5 us, 4.8 TB/s.  part: [gridDim.y][cols].
template <typename T>
__global__ __launch_bounds__(256) void k_act_grad(const T *dy, const T *pre, int act, int64_t rows, int64_t cols,
                                                  T *dp, int64_t ld_out, float *part) {
  __shared__ float red[4][512];
  const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int64_t c0 = (int64_t)blockIdx.x * 512, c = c0 + l * 8;
  const int64_t left = cols - c;
  const int nv = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  const int64_t per = cdiv(rows, (int64_t)gridDim.y), r0 = per * blockIdx.y, r1 = r0 + per < rows ? r0 + per : rows;
  float sum[8] = {};
  for (int64_t r = r0 + wave; r < r1; r += 4) {
    float v[8];
    load8(dy + r * cols + c, nv, v);
    if (act != POETX_ACT_NONE) {
      float p[8];
      load8(pre + r * cols + c, nv, p);
      act_slopes<T>(v, p, act);  // past nv: zero times a finite slope
    }
    // ld_out is a multiple of 8, so a partly valid group is stored whole, with its zeros
    if (dp && nv) store8(dp + r * ld_out + c, ld_out == cols ? nv : 8, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += v[e];
  }
  if (!part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[wave][l * 8 + e] = sum[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 512; i += 256)
    if (c0 + i < cols)
      part[(int64_t)blockIdx.y * cols + c0 + i] = ((red[0][i] + red[1][i]) + red[2][i]) + red[3][i];
}

__global__ __launch_bounds__(1024) void k_sum_parts(SumArgs a) {
  __shared__ float red[16 * 64];
  sum_parts_body<64>(a, blockIdx.x, red);
}

template <typename T>
__global__ __launch_bounds__(256) void k_fill_zero(T *out, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) out[i] = 0;
}

// The copies of a list; job k has workgroups [end[k - 1], end[k]).  Rows are walked with that range's
// stride.
struct PackArgs {
  PackJob j[3];
  int end[3];
};
template <typename T>
__global__ __launch_bounds__(256) void k_pack_rows(PackArgs a) {
  const int id = (int)blockIdx.x, k = id < a.end[0] ? 0 : id < a.end[1] ? 1 : 2;
  const int begin = k == 0 ? 0 : k == 1 ? a.end[0] : a.end[1];
  const int groups = (k == 0 ? a.end[0] : k == 1 ? a.end[1] : a.end[2]) - begin;
  const PackJob p = k == 0 ? a.j[0] : k == 1 ? a.j[1] : a.j[2];
  const int64_t cpr = cdiv(p.ld_out, 8), total = p.rows * cpr;
  for (int64_t i = (int64_t)(id - begin) * 256 + threadIdx.x; i < total; i += (int64_t)groups * 256) {
    // a 32-bit division where it reaches (a 64-bit one is a long sequence)
    const int64_t r = total <= 0xffffffff ? (int64_t)((uint32_t)i / (uint32_t)cpr) : i / cpr;
    const int64_t c = (i - r * cpr) * 8, left = p.cols - c;
    float v[8] = {};
    const bool keep = !p.target || (p.target[r] >= 0 && p.target[r] < p.vocab);
    if (keep) load8((const T *)p.in + r * p.cols + c, left >= 8 ? 8 : left > 0 ? (int)left : 0, v);
    store8((T *)p.out + r * p.ld_out + c, p.ld_out - c >= 8 ? 8 : (int)(p.ld_out - c), v);
  }
}

// The same, transposed, through 64 x 64 tiles of LDS (4096 x 4096: 14.7 us, 4.6 TB/s).
__global__ __launch_bounds__(256) void k_pack_rows_t(const bf16_t *in, int64_t rows, int64_t cols, bf16_t *out,
                                                     int64_t ld_out, const int32_t *target, int64_t vocab,
                                                     int64_t tiles_r, int64_t tiles) {
  __shared__ bf16_t t[64][66];
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = tile % tiles_r * 64, c0 = tile / tiles_r * 64;
    __syncthreads();  // the tile before has been read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = threadIdx.x + 256 * i, r = e >> 3, c = (e & 7) * 8;
      const int64_t row = r0 + r, left = cols - c0 - c;
      u32v4 u = {0u, 0u, 0u, 0u};
      if (row < rows && (!target || (target[row] >= 0 && target[row] < vocab))) {
        if (left >= 8) {
          __builtin_memcpy(&u, in + row * cols + c0 + c, 16);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < left) u[k >> 1] |= (uint32_t)in[row * cols + c0 + c + k] << (16 * (k & 1));
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) *(uint32_t *)&t[r][c + 2 * k] = u[k];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = threadIdx.x + 256 * i, c = e >> 3, r = (e & 7) * 8;
      if (c0 + c >= cols || r0 + r >= ld_out) continue;
      u32v4 u;
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = (uint32_t)t[r + 2 * k][c] | (uint32_t)t[r + 2 * k + 1][c] << 16;
      __builtin_memcpy(out + (c0 + c) * ld_out + r0 + r, &u, 16);
    }
  }
}

// Workgroups of 256 for `n` independent items, walked with the grid's stride.
static dim3 stride_grid(int64_t n) {
  const int64_t g = cdiv(n, 256);
  return dim3((unsigned)(g < 65536 ? g : 65536));
}

int pack_rows(PackList &l, int dt, hipStream_t s) {
  if (l.n == 0) return POETX_OK;
  PackArgs a = {};
  int end = 0;
  for (int k = 0; k < 3; ++k) {
    if (k < l.n) {
      a.j[k] = l.j[k];
      end += (int)stride_grid(l.j[k].rows * cdiv(l.j[k].ld_out, 8)).x;
    }
    a.end[k] = end;
  }
  l.n = 0;
  if (dt == POETX_F32) return launch_k("pack_rows", s, k_pack_rows<float>, dim3((unsigned)end), dim3(256), 0, a);
  return launch_k("pack_rows", s, k_pack_rows<bf16_t>, dim3((unsigned)end), dim3(256), 0, a);
}

int pack_rows_t(const void *in, int64_t rows, int64_t cols, void *out, int64_t ld_out, const int32_t *target,
                int64_t vocab, hipStream_t s) {
  if (rows == 0) return POETX_OK;
  const int64_t tr = cdiv(ld_out, 64), tiles = tr * cdiv(cols, 64);
  return launch_k("pack_rows_t", s, k_pack_rows_t, dim3((unsigned)(tiles < 65536 ? tiles : 65536)), dim3(256), 0,
                  (const bf16_t *)in, rows, cols, (bf16_t *)out, ld_out, target, vocab, tr, tiles);
}

int fill_zero(void *p, int64_t n, int dt, hipStream_t s) {
  if (n == 0) return POETX_OK;
  const dim3 grid = stride_grid(n);
  if (dt == POETX_F32) return launch_k("fill_zero", s, k_fill_zero<float>, grid, dim3(256), 0, (float *)p, n);
  return launch_k("fill_zero", s, k_fill_zero<bf16_t>, grid, dim3(256), 0, (bf16_t *)p, n);
}

// ------------------------------------------------------------------- host ----
namespace {

int64_t round8(int64_t v) { return (v + 7) & ~(int64_t)7; }

// A bf16 operand whose rows are not a multiple of 16 bytes is copied to padded rows, which
// the direct global -> LDS loads need; others (and float32 ones) are used as they are.
struct Packed {
  const void *p = nullptr;
  int64_t ld = 0;
};
Packed packed(const void *in, int64_t rows, int64_t cols, int dt, Arena &ar, PackList &l) {
  Packed o{in, cols};
  if (dt == POETX_F32 || cols % 8 == 0) return o;
  o.ld = round8(cols);
  void *q = ar.take((size_t)rows * o.ld * 2);
  o.p = q;
  l.add({in, rows, cols, q, o.ld, nullptr, 0});
  return o;
}

template <typename T>
int fwd_t(const LinDesc &d, Arena &ar, bool measure, hipStream_t s) {
  const LinEpi<T> epi{(T *)d.y, (T *)d.pre, (const T *)d.residual, {d.bias, d.bias_bf16}, d.act, d.d_out};
  MmDesc m;
  m.M = d.n; m.N = d.d_out; m.K = d.d_in; m.name = "linear_fwd"; m.large = "linear_fwd_large";
  m.A = d.x; m.lda = d.d_in; m.B = d.w; m.ldb = d.d_in;
  if (d.n <= 16) {  // reading W bounds these: no LDS tiles, any alignment
    if (measure) return POETX_OK;
    MmArgs a{m.M, m.N, m.K, m.A, m.lda, m.B, m.ldb, 1, 1, 1, m.K};
    const int64_t groups = cdiv(d.d_out, 16), two = groups >= 1024;
    constexpr bool B16 = sizeof(T) == 2;
    auto kern = two ? k_mm_few<T, 2, false, LinEpi<T>> : k_mm_few<T, 1, false, LinEpi<T>>;
    if (B16 && d.d_in % 2) kern = two ? k_mm_few<T, 2, B16, LinEpi<T>> : k_mm_few<T, 1, B16, LinEpi<T>>;
    return launch_k(m.name, s, kern, dim3((unsigned)(two ? cdiv(groups, 2) : groups)), dim3(512), 0, a, epi);
  }
  PackList l;
  const Packed x = packed(d.x, d.n, d.d_in, d.dt, ar, l), w = packed(d.w, d.d_out, d.d_in, d.dt, ar, l);
  m.A = x.p; m.lda = x.ld; m.B = w.p; m.ldb = w.ld;
  if (d.dt == POETX_BF16) m.K = round8(d.d_in);  // the padding is zero
  const MmPlan p = mm_plan(m.M, m.N, m.K, d.dt);
  float *part = p.part_bytes ? (float *)ar.take(p.part_bytes) : nullptr;
  if (measure) return POETX_OK;
  POETX_TRY(pack_rows(l, d.dt, s));
  return mm_run<T, false, false>(m, p, part, epi, s);
}

// dx = dp W: dp k-contiguous, W k-major;  dW = dp^T x: both k-major
template <typename T>
int bwd_t(const LinDesc &d, Arena &ar, bool measure, hipStream_t s) {
  const bool b16 = d.dt == POETX_BF16;
  const void *dp = d.dy;
  int64_t ld = d.d_out;
  const bool products = d.dx || d.dw;
  const bool copy = products && (d.act != POETX_ACT_NONE || (b16 && d.d_out % 8));
  T *dpw = nullptr;
  if (copy) {
    if (b16) ld = round8(d.d_out);
    dpw = (T *)ar.take((size_t)d.n * ld * sizeof(T));
    dp = dpw;
  }
  SumArgs sum;  // the bias gradient's partials
  if (copy || d.dbias) {
    const int64_t cb = cdiv(d.d_out, 512), cus = device_cus() > 0 ? device_cus() : 256;
    int64_t parts = cdiv(4 * cus, cb);
    if (parts > cdiv(d.n, 4)) parts = cdiv(d.n, 4);  // a row per wave at least
    if (parts > 1024) parts = 1024;
    if (d.n <= 32) parts = 1;  // the column sums of few rows are whole at once: one launch less
    const bool join = d.dbias && (parts != 1 || d.n == 0);
    float *part = join ? (float *)ar.take((size_t)(parts > 0 ? parts : 1) * d.d_out * 4) : d.dbias;
    if (!measure && d.n > 0)
      POETX_TRY(launch_k("linear_act_grad", s, k_act_grad<T>, dim3((unsigned)cb, (unsigned)parts), dim3(256), 0,
                         (const T *)d.dy, (const T *)d.saved_pre, d.act, d.n, d.d_out, dpw, ld, part));
    if (join) sum = {part, d.n > 0 ? parts : (int64_t)0, d.d_out, d.dbias};
  }
  auto run_sum = [&] {
    if (measure || !sum.out) return (int)POETX_OK;
    return launch_k("linear_bias_grad", s, k_sum_parts, dim3((unsigned)cdiv(d.d_out, 64)), dim3(1024), 0, sum);
  };
  if (d.n == 0) {
    POETX_TRY(run_sum());
    return measure || !d.dw ? POETX_OK : fill_zero(d.dw, d.d_out * d.d_in, d.dt, s);
  }
  const StoreEpi<T, LinTag> ex{(T *)d.dx, d.d_in, 0}, ew{(T *)d.dw, d.d_in, 0};
  MmDesc mx, mw;
  PackList l;
  if (d.dx) {
    const Packed w = packed(d.w, d.d_out, d.d_in, d.dt, ar, l);
    mx.M = d.n; mx.N = d.d_in; mx.K = d.d_out; mx.name = "linear_dx"; mx.large = "linear_dx_large";
    mx.A = dp; mx.lda = ld; mx.B = w.p; mx.ldb = w.ld;
  }
  const bool flip = b16 && d.dw && dw_flips(d.d_out, d.d_in, d.n, d.dt);
  if (d.dw && !flip) {
    const Packed x = packed(d.x, d.n, d.d_in, d.dt, ar, l);
    mw.M = d.d_out; mw.N = d.d_in; mw.K = d.n; mw.name = "linear_dw"; mw.large = "linear_dw_large";
    mw.A = dp; mw.lda = ld; mw.B = x.p; mw.ldb = x.ld;
  }
  const MmTwo two = mm_two(mx.M, mx.N, mx.K, mw.M, mw.N, mw.K, d.dt);
  const MmPlan &px = two.a, &pw = two.b;
  float *part_x = px.part_bytes ? (float *)ar.take(px.part_bytes) : nullptr;
  float *part_w = pw.part_bytes ? (float *)ar.take(pw.part_bytes) : nullptr;
  if (!measure) POETX_TRY(pack_rows(l, d.dt, s));
  if (two.pair)
    return measure ? POETX_OK : mm_run_pair<T>("linear_dx_dw", mx, px, part_x, ex, mw, pw, part_w, ew, sum, s);
  POETX_TRY(run_sum());
  if (!measure) {
    POETX_TRY((mm_run<T, false, true>(mx, px, part_x, ex, s)));
    POETX_TRY((mm_run<T, true, true>(mw, pw, part_w, ew, s)));
  }
  if constexpr (sizeof(T) == 2) {
    if (flip) {
      const int64_t ldt = round8(d.n);
      void *xt = ar.take((size_t)d.d_in * ldt * 2);
      if (measure) return POETX_OK;
      POETX_TRY(pack_rows_t(d.x, d.n, d.d_in, xt, ldt, nullptr, 0, s));
      MmDesc m;
      m.M = d.d_in; m.N = d.d_out; m.K = d.n; m.large = "linear_dw_large";
      m.A = xt; m.lda = ldt; m.B = dp; m.ldb = ld;
      return mm_run_flipped(m, ew, s);
    }
  }
  return POETX_OK;
}

}  // namespace

int linear_forward(const LinDesc &d, Arena &ar, bool measure, hipStream_t s) {
  if (d.n == 0) return POETX_OK;
  return d.dt == POETX_F32 ? fwd_t<float>(d, ar, measure, s) : fwd_t<bf16_t>(d, ar, measure, s);
}

int linear_backward(const LinDesc &d, Arena &ar, bool measure, hipStream_t s) {
  return d.dt == POETX_F32 ? bwd_t<float>(d, ar, measure, s) : bwd_t<bf16_t>(d, ar, measure, s);
}

}  // namespace poetx
