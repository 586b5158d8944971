// Layer norm over the last axis of row-major [n][d]:
//   forward   mu = sum_c x_c / d,  r = (sum_c (x_c - mu)^2 / d + eps)^(-1/2),
//             y = (x - mu) r gamma + beta
//   backward  xh = (x - mu) r,  g = dy gamma,
//             dx = dres + r (g - mean_c(g) - xh mean_c(g xh)),
//             dgamma = sum_rows dy xh,  dbeta = sum_rows dy
// Both directions read each row once: it stays in registers (chunks of 8 elements per
// thread) between the statistics and the result, so the variance is the two-pass one.  (Above
// 12288 columns the backward reads it twice.)
// All sums are float32.  Bound by HBM: 2 n d elements forward, 3 (4 with dres) backward.
// 8192 x 4096 bf16: forward 25.7 us (5.2 TB/s, a large copy's rate), backward with dres 44.5 us
// and 4.4 us to join its partials (268 MB of operands at 5.5 TB/s; without the row in flight
// ahead and with 4 workgroups per CU it was 84 and 17 us).  A wave per row up to 1024 columns,
// 256 threads up to 6144, 512 (the forward's last 4096 columns: 1024) above: few threads with up to
// three chunks each leave room for more rows on a CU than many threads with one (8192 rows of 5120
// bf16, forward and backward: 256 x 3 chunks 29 and 48 us, 512 x 2 34 and 67, 1024 x 1 43 and 65; of
// 12288: 512 x 3 77 and 112, 1024 x 2 111 and 349; float32 gains less, 75 and 113 us at 6144 against 79
// and 118).
#include "kernels.h"
#include "vec.h"

namespace poetx {

struct NormArgs {
  int64_t n, d;
  const void *x, *dy, *dres;
  ParamVec gamma, beta;  // p null: gamma = 1, beta = 0
  float eps, fd;         // fd: d, the divisor (a product by 1 / d would not give a constant row its mean)
  void *out;             // y or dx
  float *mean, *rstd;    // written by the forward (nullable), read by the backward
  float *part;           // [grid][2][d] partial dgamma, dbeta (nullable)
};

namespace {

// Sum of NV values over the THR threads that share a row.  `red` alternates between two
// halves from call to call (its parity), so one barrier per call is enough.
template <int THR, int NV>
__device__ inline void row_sum(float (&v)[NV], float *red, int parity) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if constexpr (THR > 64) {
    constexpr int W = THR / 64;
    float *r = red + parity * (NV * W);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) r[i * W + (threadIdx.x >> 6)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += r[i * W + w];
      v[i] = s;
    }
  }
}

__device__ inline int clamp8(int64_t left) { return left >= 8 ? 8 : left > 0 ? (int)left : 0; }

}  // namespace

// THR threads per row, CH chunks of 8 columns per thread: d <= 8 THR CH.
template <typename T, int THR, int CH>
__global__ __launch_bounds__(THR < 256 ? 256 : THR) void k_norm_fwd(NormArgs a) {
  constexpr int BLK = THR < 256 ? 256 : THR, RPB = BLK / THR;
  __shared__ float red[2 * (THR > 64 ? THR / 64 : 1)];
  const int t = threadIdx.x % THR;
  float ga[CH][8], be[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int64_t col = (int64_t)(c * THR + t) * 8;
    const int nv = clamp8(a.d - col);
#pragma unroll
    for (int e = 0; e < 8; ++e) { ga[c][e] = 1.f; be[c][e] = 0.f; }
    if (nv && a.gamma.p) a.gamma.load(col, nv, ga[c]);
    if (nv && a.beta.p) a.beta.load(col, nv, be[c]);
  }
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / THR; row < a.n; row += (int64_t)gridDim.x * RPB) {
    const T *x = (const T *)a.x + row * a.d;
    float v[CH][8];
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = (int64_t)(c * THR + t) * 8;
      load8(x + col, clamp8(a.d - col), v[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[c][e];
    }
    row_sum<THR, 1>(s, red, 0);
    const float mu = s[0] / a.fd;
    s[0] = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int nv = clamp8(a.d - (int64_t)(c * THR + t) * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = v[c][e] - mu;
        s[0] += e < nv ? z * z : 0.f;
      }
    }
    row_sum<THR, 1>(s, red, 1);
    const float r = 1.f / sqrtf(s[0] / a.fd + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = r;
    }
    T *y = (T *)a.out + row * a.d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = (int64_t)(c * THR + t) * 8;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (v[c][e] - mu) * r * ga[c][e] + be[c][e];
      store8(y + col, clamp8(a.d - col), o);
    }
  }
}

// A workgroup walks rows blockIdx.x, + gridDim.x, ... and keeps its columns' sums of
// dy xh and dy in registers; they leave once, as one partial per workgroup, and
// k_norm_params sums the partials in order.
template <typename T, int THR, int CH>
__global__ __launch_bounds__(THR < 256 ? 256 : THR) void k_norm_bwd(NormArgs a) {
  constexpr int BLK = THR < 256 ? 256 : THR, RPB = BLK / THR;
  __shared__ float red[4 * (THR > 64 ? THR / 64 : 1)];
  const int t = threadIdx.x % THR;
  float ga[CH][8], dg[CH][8], db[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int64_t col = (int64_t)(c * THR + t) * 8;
    const int nv = clamp8(a.d - col);
#pragma unroll
    for (int e = 0; e < 8; ++e) { ga[c][e] = 1.f; dg[c][e] = db[c][e] = 0.f; }
    if (nv && a.gamma.p) a.gamma.load(col, nv, ga[c]);
  }
  // The next row's loads are in flight while this row is reduced.  With four chunks the registers
  // do not hold that: LEAN loads the row once for its sums and again (from L2) for its results (8192
  // rows of 16384 bf16 224 us; with all of it in registers, which spills, 419, with the row kept as
  // it lies in memory 466).
  constexpr bool LEAN = CH == 4;
  constexpr int KEEP = LEAN ? 1 : CH;
  Raw8<T> rx[KEEP], ry[KEEP], rr[KEEP];
  float mu_n = 0.f, r_n = 0.f;
  auto fetch_chunk = [&](int64_t row, int c, int k) {
    const int64_t col = (int64_t)(c * THR + t) * 8;
    const int nv = clamp8(a.d - col);
    load_raw((const T *)a.x + row * a.d + col, nv, rx[k]);
    load_raw((const T *)a.dy + row * a.d + col, nv, ry[k]);
    if (a.dres) load_raw((const T *)a.dres + row * a.d + col, nv, rr[k]);
  };
  auto fetch = [&](int64_t row) {
    mu_n = a.mean[row];
    r_n = a.rstd[row];
#pragma unroll
    for (int c = 0; c < CH && !LEAN; ++c) fetch_chunk(row, c, c);
  };
  int parity = 0;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / THR;
  if (!LEAN && row < a.n) fetch(row);
  for (; row < a.n; row += step) {
    if (LEAN) fetch(row);
    const float mu = mu_n, r = r_n;
    float xh[KEEP][8], g[KEEP][8], q[KEEP][8], s[2] = {0.f, 0.f};
    auto expand = [&](int c, float (&xh_)[8], float (&g_)[8], float (&q_)[8]) {
      const int nv = clamp8(a.d - (int64_t)(c * THR + t) * 8);
      const int k = LEAN ? 0 : c;
      widen(rx[k], xh_);
      widen(ry[k], g_);
      if (a.dres) widen(rr[k], q_);
#pragma unroll
      for (int e = 0; e < 8; ++e) xh_[e] = e < nv ? (xh_[e] - mu) * r : 0.f;
    };
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = LEAN ? 0 : c;
      if (LEAN) fetch_chunk(row, c, k);
      expand(c, xh[k], g[k], q[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dg[c][e] += g[k][e] * xh[k][e];
        db[c][e] += g[k][e];
        g[k][e] *= ga[c][e];
        s[0] += g[k][e];
        s[1] += g[k][e] * xh[k][e];
      }
    }
    if (!LEAN && row + step < a.n) fetch(row + step);
    row_sum<THR, 2>(s, red, parity);
    if (LEAN) asm volatile("" ::: "memory");  // the second pass loads again
    parity ^= 1;
    const float m1 = s[0] / a.fd, m2 = s[1] / a.fd;
    T *dx = (T *)a.out + row * a.d;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = LEAN ? 0 : c;
      if constexpr (LEAN) {
        fetch_chunk(row, c, k);
        expand(c, xh[k], g[k], q[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[k][e] *= ga[c][e];
      }
      const int64_t col = (int64_t)(c * THR + t) * 8;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = r * (g[k][e] - m1 - xh[k][e] * m2);
        if (a.dres) o[e] += q[k][e];
      }
      store8(dx + col, clamp8(a.d - col), o);
    }
  }
  if (!a.part) return;
  float *pg = a.part + (int64_t)blockIdx.x * 2 * a.d;
  if constexpr (RPB > 1) {  // the rows' waves of one workgroup, added in wave order
    __shared__ float acc[2][CH * THR * 8];
    for (int w = 0; w < RPB; ++w) {
      if ((int)threadIdx.x / THR == w) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = (c * THR + t) * 8 + e;
            acc[0][i] = w ? acc[0][i] + dg[c][e] : dg[c][e];
            acc[1][i] = w ? acc[1][i] + db[c][e] : db[c][e];
          }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < a.d; i += BLK) {
      pg[i] = acc[0][i];
      pg[a.d + i] = acc[1][i];
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = (int64_t)(c * THR + t) * 8;
      const int nv = clamp8(a.d - col);
      store8(pg + col, nv, dg[c]);
      store8(pg + a.d + col, nv, db[c]);
    }
  }
}

// dgamma, dbeta = the sums over the workgroups' partials [parts][2 d], in a fixed order: 32
// columns per workgroup, 128 threads per 4 columns each summing every 128th partial, joined
// pairwise.
__global__ __launch_bounds__(1024) void k_norm_params(const float *part, int64_t parts, int64_t d, float *dgamma,
                                                      float *dbeta) {
  __shared__ f32v4 red[128][8];
  const int c = threadIdx.x & 7, q = threadIdx.x >> 3;
  const int64_t col = (int64_t)blockIdx.x * 32 + c * 4, left = 2 * d - col;
  f32v4 s = {0.f, 0.f, 0.f, 0.f};
  for (int64_t p = q; p < parts; p += 128) {
    const float *src = part + p * 2 * d + col;
    if (left >= 4) {
      f32v4 v;
      __builtin_memcpy(&v, src, 16);
      s += v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += e < left ? src[e] : 0.f;
    }
  }
  red[q][c] = s;
#pragma unroll
  for (int o = 64; o; o >>= 1) {
    __syncthreads();
    if (q < o) {
      s += red[q + o][c];
      red[q][c] = s;
    }
  }
  if (q) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (e >= left) break;
    float *out = col + e < d ? dgamma : dbeta;
    if (out) out[col + e < d ? col + e : col + e - d] = s[e];
  }
}

namespace {

template <typename T, int THR, int CH>
int run_fwd(const NormArgs &a, int64_t blocks, hipStream_t s) {
  constexpr int BLK = THR < 256 ? 256 : THR;
  return launch_k("layernorm_fwd", s, k_norm_fwd<T, THR, CH>, dim3((unsigned)blocks), dim3(BLK), 0, a);
}
template <typename T, int THR, int CH>
int run_bwd(const NormArgs &a, int64_t blocks, hipStream_t s) {
  constexpr int BLK = THR < 256 ? 256 : THR;
  return launch_k("layernorm_bwd", s, k_norm_bwd<T, THR, CH>, dim3((unsigned)blocks), dim3(BLK), 0, a);
}

// Workgroups that walk the n rows (a wave per row up to 1024 columns).  Forward: 8 per CU (2 above
// 8192 columns).  Backward: 2 (1 above 6144 columns) per CU, which with a row in flight ahead keep
// as much memory traffic going while they leave fewer partial sums to write and join.
int64_t norm_blocks(int64_t n, int64_t d, bool bwd) {
  const int64_t cus = device_cus() > 0 ? device_cus() : 256;
  const int64_t most = cus * (bwd ? (d <= 6144 ? 2 : 1) : (d <= 8192 ? 8 : 2));
  const int64_t need = cdiv(n, d <= 1024 ? 4 : 1);
  return need < most ? need : most;
}

template <typename T>
int fwd_t(const NormArgs &a, hipStream_t s) {
  const int64_t g = norm_blocks(a.n, a.d, false);
  if (a.d <= 512) return run_fwd<T, 64, 1>(a, g, s);
  if (a.d <= 1024) return run_fwd<T, 64, 2>(a, g, s);
  if (a.d <= 2048) return run_fwd<T, 256, 1>(a, g, s);
  if (a.d <= 4096) return run_fwd<T, 256, 2>(a, g, s);
  if (a.d <= 6144) return run_fwd<T, 256, 3>(a, g, s);
  if (a.d <= 8192) return run_fwd<T, 512, 2>(a, g, s);
  if (a.d <= 12288) return run_fwd<T, 512, 3>(a, g, s);
  return run_fwd<T, 1024, 2>(a, g, s);
}
template <typename T>
int bwd_t(const NormArgs &a, int64_t g, hipStream_t s) {
  if (a.d <= 512) return run_bwd<T, 64, 1>(a, g, s);
  if (a.d <= 1024) return run_bwd<T, 64, 2>(a, g, s);
  if (a.d <= 2048) return run_bwd<T, 256, 1>(a, g, s);
  if (a.d <= 4096) return run_bwd<T, 256, 2>(a, g, s);
  if (a.d <= 6144) return run_bwd<T, 256, 3>(a, g, s);
  if (a.d <= 8192) return run_bwd<T, 512, 2>(a, g, s);
  if (a.d <= 12288) return run_bwd<T, 512, 3>(a, g, s);
  return run_bwd<T, 512, 4>(a, g, s);
}

}  // namespace

int64_t norm_bwd_parts(int64_t n, int64_t d) { return norm_blocks(n, d, true); }

int norm_forward(const NormDesc &n, hipStream_t s) {
  if (n.n == 0) return POETX_OK;
  NormArgs a{n.n, n.d, n.x, nullptr, nullptr, {n.gamma, n.p_bf16}, {n.beta, n.p_bf16}, n.eps, (float)n.d,
             n.out, n.mean, n.rstd, nullptr};
  return n.dt == POETX_F32 ? fwd_t<float>(a, s) : fwd_t<bf16_t>(a, s);
}

int norm_backward(const NormDesc &n, float *part, float *dgamma, float *dbeta, hipStream_t s) {
  const int64_t g = norm_bwd_parts(n.n, n.d);
  if (n.n > 0) {
    NormArgs a{n.n, n.d, n.x, n.dy, n.dres, {n.gamma, n.p_bf16}, {nullptr, 0}, 0.f, (float)n.d,
               n.out, n.mean, n.rstd, part};
    POETX_TRY(n.dt == POETX_F32 ? bwd_t<float>(a, g, s) : bwd_t<bf16_t>(a, g, s));
  }
  if (!dgamma && !dbeta) return POETX_OK;
  // no rows: no partials, and the sums over nothing are zero
  return launch_k("layernorm_params", s, k_norm_params, dim3((unsigned)cdiv(2 * n.d, 32)), dim3(1024), 0,
                  (const float *)part, n.n > 0 ? g : (int64_t)0, n.d, dgamma, dbeta);
}

}  // namespace poetx
