// Softmax cross entropy of a linear head, without keeping the logits l = h W^T:
//   forward   lse_i = log sum_v exp l_iv,  loss_i = lse_i - l_i,t(i)
//   backward  dl_iv = (exp(l_iv - lse_i) - [v = t(i)]) dloss_i,  dh = dl W,  dW = dl^T h
// A row whose target lies outside the vocabulary takes no part: loss 0, dl 0.
//
// Forward: the product's epilogue reduces each row of a tile to its maximum and its sum of
// exp(l - maximum), 8 bytes per row and 256 columns; k_xent_join joins them.  (A product of so
// few tiles that it is split over k passes its partial sums, at most 2^24 floats at a time,
// through the workspace first.)  Backward: the
// logits of a piece of the vocabulary are computed again and leave the epilogue as dl (bf16
// for bf16 operands, the operand type of the two products that read it), then dh += dl W and
// dW of the piece follow while dl is in the caches.  8 n d v flops in all, chosen for the memory
// (keeping the logits would take 6 n d v and n v values).  Bound by the matrix cores for many
// tokens (4096 x 4096 x 65536: forward 1.59, dl 1.63, dh 1.55, dW 1.70 ms, 1.29 to 1.41 PFLOP/s)
// and by reading W for few.
#include "gemm_core.h"

namespace poetx {

struct XentTag {};

namespace {
// (max, sum of exp(l - max)) of two sets of logits.  An empty set has max = -inf, sum = 0.
__device__ inline void join_stats(float &m, float &s, float m2, float s2) {
  const float t = fmaxf(m, m2);
  const float ref = fabsf(t) == INFINITY ? 0.f : t;
  s = s * __expf(m - ref) + s2 * __expf(m2 - ref);
  m = t;
}
__device__ inline float safe_ref(float m) { return fabsf(m) == INFINITY ? 0.f : m; }
}  // namespace

// part[tile][row] = (max, sum) over the tile's columns; at_target[row] = l of the target.
struct XentStats {
  static constexpr bool kStats = true;
  using Tag_ = XentTag;
  float2 *part;
  const int32_t *target;
  float *at_target;
  int64_t v0;     // first vocabulary entry of this launch
  int tile0;      // first row of `part`
  __device__ const XentStats &at(int) const { return *this; }

  template <int BM, int BN, int WGM, int WGN, int FM, int FN>
  __device__ void reduce(const f32x4 (&acc)[FM][FN], int64_t m0, int64_t n0, int64_t M, int64_t N, int tn,
                         float *lds) const {
    constexpr int R = 16;
    const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int wm = (wave / WGN) * (BM / WGM), wn = (wave % WGN) * (BN / WGN);
    const int64_t nb = n0 + wn + 4 * (l / R);  // this lane's columns: nb + R j + e
    const int left = N - nb < 65536 ? (int)(N - nb) : 65536;
    float2 *st = (float2 *)lds;                // [WGN][BM]
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = wm + R * i + l % R;
      const int64_t m = m0 + r;
      const int64_t tt = m < M ? (int64_t)target[m] - v0 - nb : -1;
      const int t = tt >= 0 && tt < left && tt < 65536 ? (int)tt : -1;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = R * j + e;
          const float v = c < left ? acc[i][j][e] : -INFINITY;
          if (t == c) at_target[m] = v;
          mx = fmaxf(mx, v);
        }
      const float ref = safe_ref(mx);
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s += R * j + e < left ? __expf(acc[i][j][e] - ref) : 0.f;
#pragma unroll
      for (int o = R; o <= 32; o <<= 1) {
        const float m2 = __shfl_xor(mx, o), s2 = __shfl_xor(s, o);
        join_stats(mx, s, m2, s2);
      }
      if (l < R) st[(wave % WGN) * BM + r] = make_float2(mx, s);
    }
    __syncthreads();
    for (int r = threadIdx.x; r < BM; r += 64 * WGM * WGN) {
      if (m0 + r >= M) continue;
      float2 p = st[r];
#pragma unroll
      for (int w = 1; w < WGN; ++w) join_stats(p.x, p.y, st[w * BM + r].x, st[w * BM + r].y);
      part[(int64_t)(tile0 + tn) * M + m0 + r] = p;
    }
  }
};

// dl of a piece of the vocabulary, rows of ld elements (a multiple of 8 for bf16, zeros
// past the piece).  Rounding dl to bf16 is the products' operand precision.  So that the errors
// are independent from row to row, bf16 rows carry dloss_i / G with G the largest |dloss| (the
// products' epilogues multiply by G): rounded as they are, the rows of a mean, whose dl at the
// target is nearly -dloss_i = -1 / count for all of them, would share one rounding error.
template <typename T>
struct XentDl {
  static constexpr bool kStats = false;
  static constexpr int kRows = 3;
  using Tag_ = XentTag;
  struct Cols { const float *rows; };
  T *dl;
  int64_t ld;
  const int32_t *target;
  const float *lse, *dloss, *scale;  // scale: G, or null for 1
  int64_t v0, vocab;
  __device__ const XentDl &at(int) const { return *this; }
  __device__ Cols cols(int64_t, int, const float *rows) const { return {rows}; }
  // lse, dloss and the target of each row of the tile; a row that takes no part has target -1
  __device__ float stage(int64_t m0, int64_t M, int i) const {
    const int64_t m = m0 + i / 3;
    if (m >= M) return 0.f;
    if (i % 3 == 0) return lse[m];
    if (i % 3 == 1) return scale ? dloss[m] / *scale : dloss[m];
    const int32_t t = target[m];
    return __int_as_float(t >= 0 && t < vocab ? t : -1);
  }
  __device__ void put(const Cols &c, int64_t m, int64_t n, float (&v)[8], int nv) const {
    // from the tile's staged rows, or (where partials are joined) from memory
    const float *r = c.rows + m * 3;
    const float z = c.rows ? r[0] : stage(m, m + 1, 0), g = c.rows ? r[1] : stage(m, m + 1, 1);
    const int t = __float_as_int(c.rows ? r[2] : stage(m, m + 1, 2));
    const int64_t q = t - v0 - n;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = __expf(v[e] - z) - (q == e ? 1.f : 0.f);
      v[e] = t >= 0 && e < nv ? p * g : 0.f;
    }
    store8(dl + m * ld + n, sizeof(T) == 2 ? 8 : nv, v);
  }
};

// dh over the pieces: float32 sums in `sum` between the first and the last piece.  A row that takes
// no part is written as zeros: its dl is zero, but zero times an infinity of W would not be.
template <typename T>
struct XentDh {
  static constexpr bool kStats = false;
  static constexpr int kRows = 1;
  using Tag_ = XentTag;
  struct Cols { float g; const float *rows; };
  float *sum;
  T *dh;
  const float *scale;
  const int32_t *target;
  int64_t vocab, ld;
  int first, last;
  __device__ const XentDh &at(int) const { return *this; }
  __device__ Cols cols(int64_t, int, const float *rows) const { return {scale ? *scale : 1.f, rows}; }
  __device__ float stage(int64_t m0, int64_t M, int i) const {  // whether the row takes part
    const int64_t m = m0 + i;
    return m < M && target[m] >= 0 && target[m] < vocab ? 1.f : 0.f;
  }
  __device__ void put(const Cols &c, int64_t m, int64_t n, float (&v)[8], int nv) const {
    const int64_t o = m * ld + n;
    if (!first) {
      float w[8];
      load8(sum + o, nv, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
    if (last) {
      const bool on = (c.rows ? c.rows[m] : stage(m, m + 1, 0)) != 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = on ? v[e] * c.g : 0.f;
      store8(dh + o, nv, v);
    } else {
      store8(sum + o, nv, v);
    }
  }
};

// dW of a piece.
template <typename T>
struct XentDw {
  static constexpr bool kStats = false;
  static constexpr int kRows = 0;
  using Tag_ = XentTag;
  struct Cols { float g; };
  T *dw;
  const float *scale;
  int64_t ld;
  __device__ const XentDw &at(int) const { return *this; }
  __device__ Cols cols(int64_t, int, const float *) const { return {scale ? *scale : 1.f}; }
  __device__ void put(const Cols &c, int64_t m, int64_t n, float (&v)[8], int nv) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= c.g;
    store8(dw + m * ld + n, nv, v);
  }
};

// G: the largest |dloss| of the tokens that take part, 1 where that is 0 or not finite.
__global__ __launch_bounds__(1024) void k_xent_scale(const float *dloss, const int32_t *target, int64_t n, int64_t vocab,
                                                     float *scale) {
  __shared__ float red[16];
  float g = 0.f;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < n; i += 1024) {
    const int32_t t = target[i];
    const float a = fabsf(dloss[i]);
    if (t >= 0 && t < vocab && a > g && a < INFINITY) g = a;
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) g = fmaxf(g, __shfl_xor(g, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = g;
  __syncthreads();
  if (threadIdx.x) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) g = fmaxf(g, red[w]);
  *scale = g > 0.f ? g : 1.f;
}

// Row statistics of a split product: its partials [splits][n][v] summed in split order, a wave
// per row and 256 columns.
__global__ __launch_bounds__(256) void k_xent_parts(const float *src, int splits, int64_t n, int64_t v, XentStats epi) {
  const int l = threadIdx.x & 63;
  const int64_t m = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6), c = (int64_t)blockIdx.x * 256 + l * 4, left = v - c;
  if (m >= n) return;
  f32v4 s = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < splits; ++k) {
    const float *p = src + ((int64_t)k * n + m) * v + c;
    if (left >= 4) {
      f32v4 w;
      __builtin_memcpy(&w, p, 16);
      s += w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += e < left ? p[e] : 0.f;
    }
  }
  const int64_t t = (int64_t)epi.target[m] - epi.v0 - c;
  float mx = -INFINITY, sum = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (e >= left) continue;
    if (t == e) epi.at_target[m] = s[e];
    mx = fmaxf(mx, s[e]);
  }
  const float ref = safe_ref(mx);
#pragma unroll
  for (int e = 0; e < 4; ++e) sum += e < left ? __expf(s[e] - ref) : 0.f;
#pragma unroll
  for (int o = 1; o <= 32; o <<= 1) {
    const float m2 = __shfl_xor(mx, o), s2 = __shfl_xor(sum, o);
    join_stats(mx, sum, m2, s2);
  }
  if (l == 0) epi.part[(int64_t)(epi.tile0 + (int)blockIdx.x) * n + m] = make_float2(mx, sum);
}

// Few tokens (n <= 16): bound by reading W once.  KW waves share a group of 16 vocabulary rows:
// each takes every KW-th turn of the group's k (the next U fragments in flight while these
// multiply) and keeps (max, sum) per lane (row l % 16, its 4 columns of the group); one partial per
// workgroup.  KW = 1 walks groups and keeps a running (max, sum): 8 tokens, d = 4096, 131072 rows,
// bf16: 206 us, 5.2 TB/s, the rate of a large copy (242 us without the loads ahead; 222 us with
// half or twice the workgroups).
template <typename T, int KW, bool ODD>
__global__ __launch_bounds__(512) void k_xent_few(MmArgs a, XentStats epi) {
  constexpr int NG = 8 / KW, U = 8, E = RowFrag<T>::E, D = 4 * E;  // fragments of D k per turn
  using V = typename RowFrag<T>::V;
  __shared__ float2 st[8][16];
  const int wave = threadIdx.x >> 6, l = threadIdx.x & 63, kw = wave % KW;
  const int64_t m = l & 15;
  const T *pa = (const T *)a.A + (m < a.M ? m : a.M - 1) * a.lda + E * (l >> 4);
  const int64_t t = m < a.M ? (int64_t)epi.target[m] : -1;
  const int64_t groups = cdiv(a.N, 16), whole = a.K / (D * U);  // whole turns of k
  float mx = -INFINITY, s = 0.f;
  auto dot = [&](int64_t g) {
    const int64_t n = g * 16 + (l & 15);
    const T *pb = (const T *)a.B + (n < a.N ? n : a.N - 1) * a.ldb + E * (l >> 4);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    V fb[2][U], fa[2][U];
    auto load = [&](int64_t q, V (&b_)[U], V (&a_)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) b_[u] = row_frag<ODD>(pb + (q * U + u) * D, E);
#pragma unroll
      for (int u = 0; u < U; ++u) a_[u] = row_frag<ODD>(pa + (q * U + u) * D, E);
    };
    auto mul = [&](const V (&b_)[U], const V (&a_)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) acc = mul_frag(b_[u], a_[u], acc);
    };
    if (kw < whole) load(kw, fb[0], fa[0]);
    for (int64_t q = kw; q < whole; q += 2 * KW) {
      if (q + KW < whole) load(q + KW, fb[1], fa[1]);
      mul(fb[0], fa[0]);
      if (q + 2 * KW < whole) load(q + 2 * KW, fb[0], fa[0]);
      if (q + KW < whole) mul(fb[1], fa[1]);
    }
    for (int64_t k = (whole * U + kw) * D; k < a.K; k += KW * D) {  // the rest, a fragment at a time
      const int64_t left = a.K - k - E * (l >> 4);
      acc = mul_frag(row_frag<ODD>(pb + k, left), row_frag<ODD>(pa + k, left), acc);
    }
    return acc;
  };
  auto stats = [&](int64_t g, f32x4 acc) {
    // lane l: row l % 16, columns n0 .. n0 + 3
    const int64_t n0 = g * 16 + 4 * (l >> 4);
    float m2 = -INFINITY, s2 = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n0 + e >= a.N) continue;
      if (t == n0 + e) epi.at_target[m] = acc[e];
      m2 = fmaxf(m2, acc[e]);
    }
    const float ref = safe_ref(m2);
#pragma unroll
    for (int e = 0; e < 4; ++e) s2 += n0 + e < a.N ? __expf(acc[e] - ref) : 0.f;
    join_stats(mx, s, m2, s2);
  };
  const int64_t g0 = (int64_t)blockIdx.x * NG + wave / KW;
  if constexpr (KW == 1) {
    for (int64_t g = g0; g < groups; g += (int64_t)gridDim.x * NG) stats(g, dot(g));
  } else {  // one group each; the parts of its k, summed in wave order by its first wave
    __shared__ f32x4 red[8][64];
    f32x4 acc = dot(g0);
    red[wave][l] = acc;
    __syncthreads();
    if (kw == 0 && g0 < groups) {
#pragma unroll
      for (int w = 1; w < KW; ++w) acc += red[wave + w][l];
      stats(g0, acc);
    }
  }
#pragma unroll
  for (int o = 16; o <= 32; o <<= 1) {
    const float m2 = __shfl_xor(mx, o), s2 = __shfl_xor(s, o);
    join_stats(mx, s, m2, s2);
  }
  if (l < 16) st[wave][l] = make_float2(mx, s);
  __syncthreads();
  if (threadIdx.x < a.M) {
    float2 p = st[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) join_stats(p.x, p.y, st[w][threadIdx.x].x, st[w][threadIdx.x].y);
    epi.part[(int64_t)blockIdx.x * a.M + threadIdx.x] = p;
  }
}

// lse and loss from the partials [tiles][n]: C rows per turn of a workgroup of 256, 256 / C threads
// per row (16 rows read whole 128-byte lines; few rows take all threads each).  The grid is capped
// and walks the rows: one workgroup per 16 of 2^28 rows would be more than a grid holds.
template <int C>
__global__ __launch_bounds__(256) void k_xent_join(const float2 *part, int64_t tiles, int64_t n, const int32_t *target,
                                                   int64_t vocab, const float *at_target, float *loss, float *lse) {
  constexpr int Q = 256 / C;
  __shared__ float2 red[Q][C];
  const int c = threadIdx.x % C, q = threadIdx.x / C;
  for (int64_t row0 = (int64_t)blockIdx.x * C; row0 < n; row0 += (int64_t)gridDim.x * C) {
    const int64_t row = row0 + c;
    float m = -INFINITY, s = 0.f;
    if (row < n)
      for (int64_t t = q; t < tiles; t += Q) {
        const float2 p = part[t * n + row];
        join_stats(m, s, p.x, p.y);
      }
    __syncthreads();  // the turn before has been read
    red[q][c] = make_float2(m, s);
#pragma unroll
    for (int o = Q / 2; o; o >>= 1) {
      __syncthreads();
      if (q < o) {
        join_stats(m, s, red[q + o][c].x, red[q + o][c].y);
        red[q][c] = make_float2(m, s);
      }
    }
    if (q || row >= n) continue;
    const float z = safe_ref(m) + logf(s);
    lse[row] = z;
    const int32_t t = target[row];
    loss[row] = t >= 0 && t < vocab ? z - at_target[row] : 0.f;
  }
}

namespace {

int64_t round8(int64_t v) { return (v + 7) & ~(int64_t)7; }

// Vocabulary entries per piece of the backward: dl of a piece takes at most 512 MB (more
// only where 2048 entries already do), a multiple of 256 entries.
int64_t piece_of(const XentDesc &d) {
  const int64_t es = d.dt == POETX_F32 ? 4 : 2;
  int64_t p = ((int64_t)512 << 20) / (d.n * es) & ~(int64_t)255;
  if (p < 2048) p = 2048;
  if (p > kMaxWidth) p = kMaxWidth;  // a row stride of the products that read dl
  return p < d.v ? p : d.v;
}

// A bf16 operand whose rows are not a multiple of 16 bytes is read from padded copies: h
// whole, W one piece at a time.
bool pads(const XentDesc &d) { return d.dt == POETX_BF16 && d.d % 8; }

struct Operands {
  const void *h = nullptr;
  int64_t ld = 0;
  void *wp = nullptr;  // one padded piece of W
};
Operands operands(const XentDesc &d, int64_t piece, Arena &ar, PackList &l) {
  Operands o{d.h, d.d, nullptr};
  if (!pads(d)) return o;
  o.ld = round8(d.d);
  void *hp = ar.take((size_t)d.n * o.ld * 2);
  o.wp = ar.take((size_t)piece * o.ld * 2);
  o.h = hp;
  l.add({d.h, d.n, d.d, hp, o.ld, nullptr, 0});
  return o;
}
// The piece of W from v0 on, after the copies still to be made (h's, before the first piece).
int w_piece(const XentDesc &d, const Operands &o, int64_t v0, int64_t vc, PackList &l, hipStream_t s, const void **w) {
  const int64_t es = d.dt == POETX_F32 ? 4 : 2;
  *w = (const char *)d.w + v0 * d.d * es;
  if (o.wp) {
    l.add({*w, vc, d.d, o.wp, o.ld, nullptr, 0});
    *w = o.wp;
  }
  return pack_rows(l, d.dt, s);
}

MmDesc logits_desc(const XentDesc &d, const Operands &o, const void *w, int64_t vc, const char *name,
                   const char *large) {
  MmDesc m;
  m.M = d.n; m.N = vc; m.K = pads(d) ? o.ld : d.d; m.name = name; m.large = large;
  m.A = o.h; m.lda = o.ld; m.B = w; m.ldb = o.ld;
  return m;
}

// dh and dW of a piece of vc entries; `flip`: dW goes its own way
MmTwo products(const XentDesc &d, int64_t vc, bool flip) {
  return mm_two(d.dh ? d.n : 0, d.d, vc, d.dw && !flip ? vc : 0, d.d, d.n, d.dt);
}

template <typename T>
int bwd_t(const XentDesc &d, Arena &ar, bool measure, hipStream_t s) {
  const int64_t piece = piece_of(d);
  PackList l;
  const Operands o = operands(d, piece, ar, l);
  // dW reads h with the rows that take no part as zeros: their dl is zero, but zero times an
  // infinity or a NaN in such a row would not be.  The copy is transposed where the product's
  // kernel gains by it.
  const int64_t last = d.v % piece ? d.v % piece : piece;
  const bool flip = sizeof(T) == 2 && d.dw && dw_flips(piece, d.d, d.n, d.dt) && dw_flips(last, d.d, d.n, d.dt);
  const int64_t ldt = round8(d.n);
  void *hz = nullptr;
  if (d.dw) {
    hz = ar.take((flip ? (size_t)d.d * ldt : (size_t)d.n * o.ld) * sizeof(T));
    if (!flip) l.add({d.h, d.n, d.d, hz, o.ld, d.target, d.v});
    else if (!measure) POETX_TRY(pack_rows_t(d.h, d.n, d.d, hz, ldt, d.target, d.v, s));
  }
  float *scale = sizeof(T) == 2 ? (float *)ar.take(4) : nullptr;
  if (scale && !measure)
    POETX_TRY(launch_k("xent_scale", s, k_xent_scale, dim3(1), dim3(1024), 0, d.dloss, d.target, d.n, d.v, scale));
  const int64_t ldl = sizeof(T) == 2 ? round8(piece) : piece;
  T *dl = (T *)ar.take((size_t)d.n * ldl * sizeof(T));
  float *sum = d.dh && piece < d.v ? (float *)ar.take((size_t)d.n * d.d * 4) : nullptr;
  // partials of split products: of whole pieces and of the last one
  size_t part_bytes = 0, part_w_bytes = 0;
  const int64_t kd = pads(d) ? o.ld : d.d;
  for (const int64_t vc : {piece, last}) {
    const size_t l = mm_plan(d.n, vc, kd, d.dt).part_bytes;
    part_bytes = l > part_bytes ? l : part_bytes;
    const MmTwo q = products(d, vc, flip);
    part_bytes = q.a.part_bytes > part_bytes ? q.a.part_bytes : part_bytes;
    part_w_bytes = q.b.part_bytes > part_w_bytes ? q.b.part_bytes : part_w_bytes;
  }
  float *part = part_bytes ? (float *)ar.take(part_bytes) : nullptr;
  float *part_w = part_w_bytes ? (float *)ar.take(part_w_bytes) : nullptr;
  if (measure) return POETX_OK;
  for (int64_t v0 = 0; v0 < d.v; v0 += piece) {
    const int64_t vc = d.v - v0 < piece ? d.v - v0 : piece;
    const void *w = nullptr;
    POETX_TRY(w_piece(d, o, v0, vc, l, s, &w));
    const MmDesc m = logits_desc(d, o, w, vc, "xent_dlogits", "xent_dlogits_large");
    POETX_TRY((mm_run<T, false, false>(m, mm_plan(m.M, m.N, m.K, d.dt), part,
                                    XentDl<T>{dl, ldl, d.target, d.lse_in, d.dloss, scale, v0, d.v}, s)));
    const MmTwo q = products(d, vc, flip);
    const XentDh<T> eh{sum, (T *)d.dh, scale, d.target, d.v, d.d, v0 == 0, v0 + vc == d.v};
    const XentDw<T> ew{d.dw ? (T *)d.dw + v0 * d.d : nullptr, scale, d.d};
    MmDesc gh, gw;
    gh.M = d.n; gh.N = d.d; gh.K = vc; gh.name = "xent_dh"; gh.large = "xent_dh_large";
    gh.A = dl; gh.lda = ldl; gh.B = w; gh.ldb = o.ld;
    gw.M = vc; gw.N = d.d; gw.K = d.n; gw.name = "xent_dw"; gw.large = "xent_dw_large";
    gw.A = dl; gw.lda = ldl; gw.B = hz; gw.ldb = o.ld;
    if (q.pair) {
      POETX_TRY(mm_run_pair<T>("xent_dh_dw", gh, q.a, part, eh, gw, q.b, part_w, ew, {}, s));
      continue;
    }
    if (d.dh) POETX_TRY((mm_run<T, false, true>(gh, q.a, part, eh, s)));
    if constexpr (sizeof(T) == 2) {
      if (flip) {
        MmDesc g;
        g.M = d.d; g.N = vc; g.K = d.n; g.large = "xent_dw_large";
        g.A = hz; g.lda = ldt; g.B = dl; g.ldb = ldl;
        POETX_TRY(mm_run_flipped(g, ew, s));
      }
    }
    if (d.dw && !flip) POETX_TRY((mm_run<T, true, true>(gw, q.b, part_w, ew, s)));
  }
  return POETX_OK;
}

template <typename T>
int fwd_t(const XentDesc &d, Arena &ar, bool measure, hipStream_t s) {
  const int64_t cus = device_cus() > 0 ? device_cus() : 256;
  float *at = (float *)ar.take((size_t)d.n * 4);
  int64_t tiles = 0;
  float2 *part = nullptr;
  if (d.n <= 16) {
    const int64_t groups = cdiv(d.v, 16);
    // Waves that share a group's k: all eight while that makes at most two workgroups per CU,
    // two while a wave per group would load the CUs unevenly.  With 1, 2 and 8: 1734 rows of 3200
    // float32 64, 35 and 15 us; 12000 of 4096 93, 51 and 51; 42114 of 4608 248, 190 and 197;
    // 131072 of 4096 396, 411 and 480.
    const int64_t share = groups <= 2 * cus ? 8 : groups <= 12 * cus ? 2 : 1;
    tiles = cdiv(groups * share, 8);  // workgroups
    if (share == 1 && tiles > 2 * cus) tiles = 2 * cus;
    part = (float2 *)ar.take((size_t)tiles * d.n * 8);
    if (measure) return POETX_OK;
    const MmArgs a{d.n, d.v, d.d, d.h, d.d, d.w, d.d, 1, 1, 1, d.d};
    constexpr bool B16 = sizeof(T) == 2;
    auto kern = share == 8   ? k_xent_few<T, 8, false>
                : share == 2 ? k_xent_few<T, 2, false>
                             : k_xent_few<T, 1, false>;
    if (B16 && d.d % 2)
      kern = share == 8 ? k_xent_few<T, 8, B16> : share == 2 ? k_xent_few<T, 2, B16> : k_xent_few<T, 1, B16>;
    POETX_TRY(launch_k("xent_few", s, kern, dim3((unsigned)tiles), dim3(512), 0, a,
                       XentStats{part, d.target, at, 0, 0}));
  } else {
    const int64_t piece = pads(d) ? piece_of(d) : d.v;
    PackList l;
    const Operands o = operands(d, piece, ar, l);
    // one row of statistics per n-tile of every piece (pieces are multiples of the tile width;
    // 256 columns where the product is split over k)
    const int64_t kd = pads(d) ? o.ld : d.d;
    size_t split_bytes = 0;
    for (int64_t v0 = 0; v0 < d.v; v0 += piece) {
      const int64_t vc = d.v - v0 < piece ? d.v - v0 : piece;
      const MmPlan p = mm_plan(d.n, vc, kd, d.dt, true, false);
      tiles += p.splits > 1 ? cdiv(vc, 256) : p.tiles_n;
      split_bytes = p.part_bytes > split_bytes ? p.part_bytes : split_bytes;
    }
    part = (float2 *)ar.take((size_t)tiles * d.n * 8);
    float *split = split_bytes ? (float *)ar.take(split_bytes) : nullptr;
    if (measure) return POETX_OK;
    int64_t t0 = 0;
    for (int64_t v0 = 0; v0 < d.v; v0 += piece) {
      const int64_t vc = d.v - v0 < piece ? d.v - v0 : piece;
      const void *w = nullptr;
      POETX_TRY(w_piece(d, o, v0, vc, l, s, &w));
      const MmDesc m = logits_desc(d, o, w, vc, "xent_fwd", "xent_fwd_large");
      const MmPlan p = mm_plan(m.M, m.N, m.K, d.dt, true, false);
      const XentStats epi{part, d.target, at, v0, (int)t0};
      POETX_TRY((mm_run<T, false, false>(m, p, split, epi, s)));
      if (p.splits > 1)
        POETX_TRY(launch_k("xent_parts", s, k_xent_parts, dim3((unsigned)cdiv(vc, 256), (unsigned)cdiv(d.n, 4)),
                           dim3(256), 0, (const float *)split, (int)p.splits, d.n, vc, epi));
      t0 += p.splits > 1 ? cdiv(vc, 256) : p.tiles_n;
    }
  }
  if (d.n <= 256)
    return launch_k("xent_join", s, k_xent_join<1>, dim3((unsigned)d.n), dim3(256), 0, (const float2 *)part, tiles,
                    d.n, d.target, d.v, (const float *)at, d.loss, d.lse);
  const int64_t turns = cdiv(d.n, 16);
  return launch_k("xent_join", s, k_xent_join<16>, dim3((unsigned)(turns < 65536 ? turns : 65536)), dim3(256), 0,
                  (const float2 *)part, tiles, d.n, d.target, d.v, (const float *)at, d.loss, d.lse);
}

}  // namespace

int xent_forward(const XentDesc &d, Arena &ar, bool measure, hipStream_t s) {
  if (d.n == 0) return POETX_OK;
  return d.dt == POETX_F32 ? fwd_t<float>(d, ar, measure, s) : fwd_t<bf16_t>(d, ar, measure, s);
}

int xent_backward(const XentDesc &d, Arena &ar, bool measure, hipStream_t s) {
  if (d.n == 0) return measure || !d.dw ? POETX_OK : fill_zero(d.dw, d.v * d.d, d.dt, s);
  return d.dt == POETX_F32 ? bwd_t<float>(d, ar, measure, s) : bwd_t<bf16_t>(d, ar, measure, s);
}

}  // namespace poetx
