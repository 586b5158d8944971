// Products C[m][n] = sum_k A(m, k) B(n, k) whose results go straight into an epilogue:
// the dense linear layer's and the cross entropy's kernels.  Internal to libpoetx.
//
// bf16 operands run on v_mfma_f32_16x16x32_bf16, float32 ones on v_mfma_f32_16x16x4f32,
// both with float32 accumulators.  An operand is k-contiguous (element (r, k) at
// base + r ld + k) or k-major (base + k ld + r).
//
// What a kernel does with its tile is an epilogue type:
//   kStats == false: put(c, m, n, v, nv) takes 8 (nv <= 8 valid) consecutive columns of row m;
//     the accumulators pass through a wave's own piece of LDS so that a row's 64 columns
//     leave as whole 128-byte lines.  c = cols(n, nv, rows): what a lane keeps for its 8
//     columns over all its rows.  kRows > 0: floats per row that stage(m0, M, i) supplies; the
//     kernel puts them into LDS for the tile's rows first (`rows` points at row m0's).
//   kStats == true: reduce() gets the whole tile's accumulators (row statistics).  A product
//     split over k leaves its partials to the caller then (no epilogue runs).
#pragma once

#include "lds_tiles.h"
#include "vec.h"

namespace poetx {

struct MmArgs {
  int64_t M, N, K;
  const void *A; int64_t lda;
  const void *B; int64_t ldb;
  int tiles_m, tiles_n;
  int splits;   // k ranges; split s covers k in [s kc, (s+1) kc)
  int64_t kc;   // a multiple of 64 when splits > 1
  // k_mm8: tiles at or past `full` (in tile order) are each shared by tail_splits workgroups,
  // k ranges of tail_kc; their float32 tiles go to tail_part[tile - full][range] (256 x 256)
  int full = 0x7fffffff, tail_splits = 1;
  int64_t tail_kc = 0;
  float *tail_part = nullptr;
};

namespace {

// Tile and split of a workgroup.  Workgroups go to the 8 XCDs round-robin; ids are dealt
// so that each XCD gets one contiguous run of the tile order (any count), in which groups
// of 4 m-tiles sweep n: the workgroups running together on an XCD share their panels in
// its L2.
struct MmTile { int tm, tn, split, tail; };  // tail: index of a shared tile, or -1
__device__ inline void tile_at(const MmArgs &a, int L, int &tm, int &tn) {
  const int GM = a.tiles_m < 4 ? a.tiles_m : 4, per = GM * a.tiles_n;
  const int grp = L / per, first = grp * GM, gm = a.tiles_m - first < GM ? a.tiles_m - first : GM, loc = L - grp * per;
  // divisions run on the vector ALU: back to scalars, so that operand bases stay uniform
  tm = __builtin_amdgcn_readfirstlane(first + loc % gm);
  tn = __builtin_amdgcn_readfirstlane(loc / gm);
}
__device__ inline MmTile mm_tile(const MmArgs &a, int id) {
  const int T = a.tiles_m * a.tiles_n;
  MmTile t;
  int L;
  if (id >= a.full) {
    const int u = (id - a.full) / a.tail_splits;
    t.tail = __builtin_amdgcn_readfirstlane(u);
    t.split = __builtin_amdgcn_readfirstlane(id - a.full - u * a.tail_splits);
    L = a.full + u;
  } else {
    const int tot = a.full < T ? a.full : T * a.splits, x = id & 7, q = tot >> 3, r = tot & 7;
    L = x * q + (x < r ? x : r) + (id >> 3);
    t.tail = -1;
    t.split = __builtin_amdgcn_readfirstlane(L / T);
    L -= t.split * T;
  }
  tile_at(a, L, t.tm, t.tn);
  return t;
}

// Global -> LDS loads of one operand's [R rows] x [64 k] stage.  k-contiguous: the base is
// the tile's first row; chunks of 8 k past the range read as zero (their offset is past
// the buffer), rows past the operand too.  k-major: the base moves with k.
constexpr int kPast = 0x7ffffff0;  // beyond every buffer extent used here

template <int R, int NW>
struct StageKC {
  static constexpr int INSTR = R / 8 / NW;
  int voff[INSTR];
  __amdgpu_buffer_rsrc_t rs;
  __device__ void init(const bf16_t *P, int64_t ld, int64_t row0, int64_t rows, int64_t kbeg) {
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t left = rows - row0 < R ? rows - row0 : R;
    rs = make_rsrc(P + row0 * ld, left * ld * 2);
#pragma unroll
    for (int i = 0; i < INSTR; ++i) {
      const int row = (w * INSTR + i) * 8 + (l >> 3);
      voff[i] = (int)((row * ld + kbeg) * 2) + (((l & 7) ^ kc_key<64>(row)) << 4);
    }
  }
  // step t (64 k); left: k of the range from this step on
  __device__ void issue(int t, int64_t left, bf16_t *tile, int i) const {
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), l = threadIdx.x & 63;
    int off = voff[i] + t * 128;
    if (left < 64) {
      const int row = (w * INSTR + i) * 8 + (l >> 3);
      if ((((l & 7) ^ kc_key<64>(row)) << 3) >= left) off = kPast;
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(tile + (w * INSTR + i) * 512), 16, off, 0, 0, 0);
  }
  __device__ void issue_all(int t, int64_t left, bf16_t *tile) const {
#pragma unroll
    for (int i = 0; i < INSTR; ++i) issue(t, left, tile, i);
  }
};

template <int R, int NW>
struct StageKM {
  static constexpr int CH = R / 8, RPI = 64 / CH, INSTR = 64 / RPI / NW;
  int voff[INSTR];
  const bf16_t *base;
  int64_t ld;
  __device__ void init(const bf16_t *P, int64_t ld_, int64_t col0, int64_t, int64_t kbeg) {
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    ld = ld_;
    base = P + kbeg * ld;
#pragma unroll
    for (int i = 0; i < INSTR; ++i) {
      const int row = (w * INSTR + i) * RPI + l / CH;
      voff[i] = (int)((row * ld + col0) * 2) + (((l % CH) ^ km_xor<R>(row)) << 4);
    }
  }
  __device__ void issue(int t, int64_t left, bf16_t *tile, int i) const {
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(base + (int64_t)t * 64 * ld, (left < 64 ? left : 64) * ld * 2);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(tile + (w * INSTR + i) * RPI * R), 16, voff[i], 0, 0, 0);
  }
  __device__ void issue_all(int t, int64_t left, bf16_t *tile) const {
#pragma unroll
    for (int i = 0; i < INSTR; ++i) issue(t, left, tile, i);
  }
};

// Accumulator layout of one 16 x 16 MFMA result with the operands swapped (B fragment first):
// lane l holds row l % 16; element e is column 4 (l / 16) + e.

// The accumulators of a wave's patch (FM x FN results), handed to the epilogue as rows.  One
// row of results at a time goes through `st`, this wave's own 16 x (columns + 4) floats.
template <int FM, int FN, class Epi>
__device__ inline void put_rows(const f32x4 (&acc)[FM][FN], int64_t m0, int64_t n0, int64_t M, int64_t N, float *st,
                                const Epi &epi, const float *rows = nullptr) {
  constexpr int R = 16, W = FN * R, LD = W + 4, LPR = W / 8, RPP = 64 / LPR;  // lanes per row, rows per pass
  const int l = threadIdx.x & 63, c = (l % LPR) * 8;
  const int64_t n = n0 + c;
  const int nv = N - n >= 8 ? 8 : N - n > 0 ? (int)(N - n) : 0;
  const auto ctx = epi.cols(n, nv, rows);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j) *(f32x4 *)(st + (l % R) * LD + R * j + 4 * (l / R)) = acc[i][j];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < R / RPP; ++p) {
      const int r = p * RPP + l / LPR;
      const f32x4 a = *(const f32x4 *)(st + r * LD + c), b = *(const f32x4 *)(st + r * LD + c + 4);
      const int64_t m = m0 + R * i + r;
      if (m < M && nv) {
        float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        epi.put(ctx, m, n, v, nv);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// The epilogue of a kernel's BM x BN tile; lds: free, at least 16 (columns + 4) floats per wave
// and kRows BM floats more.
template <int BM, int BN, int WGM, int WGN, int FM, int FN, class Epi>
__device__ inline void finish(const f32x4 (&acc)[FM][FN], const MmArgs &a, const MmTile &tile, float *lds,
                              const Epi &epi) {
  constexpr int R = 16, WTM = BM / WGM, WTN = BN / WGN;
  const int64_t m0 = (int64_t)tile.tm * BM, n0 = (int64_t)tile.tn * BN;
  if constexpr (Epi::kStats) {
    epi.template reduce<BM, BN, WGM, WGN>(acc, m0, n0, a.M, a.N, tile.tn, lds);
  } else {
    const int wave = threadIdx.x >> 6, wm = (wave / WGN) * WTM, wn = (wave % WGN) * WTN;
    float *rows = lds + WGM * WGN * R * (WTN + 4);
    if constexpr (Epi::kRows > 0) {
      for (int i = threadIdx.x; i < BM * Epi::kRows; i += 64 * WGM * WGN) rows[i] = epi.stage(m0, a.M, i);
      __syncthreads();
    }
    put_rows<FM, FN>(acc, m0 + wm, n0 + wn, a.M, a.N, lds + wave * R * (WTN + 4), epi.at(tile.split),
                     Epi::kRows > 0 ? rows + wm * Epi::kRows - (m0 + wm) * Epi::kRows : nullptr);
  }
}

}  // namespace

// Epilogue that only writes: C[m][n] in T, split s at C + s * stride.  Tag (every epilogue
// names one, as Tag_) keeps the kernels of two source files apart.
template <typename T, class Tag>
struct StoreEpi {
  static constexpr bool kStats = false;
  static constexpr int kRows = 0;
  using Tag_ = Tag;
  struct Cols {};
  T *C; int64_t ld, stride;
  __device__ Cols cols(int64_t, int, const float *) const { return {}; }
  __device__ StoreEpi at(int split) const { return StoreEpi{C + split * stride, ld, stride}; }
  __device__ void put(const Cols &, int64_t m, int64_t n, float (&v)[8], int nv) const { store8(C + m * ld + n, nv, v); }
};

// bf16 kernel of the smaller products: 128 x 128 tile over 2 x 2 waves (64 x 64 each), 64-deep k
// steps, two LDS stages filled by direct global -> LDS loads, one barrier per step, two
// workgroups per CU that fill each other's waits.  2048^3: 27-30 us, 0.6 PFLOP/s (the vendor
// library 21-27 us); a handful of tokens or columns is bound by the load latency of its k range.
template <int BM, int BN, int WGM, int WGN, bool AKM, bool BKM, class Epi>
__device__ inline void mm_body(const MmArgs &a, const Epi &epi, int id, bf16_t *smem) {
  constexpr int NW = WGM * WGN, BK = 64;
  constexpr int WTM = BM / WGM, WTN = BN / WGN, FM = WTM / 16, FN = WTN / 16;
  constexpr int AE = BM * BK, BE = BN * BK;

  const MmTile tile = mm_tile(a, id);
  const int64_t m0 = (int64_t)tile.tm * BM, n0 = (int64_t)tile.tn * BN;
  const int64_t kbeg = tile.split * a.kc, kend = a.splits > 1 && kbeg + a.kc < a.K ? kbeg + a.kc : a.K;
  const int wave = threadIdx.x >> 6;
  const int wm = (wave / WGN) * WTM, wn = (wave % WGN) * WTN;

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  using SA = typename std::conditional<AKM, StageKM<BM, NW>, StageKC<BM, NW>>::type;
  using SB = typename std::conditional<BKM, StageKM<BN, NW>, StageKC<BN, NW>>::type;
  SA sa;
  SB sb;
  sa.init((const bf16_t *)a.A, a.lda, m0, a.M, kbeg);
  sb.init((const bf16_t *)a.B, a.ldb, n0, a.N, kbeg);
  const int64_t span = kend - kbeg;
  const int nk = (int)((span + BK - 1) / BK);
  auto issue = [&](int t) {
    sa.issue_all(t, span - (int64_t)t * BK, smem + (t & 1) * AE);
    sb.issue_all(t, span - (int64_t)t * BK, smem + 2 * AE + (t & 1) * BE);
  };
  if (nk > 0) issue(0);
  for (int t = 0; t < nk; ++t) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();  // stage t is in LDS for every wave; the other stage is no longer read
    const bf16_t *ta = smem + (t & 1) * AE, *tb = smem + 2 * AE + (t & 1) * BE;
    bf16x8 fa[2][FM], fb[2][FN];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[h][i] = AKM ? frag_km<BM>(ta, wm + 16 * i, 32 * h) : frag_kc<BK>(ta, wm + 16 * i, 32 * h);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fb[h][j] = BKM ? frag_km<BN>(tb, wn + 16 * j, 32 * h) : frag_kc<BK>(tb, wn + 16 * j, 32 * h);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (t + 1 < nk) issue(t + 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          // operands swapped: lane l then holds C[m = l % 16][n = 4 (l / 16) + 0..3]
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[h][j], fa[h][i], acc[i][j], 0, 0, 0);
  }
  __syncthreads();  // every wave is done with the last stage: the epilogue reuses the LDS
  finish<BM, BN, WGM, WGN>(acc, a, tile, (float *)smem, epi);
}
template <int BM, int BN, int WGM, int WGN, bool AKM, bool BKM, class Epi>
__global__ __launch_bounds__(64 * WGM * WGN) void k_mm(MmArgs a, Epi epi) {
  extern __shared__ __align__(16) bf16_t smem[];
  mm_body<BM, BN, WGM, WGN, AKM, BKM>(a, epi, blockIdx.x, smem);
}

// 256 x 256 tile, 8 waves (2 x 4, 128 x 64 each), 64-deep k steps: the large products.
//
// The tile's operands are kept in LDS as half tiles of 128 rows (A0, A1, B0, B1; 16 KB each),
// two k steps of them.  A wave owns 64 rows of each A half and 32 columns of each B half, so a
// k step is two phases of 32 MFMAs, one per A half:
//
//     phase   reads             loads                multiplies
//       0     A0(t), B1(t)      A1(t+1), B0(t+2)     A0 B0, A0 B1
//       1     A1(t), B0(t+1)    A0(t+2), B1(t+2)     A1 B0, A1 B1
//
// The waves form two groups of four (one wave of each per SIMD); group 1 runs one barrier
// behind group 0, so while one group multiplies the other reads: the matrix cores of every
// SIMD stay fed.  Every half tile is loaded three phases before it is read, into LDS that was
// last read in the phase before.  A phase ends its reading part by waiting for its own LDS
// reads and for all but its 8 newest loads (two phases'), so after the barrier the halves that
// the next phase reads have landed for all waves, and those just read may be overwritten.
// Loads past the k range read zeros.
//
// What bounds it: the chip's power.  At 8192^3, 20 calls in a row, it runs at 1.45 PFLOP/s at best
// and 1.31 in the median with both operands k-contiguous (the vendor library 1.56 and 1.42), the
// matrix cores busy 0.82 of the time (library 0.87) at a clock that falls to about 1.4 GHz under
// either; with a k-major B 1.40 and 1.38 (library 1.36 and 1.24), with both k-major 1.33 and 1.32
// (those issue two 8-byte transposing LDS reads per fragment instead of one of 16 bytes).  Where
// the three forms ran at 1.47, 1.40 and 1.34, one phase of 16 MFMAs per pair of halves instead of
// one of 32 per A half gave 1.40, 1.30 and 1.25; 32 x 32 x 16 MFMAs in the same schedule were 2 to
// 6 % slower, four waves of 128 x 128 30 % (the compiler moves accumulators between register files).
template <int HALF_ROWS, bool KM>
struct Half;

// rows of a half tile: local row r of half h is tile row (r / RUN) 2 RUN + h RUN + r % RUN
// (RUN = 64 for A, 32 for B), so that a wave's rows of both halves are consecutive
template <int RUN>
struct Half<RUN, false> {
  int voff[2], step;
  int64_t span;
  __amdgpu_buffer_rsrc_t rs;
  __device__ void init(const bf16_t *P, int64_t ld, int64_t row0, int64_t rows, int64_t kbeg, int64_t span_) {
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t left = rows - row0 < 256 ? rows - row0 : 256;
    rs = make_rsrc(P + row0 * ld, left * ld * 2);
    step = (int)(RUN * ld * 2);
    span = span_;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (w * 2 + i) * 8 + (l >> 3), row = (r / RUN) * 2 * RUN + r % RUN;
      voff[i] = (int)((row * ld + kbeg) * 2) + (((l & 7) ^ kc_key<64>(r)) << 4);
    }
  }
  // branch-free: a lane whose k lies past the range takes an offset past the buffer
  __device__ void issue(int t, int h, bf16_t *tile) const {
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), l = threadIdx.x & 63;
    const int64_t left64 = span - (int64_t)t * 64;
    const int left = left64 < 64 ? (int)left64 : 64;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (w * 2 + i) * 8 + (l >> 3);
      const int off = (((l & 7) ^ kc_key<64>(r)) << 3) < left ? voff[i] + t * 128 + h * step : kPast;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(tile + (w * 2 + i) * 512), 16, off, 0, 0, 0);
    }
  }
  __device__ static bf16x8 frag(const bf16_t *tile, int r0, int ks) { return frag_kc<64>(tile, r0, ks); }
};

template <int RUN>
struct Half<RUN, true> {
  int voff[2];
  const bf16_t *base;
  int64_t ld, span;
  __device__ void init(const bf16_t *P, int64_t ld_, int64_t col0, int64_t, int64_t kbeg, int64_t span_) {
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    ld = ld_;
    span = span_;
    base = P + kbeg * ld;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (w * 2 + i) * 4 + (l >> 4), c = ((l & 15) ^ km_xor<128>(row)) * 8;
      voff[i] = (int)((row * ld + col0 + (c / RUN) * 2 * RUN + c % RUN) * 2);
    }
  }
  __device__ void issue(int t, int h, bf16_t *tile) const {
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t left = span - (int64_t)t * 64;
    const __amdgpu_buffer_rsrc_t rs =
        make_rsrc(base + (int64_t)t * 64 * ld, (left < 0 ? 0 : left < 64 ? left : 64) * ld * 2);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(tile + (w * 2 + i) * 512), 16, voff[i] + h * RUN * 2, 0,
                                               0, 0);
  }
  __device__ static bf16x8 frag(const bf16_t *tile, int r0, int ks) { return frag_km<128>(tile, r0, ks); }
};

namespace {
// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ inline void wait_vm_lds() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (((N >> 4) & 3) << 14));
}
// a barrier that nothing is moved across and that waits for no memory operation by itself
__device__ inline void phase_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
}  // namespace

// FLIP: the results leave as C^T, rows n and columns m: the roles of the operands (128 rows of
// A and 64 of B per wave) are then the caller's choice.
template <bool AKM, bool BKM, bool FLIP, class Epi>
__global__ __launch_bounds__(512) void k_mm8(MmArgs a, Epi epi) {
  constexpr int HE = 128 * 64, FM = 8, FN = 4;  // elements of a half tile; 16 x 16 results per wave
  extern __shared__ __align__(16) bf16_t smem[];  // [A0 A1 B0 B1][2 steps]
  const MmTile tile = mm_tile(a, blockIdx.x);
  const int64_t m0 = (int64_t)tile.tm * 256, n0 = (int64_t)tile.tn * 256;
  const int64_t kc = tile.tail >= 0 ? a.tail_kc : a.splits > 1 ? a.kc : a.K;
  const int64_t kbeg = tile.split * kc, kend = kbeg + kc < a.K ? kbeg + kc : a.K;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wr = wave >> 2, wc = wave & 3;

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  using HA = Half<64, AKM>;
  using HB = Half<32, BKM>;
  HA ha;
  HB hb;
  ha.init((const bf16_t *)a.A, a.lda, m0, a.M, kbeg, kend - kbeg);
  hb.init((const bf16_t *)a.B, a.ldb, n0, a.N, kbeg, kend - kbeg);
  const int nk = (int)((kend - kbeg + 63) / 64);
  // all of A's halves within 64 KB of one base, and all of B's: the reach of a DS offset
  auto sA = [&](int s, int h) { return smem + (2 * h + s) * HE; };
  auto sB = [&](int s, int h) { return smem + (4 + 2 * h + s) * HE; };

  bf16x8 fa[2][4], fb0[2][2][2], fb1[2][2];  // [32-deep half of the step][fragment]; fb0 by step parity
  auto read_a = [&](const bf16_t *t) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) fa[q][i] = HA::frag(t, wr * 64 + 16 * i, 32 * q);
  };
  auto read_b = [&](const bf16_t *t, bf16x8 (&f)[2][2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j) f[q][j] = HB::frag(t, wc * 32 + 16 * j, 32 * q);
  };
  // phase P of k step t, whose halves are in LDS buffer S = t % 2
  auto phase = [&](auto pc, auto sc, int t) {
    constexpr int P = decltype(pc)::value, S = decltype(sc)::value;
    read_a(sA(S, P));
    if constexpr (P == 0) {
      read_b(sB(S, 1), fb1);
      ha.issue(t + 1, 1, sA(S ^ 1, 1));
      hb.issue(t + 2, 0, sB(S, 0));
    } else {
      read_b(sB(S ^ 1, 0), fb0[S ^ 1]);
      ha.issue(t + 2, 0, sA(S, 0));
      hb.issue(t + 2, 1, sB(S, 1));
    }
    wait_vm_lds<8>();
    phase_barrier();
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
        {
          // operands swapped (B first): lane l then holds C[m = l % 16][n = 4 (l / 16) + 0..3]
          const bf16x8 b = j < 2 ? fb0[S][q][j] : fb1[q][j - 2];
          acc[4 * P + i][j] = FLIP ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[q][i], b, acc[4 * P + i][j], 0, 0, 0)
                                   : __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, fa[q][i], acc[4 * P + i][j], 0, 0, 0);
        }
    __builtin_amdgcn_s_setprio(0);
    phase_barrier();
  };
  using I0_ = std::integral_constant<int, 0>;
  using I1_ = std::integral_constant<int, 1>;
  auto step = [&](auto sc, int t) {
    phase(I0_{}, sc, t);
    phase(I1_{}, sc, t);
  };

  // what the phases before the first would have loaded, in their order
  hb.issue(0, 0, sB(0, 0));
  ha.issue(0, 0, sA(0, 0));
  hb.issue(0, 1, sB(0, 1));
  ha.issue(0, 1, sA(0, 1));
  hb.issue(1, 0, sB(1, 0));
  ha.issue(1, 0, sA(1, 0));
  hb.issue(1, 1, sB(1, 1));
  wait_vmcnt<8>();  // B0(0), A0(0), B1(0) have landed
  phase_barrier();
  read_b(sB(0, 0), fb0[0]);
  wait_vm_lds<8>();
  phase_barrier();          // B0(0) is read: phase 0 loads into it
  if (wr) phase_barrier();  // group 1 runs one barrier behind
  int t = 0;
  for (; t + 1 < nk; t += 2) {
    step(I0_{}, t);
    step(I1_{}, t + 1);
  }
  if (t < nk) step(I0_{}, t);
  if (!wr) phase_barrier();
  __builtin_amdgcn_s_waitcnt(0);  // the loads past the range have written their zeros
  __syncthreads();                // the epilogue reuses the LDS
  if constexpr (!Epi::kStats) {
    if (tile.tail >= 0) {
      float *part = a.tail_part + ((int64_t)tile.tail * a.tail_splits + tile.split) * 65536;
      put_rows<FM, FN>(acc, wr * 128, wc * 64, 256, 256, (float *)smem + wave * 16 * 68,
                       StoreEpi<float, typename Epi::Tag_>{part, 256, 0});
      return;
    }
  }
  if constexpr (FLIP) {
    f32x4 tr[FN][FM];  // the same registers, rows and columns exchanged
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) tr[j][i] = acc[i][j];
    put_rows<FN, FM>(tr, n0 + wc * 64, m0 + wr * 128, a.N, a.M, (float *)smem + wave * 16 * 132, epi);
  } else {
    finish<256, 256, 2, 4>(acc, a, tile, (float *)smem, epi);
  }
}

// float32 kernel: BT x BT tile (128 or 64) over 2 x 2 waves, BK-deep k steps (16 or 32), two
// LDS stages, operands through registers (any alignment, any tail).  An MFMA of 16 x 16 takes
// four k; the four of one 16-deep block take k = 4 g + s (lane group g, MFMA s) instead of
// 4 s + g, so that a k-contiguous operand is read 16 bytes (its lane's four MFMAs) at a time
// from rows as they lie in memory, chunks XORed as in the bf16 tiles, and a k-major one, in
// rows of BT + 4 floats, meets four different 16-bank groups.  Bound by the float32 matrix
// rate (157 TFLOP/s).
constexpr int f32_lds(int bt, int bk) { return 4 * bk * (bt + 4); }  // floats
template <int BT, int BK, bool AKM, bool BKM, class Epi>
__device__ inline void mm_f32_body(const MmArgs &a, const Epi &epi, int id, float *smem) {
  constexpr int LD = BT + 4, ST = BK * LD, WT = BT / 2, F = WT / 16;  // a stage of either layout fits ST
  constexpr int PC = BT * BK / 4 / 256;  // 4-float pieces per thread and operand stage
  const MmTile tile = mm_tile(a, id);
  const int64_t m0 = (int64_t)tile.tm * BT, n0 = (int64_t)tile.tn * BT;
  const int64_t kbeg = tile.split * a.kc, kend = a.splits > 1 && kbeg + a.kc < a.K ? kbeg + a.kc : a.K;
  const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63;
  const int wm = (wave >> 1) * WT, wn = (wave & 1) * WT;
  f32x4 acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Global loads go through a buffer that ends with the operand's valid rows, so what lies past
  // them reads as zero.  k-contiguous: the base is the tile's first row and only a last step
  // that is not whole needs its elements past k cleared; k-major: the base moves with k.
  const int64_t span = kend - kbeg;
  auto offsets = [&](int64_t ld, bool km, int (&off)[PC]) {
#pragma unroll
    for (int i = 0; i < PC; ++i) {
      const int e = tid + 256 * i;
      off[i] = km ? (int)((e / (BT / 4) * ld + e % (BT / 4) * 4) * 4)
                  : (int)((e / (BK / 4) * ld + e % (BK / 4) * 4) * 4);
    }
  };
  auto fetch = [&](const float *P, int64_t ld, int64_t r0, int64_t rows, bool km, int t, const int (&off)[PC],
                   f32x4 (&v)[PC]) {
    const int64_t left = span - (int64_t)t * BK;
    const int64_t nr = rows - r0 < BT ? rows - r0 : BT;
    const __amdgpu_buffer_rsrc_t rs =
        km ? make_rsrc(P + (kbeg + (int64_t)t * BK) * ld + r0, ((left < BK ? left : BK) * ld - r0) * 4)
           : make_rsrc(P + r0 * ld + kbeg + (int64_t)t * BK, (nr * ld - kbeg - (int64_t)t * BK) * 4);
#pragma unroll
    for (int i = 0; i < PC; ++i)
      v[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off[i], 0, 0));
    if (!km && left < BK) {
#pragma unroll
      for (int i = 0; i < PC; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if ((tid + 256 * i) % (BK / 4) * 4 + q >= left) v[i][q] = 0.f;
    }
  };
  auto stash = [&](float *st, bool km, const f32x4 (&v)[PC]) {
#pragma unroll
    for (int i = 0; i < PC; ++i) {
      const int e = tid + 256 * i;
      if (km) {
        *(f32x4 *)(st + e / (BT / 4) * LD + e % (BT / 4) * 4) = v[i];
      } else {
        const int r = e / (BK / 4), c = e % (BK / 4);
        *(f32x4 *)(st + r * BK + (c ^ kc_key<2 * BK>(r)) * 4) = v[i];
      }
    }
  };
  const float *A = (const float *)a.A, *B = (const float *)a.B;
  const int nk = (int)((span + BK - 1) / BK);
  f32x4 va[PC], vb[PC];
  int oa[PC], ob[PC];
  offsets(a.lda, AKM, oa);
  offsets(a.ldb, BKM, ob);
  if (nk > 0) {
    fetch(A, a.lda, m0, a.M, AKM, 0, oa, va);
    fetch(B, a.ldb, n0, a.N, BKM, 0, ob, vb);
  }
  for (int t = 0; t < nk; ++t) {
    float *ta = smem + (t & 1) * 2 * ST, *tb = ta + ST;
    stash(ta, AKM, va);
    stash(tb, BKM, vb);
    // one barrier per step: stage t-1 may still be read by a slower wave, stage t-2, whose
    // LDS this step has just overwritten, may not (its readers passed the last barrier)
    __syncthreads();
    if (t + 1 < nk) {
      fetch(A, a.lda, m0, a.M, AKM, t + 1, oa, va);
      fetch(B, a.ldb, n0, a.N, BKM, t + 1, ob, vb);
    }
    // the four MFMAs' elements of 16 rows from r0 in 16-deep block h
    auto frag = [&](const float *st, bool km, int r0, int h) {
      const int r = r0 + (l & 15), g = l >> 4;
      if (!km) return *(const f32x4 *)(st + r * BK + ((4 * h + g) ^ kc_key<2 * BK>(r)) * 4);
      f32x4 v;
#pragma unroll
      for (int s = 0; s < 4; ++s) v[s] = st[(16 * h + 4 * g + s) * LD + r];
      return v;
    };
#pragma unroll
    for (int h = 0; h < BK / 16; ++h) {
      f32x4 fa[F], fb[F];
#pragma unroll
      for (int i = 0; i < F; ++i) fa[i] = frag(ta, AKM, wm + 16 * i, h);
#pragma unroll
      for (int j = 0; j < F; ++j) fb[j] = frag(tb, BKM, wn + 16 * j, h);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < F; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j][s], fa[i][s], acc[i][j], 0, 0, 0);
    }
  }
  __syncthreads();
  finish<BT, BT, 2, 2>(acc, a, tile, smem, epi);
}
template <int BT, int BK, bool AKM, bool BKM, class Epi>
__global__ __launch_bounds__(256) void k_mm_f32(MmArgs a, Epi epi) {
  __shared__ __align__(16) float smem[f32_lds(BT, BK)];
  mm_f32_body<BT, BK, AKM, BKM>(a, epi, blockIdx.x, smem);
}

// An epilogue whose product may be split over k: partials where `part` is set.
template <class Epi>
struct MaybePart {
  static constexpr bool kStats = false;
  static constexpr int kRows = Epi::kRows;
  using Tag_ = typename Epi::Tag_;
  using Cols = typename Epi::Cols;
  Epi epi;
  float *part; int64_t N, stride;
  __device__ MaybePart at(int split) const { return MaybePart{epi, part ? part + split * stride : nullptr, N, stride}; }
  __device__ Cols cols(int64_t n, int nv, const float *rows) const { return epi.cols(n, nv, rows); }
  __device__ float stage(int64_t m0, int64_t M, int i) const { return epi.stage(m0, M, i); }
  __device__ void put(const Cols &c, int64_t m, int64_t n, float (&v)[8], int nv) const {
    if (part) store8(part + m * N + n, nv, v);
    else epi.put(c, m, n, v, nv);
  }
};

// out[c] = sum over the parts [parts][cols], in a fixed order: C columns per workgroup, 16 threads
// per column each summing every 16th part.
struct SumArgs {
  const float *part = nullptr;
  int64_t parts = 0, cols = 0;
  float *out = nullptr;
};
template <int C>
__device__ inline void sum_parts_body(const SumArgs &a, int64_t id, float *red) {
  const int c = threadIdx.x % C, q = threadIdx.x / C;
  const int64_t col = id * C + c;
  float s = 0.f;
  if (col < a.cols)
    for (int64_t p = q; p < a.parts; p += 16) s += a.part[p * a.cols + col];
  red[q * C + c] = s;
  __syncthreads();
  if (q || col >= a.cols) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += red[i * C + c];
  a.out[col] = s;
}

// The two products of a backward pass, D W (W k-major) and D^T X (both k-major), in one launch:
// small ones fill the GPU together and wait for one launch and one fill instead of two.  513 x
// 1001 x 777 float32: 32 us for both.  The first has workgroups [0, ga), ga a multiple of 8 so that
// both deal their tiles to the XCDs alike.
template <typename T, class EA, class EB>
__global__ __launch_bounds__(256) void k_mm_pair(MmArgs a, EA ea, MmArgs b, EB eb, SumArgs sum, int ga,
                                                 int gb) {
  extern __shared__ __align__(16) bf16_t smem[];
  const int id = (int)blockIdx.x;
  if (id < ga) {
    if (id >= a.tiles_m * a.tiles_n * a.splits) return;
    if constexpr (sizeof(T) == 4) mm_f32_body<64, 32, false, true>(a, ea, id, (float *)smem);
    else mm_body<128, 128, 2, 2, false, true>(a, ea, id, smem);
  } else if (id >= gb) {
    sum_parts_body<16>(sum, id - gb, (float *)smem);
  } else {
    if constexpr (sizeof(T) == 4) mm_f32_body<64, 32, true, true>(b, eb, id - ga, (float *)smem);
    else mm_body<128, 128, 2, 2, true, true>(b, eb, id - ga, smem);
  }
}

// 16 bytes of an operand row as an MFMA fragment (8 bf16 or 4 floats), the first `left` in range.
// ODD: the rows are an odd number of bf16 apart.  A 16-byte load off its 4-byte alignment takes
// three times as long (14 tokens, 100793 rows of 641: 98 us, of 642: 40), so every load starts at
// the element before where the address is odd, the last element is loaded by itself, and the
// words are shifted into place.  (An odd address is never the operand's first.)
template <typename T> struct RowFrag;
template <> struct RowFrag<bf16_t> { using V = bf16x8; static constexpr int E = 8; };
template <> struct RowFrag<float> { using V = f32x4; static constexpr int E = 4; };
template <bool ODD, typename T>
__device__ inline typename RowFrag<T>::V row_frag(const T *p, int64_t left) {
  constexpr int E = RowFrag<T>::E, PER = E / 4;
  u32v4 u = {0u, 0u, 0u, 0u};
  if (left >= E) {
    if constexpr (ODD) {
      const uint32_t sh = (uint32_t)((uintptr_t)p & 2) * 8;
      u32v4 w;
      __builtin_memcpy(&w, p - (sh ? 1 : 0), 16);
      const uint32_t last = p[E - 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __builtin_amdgcn_alignbit(i < 3 ? w[i < 3 ? i + 1 : 3] : last, w[i], sh);
    } else {
      __builtin_memcpy(&u, p, 16);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < left) {
        if constexpr (PER == 2) u[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
        else u[e] = __float_as_uint(p[e]);
      }
  }
  return __builtin_bit_cast(typename RowFrag<T>::V, u);
}
// acc += the fragments' product over their four lane groups' k: 32 (one MFMA) or 16 (four, the
// s-th over element s of every group); operands swapped as everywhere
__device__ inline f32x4 mul_frag(bf16x8 b, bf16x8 a, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, acc, 0, 0, 0);
}
__device__ inline f32x4 mul_frag(f32x4 b, f32x4 a, f32x4 acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(b[s], a[s], acc, 0, 0, 0);
  return acc;
}

// Few rows (M <= 16, both operands k-contiguous): bound by reading B once (one token, 13824 x
// 5120 bf16: 26.7 us, 5.3 TB/s).  Each
// workgroup takes 16 NG rows of B; its 8 waves are NG groups of 8 / NG, which share a
// group's k range in turns of U fragments and are joined in LDS.  Operands go from memory into
// fragments: lane l reads 16 bytes of row l % 16 in its quarter (l / 16) of each fragment's k.
template <typename T, int NG, bool ODD, class Epi>
__global__ __launch_bounds__(512) void k_mm_few(MmArgs a, Epi epi) {
  constexpr int KW = 8 / NG, U = 4, E = RowFrag<T>::E, D = 4 * E;  // U fragments of D k in flight per wave
  __shared__ __align__(16) float red[8 * 16 * 20];  // the parts (8 x 256), then the rows (8 x 320)
  const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int ng = wave / KW, kw = wave % KW;
  const int64_t n0 = ((int64_t)blockIdx.x * NG + ng) * 16, n = n0 + (l & 15), m = l & 15;
  const T *pb = (const T *)a.B + (n < a.N ? n : a.N - 1) * a.ldb;
  const T *pa = (const T *)a.A + (m < a.M ? m : a.M - 1) * a.lda;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const int64_t steps = cdiv(a.K, D * U);
  for (int64_t t = kw; t < steps; t += KW) {
    const int64_t k0 = t * D * U + E * (l >> 4);
    typename RowFrag<T>::V fb[U], fa[U];
    if ((t + 1) * D * U <= a.K) {
#pragma unroll
      for (int u = 0; u < U; ++u) fb[u] = row_frag<ODD>(pb + k0 + D * u, E);
#pragma unroll
      for (int u = 0; u < U; ++u) fa[u] = row_frag<ODD>(pa + k0 + D * u, E);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        fb[u] = row_frag<ODD>(pb + k0 + D * u, a.K - k0 - D * u);
        fa[u] = row_frag<ODD>(pa + k0 + D * u, a.K - k0 - D * u);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc = mul_frag(fb[u], fa[u], acc);
  }
  // the k parts of a group, summed in wave order by its first wave
  if constexpr (KW > 1) {
    *(f32x4 *)(red + (wave * 64 + l) * 4) = acc;
    __syncthreads();
    if (kw == 0) {
#pragma unroll
      for (int w = 1; w < KW; ++w) acc += *(const f32x4 *)(red + ((wave + w) * 64 + l) * 4);
    }
    __syncthreads();
  }
  if (kw) return;
  // lane l: row l % 16, columns 4 (l / 16) .. +3; pairs of lanes make 8 columns
  float *st = red + wave * 16 * 20;
  *(f32x4 *)(st + (l & 15) * 20 + 4 * (l >> 4)) = acc;
  __builtin_amdgcn_wave_barrier();
  const int r = l >> 1, c = (l & 1) * 8;
  if (l < 32 && r < a.M && n0 + c < a.N) {
    const f32x4 p = *(const f32x4 *)(st + r * 20 + c), q = *(const f32x4 *)(st + r * 20 + c + 4);
    float v[8] = {p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
    const int nv = a.N - n0 - c >= 8 ? 8 : (int)(a.N - n0 - c);
    epi.put(epi.cols(n0 + c, nv, nullptr), r, n0 + c, v, nv);
  }
}

// Sum of the float32 partials of a split product, [splits][M][N] in split order, into the
// epilogue; one thread per 8 columns.
template <class Epi>
__device__ inline void join_body(const float *part, int splits, int64_t M, int64_t N, const Epi &epi, uint32_t id) {
  // (a split product has fewer than 2^32 results)
  const uint32_t cpr = (uint32_t)cdiv(N, 8), i = id * 256 + threadIdx.x;
  if (i >= M * cpr) return;
  const int64_t m = i / cpr, n = (int64_t)(i - (uint32_t)m * cpr) * 8;
  const int nv = N - n >= 8 ? 8 : (int)(N - n);
  float v[8];
  load8(part + m * N + n, nv, v);
#pragma unroll 4
  for (int s = 1; s < splits; ++s) {
    float w[8];
    load8(part + ((int64_t)s * M + m) * N + n, nv, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += w[e];
  }
  epi.put(epi.cols(n, nv, nullptr), m, n, v, nv);
}
template <class Epi>
__global__ __launch_bounds__(256) void k_mm_join(const float *part, int splits, int64_t M, int64_t N, Epi epi) {
  join_body(part, splits, M, N, epi, blockIdx.x);
}
// both products of a pair; the first has workgroups [0, ja)
template <class EA, class EB>
__global__ __launch_bounds__(256) void k_mm_join_pair(const float *pa, int sa, int64_t Ma, int64_t Na, EA ea,
                                                      const float *pb, int sb, int64_t Mb, int64_t Nb, EB eb,
                                                      uint32_t ja) {
  if (blockIdx.x < ja) join_body(pa, sa, Ma, Na, ea, blockIdx.x);
  else join_body(pb, sb, Mb, Nb, eb, blockIdx.x - ja);
}

// The same for the shared tiles of k_mm8: 32 workgroups per tile, one thread per 8 columns.
template <class Epi>
__global__ __launch_bounds__(256) void k_mm_tail(MmArgs a, Epi epi) {
  const int tail = blockIdx.x / 32, i = (int)(blockIdx.x % 32) * 256 + threadIdx.x;
  int tm, tn;
  tile_at(a, a.full + tail, tm, tn);
  const int64_t m = (int64_t)tm * 256 + i / 32, n = (int64_t)tn * 256 + i % 32 * 8;
  if (m >= a.M || n >= a.N) return;
  const float *p = a.tail_part + (int64_t)tail * a.tail_splits * 65536 + i * 8;
  float v[8];
  load8(p, 8, v);
#pragma unroll 2
  for (int s = 1; s < a.tail_splits; ++s) {
    float w[8];
    load8(p + (int64_t)s * 65536, 8, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += w[e];
  }
  const int nv = a.N - n >= 8 ? 8 : (int)(a.N - n);
  epi.put(epi.cols(n, nv, nullptr), m, n, v, nv);
}

// ------------------------------------------------------------------ host side ----
// A grid holds fewer than 2^32 threads: 2^24 - 1 workgroups of 256.  (The callers admit 2^22 tiles of
// 128 x 128; those of 256 x 256, of 512 threads, are no more, and 64 x 64 ones are taken where they
// are less than 3.75 times as many.)
constexpr int64_t kMaxTiles = ((int64_t)1 << 24) - 1;

// How a product is tiled (bt x bt results per workgroup), and over how many k ranges.
struct MmPlan {
  int64_t bt = 64, splits = 1, kc = 0;
  int64_t tiles_m = 0, tiles_n = 0;
  int64_t full = 0, tail_splits = 1, tail_kc = 0;  // 256 x 256 tiles from `full` on share their k
  size_t part_bytes = 0;  // workspace of a split product
};

struct MmDesc {
  int64_t M = 0, N = 0, K = 0;
  const void *A = nullptr; int64_t lda = 0;
  const void *B = nullptr; int64_t ldb = 0;
  const char *name = "mm", *large = "mm_large";  // launch labels: of the smaller and the larger tile
};

// float32: the kernels are bound by the matrix cores, so a CU's time is that of the tiles dealt to
// it: w = ceil(workgroups / CUs) of them, a 32-deep step of a 64 x 64 tile taking 0.55 us (0.83
// where the CU has one workgroup, which waits for its loads), a 16-deep one of 128 x 128 1.03 us.
// 128 x 128 tiles are taken where that comes out lower, which asks for enough of them to spread
// evenly (4096^3: 974-1114 us against 1078; 3000^3, 2.2 tiles per CU: 573 against 457).  Of the 64 x
// 64 ones, k is split where that spreads the work better by more than the partials' write, read
// and join (6 us, 5 TB/s) and a tenth of the time: 896 x 2573 x 3056, 2.2 tiles per CU, 166 us
// whole, 132 in 4 ranges; 64 x 4096 x 4096 105 and 33; 1024^3 stays whole, 29 against 34.
constexpr size_t kMaxPart = (size_t)64 << 20;
inline void plan_f32(int64_t M, int64_t N, int64_t K, int64_t cus, int halves, bool may_split, MmPlan &p) {
  const int64_t t64 = cdiv(M, 64) * cdiv(N, 64), t128 = cdiv(M, 128) * cdiv(N, 128);
  auto cost = [&](int64_t kc, int64_t sp) {
    const int64_t w = cdiv(t64 * sp, cus);
    return (double)cdiv(kc, 32) * (w == 1 ? 0.83 : 0.55 * w) + (sp > 1 ? 6 + (double)sp * M * N * 4 / 5e6 : 0);
  };
  const double whole = cost(K, 1);
  if (t128 >= 2 * cus && (double)cdiv(K, 16) * 1.03 * cdiv(t128, cus) < whole) {
    p.bt = 128;
    return;
  }
  if (!may_split || t64 >= 8 * cus) return;
  cus /= halves;
  double best = 0.9 * cost(K, 1);
  for (int64_t want = 2; want <= 32 && want <= K / 128; ++want) {
    const int64_t kc = cdiv(cdiv(K, want), 64) * 64, sp = cdiv(K, kc);
    const size_t bytes = (size_t)sp * M * N * 4;
    if (sp < 2 || bytes > kMaxPart || cost(kc, sp) >= best) continue;
    best = cost(kc, sp);
    p.kc = kc;
    p.splits = sp;
    p.part_bytes = bytes;
  }
}

// bf16: 256 x 256 tiles (one workgroup per CU), or 128 x 128 (two per CU, one of which multiplies
// while the other loads its first step or stores) for smaller products.  The larger are taken from
// 384 deep
//   - where they fill three quarters of the GPU (8192 x 4096 x 1024 with GELU 95 -> 81 us, x 512 63 ->
//     61; not x 128, 42 -> 43, nor 1102 x 40000 x 256, 67 -> 90),
//   - where 128 x 128 ones would begin a second round (3000^3 102 -> 62 us, 8192 x 1032 x 4096 105 ->
//     86, 2560 x 4096 x 512 equal),
//   - where k can be split over the GPU into ranges of 2304 at least (1024 x 1024 x 65536 175 -> 129 us,
//     768 x 3000 x 16384 80 -> 77; 2048 x 2048 x 8192, ranges of 2048, equal), or of 1792 where 128 x
//     128 ones load the CUs unevenly (weights not in the caches: 190 x 17792 x 5384 128 -> 76 us, 512 x
//     14336 x 4096 77 -> 66; ranges of 1024, 384 x 16000 x 2048, 40 -> 43).
// may_split, may_share: whether k may be split, the last round's tiles shared.  halves = 2: k is split
// as for half the GPU, which another product fills at the same time.
inline MmPlan mm_plan(int64_t M, int64_t N, int64_t K, int dt, bool may_split = true, bool may_share = true,
                      int halves = 1) {
  MmPlan p;
  if (M <= 0 || N <= 0) return p;  // nothing to launch
  const int64_t cus = device_cus() > 0 ? device_cus() : 256;
  p.kc = K;
  if (dt == POETX_F32) {
    plan_f32(M, N, K, cus, halves, may_split, p);
  } else {
    const int64_t t256 = cdiv(M, 256) * cdiv(N, 256), ranges = cus / t256 < 32 ? cus / t256 : 32;
    const int64_t t128 = cdiv(M, 128) * cdiv(N, 128);
    const bool many = 4 * t256 >= 3 * cus || t128 > 2 * cus;
    const bool deep = may_split && ranges >= 2 && K >= (t128 > cus ? 1792 : 2304) * ranges;
    p.bt = (many && K >= 384) || deep ? 256 : 128;
  }
  p.tiles_m = cdiv(M, p.bt);
  p.tiles_n = cdiv(N, p.bt);
  const int64_t tiles = p.tiles_m * p.tiles_n, slots = (p.bt == 256 ? cus : 2 * cus) / halves;
  // Too few bf16 tiles to fill the GPU: split k, each range at least 256 deep.  The partials'
  // join costs about 5 us, so a product with tiles for a quarter of the CUs and no more than 32
  // steps of 64 stays whole: 1024 x 2048 x 2048 24.5 -> 22.3 us, 1024^3 20 -> 14 us, while 64 x 4096
  // x 4096 takes 18 us split and 45 us whole.
  if (may_split && dt == POETX_BF16 && tiles < slots && !(4 * halves * tiles >= cus && K <= 32 * 64)) {
    int64_t sp = slots / tiles;
    if (sp > K / 256) sp = K / 256;
    if (sp > 32) sp = 32;
    if (sp >= 2) {
      p.kc = cdiv(cdiv(K, sp), 64) * 64;
      p.splits = cdiv(K, p.kc);
      if (p.splits < 2) { p.splits = 1; p.kc = K; }
      else p.part_bytes = (size_t)p.splits * M * N * 4;
    }
  }
  // 256 x 256 tiles past the last whole round of one per CU: where at most half the CUs would
  // have one, its k is shared by as many as fill the round.  Kept where the round's time (a CU
  // does 5.6 TFLOP/s) shrinks by more than the partials' write, read and join (4.5 TB/s, 6 us).
  p.full = tiles;
  const int64_t left = tiles % cus;
  if (may_split && may_share && p.bt == 256 && tiles > cus && left && 2 * left <= cus) {
    int64_t sp = cus / left;
    if (sp > K / 256) sp = K / 256;
    if (sp > 8) sp = 8;
    const double round_us = (double)K * 131072 / 5.6e6, parts_us = (double)left * sp * 524288 / 4.5e6 + 6;
    if (sp >= 2 && round_us * (sp - 1) / sp > 1.2 * parts_us) {
      p.full = tiles - left;
      p.tail_kc = cdiv(cdiv(K, sp), 64) * 64;
      p.tail_splits = cdiv(K, p.tail_kc);
      p.part_bytes = (size_t)left * p.tail_splits * 65536 * 4;
    }
  }
  return p;
}

template <bool AKM, bool BKM, class Epi>
int mm_launch(const MmArgs &a, int64_t bt, const MmDesc &d, const Epi &epi, hipStream_t s) {
  const int tiles = a.tiles_m * a.tiles_n;
  const dim3 grid((unsigned)(a.full < tiles ? a.full + (tiles - a.full) * a.tail_splits : tiles * a.splits));
  if (bt == 256) {
    constexpr size_t lds = (size_t)2 * 4 * 128 * 64 * 2;
    auto kern = &k_mm8<AKM, BKM, false, Epi>;
    static std::atomic<uint64_t> attr{0};  // dynamic-LDS limit, per device
    POETX_TRY(lds_limit(reinterpret_cast<const void *>(kern), lds, attr));
    return launch_k(d.large, s, kern, grid, dim3(512), lds, a, epi);
  }
  constexpr size_t lds = (size_t)2 * 2 * 128 * 64 * 2;
  auto kern = &k_mm<128, 128, 2, 2, AKM, BKM, Epi>;
  static std::atomic<uint64_t> attr{0};
  POETX_TRY(lds_limit(reinterpret_cast<const void *>(kern), lds, attr));
  return launch_k(d.name, s, kern, grid, dim3(256), lds, a, epi);
}

template <typename T, bool AKM, bool BKM, class Epi>
int mm_run_as(const MmArgs &a, const MmPlan &p, const MmDesc &d, const Epi &epi, hipStream_t s) {
  if constexpr (sizeof(T) == 4) {
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n * a.splits));
    if (p.bt == 128) return launch_k(d.large, s, k_mm_f32<128, 16, AKM, BKM, Epi>, grid, dim3(256), 0, a, epi);
    return launch_k(d.name, s, k_mm_f32<64, 32, AKM, BKM, Epi>, grid, dim3(256), 0, a, epi);
  } else {
    return mm_launch<AKM, BKM>(a, p.bt, d, epi, s);
  }
}

// The product of operands of type T (float or bf16_t) through its plan; `part` holds
// p.part_bytes when the plan splits k.
template <typename T, bool AKM, bool BKM, class Epi>
int mm_run(const MmDesc &d, const MmPlan &p, float *part, const Epi &epi, hipStream_t s) {
  if (d.M <= 0 || d.N <= 0) return POETX_OK;
  MmArgs a{d.M, d.N, d.K, d.A, d.lda, d.B, d.ldb, (int)p.tiles_m, (int)p.tiles_n, (int)p.splits, p.kc};
  const int64_t tiles = p.tiles_m * p.tiles_n;
  if (tiles * p.splits > kMaxTiles) return POETX_ERR_UNSUPPORTED;
  if constexpr (!Epi::kStats && sizeof(T) == 2) {
    if (p.full < tiles) {
      a.full = (int)p.full; a.tail_splits = (int)p.tail_splits; a.tail_kc = p.tail_kc; a.tail_part = part;
      POETX_TRY((mm_run_as<T, AKM, BKM>(a, p, d, epi, s)));
      return launch_k("mm_tail", s, k_mm_tail<Epi>, dim3((unsigned)((tiles - p.full) * 32)), dim3(256), 0, a, epi);
    }
  }
  if (p.splits == 1) return mm_run_as<T, AKM, BKM>(a, p, d, epi, s);
  POETX_TRY((mm_run_as<T, AKM, BKM>(a, p, d, StoreEpi<float, typename Epi::Tag_>{part, d.N, d.M * d.N}, s)));
  if constexpr (Epi::kStats) {
    return POETX_OK;
  } else {
    return launch_k("mm_join", s, k_mm_join<Epi>, dim3((unsigned)cdiv(d.M * cdiv(d.N, 8), 256)), dim3(256), 0,
                    (const float *)part, (int)p.splits, d.M, d.N, epi);
  }
}

// Plans of a backward pass's two products (D W, D^T X; one that is not wanted has no rows), and
// whether they run as a pair: both on the smaller tiles, and not slower so by the steps that their
// workgroups take (0.94 us for 64 deep in bf16, float32 as in plan_f32; a join 6 us, a launch 5).
// 7808 tokens, 768 -> 2816 bf16, where the pair would leave one product's k unsplit: 121 us apart, 137
// as a pair; 2112 tokens, 248 -> 9984 81 and 66; 145 tokens, 1807 -> 606 float32 34 and 30.
struct MmTwo {
  MmPlan a, b;
  bool pair = false;
};
inline MmTwo mm_two(int64_t Ma, int64_t Na, int64_t Ka, int64_t Mb, int64_t Nb, int64_t Kb, int dt) {
  MmTwo t;
  t.a = mm_plan(Ma, Na, Ka, dt);
  t.b = mm_plan(Mb, Nb, Kb, dt);
  const bool b16 = dt == POETX_BF16;
  const int64_t bt = b16 ? 128 : 64, cus = device_cus() > 0 ? device_cus() : 256;
  if (t.a.bt != bt || t.b.bt != bt || t.a.tiles_m == 0 || t.b.tiles_m == 0) return t;
  const MmPlan a = mm_plan(Ma, Na, Ka, dt, true, true, 2), b = mm_plan(Mb, Nb, Kb, dt, true, true, 2);
  auto wgs = [](const MmPlan &p) { return p.tiles_m * p.tiles_n * p.splits; };
  auto steps = [&](const MmPlan &p) { return cdiv(p.kc, b16 ? 64 : 32); };
  auto alone = [&](const MmPlan &p) {
    const int64_t w = cdiv(wgs(p), b16 ? 2 * cus : cus);
    return steps(p) * (b16 ? 0.94 * w : w == 1 ? 0.83 : 0.55 * w) + (p.splits > 1 ? 6 : 0);
  };
  const double longest = (b16 ? 0.94 : 0.83) * (steps(a) > steps(b) ? steps(a) : steps(b));
  const double shared = 1.1 * (b16 ? 0.47 : 0.55) * ((double)wgs(a) * steps(a) + (double)wgs(b) * steps(b)) / cus;
  const double both = (longest > shared ? longest : shared) + (a.splits > 1 || b.splits > 1 ? 6 : 0);
  if (both > alone(t.a) + alone(t.b) + 5 || wgs(a) + wgs(b) > kMaxTiles / 2) return t;  // one grid holds both
  t.a = a;
  t.b = b;
  t.pair = true;
  return t;
}
// The pair of mm_run<T, false, true>(da, ..) and mm_run<T, true, true>(db, ..); plans with halves = 2.
template <typename T, class EA, class EB>
int mm_run_pair(const char *name, const MmDesc &da, const MmPlan &pa, float *part_a, const EA &ea, const MmDesc &db,
                const MmPlan &pb, float *part_b, const EB &eb, const SumArgs &sum, hipStream_t s) {
  const int64_t na = pa.tiles_m * pa.tiles_n * pa.splits, nb = pb.tiles_m * pb.tiles_n * pb.splits;
  const int64_t ga = cdiv(na, 8) * 8;
  const int64_t ns = cdiv(sum.cols, 16);
  if (ga + nb + ns > kMaxTiles) return POETX_ERR_UNSUPPORTED;
  const MmArgs a{da.M, da.N, da.K, da.A, da.lda, da.B, da.ldb, (int)pa.tiles_m, (int)pa.tiles_n, (int)pa.splits, pa.kc};
  const MmArgs b{db.M, db.N, db.K, db.A, db.lda, db.B, db.ldb, (int)pb.tiles_m, (int)pb.tiles_n, (int)pb.splits, pb.kc};
  const bool sa = pa.splits > 1, sb = pb.splits > 1;
  constexpr size_t lds = sizeof(T) == 4 ? f32_lds(64, 32) * 4 : (size_t)2 * 2 * 128 * 64 * 2;
  auto kern = &k_mm_pair<T, MaybePart<EA>, MaybePart<EB>>;
  static std::atomic<uint64_t> attr{0};  // dynamic-LDS limit, per device
  POETX_TRY(lds_limit(reinterpret_cast<const void *>(kern), lds, attr));
  POETX_TRY(launch_k(name, s, kern, dim3((unsigned)(ga + nb + ns)), dim3(256), lds, a,
                     MaybePart<EA>{ea, sa ? part_a : nullptr, da.N, da.M * da.N}, b,
                     MaybePart<EB>{eb, sb ? part_b : nullptr, db.N, db.M * db.N}, sum, (int)ga, (int)(ga + nb)));
  if (!sa && !sb) return POETX_OK;
  const unsigned ja = sa ? (unsigned)cdiv(da.M * cdiv(da.N, 8), 256) : 0;
  const unsigned jb = sb ? (unsigned)cdiv(db.M * cdiv(db.N, 8), 256) : 0;
  return launch_k("mm_join", s, k_mm_join_pair<EA, EB>, dim3(ja + jb), dim3(256), 0, (const float *)part_a,
                  (int)pa.splits, da.M, da.N, ea, (const float *)part_b, (int)pb.splits, db.M, db.N, eb, (uint32_t)ja);
}

// dW = D^T X (D [K][M] and X [K][N], both k-major) for bf16: the kernels read a k-major operand
// with twice the LDS instructions of a k-contiguous one.  Where a transposed copy of X costs
// less than that (one pass over X, against a product M times as large), X^T takes the kernel's
// 128-row role k-contiguous and D its 64-row role.  M, N, K = 65536, 4096, 4096: 1790 us as it
// lies, 1560 us so; below about M = 8192 the copy eats the gain (8192 tokens, 4096 x 4096: 208 us,
// of which it would take 27).  K is a row stride of the copy: not past the widths whose offsets
// within a tile's rows fit 32 bits.
inline bool dw_flips(int64_t M, int64_t N, int64_t K, int dt) {
  const MmPlan p = mm_plan(N, M, K, dt, false);
  return dt == POETX_BF16 && M >= 8192 && K <= kMaxWidth && p.bt == 256;
}
// C^T of the product: A is X^T, [M][lda] with lda a multiple of 8 and zeros past K, B is D
template <class Epi>
int mm_run_flipped(const MmDesc &d, const Epi &epi, hipStream_t s) {
  const MmPlan p = mm_plan(d.M, d.N, d.K, POETX_BF16, false);
  const MmArgs a{d.M, d.N, d.K, d.A, d.lda, d.B, d.ldb, (int)p.tiles_m, (int)p.tiles_n, 1, d.K};
  if (p.tiles_m * p.tiles_n > kMaxTiles) return POETX_ERR_UNSUPPORTED;
  constexpr size_t lds = (size_t)2 * 4 * 128 * 64 * 2;
  auto kern = &k_mm8<false, true, true, Epi>;
  static std::atomic<uint64_t> attr{0};  // dynamic-LDS limit, per device
  POETX_TRY(lds_limit(reinterpret_cast<const void *>(kern), lds, attr));
  return launch_k(d.large, s, kern, dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(512), lds, a, epi);
}

}  // namespace poetx
