// Device helpers of the row-wise kernels and of the products' epilogues: 8-element loads
// and stores of any alignment, rounding to bf16, wave reductions.  Internal to libpoetx.
#pragma once

#include "common.h"

namespace poetx {

typedef float f32v4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));

namespace {

// Two floats rounded to nearest even (one v_cvt_pk_bf16_f32); NaN stays NaN, unlike
// f32_to_bf16, whose inputs are finite.
__device__ inline uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ inline bf16_t round_bf16(float f) { return __builtin_bit_cast(bf16_t, (__bf16)f); }

// Eight consecutive elements from p, the first nv of them in range (the others read as
// zero).  p is aligned to its element only: gfx950's vector memory takes 16-byte accesses
// at any such address, so rows of odd widths need no path of their own.
__device__ inline void load8(const bf16_t *p, int nv, float (&v)[8]) {
  if (nv >= 8) {
    u32v4 u;
    __builtin_memcpy(&u, p, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < nv ? bf16_to_f32(p[e]) : 0.f;
  }
}
__device__ inline void load8(const float *p, int nv, float (&v)[8]) {
  if (nv >= 8) {
    f32v4 a, b;
    __builtin_memcpy(&a, p, 16);
    __builtin_memcpy(&b, p + 4, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < nv ? p[e] : 0.f;
  }
}
__device__ inline void store8(bf16_t *p, int nv, const float (&v)[8]) {
  if (nv >= 8) {
    const u32v4 u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    __builtin_memcpy(p, &u, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < nv) p[e] = round_bf16(v[e]);
  }
}
__device__ inline void store8(float *p, int nv, const float (&v)[8]) {
  if (nv >= 8) {
    const f32v4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    __builtin_memcpy(p, &a, 16);
    __builtin_memcpy(p + 4, &b, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < nv) p[e] = v[e];
  }
}

// Eight elements as they lie in memory, so that a load can stay in flight before it is widened.
template <typename T> struct Raw8 { u32v4 u[sizeof(T) / 2]; };
template <typename T>
__device__ inline void load_raw(const T *p, int nv, Raw8<T> &r) {
  if (nv >= 8) {
    __builtin_memcpy(&r, p, sizeof(r));
  } else {
    float v[8];
    load8(p, nv, v);
    if constexpr (sizeof(T) == 2) {
      r.u[0] = u32v4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.u[e >> 2][e & 3] = __float_as_uint(v[e]);
    }
  }
}
template <typename T>
__device__ inline void widen(const Raw8<T> &r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (sizeof(T) == 2)
      v[e] = __uint_as_float(e & 1 ? r.u[0][e >> 1] & 0xffff0000u : r.u[0][e >> 1] << 16);
    else
      v[e] = __uint_as_float(r.u[e >> 2][e & 3]);
  }
}

// A parameter vector (gamma, beta, bias) stored as float32 or bf16.
struct ParamVec {
  const void *p;
  int bf16;
  __device__ void load(int64_t i, int nv, float (&v)[8]) const {
    if (bf16) load8((const bf16_t *)p + i, nv, v);
    else load8((const float *)p + i, nv, v);
  }
};

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

}  // namespace
}  // namespace poetx
