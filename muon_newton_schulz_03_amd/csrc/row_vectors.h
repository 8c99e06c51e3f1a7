// Rows of bf16 or fp32 elements in vectors of 16 bytes: loads and stores that
// the row operators (layer norm, embedding) share.
#pragma once

#include "device_common.h"

namespace muon {

// --------------------------------------------------------------- elements --
// A row is read and written in vectors of 16 bytes, wherever it starts: global
// accesses of gfx950 need no alignment, and on rows of 1001 fp32 elements
// 16-byte accesses off their boundaries take half the time of 4-byte ones.
// The types below only promise an element's alignment.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

template <class T, int N>
__device__ __forceinline__ void load_n(const T* p, float* v) {
  if constexpr (sizeof(T) == 2 && N == 8) {
    unpack8_bf16(*gv<u32x4_any>(p), v);
  } else if constexpr (sizeof(T) == 2) {
    unpack4_bf16(*gv<u32x2_any>(p), v);
  } else {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const f32x4 r = *gv<f32x4_any>(p + 4 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] = r[e];
    }
  }
}
template <class T, int N>
__device__ __forceinline__ void store_n(T* p, const float* v) {
  if constexpr (sizeof(T) == 2 && N == 8) {
    *gv<u32x4_any>(p) = pack8_bf16(v);
  } else if constexpr (sizeof(T) == 2) {
    *gv<u32x2_any>(p) = pack4_bf16(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int q = 0; q < N / 4; ++q)
      *gv<f32x4_any>(p + 4 * q) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
  }
}
// N elements at p of which `n` are inside the row: the others read as 0 and
// are not written.  PART: rows are no whole number of vectors (without it n is
// N, and the loads of a row stay in one block of code: with the branch, a
// backward pass over 65536 x 768 took 77 us instead of 57).
template <class T, int N, bool PART>
__device__ __forceinline__ void load_part(const T* p, int n, float* v) {
  if (!PART || n >= N) return load_n<T, N>(p, v);
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = e < n ? (float)*gv<T>(p + e) : 0.f;
}
template <class T, int N, bool PART>
__device__ __forceinline__ void store_part(T* p, int n, const float* v) {
  if (!PART || n >= N) return store_n<T, N>(p, v);
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (e < n) *gv<T>(p + e) = (T)v[e];
}
// Parameters are bf16 or fp32 independently of the activations.
template <class P, int N, bool PART>
__device__ __forceinline__ void load_param(const void* p, int64_t at, int n, float* v, float none) {
  if (p) return load_part<P, N, PART>((const P*)p + at, n, v);
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = none;
}

}  // namespace muon
