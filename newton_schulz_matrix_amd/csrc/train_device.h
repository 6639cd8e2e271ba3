// Device helpers of the operators around the matrix update: eight
// consecutive elements of a row as fp32, wavefront sums, typed scalars.
//
// A vector is loaded and stored with the alignment of its elements only:
// gfx950 runs in unaligned access mode, so a 16-byte access at any element
// address is one instruction. Rows of odd width or odd leading dimension
// therefore take the same path as aligned ones.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nsmi {

constexpr int VEC = 8;   // elements per lane and access

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[VEC]) {
  T r[VEC];
  __builtin_memcpy(r, p, sizeof(r));
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = static_cast<float>(r[e]);
}

template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[VEC]) {
  T r[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) r[e] = static_cast<T>(v[e]);
  __builtin_memcpy(p, r, sizeof(r));
}

// The first `left` (any number) of eight elements; the others read as 0.
template <class T>
__device__ __forceinline__ void load8_upto(const T* p, int left, float (&v)[VEC]) {
  if (left >= VEC) {
    load8(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = e < left ? static_cast<float>(p[e]) : 0.f;
  }
}

template <class T>
__device__ __forceinline__ void store8_upto(T* p, int left, const float (&v)[VEC]) {
  if (left >= VEC) {
    store8(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < left) p[e] = static_cast<T>(v[e]);
  }
}

// v as it reads back after being stored as T.
template <class T>
__device__ __forceinline__ float rounded(float v) {
  return static_cast<float>(static_cast<T>(v));
}

// Sum and maximum over the 64 lanes (every lane gets the result; the order is fixed).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

// One of three element types chosen at run time: the switch goes once around
// a whole kernel launch, on the host.
template <class F>
inline hipError_t by_type(int type, F f) {
  switch (type) {
    case 0: return f(float{});
    case 1: return f(__bf16{});
    default: return f(_Float16{});
  }
}

}  // namespace nsmi
