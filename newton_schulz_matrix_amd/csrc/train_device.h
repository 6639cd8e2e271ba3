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

// How a vector is read. ONCE marks data that a call reads a single time
// (non-temporal loads): large streams run at 6.5 instead of 6.1 TB/s with it,
// copied by workgroups of 256 threads that take 4 KB each, in order.
enum class Use { AGAIN, ONCE };

// Eight elements of type T as loaded. Loading and converting are separate
// steps, so that a kernel can have all the loads of several operands in
// flight before the first conversion waits for one.
// (any element's address; other types' memory)
typedef uint32_t Quad __attribute__((ext_vector_type(4), aligned(2), may_alias));
template <class T>
struct Raw {
  Quad q[sizeof(T) * VEC / 16];
};

template <Use U = Use::AGAIN, class T>
__device__ __forceinline__ Raw<T> fetch(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) {
    const Quad* from = reinterpret_cast<const Quad*>(p) + i;
    if constexpr (U == Use::ONCE) r.q[i] = __builtin_nontemporal_load(from);
    else r.q[i] = *from;
  }
  return r;
}

template <class T>
__device__ __forceinline__ void widen(const Raw<T>& raw, float (&v)[VEC]) {
  T r[VEC];
  __builtin_memcpy(r, &raw, sizeof(r));
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = static_cast<float>(r[e]);
}

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[VEC]) {
  widen(fetch(p), v);
}

// Stored as vectors by type: written as a copy of eight elements, it would be
// taken apart and merged with the element stores of store8_upto below, into
// two-byte and twelve-byte stores at two thirds of the rate.
// With ONCE the stores are non-temporal: for large outputs that this call does
// not read back. Eight 16-bit elements a lane make whole lines of a wave's store;
// in fp32 it is two stores of every second 16 bytes, which pays in some kernels and
// costs in others (measured beside each use).
template <Use U = Use::AGAIN, class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[VEC]) {
  T r[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) r[e] = static_cast<T>(v[e]);
  Quad q[sizeof(r) / 16];
  __builtin_memcpy(q, r, sizeof(r));
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) {
    Quad* to = reinterpret_cast<Quad*>(p) + i;
    if constexpr (U == Use::ONCE) __builtin_nontemporal_store(q[i], to);
    else *to = q[i];
  }
}

// The eight columns at `at` of a row of `dim`, in two steps. The vector that
// crosses the row's end is read so that it ends there and moved into place
// afterwards, and lanes past the row read its end too: every lane makes the
// same one access, without a branch. Elements past the row in the crossing
// vector come out as 0; a vector that begins past the row holds something else,
// finite or not, which the caller leaves out. Rows narrower than a vector
// (dim < VEC) are read by element in the second step.
template <Use U = Use::AGAIN, class T>
__device__ __forceinline__ Raw<T> fetch_at(const T* row, int dim, int at) {
  return fetch<U>(row + min(at, dim - VEC));
}
template <class T>
__device__ __forceinline__ void widen_ragged(const Raw<T>& raw, int dim, int at, float (&v)[VEC]) {
  widen(raw, v);
  const int past = max(at + VEC - dim, 0);
  if (!__any(past > 0 && past < VEC)) return;   // most waves have no vector that crosses
#pragma unroll
  for (int by = VEC / 2; by >= 1; by /= 2)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float from = e + by < VEC ? v[(e + by) % VEC] : 0.f;
      v[e] = past & by ? from : v[e];
    }
}
template <class T>
__device__ __forceinline__ void widen_narrow(const T* row, int dim, int at, float (&v)[VEC]) {
  float one[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) one[e] = static_cast<float>(row[min(e, dim - 1)]);
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = at + e < dim ? one[e] : 0.f;
}
template <class T>
__device__ __forceinline__ void widen_at(const Raw<T>& raw, const T* row, int dim, int at,
                                         float (&v)[VEC]) {
  if (dim < VEC) widen_narrow(row, dim, at, v);
  else if (dim % VEC == 0) widen(raw, v);
  else widen_ragged(raw, dim, at, v);
}

template <Use U = Use::AGAIN, class T>
__device__ __forceinline__ void store8_upto(T* p, int left, const float (&v)[VEC]) {
  if (left >= VEC) {
    store8<U>(p, v);
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

constexpr float FAR = 150.f;   // exp(-FAR) is 0 in fp32

// exp(x) by the hardware's 2^x, without the rounding of the product
// p = x log2(e): exp(x) = 2^p exp(x - p ln 2), where the second factor is 1 + c. That
// rounding is up to |x| half steps of the result. bf16 logits take few
// values, so the roundings of p do not average out over a row: left alone they
// put 2e-8 on its sum, much the same for every row, which the difference of
// two sequences' sums keeps. x is not below -FAR.
__device__ __forceinline__ float exp_exact(float x) {
  const float p = x * 1.442695041f;
  const float c = fmaf(p, 1.904654299e-9f, fmaf(-p, 0.693147182f, x));
  const float t = __builtin_amdgcn_exp2f(p);
  return fmaf(t, c, t);
}
// The same with ln 2 in one fp32 number, which is 1.9e-9 above it: a power of
// e^(1 - OF_E), so that sums of such powers are brought from one reference to another by
// them, and sum exp x is sum e^((1 - OF_E) x) plus OF_E times the sum of those terms times x.
constexpr double OF_E = 1.904654299e-9 * 1.442695041;
__device__ __forceinline__ float exp_near(float x) {
  const float p = x * 1.442695041f;
  const float t = __builtin_amdgcn_exp2f(p);
  return fmaf(t, fmaf(-p, 0.693147182f, x), t);
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
