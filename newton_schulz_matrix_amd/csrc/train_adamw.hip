// AdamW step of several tensors in one launch.
//
//   m <- b1 m + (1 - b1) g;  v <- b2 v + (1 - b2) g^2
//   w <- w - lr (decay w + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// Bound by memory: each of w, g, m, v is read once and each of w, m, v
// written once. The tensors' table is a kernel argument, so a step of small
// tensors is one launch and nothing else. Types differ by tensor; the
// switches on them are uniform over a workgroup, and all loads of an element
// group are issued before its first conversion.
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int THREADS = 256;
constexpr int GROUPS = 2;                              // vectors of a thread
constexpr int BLOCK_ELEMS = THREADS * VEC * GROUPS;

// Eight elements as loaded, in 16 or 32 bytes.
struct Raw {
  uint4 lo, hi;
};
__device__ __forceinline__ Raw load_raw(const void* p, int type, int64_t at) {
  Raw r;
  r.hi = make_uint4(0, 0, 0, 0);
  if (type == OUT_F32) {
    const float* f = static_cast<const float*>(p) + at;
    __builtin_memcpy(&r.lo, f, 16);
    __builtin_memcpy(&r.hi, f + 4, 16);
  } else {
    __builtin_memcpy(&r.lo, static_cast<const uint16_t*>(p) + at, 16);
  }
  return r;
}
__device__ __forceinline__ void widen(const Raw& r, int type, float (&v)[VEC]) {
  if (type == OUT_F32) {
    __builtin_memcpy(v, &r, 32);
  } else if (type == OUT_BF16) {
    __bf16 b[VEC];
    __builtin_memcpy(b, &r.lo, 16);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = static_cast<float>(b[e]);
  } else {
    _Float16 b[VEC];
    __builtin_memcpy(b, &r.lo, 16);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = static_cast<float>(b[e]);
  }
}
__device__ __forceinline__ void store_as(void* p, int type, int64_t at, const float (&v)[VEC]) {
  if (type == OUT_F32) store8(static_cast<float*>(p) + at, v);
  else if (type == OUT_BF16) store8(static_cast<__bf16*>(p) + at, v);
  else store8(static_cast<_Float16*>(p) + at, v);
}
__device__ __forceinline__ float load_one(const void* p, int type, int64_t at) {
  if (type == OUT_F32) return static_cast<const float*>(p)[at];
  if (type == OUT_BF16) return static_cast<float>(static_cast<const __bf16*>(p)[at]);
  return static_cast<float>(static_cast<const _Float16*>(p)[at]);
}
__device__ __forceinline__ void store_one(void* p, int type, int64_t at, float v) {
  if (type == OUT_F32) static_cast<float*>(p)[at] = v;
  else if (type == OUT_BF16) static_cast<__bf16*>(p)[at] = static_cast<__bf16>(v);
  else static_cast<_Float16*>(p)[at] = static_cast<_Float16>(v);
}

__device__ __forceinline__ void update(const AdamwArgs& a, float decay, float g, float& w,
                                       float& m, float& v) {
  m = fmaf(a.beta1, m, a.rest1 * g);
  v = fmaf(a.beta2, v, a.rest2 * g * g);
  const float root = fmaf(sqrtf(v), a.root_scale, a.eps);
  w = fmaf(-decay, w, w) - a.step_size * m / root;
}

__global__ __launch_bounds__(THREADS) void adamw_kernel(const AdamwArgs a) {
  int i = 0;
  while (i + 1 < a.count && a.t[i + 1].block_begin <= blockIdx.x) ++i;
  const AdamwTensor& t = a.t[i];
  const int64_t base = static_cast<int64_t>(blockIdx.x - t.block_begin) * BLOCK_ELEMS;
  const void* from = t.master ? t.master : t.param;
  const int from_type = t.master ? static_cast<int>(OUT_F32) : t.param_type;
  if (base + BLOCK_ELEMS <= t.elems) {
    Raw rw[GROUPS], rg[GROUPS], rm[GROUPS], rv[GROUPS];
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
      const int64_t at = base + (j * THREADS + threadIdx.x) * VEC;
      rg[j] = load_raw(t.grad, t.grad_type, at);
      rm[j] = load_raw(t.exp_avg, t.exp_avg_type, at);
      rv[j] = load_raw(t.exp_avg_sq, t.exp_avg_sq_type, at);
      rw[j] = load_raw(from, from_type, at);
    }
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
      const int64_t at = base + (j * THREADS + threadIdx.x) * VEC;
      float w[VEC], g[VEC], m[VEC], v[VEC];
      widen(rw[j], from_type, w);
      widen(rg[j], t.grad_type, g);
      widen(rm[j], t.exp_avg_type, m);
      widen(rv[j], t.exp_avg_sq_type, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) update(a, t.decay, g[e], w[e], m[e], v[e]);
      store_as(t.exp_avg, t.exp_avg_type, at, m);
      store_as(t.exp_avg_sq, t.exp_avg_sq_type, at, v);
      if (t.master) store8(t.master + at, w);
      store_as(t.param, t.param_type, at, w);
    }
    return;
  }
  // the last workgroup of a tensor: neighbouring threads take neighbouring elements
  for (int64_t at = base + threadIdx.x; at < t.elems; at += THREADS) {
    float w = load_one(from, from_type, at), m = load_one(t.exp_avg, t.exp_avg_type, at);
    float v = load_one(t.exp_avg_sq, t.exp_avg_sq_type, at);
    update(a, t.decay, load_one(t.grad, t.grad_type, at), w, m, v);
    store_one(t.exp_avg, t.exp_avg_type, at, m);
    store_one(t.exp_avg_sq, t.exp_avg_sq_type, at, v);
    if (t.master) t.master[at] = w;
    store_one(t.param, t.param_type, at, w);
  }
}

}  // namespace

unsigned adamw_blocks(int64_t elems) {
  return static_cast<unsigned>((elems + BLOCK_ELEMS - 1) / BLOCK_ELEMS);
}

hipError_t launch_adamw(const AdamwArgs& a, unsigned blocks, hipStream_t stream) {
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(adamw_kernel, dim3(blocks), dim3(THREADS), 0, stream, a);
  return hipGetLastError();
}

}  // namespace nsmi
