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
//
// A thread takes four elements, 16 bytes of fp32 side by side with its
// neighbours', and a workgroup 1024, once: a table of 64000 x 4096 (bf16 with
// fp32 copy and states, 7.3 GB) takes 1.20 ms, 6.1 TB/s, with loads and stores
// non-temporal; 1.32 ms with cached stores, 1.43 with eight elements twice.
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int THREADS = 256;
constexpr int LANE = 4;                                // elements of a thread
constexpr int BLOCK_ELEMS = THREADS * LANE;

// LANE elements as loaded, in 16 or 8 bytes; each is read once in a call.
typedef uint32_t Words __attribute__((ext_vector_type(4)));
__device__ __forceinline__ Words load_raw(const void* p, int type, int64_t at) {
  typedef uint32_t Pair __attribute__((ext_vector_type(2), aligned(2), may_alias));
  if (type == OUT_F32)
    return __builtin_nontemporal_load(reinterpret_cast<const Quad*>(static_cast<const float*>(p) + at));
  const Pair h =
      __builtin_nontemporal_load(reinterpret_cast<const Pair*>(static_cast<const uint16_t*>(p) + at));
  return Words{h.x, h.y, 0, 0};
}
template <class T>
__device__ __forceinline__ void widen_from(const Words& r, float (&v)[LANE]) {
  T b[LANE];
  __builtin_memcpy(b, &r, sizeof(b));
#pragma unroll
  for (int e = 0; e < LANE; ++e) v[e] = static_cast<float>(b[e]);
}
__device__ __forceinline__ void widen(const Words& r, int type, float (&v)[LANE]) {
  if (type == OUT_F32) widen_from<float>(r, v);
  else if (type == OUT_BF16) widen_from<__bf16>(r, v);
  else widen_from<_Float16>(r, v);
}
template <class T>
__device__ __forceinline__ void store_lane(T* p, const float (&v)[LANE]) {
  T b[LANE];
#pragma unroll
  for (int e = 0; e < LANE; ++e) b[e] = static_cast<T>(v[e]);
  typedef uint32_t Word __attribute__((ext_vector_type(sizeof(b) / 4), aligned(2), may_alias));
  Word w;
  __builtin_memcpy(&w, b, sizeof(b));
  __builtin_nontemporal_store(w, reinterpret_cast<Word*>(p));
}
__device__ __forceinline__ void store_as(void* p, int type, int64_t at, const float (&v)[LANE]) {
  if (type == OUT_F32) store_lane(static_cast<float*>(p) + at, v);
  else if (type == OUT_BF16) store_lane(static_cast<__bf16*>(p) + at, v);
  else store_lane(static_cast<_Float16*>(p) + at, v);
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
  // the tensors that begin at or before this workgroup, counted by the lanes of a wave
  const int lane = threadIdx.x & 63;
  const bool begun = lane < a.count && a.begin[min(lane, ADAMW_TENSORS - 1)] <= blockIdx.x;
  const int i = __popcll(__ballot(begun)) - 1;
  const AdamwTensor& t = a.t[i];
  const int64_t base = static_cast<int64_t>(blockIdx.x - a.begin[i]) * BLOCK_ELEMS;
  const void* from = t.master ? t.master : t.param;
  const int from_type = t.master ? static_cast<int>(OUT_F32) : t.param_type;
  if (base + BLOCK_ELEMS <= t.elems) {
    const int64_t at = base + threadIdx.x * LANE;
    const Words rg = load_raw(t.grad, t.grad_type, at);
    const Words rm = load_raw(t.exp_avg, t.exp_avg_type, at);
    const Words rv = load_raw(t.exp_avg_sq, t.exp_avg_sq_type, at);
    const Words rw = load_raw(from, from_type, at);
    float w[LANE], g[LANE], m[LANE], v[LANE];
    widen(rg, t.grad_type, g);
    widen(rm, t.exp_avg_type, m);
    widen(rv, t.exp_avg_sq_type, v);
    widen(rw, from_type, w);
#pragma unroll
    for (int e = 0; e < LANE; ++e) update(a, t.decay, g[e], w[e], m[e], v[e]);
    store_as(t.exp_avg, t.exp_avg_type, at, m);
    store_as(t.exp_avg_sq, t.exp_avg_sq_type, at, v);
    if (t.master) store_lane(t.master + at, w);
    store_as(t.param, t.param_type, at, w);
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
