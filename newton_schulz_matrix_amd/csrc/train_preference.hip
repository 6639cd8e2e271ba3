// Preference loss on the logits of paired sequences, and its gradient.
//
//   lse = log sum_v exp z_v;   logp_s = sum_t z[label] - lse
//   margin = beta ((logp_l - ref_l) - (logp_r - ref_r))
//   loss = -(1 - s) log sigmoid(margin) - s log sigmoid(-margin)
//   dz = k ([v == label] - exp(z - lse)),  k = +- dloss beta (s sigmoid(margin) - (1 - s) sigmoid(-margin))
//
// Bound by memory. The forward pass reads the counted rows once, with a
// running maximum and sum, cut into pieces where the rows alone would not
// fill the chip; the factor k of a row needs its whole sequence, so the
// gradient reads the logits a second time. Rows begin at any element: all
// accesses are vectors with element alignment.
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;                           // vectors of a thread in flight
constexpr int STEP = THREADS * VEC * UNROLL;        // elements of a workgroup's step

// exp(x), x <= 0, by the hardware's 2^x. The product with log2(e) carries the
// constant's next 24 bits: without them every term of a sum would be off to
// the same side, and the sums over a sequence would keep that error.
__device__ __forceinline__ float exp_neg(float x) {
  return __builtin_amdgcn_exp2f(fmaf(x, 1.925963033e-8f, x * 1.442695041f));
}

// Joins (m, s) with (m2, s2): sums of exp relative to their maxima. A maximum
// of -inf stands for no terms (its sum is 0).
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float safe = top == -INFINITY ? 0.f : top;
  s = s * exp_neg(m - safe) + s2 * exp_neg(m2 - safe);
  m = top;
}

template <class I>
__device__ __forceinline__ int64_t label_at(const PrefArgs& a, int64_t row) {
  return static_cast<int64_t>(static_cast<const I*>(a.labels)[row]);
}
__device__ __forceinline__ bool counted(const PrefArgs& a, int64_t label) {
  return label >= 0 && label < a.vocab;
}

// Maximum and sum of one piece of a row.
template <class T, class I>
__global__ __launch_bounds__(THREADS) void pieces_kernel(PrefArgs a, PrefSplit sp, float2* parts) {
  __shared__ float red_m[THREADS / 64], red_s[THREADS / 64];
  const int64_t row = blockIdx.x;
  if (!counted(a, label_at<I>(a, row))) return;
  const int begin = blockIdx.y * sp.piece, end = min(a.vocab, begin + sp.piece);
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  float m = -INFINITY, s = 0.f;
  for (int base = begin; base < end; base += STEP) {
    float v[UNROLL][VEC];
    const bool whole = base + STEP <= end;
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int at = base + (j * THREADS + threadIdx.x) * VEC;
      if (whole || at + VEC <= end) {
        load8(z + at, v[j]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j][e] = at + e < end ? static_cast<float>(z[at + e]) : -INFINITY;
      }
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < UNROLL; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) top = fmaxf(top, v[j][e]);
    const float safe = top == -INFINITY ? 0.f : top;
    float add = 0.f;
#pragma unroll
    for (int j = 0; j < UNROLL; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) add += exp_neg(v[j][e] - safe);
    s = fmaf(s, exp_neg(m - safe), add);
    m = top;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) join(m, s, __shfl_xor(m, off, 64), __shfl_xor(s, off, 64));
  if ((threadIdx.x & 63) == 0) {
    red_m[threadIdx.x >> 6] = m;
    red_s[threadIdx.x >> 6] = s;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < THREADS / 64; ++w) join(m, s, red_m[w], red_s[w]);
  parts[row * sp.pieces + blockIdx.y] = make_float2(m, s);
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// log(1 + exp(x)) = -log sigmoid(-x)
__device__ __forceinline__ double softplus(double x) {
  return fmax(x, 0.0) + log1p(exp(-fabs(x)));
}

// One workgroup for each pair: the rows' lse, the sequences' sums, the loss.
constexpr int PAIR_THREADS = 1024;
template <class T, class I>
__global__ __launch_bounds__(PAIR_THREADS) void pairs_kernel(PrefArgs a, PrefSplit sp,
                                                             const float2* parts,
                                                             const float* ref_logps, float* losses,
                                                             float* margins, float* logps,
                                                             float* lse) {
  __shared__ double red[2][PAIR_THREADS / 64];
  double sums[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int64_t first = static_cast<int64_t>(side * a.pairs + blockIdx.x) * a.length;
    double sum = 0.0;
    for (int t = threadIdx.x; t < a.length; t += PAIR_THREADS) {
      const int64_t row = first + t;
      const int64_t label = label_at<I>(a, row);
      float l = 0.f;
      if (counted(a, label)) {
        float m = -INFINITY, s = 0.f;
        for (int k = 0; k < sp.pieces; ++k) {
          const float2 p = parts[row * sp.pieces + k];
          join(m, s, p.x, p.y);
        }
        const double wide = static_cast<double>(m) + log(static_cast<double>(s));
        l = static_cast<float>(wide);
        sum += static_cast<double>(static_cast<float>(static_cast<const T*>(a.logits)[row * a.ld + label])) - wide;
      }
      lse[row] = l;
    }
    sum = wave_sum64(sum);
    if ((threadIdx.x & 63) == 0) red[side][threadIdx.x >> 6] = sum;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    double sum = 0.0;
    for (int w = 0; w < PAIR_THREADS / 64; ++w) sum += red[side][w];
    const int s = side * a.pairs + blockIdx.x;
    logps[s] = static_cast<float>(sum);
    sums[side] = sum - static_cast<double>(ref_logps[s]);
  }
  const double margin = static_cast<double>(a.beta) * (sums[0] - sums[1]);
  const double eps = a.smoothing;
  margins[blockIdx.x] = static_cast<float>(margin);
  // a weight of 0 leaves its term out, also where that term is infinite
  double loss = 0.0;
  if (eps != 1.0) loss += (1.0 - eps) * softplus(-margin);
  if (eps != 0.0) loss += eps * softplus(margin);
  losses[blockIdx.x] = static_cast<float>(loss);
}

// --------------------------------------------------------------- gradient

__device__ __forceinline__ float sigmoid(float x) {
  const float e = expf(-fabsf(x));
  return x >= 0.f ? 1.f / (1.f + e) : e / (1.f + e);
}

// One step of STEP elements of a row.
template <class T, class I>
__global__ __launch_bounds__(THREADS) void grad_kernel(PrefArgs a, const float* margins,
                                                       const float* lse, const float* dlosses,
                                                       T* dlogits, int64_t ld_dlogits) {
  const int64_t row = blockIdx.x;
  const int base = blockIdx.y * STEP;
  const int64_t label = label_at<I>(a, row);
  T* d = dlogits + row * ld_dlogits;
  const bool whole = base + STEP <= a.vocab;
  if (!counted(a, label)) {
    const float zero[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int at = base + (j * THREADS + threadIdx.x) * VEC;
      store8_upto(d + at, a.vocab - at, zero);
    }
    return;
  }
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  float v[UNROLL][VEC];
#pragma unroll
  for (int j = 0; j < UNROLL; ++j) {
    const int at = base + (j * THREADS + threadIdx.x) * VEC;
    if (whole) load8(z + at, v[j]);
    else load8_upto(z + at, a.vocab - at, v[j]);
  }
  const int seq = static_cast<int>(blockIdx.x) / a.length;
  const int pair = seq < a.pairs ? seq : seq - a.pairs;
  const float margin = margins[pair];
  float k = dlosses[pair] * a.beta *
            (a.smoothing * sigmoid(margin) - (1.f - a.smoothing) * sigmoid(-margin));
  if (seq >= a.pairs) k = -k;
  const float l = lse[row];
#pragma unroll
  for (int j = 0; j < UNROLL; ++j) {
    const int at = base + (j * THREADS + threadIdx.x) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float p = exp_neg(v[j][e] - l);
      v[j][e] = at + e == label ? k * (1.f - p) : -k * p;
    }
    if (whole) store8(d + at, v[j]);
    else store8_upto(d + at, a.vocab - at, v[j]);
  }
}

}  // namespace

PrefSplit pref_split(int64_t rows, int64_t vocab) {
  // pieces of at least one step; as many as give every CU a few workgroups
  const int64_t steps = (vocab + STEP - 1) / STEP;
  const int64_t want = rows > 0 ? std::max<int64_t>(1, 2048 / rows) : 1;
  const int64_t pieces = std::min(steps, want);
  const int64_t each = (steps + pieces - 1) / pieces;
  PrefSplit sp;
  sp.piece = static_cast<int>(each * STEP);
  sp.pieces = static_cast<int>((steps + each - 1) / each);
  return sp;
}

hipError_t launch_preference_loss(const PrefArgs& a, int type, bool labels64, const PrefSplit& sp,
                                  float2* parts, const float* ref_logps, float* losses,
                                  float* margins, float* logps, float* lse, hipStream_t stream) {
  const int64_t rows = int64_t{2} * a.pairs * a.length;
  auto on = [&](auto t, auto i) {
    using T = decltype(t);
    using I = decltype(i);
    if (rows > 0) {
      hipLaunchKernelGGL((pieces_kernel<T, I>), dim3(static_cast<unsigned>(rows), sp.pieces),
                         dim3(THREADS), 0, stream, a, sp, parts);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((pairs_kernel<T, I>), dim3(a.pairs), dim3(PAIR_THREADS), 0, stream, a, sp,
                       parts, ref_logps, losses, margins, logps, lse);
    return hipGetLastError();
  };
  return by_type(type, [&](auto t) { return labels64 ? on(t, int64_t{}) : on(t, int32_t{}); });
}

hipError_t launch_preference_grad(const PrefArgs& a, int type, bool labels64,
                                  const float* margins, const float* lse, const float* dlosses,
                                  void* dlogits, int64_t ld_dlogits, hipStream_t stream) {
  const int64_t rows = int64_t{2} * a.pairs * a.length;
  if (rows <= 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(rows), (a.vocab + STEP - 1) / STEP);
  auto on = [&](auto t, auto i) {
    using T = decltype(t);
    hipLaunchKernelGGL((grad_kernel<T, decltype(i)>), grid, dim3(THREADS), 0, stream, a, margins,
                       lse, dlosses, static_cast<T*>(dlogits), ld_dlogits);
    return hipGetLastError();
  };
  return by_type(type, [&](auto t) { return labels64 ? on(t, int64_t{}) : on(t, int32_t{}); });
}

}  // namespace nsmi
