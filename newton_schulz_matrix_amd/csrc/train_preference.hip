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
//
// 2 pairs of 1024 positions, 128000 entries, bf16 (65% counted): 128 us for the
// pieces (0.70 GB, 5.5 TB/s; the exponentials keep the vector units half
// busy), 9 for the pairs, 286 for the gradient (0.70 GB in, 1.05 out, 6.1 TB/s).
// The logits are read with cached loads in the forward pass: it is 8 us
// slower so, and the gradient 19 us faster, which finds a part of them. The
// gradient is stored non-temporally, which pays in fp32 too (1024 rows of 128000,
// loss and gradient: 273 us, 299 with cached stores).
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

// A workgroup is one wave for short vocabularies, else four: loss and gradient
// of 32000 rows of 1001 take 57 us with the one, 116 with the four, which the
// long rows need.
constexpr int UNROLL = 8;                           // vectors of a thread in flight
constexpr int SHORT_VOCAB = 64 * VEC * UNROLL / 2;
constexpr int step_of(int threads) { return threads * VEC * UNROLL; }   // elements of a step
constexpr float FAR = 150.f;                        // exp(-FAR) is 0 in fp32

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

// The exponent's base for a maximum m: exp(z - m) for m = -inf (no terms yet,
// or none but masked ones) is taken against 0 instead, which gives 0.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

template <class I>
__device__ __forceinline__ int64_t label_at(const PrefArgs& a, int64_t row) {
  return static_cast<int64_t>(static_cast<const I*>(a.labels)[row]);
}
__device__ __forceinline__ bool counted(const PrefArgs& a, int64_t label) {
  return label >= 0 && label < a.vocab;
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// exp(m - base), 0 for m = -inf.
__device__ __forceinline__ float factor(float m, float base) {
  const float x = m - base;
  return x < -FAR ? 0.f : exp_exact(x);
}

// Maximum and sum of one piece of a row. A thread keeps its own running
// maximum and rescales its sum once a step; the threads' sums are brought to
// the piece's maximum once, at the end, and added and kept in 64 bits: a
// sequence adds up the roundings of hundreds of rows, and the difference of two
// sequences is small beside them.
template <int U>
__device__ __forceinline__ void take(const float (&v)[U][VEC], float& m, float& s) {
  float top = m, low = INFINITY;
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      top = fmaxf(top, v[j][e]);
      low = fminf(low, v[j][e]);
    }
  const float base = base_of(top);
  float add = 0.f;
  if (__any(low - base < -FAR)) {   // -inf - (-inf) in the correction: terms this far off are 0
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float x = v[j][e] - base;
        add += exp_exact(x < -FAR ? -FAR : x);   // (a NaN stays one)
      }
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) add += exp_exact(v[j][e] - base);
  }
  s = fmaf(s, factor(m, base), add);
  m = top;
}
template <class T, class I, int THREADS>
__global__ __launch_bounds__(THREADS) void pieces_kernel(PrefArgs a, PrefSplit sp,
                                                         double2* parts) {
  constexpr int STEP = step_of(THREADS);
  __shared__ float red_m[THREADS / 64];
  __shared__ double red_s[THREADS / 64];
  const int row = blockIdx.x, seq = row / a.length;
  if (!counted(a, label_at<I>(a, row))) return;
  const int begin = blockIdx.y * sp.piece, end = min(a.vocab, begin + sp.piece);
  const T* z = static_cast<const T*>(a.logits) + seq * a.ld_seq + (row - seq * a.length) * a.ld;
  float m = -INFINITY, s = 0.f;
  const int col0 = threadIdx.x * VEC;
  int base = begin;
  for (; base + STEP <= end; base += STEP) {
    float v[UNROLL][VEC];
    Raw<T> raw[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) raw[j] = fetch(z + base + j * THREADS * VEC + col0);
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) widen(raw[j], v[j]);
    take(v, m, s);
  }
  if (base < end) {   // the vectors left, all in flight, then one after the other
    Raw<T> raw[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int at = base + j * THREADS * VEC;
      if (at < end && end >= VEC) raw[j] = fetch_at(z, end, at + col0);
    }
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int at = base + j * THREADS * VEC;
      if (at >= end) break;
      float v[1][VEC];
      widen_at(raw[j], z, end, at + col0, v[0]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[0][e] = at + col0 + e < end ? v[0][e] : -INFINITY;
      take(v, m, s);
    }
  }
  const int wave = threadIdx.x >> 6;
  const float wave_top = wave_max(m);
  if ((threadIdx.x & 63) == 0) red_m[wave] = wave_top;
  __syncthreads();
  float top = red_m[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) top = fmaxf(top, red_m[w]);
  const double sum = wave_sum64(static_cast<double>(s * factor(m, base_of(top))));
  if ((threadIdx.x & 63) == 0) red_s[wave] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double total = 0.0;
  for (int w = 0; w < THREADS / 64; ++w) total += red_s[w];
  parts[static_cast<int64_t>(row) * sp.pieces + blockIdx.y] = make_double2(top, total);
}

// log(1 + exp(x)) = -log sigmoid(-x)
__device__ __forceinline__ double softplus(double x) {
  return fmax(x, 0.0) + log1p(exp(-fabs(x)));
}

// One workgroup for each pair: the rows' lse, the sequences' sums, the loss. A
// wave for sequences that short, of which there can be millions.
constexpr int SHORT_LENGTH = 64;
template <class T, class I, int PAIR_THREADS>
__global__ __launch_bounds__(PAIR_THREADS) void pairs_kernel(PrefArgs a, PrefSplit sp,
                                                             const double2* parts,
                                                             const float* ref_logps, float* losses,
                                                             float* margins, float* logps,
                                                             float* lse) {
  __shared__ double red[2][PAIR_THREADS / 64];
  double sums[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int seq = side * a.pairs + blockIdx.x;
    const int64_t first = static_cast<int64_t>(seq) * a.length;
    const T* z = static_cast<const T*>(a.logits) + seq * a.ld_seq;
    double sum = 0.0;
    for (int t = threadIdx.x; t < a.length; t += PAIR_THREADS) {
      const int64_t row = first + t;
      const int64_t label = label_at<I>(a, row);
      float l = 0.f;
      if (counted(a, label)) {
        const double2* p = parts + row * sp.pieces;
        double m = p[0].x;
        for (int k = 1; k < sp.pieces; ++k) m = fmax(m, p[k].x);
        double s = 0.0;
        for (int k = 0; k < sp.pieces; ++k)
          s += p[k].y * exp(p[k].x - static_cast<double>(base_of(static_cast<float>(m))));
        const double wide = m + log(s);
        // lse is an fp32 output: its rounding, at most |lse| / 2^24, multiplies the
        // row's gradient, which 16-bit gradients do not show
        l = static_cast<float>(wide);
        sum += static_cast<double>(static_cast<float>(z[t * a.ld + label])) - wide;
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

// s sigmoid(m) - (1 - s) sigmoid(-m), in 64 bits: the two terms all but cancel
// where the smoothed loss is flat, and a whole row is multiplied by this.
__device__ __forceinline__ double slope(double m, double s) {
  const double e = exp(-fabs(m));
  return (m >= 0.0 ? s - (1.0 - s) * e : s * e - (1.0 - s)) / (1.0 + e);
}

// Workgroups take a step each, in the order of the addresses.
template <class T, class I, int THREADS>
__global__ __launch_bounds__(THREADS) void grad_kernel(PrefArgs a, const float* margins,
                                                       const float* lse, const float* dlosses,
                                                       T* dlogits, int64_t ld_dlogits,
                                                       int64_t ld_dseq, int steps) {
  const int64_t all = int64_t{2} * a.pairs * a.length * steps;
  for (int64_t block = blockIdx.x; block < all; block += gridDim.x) {
    const int row = static_cast<int>(block / steps);
    const int base = static_cast<int>(block - static_cast<int64_t>(row) * steps) * step_of(THREADS);
    const int seq = row / a.length, t = row - seq * a.length;
    const int64_t label = label_at<I>(a, row);
    T* d = dlogits + seq * ld_dseq + t * ld_dlogits;
    const int col0 = static_cast<int>(threadIdx.x) * VEC;
    if (!counted(a, label)) {
      const float zero[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        const int at = base + j * THREADS * VEC;
        if (at >= a.vocab) break;
        store8_upto<Use::ONCE>(d + at + col0, a.vocab - at - col0, zero);
      }
      continue;
    }
    // read first: k is computed while the logits are on their way
    const int pair = seq < a.pairs ? seq : seq - a.pairs;
    const float margin = margins[pair], dloss = dlosses[pair], l = lse[row];
    const T* z = static_cast<const T*>(a.logits) + seq * a.ld_seq + t * a.ld;
    Raw<T> raw[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int at = base + j * THREADS * VEC;
      if (at < a.vocab && a.vocab >= VEC) raw[j] = fetch_at<Use::ONCE>(z, a.vocab, at + col0);
    }
    float k = static_cast<float>(static_cast<double>(dloss) * a.beta * slope(margin, a.smoothing));
    if (seq >= a.pairs) k = -k;
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int at = base + j * THREADS * VEC;
      if (at >= a.vocab) break;
      float v[VEC];
      widen_at(raw[j], z, a.vocab, at + col0, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float x = v[e] - l;
        const float p = exp_exact(x < -FAR ? -FAR : x);   // (a NaN stays one)
        v[e] = at + col0 + e == label ? k * (1.f - p) : -k * p;
      }
      store8_upto<Use::ONCE>(d + at + col0, a.vocab - at - col0, v);
    }
  }
}

}  // namespace

PrefSplit pref_split(int64_t rows, int64_t vocab) {
  // pieces of at least one step; as many as give every CU a few workgroups
  const int STEP = step_of(vocab <= SHORT_VOCAB ? 64 : 256);
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
                                  double2* parts, const float* ref_logps, float* losses,
                                  float* margins, float* logps, float* lse, hipStream_t stream) {
  const int64_t rows = int64_t{2} * a.pairs * a.length;
  auto on = [&](auto t, auto i) {
    using T = decltype(t);
    using I = decltype(i);
    if (rows > 0) {
      const dim3 grid(static_cast<unsigned>(rows), sp.pieces);
      if (a.vocab <= SHORT_VOCAB)
        hipLaunchKernelGGL((pieces_kernel<T, I, 64>), grid, dim3(64), 0, stream, a, sp, parts);
      else
        hipLaunchKernelGGL((pieces_kernel<T, I, 256>), grid, dim3(256), 0, stream, a, sp, parts);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (a.length <= SHORT_LENGTH)
      hipLaunchKernelGGL((pairs_kernel<T, I, 64>), dim3(a.pairs), dim3(64), 0, stream, a, sp, parts,
                         ref_logps, losses, margins, logps, lse);
    else
      hipLaunchKernelGGL((pairs_kernel<T, I, 1024>), dim3(a.pairs), dim3(1024), 0, stream, a, sp,
                         parts, ref_logps, losses, margins, logps, lse);
    return hipGetLastError();
  };
  return by_type(type, [&](auto t) { return labels64 ? on(t, int64_t{}) : on(t, int32_t{}); });
}

hipError_t launch_preference_grad(const PrefArgs& a, int type, bool labels64,
                                  const float* margins, const float* lse, const float* dlosses,
                                  void* dlogits, int64_t ld_dlogits, int64_t ld_dseq,
                                  hipStream_t stream) {
  const int64_t rows = int64_t{2} * a.pairs * a.length;
  if (rows <= 0) return hipSuccess;
  const int threads = a.vocab <= SHORT_VOCAB ? 64 : 256, step = step_of(threads);
  const int steps = (a.vocab + step - 1) / step;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(rows * steps, 1 << 23)));
  auto on = [&](auto t, auto i) {
    using T = decltype(t);
    using I = decltype(i);
    if (threads == 64)
      hipLaunchKernelGGL((grad_kernel<T, I, 64>), grid, dim3(64), 0, stream, a, margins, lse,
                         dlosses, static_cast<T*>(dlogits), ld_dlogits, ld_dseq, steps);
    else
      hipLaunchKernelGGL((grad_kernel<T, I, 256>), grid, dim3(256), 0, stream, a, margins, lse,
                         dlosses, static_cast<T*>(dlogits), ld_dlogits, ld_dseq, steps);
    return hipGetLastError();
  };
  return by_type(type, [&](auto t) { return labels64 ? on(t, int64_t{}) : on(t, int32_t{}); });
}

}  // namespace nsmi
