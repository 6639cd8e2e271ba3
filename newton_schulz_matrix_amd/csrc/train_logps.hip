// Log probabilities of given tokens from rows of logits, with the entropy of
// each row and its likeliest entries, and their gradient.
//
//   m = max z,  x = z - m,  s = sum exp x,  t = sum x exp x
//   lse = m + log s,   logp = z[token] - lse,   entropy = log s - t / s
//   gradient: dz = dlogp ([v == token] - p) - dentropy p (log p + entropy),   p = exp(z - lse)
//
// Bound by memory. A row is read once: every thread keeps a running maximum
// and both sums (each term of the entropy has the same sign, nothing cancels),
// and every wave the candidates for the likeliest entries, which are few once
// it knows a threshold that `top` entries reach. Few rows are cut into pieces
// of which a second kernel makes one. Rows begin at any element.
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int UNROLL = 8;                           // vectors of a thread in flight
constexpr int SHORT_VOCAB = 64 * VEC * UNROLL / 2;  // rows up to this long are one wave's
constexpr int step_of(int threads) { return threads * VEC * UNROLL; }
constexpr float FAR = 150.f;                        // exp(-FAR) is 0 in fp32
constexpr float LOG2E = 1.442695041f;

__device__ __forceinline__ int64_t token_at(const LogpsArgs& a, int64_t row) {
  return a.tokens64 ? static_cast<const int64_t*>(a.tokens)[row]
                    : static_cast<const int32_t*>(a.tokens)[row];
}
__device__ __forceinline__ bool counted(const LogpsArgs& a, int64_t token) {
  return token >= 0 && token < a.vocab;
}
// The exponent's base for a maximum m: -inf (nothing but masked entries) is replaced by 0.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * LOG2E); }

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Running maximum and sums of a thread.
struct Sums {
  float m, s, t;
};
// Brings the sums to another maximum.
__device__ __forceinline__ void rebase(Sums& r, float m) {
  const float d = base_of(r.m) - base_of(m);   // <= 0 (r.m = -inf: both sums are 0)
  const float f = r.m == -INFINITY ? 0.f : exp_of(d);
  r.t = f == 0.f ? 0.f : f * fmaf(r.s, d, r.t);
  r.s *= f;
  r.m = m;
}
// Takes in a step; `high` receives the maximum of each vector.
template <int U>
__device__ __forceinline__ void take(const float (&v)[U][VEC], Sums& r, float (&high)[U]) {
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    high[j] = v[j][0];
#pragma unroll
    for (int e = 1; e < VEC; ++e) high[j] = fmaxf(high[j], v[j][e]);
    top = fmaxf(top, high[j]);
  }
  if (top > r.m) rebase(r, top);
  const float base = base_of(r.m);
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float x = v[j][e] - base, w = exp_of(x);   // (a NaN stays one in w)
      r.s += w;
      r.t = fmaf(w, fmaxf(x, -FAR), r.t);              // 0 for an entry at -inf
    }
}

// ------------------------------------------------------- likeliest entries

// A value's place in the order as a whole number: 0 for a NaN, which is never
// chosen, then -inf up to inf; -0 and 0 are equal.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.f);
  const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
  return v != v ? 0u : k;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  const uint32_t b = k & 0x80000000u ? k & 0x7fffffffu : ~k;
  return k == 0u ? NAN : __builtin_bit_cast(float, b);
}
// Orders by value, and the lowest index first among equals.
__device__ __forceinline__ uint64_t entry_of(uint32_t order, int index) {
  return static_cast<uint64_t>(order) << 32 | static_cast<uint32_t>(~index);
}

// A wave's candidates, in LDS. A vector brings at most 512; `top` and those fit.
constexpr int CANDIDATES = LOGPS_MAX_TOP + 64 * VEC;

// Orders of the list's first `count` entries: those of rank < top move to their
// ranks. Every entry is another number, so ranks are distinct.
__device__ __forceinline__ void compact(uint64_t* list, int& count, int top, uint32_t& above) {
  constexpr int MINE = (CANDIDATES + 63) / 64;
  const int lane = threadIdx.x & 63;
  uint64_t mine[MINE];
  int rank[MINE];
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    mine[i] = lane + 64 * i < count ? list[lane + 64 * i] : 0;
    rank[i] = 0;
  }
  for (int k = 0; k < count; ++k) {
    const uint64_t other = list[k];
#pragma unroll
    for (int i = 0; i < MINE; ++i) rank[i] += other > mine[i];
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < MINE; ++i)
    if (lane + 64 * i < count && rank[i] < top) list[rank[i]] = mine[i];
  __builtin_amdgcn_wave_barrier();
  if (count >= top) {
    count = top;
    above = max(above, static_cast<uint32_t>(list[top - 1] >> 32));
  }
}

// Offers a step's entries: those whose order is more than `above` become
// candidates. `high` is the maximum of each of the lane's vectors. Indices rise
// from one vector of a wave to the next, so an entry equal to the last of `top`
// earlier ones is behind them.
template <int U, int THREADS>
__device__ __forceinline__ void offer(const float (&v)[U][VEC], const float (&high)[U], int at, int end,
                                      int top, uint64_t* list, int& count, uint32_t& above) {
  const int lane = threadIdx.x & 63;
  uint32_t most = 0;
  int hits = 0;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const uint32_t order = order_of(high[j]);
    most = max(most, order);
    hits += __popcll(__ballot(order > above));
  }
  if (hits == 0) return;
  if (hits > top + 32) {
    // the lane of rank top - 1 by its greatest entry: that many entries reach its order
    int rank = 0;
    for (int i = 0; i < 64; ++i) {
      const uint32_t other = __builtin_amdgcn_readlane(most, i);
      rank += other > most || (other == most && i < lane);
    }
    const int at_rank = __ffsll(static_cast<unsigned long long>(__ballot(rank == top - 1))) - 1;
    const uint32_t reached = __builtin_amdgcn_readlane(most, at_rank);
    above = max(above, reached > 0 ? reached - 1 : 0u);
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (!__any(order_of(high[j]) > above)) continue;
    const int first = at + j * THREADS * VEC;
    int more = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) more += __popcll(__ballot(order_of(v[j][e]) > above && first + e < end));
    if (count + more > CANDIDATES) compact(list, count, top, above);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const uint32_t order = order_of(v[j][e]);
      const bool in = order > above && first + e < end;
      const unsigned long long all = __ballot(in);
      if (in)
        list[count + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(all >> 32),
                                               __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(all), 0))] =
            entry_of(order, first + e);
      count += __popcll(all);
    }
  }
}

// What is known of a row in the end. Differences from the maximum come first: beside
// entries of the type's lowest value the log of the sum would be lost in lse.
__device__ __forceinline__ void write_row(const LogpsOut& o, int64_t row, float token_logit, double m, double s,
                                          double t) {
  const double log_s = log(s);
  o.logps[row] = static_cast<float>(static_cast<double>(token_logit) - m - log_s);
  o.lse[row] = static_cast<float>(m + log_s);
  o.entropy[row] = static_cast<float>(log_s - t / s);
}
__device__ __forceinline__ void write_entry(const LogpsArgs& a, const LogpsOut& o, int64_t row, int rank,
                                            uint64_t entry, double m, double log_s) {
  const uint32_t order = static_cast<uint32_t>(entry >> 32);
  const int64_t at = row * a.top + rank;
  o.top_logps[at] = static_cast<float>(static_cast<double>(value_of(order)) - m - log_s);
  const int id = order == 0u ? -1 : ~static_cast<int>(static_cast<uint32_t>(entry));
  if (a.tokens64) static_cast<int64_t*>(o.top_ids)[at] = id;
  else static_cast<int32_t*>(o.top_ids)[at] = id;
}
__device__ __forceinline__ void write_nothing(const LogpsArgs& a, const LogpsOut& o, int64_t row) {
  if (threadIdx.x == 0) o.logps[row] = o.lse[row] = o.entropy[row] = 0.f;
  for (int k = threadIdx.x; k < a.top; k += blockDim.x) {
    o.top_logps[row * a.top + k] = 0.f;
    if (a.tokens64) static_cast<int64_t*>(o.top_ids)[row * a.top + k] = -1;
    else static_cast<int32_t*>(o.top_ids)[row * a.top + k] = -1;
  }
}

// One piece of a row, or a whole one, whose results it then writes.
template <class T, int THREADS, bool TOP>
__global__ __launch_bounds__(THREADS) void logps_kernel(LogpsArgs a, PrefSplit sp, LogpsPart* parts,
                                                        uint64_t* entries, LogpsOut o) {
  constexpr int STEP = step_of(THREADS), WAVES = THREADS / 64;
  __shared__ float red_m[WAVES];
  __shared__ double red_s[WAVES], red_t[WAVES];
  __shared__ uint64_t lists[TOP ? WAVES : 1][TOP ? CANDIDATES : 1];
  __shared__ int counts[WAVES];
  const int64_t row = blockIdx.x;
  const int64_t token = token_at(a, row);
  if (!counted(a, token)) {
    if (blockIdx.y == 0) write_nothing(a, o, row);
    return;
  }
  const int begin = blockIdx.y * sp.piece, end = min(a.vocab, begin + sp.piece);
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int col0 = threadIdx.x * VEC;
  const float token_logit = static_cast<float>(z[token]);
  Sums r = {-INFINITY, 0.f, 0.f};
  int count = 0;
  uint32_t above = 0;
  int base = begin;
  for (; base + STEP <= end; base += STEP) {
    float v[UNROLL][VEC];
    Raw<T> raw[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) raw[j] = fetch(z + base + j * THREADS * VEC + col0);
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) widen(raw[j], v[j]);
    float high[UNROLL];
    take(v, r, high);
    if constexpr (TOP) offer<UNROLL, THREADS>(v, high, base + col0, end, a.top, lists[wave], count, above);
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
      float high[1];
      take(v, r, high);
      if constexpr (TOP) offer<1, THREADS>(v, high, at + col0, end, a.top, lists[wave], count, above);
    }
  }
  const float wave_top = wave_max(r.m);
  if (lane == 0) {
    red_m[wave] = wave_top;
    counts[wave] = count;
  }
  __syncthreads();
  float m = red_m[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) m = fmaxf(m, red_m[w]);
  rebase(r, m);
  const double ws = wave_sum64(static_cast<double>(r.s)), wt = wave_sum64(static_cast<double>(r.t));
  if (lane == 0) {
    red_s[wave] = ws;
    red_t[wave] = wt;
  }
  __syncthreads();
  double s = 0.0, t = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    s += red_s[w];
    t += red_t[w];
  }
  const bool whole = sp.pieces == 1;
  const int64_t part = row * sp.pieces + blockIdx.y;
  if (threadIdx.x == 0) {
    if (whole) write_row(o, row, token_logit, m, s, t);
    else parts[part] = {m, s, t};
  }
  if constexpr (TOP) {
    // ranks among all waves' candidates
    const double log_s = whole ? log(s) : 0.0;
    int all = 0;
    for (int w = 0; w < WAVES; ++w) {
      all += counts[w];
      for (int i = threadIdx.x; i < counts[w]; i += THREADS) {
        const uint64_t mine = lists[w][i];
        int rank = 0;
        for (int u = 0; u < WAVES; ++u)
          for (int k = 0; k < counts[u]; ++k) rank += lists[u][k] > mine;
        if (rank >= a.top) continue;
        if (whole) write_entry(a, o, row, rank, mine, m, log_s);
        else entries[part * a.top + rank] = mine;
      }
    }
    for (int rank = all + threadIdx.x; rank < a.top; rank += THREADS) {   // short, or NaN
      if (whole) write_entry(a, o, row, rank, 0, m, log_s);
      else entries[part * a.top + rank] = 0;
    }
  }
}

// Makes one row of its pieces.
constexpr int JOIN_THREADS = 256;
template <class T>
__global__ __launch_bounds__(JOIN_THREADS) void join_kernel(LogpsArgs a, int pieces,
                                                            const LogpsPart* parts,
                                                            const uint64_t* entries, LogpsOut o) {
  __shared__ uint64_t list[LOGPS_JOIN];
  const int64_t row = blockIdx.x;
  const int64_t token = token_at(a, row);
  if (!counted(a, token)) return;   // written by the row's first piece
  const LogpsPart* p = parts + row * pieces;
  const int all = pieces * a.top;
  for (int i = threadIdx.x; i < all; i += JOIN_THREADS) list[i] = entries[row * all + i];
  double m = -INFINITY, s = 0.0, t = 0.0;
  for (int k = 0; k < pieces; ++k) m = fmax(m, p[k].m);
  const double base = base_of(static_cast<float>(m));
  for (int k = 0; k < pieces; ++k) {
    if (p[k].m == -INFINITY) {   // sums of 0, or NaN
      s += p[k].s;
      t += p[k].t;
      continue;
    }
    const double d = p[k].m - base, f = exp(d);
    s += f * p[k].s;
    t += f == 0.0 ? 0.0 * p[k].s : f * (p[k].t + d * p[k].s);
  }
  if (threadIdx.x == 0)
    write_row(o, row, static_cast<float>(static_cast<const T*>(a.logits)[row * a.ld + token]), m, s, t);
  __syncthreads();
  const double log_s = log(s);
  for (int i = threadIdx.x; i < all; i += JOIN_THREADS) {
    const uint64_t mine = list[i];
    int rank = 0;
    // empty places are equal; they are told apart by where they stand
    for (int k = 0; k < all; ++k) rank += list[k] > mine || (list[k] == mine && k < i);
    if (rank < a.top) write_entry(a, o, row, rank, mine, m, log_s);
  }
}

// --------------------------------------------------------------- gradient

// Workgroups take a step each, in the order of the addresses.
template <class T, int THREADS, bool ENTROPY>
__global__ __launch_bounds__(THREADS) void logps_grad_kernel(LogpsArgs a, const float* lse,
                                                             const float* entropy, const float* dlogps,
                                                             const float* dentropy, T* dlogits,
                                                             int64_t ld_dlogits, int steps) {
  const int64_t all = static_cast<int64_t>(a.rows) * steps;
  for (int64_t block = blockIdx.x; block < all; block += gridDim.x) {
    const int row = static_cast<int>(block / steps);
    const int base = static_cast<int>(block - static_cast<int64_t>(row) * steps) * step_of(THREADS);
    const int64_t token = token_at(a, row);
    T* d = dlogits + row * ld_dlogits;
    const int col0 = static_cast<int>(threadIdx.x) * VEC;
    if (!counted(a, token)) {
      const float zero[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        const int at = base + j * THREADS * VEC;
        if (at >= a.vocab) break;
        store8_upto<Use::ONCE>(d + at + col0, a.vocab - at - col0, zero);
      }
      continue;
    }
    const T* z = static_cast<const T*>(a.logits) + row * a.ld;
    Raw<T> raw[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int at = base + j * THREADS * VEC;
      if (at < a.vocab && a.vocab >= VEC) raw[j] = fetch_at<Use::ONCE>(z, a.vocab, at + col0);
    }
    const float l = lse[row], g = dlogps ? dlogps[row] : 0.f;
    const float h = ENTROPY ? dentropy[row] : 0.f, H = ENTROPY ? entropy[row] : 0.f;
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const int at = base + j * THREADS * VEC;
      if (at >= a.vocab) break;
      float v[VEC];
      widen_at(raw[j], z, a.vocab, at + col0, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float x = v[e] - l, p = exp_of(x);
        // an entry at -inf has no share, and p log p goes to 0 there
        const float slope = ENTROPY ? fmaf(h, fmaxf(x, -FAR) + H, g) : g;
        v[e] = fmaf(-p, slope, at + col0 + e == token ? g : 0.f);
      }
      store8_upto<Use::ONCE>(d + at + col0, a.vocab - at - col0, v);
    }
  }
}

}  // namespace

PrefSplit logps_split(int64_t rows, int64_t vocab, int top) {
  PrefSplit sp = pref_split(rows, vocab);
  const int64_t most = top > 0 ? std::max(1, LOGPS_JOIN / top) : sp.pieces;
  if (sp.pieces > most) {   // a row's entries meet in one workgroup's list
    const int64_t step = step_of(vocab <= SHORT_VOCAB ? 64 : 256);
    const int64_t steps = (vocab + step - 1) / step, each = (steps + most - 1) / most;
    sp.piece = static_cast<int>(each * step);
    sp.pieces = static_cast<int>((steps + each - 1) / each);
  }
  return sp;
}

hipError_t launch_token_logps(const LogpsArgs& a, int type, const PrefSplit& sp, LogpsPart* parts,
                              uint64_t* entries, const LogpsOut& o, hipStream_t stream) {
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    const dim3 grid(static_cast<unsigned>(a.rows), sp.pieces);
    auto go = [&](auto threads, auto top) {
      constexpr int N = threads();
      constexpr bool TOP = top();
      hipLaunchKernelGGL((logps_kernel<T, N, TOP>), grid, dim3(N), 0, stream, a, sp, parts, entries, o);
      return hipGetLastError();
    };
    auto shaped = [&](auto threads) {
      return a.top > 0 ? go(threads, std::true_type{}) : go(threads, std::false_type{});
    };
    hipError_t e = a.vocab <= SHORT_VOCAB ? shaped(std::integral_constant<int, 64>{})
                                          : shaped(std::integral_constant<int, 256>{});
    if (e != hipSuccess || sp.pieces == 1) return e;
    hipLaunchKernelGGL(join_kernel<T>, dim3(static_cast<unsigned>(a.rows)), dim3(JOIN_THREADS), 0, stream,
                       a, sp.pieces, parts, entries, o);
    return hipGetLastError();
  });
}

hipError_t launch_token_logps_grad(const LogpsArgs& a, int type, const float* lse, const float* entropy,
                                   const float* dlogps, const float* dentropy, void* dlogits,
                                   int64_t ld_dlogits, hipStream_t stream) {
  const int threads = a.vocab <= SHORT_VOCAB ? 64 : 256, step = step_of(threads);
  const int steps = (a.vocab + step - 1) / step;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(a.rows) * steps, 1 << 23)));
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto n, auto with) {
      constexpr int N = n();
      constexpr bool E = with();
      hipLaunchKernelGGL((logps_grad_kernel<T, N, E>), grid, dim3(N), 0, stream, a, lse, entropy, dlogps,
                         dentropy, static_cast<T*>(dlogits), ld_dlogits, steps);
      return hipGetLastError();
    };
    auto shaped = [&](auto n) { return dentropy ? go(n, std::true_type{}) : go(n, std::false_type{}); };
    return threads == 64 ? shaped(std::integral_constant<int, 64>{})
                         : shaped(std::integral_constant<int, 256>{});
  });
}

}  // namespace nsmi
