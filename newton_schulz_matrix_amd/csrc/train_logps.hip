// Log probabilities of given tokens from rows of logits, with the entropy of
// each row and its likeliest entries, and their gradient.
//
//   m = max z,  x = z - m,  s = sum exp x,  t = sum x exp x
//   lse = m + log s,   logp = z[token] - lse,   entropy = log s - t / s
//   gradient: dz = dlogp ([v == token] - p) - dentropy p (log p + entropy),   p = exp(z - lse)
//
// Bound by memory, and nearly as much by the vector units. Exponentials are taken without the
// rounding of their argument's product (exp_near, exp_exact), as those of the preference
// loss: log probabilities are added up over sequences and the sums subtracted. It costs 2 to
// 6% (4096 rows of 128000 without alternatives 161 and 164 us, with 5 177 and 188).
//
// A row is read once: every thread keeps a running maximum
// and both sums (each term of the entropy has the same sign, nothing cancels),
// and every wave the candidates for the likeliest entries, which are few once
// it knows a threshold that `top` entries reach. Few rows are cut into pieces
// of which a second kernel makes one. Rows begin at any element.
//
// Measured, bf16: 4096 rows of 128000, a fifth of them not counted, 5 alternatives, 185 us (0.84
// GB read: 4.5 TB/s); its gradient with entropy 338 (1.89 GB: 5.6); 8 rows
// of 50021 with 20 alternatives 12 + 5, the latency of the two kernels.
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int UNROLL = 8;                           // vectors of a thread in flight
constexpr int SHORT_VOCAB = 64 * VEC * UNROLL / 2;  // rows up to this long are one wave's
// Many rows are one wave's up to longer ones: nothing is brought together between waves
// then (bf16, us with one wave and with four: 16000 rows of 4096, top 5, 45 and 121; 4096 of
// 40000 76 and 88; 8192 of 50021 194 and 223; without top 4096 of 12000 26 and 28, 12000 of 21273
// 119 and 120, 4096 of 128000 201 and 194). Few rows are done sooner by four. With alternatives
// one wave is 4 to 15% faster on longer rows too (4096 of 128000, top 5, 209 and 219; 16384 of
// 70000 442 and 517), but 60% slower where they rise throughout (4096 of 128000 765 and 473):
// four from there on.
constexpr int MANY_ROWS = 4096, MANY_VOCAB = 1 << 14, MANY_VOCAB_TOP = 1 << 16;
constexpr int one_wave_vocab(int rows, int top) {
  return rows < MANY_ROWS ? SHORT_VOCAB : top > 0 ? MANY_VOCAB_TOP : MANY_VOCAB;
}
constexpr int step_of(int threads) { return threads * VEC * UNROLL; }

__device__ __forceinline__ int64_t token_at(const LogpsArgs& a, int64_t row) {
  return a.tokens64 ? static_cast<const int64_t*>(a.tokens)[row]
                    : static_cast<const int32_t*>(a.tokens)[row];
}
// Offset of a row in sequences `apart`, rows `ld` apart.
__device__ __forceinline__ int64_t offset_of(const LogpsArgs& a, int row, int64_t apart, int64_t ld) {
  const int seq = row / a.length;
  return seq * apart + (row - seq * a.length) * ld;
}
__device__ __forceinline__ bool counted(const LogpsArgs& a, int64_t token) {
  return token >= 0 && token < a.vocab;
}
// The exponent's base for a maximum m: -inf (nothing but masked entries) is replaced by 0.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// bf16 as one step each: taken from the halves by type, the upper ones are shifted
// down and up again.
__device__ __forceinline__ void widen(const Raw<__bf16>& raw, float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    const uint32_t word = raw.q[0][i];
    v[2 * i] = __builtin_bit_cast(float, word << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, word & 0xffff0000u);
  }
}

// Sums of a thread against a reference m, which is at most LAG below its
// greatest entry: x is at most LAG, and the entropy's two terms do not cancel.
// s and t are those of a step's terms, which go to all_s and all_t at its end: beside the sum of
// a thousand terms the small ones would be lost, in every row alike (rows of 65536, standard
// deviation 4, lse too low by 21 half steps of 1, by 1 so; it costs 1%).
constexpr float LAG = 1.f;
struct Sums {
  float m = -INFINITY, s = 0.f, t = 0.f, all_s = 0.f, all_t = 0.f;
};
__device__ __forceinline__ void end_step(Sums& r) {
  r.all_s += r.s;
  r.all_t += r.t;
  r.s = r.t = 0.f;
}
// Brings the sums to another reference.
__device__ __forceinline__ void rebase(Sums& r, float m) {
  const float d = base_of(r.m) - base_of(m);   // (r.m = -inf: all sums are 0)
  const float f = r.m == -INFINITY || d < -FAR ? 0.f : exp_near(d);
  r.t = f == 0.f ? 0.f : f * fmaf(r.s, d, r.t);
  r.all_t = f == 0.f ? 0.f : f * fmaf(r.all_s, d, r.all_t);
  r.s *= f;
  r.all_s *= f;
  r.m = m;
}
// Takes in one vector, whose greatest entry is `high`.
__device__ __forceinline__ void take(const float (&v)[VEC], float high, Sums& r) {
  if (__any(high > r.m + LAG)) rebase(r, fmaxf(r.m, high));
  const float base = base_of(r.m);
  float low = v[0];
#pragma unroll
  for (int e = 1; e < VEC; ++e) low = fminf(low, v[e]);
  auto add = [&](float x) {
    const float w = exp_near(x);
    r.s += w;
    r.t = fmaf(w, x, r.t);
  };
  if (__any(low - base < -FAR)) {   // an entry at -inf has no share; a NaN stays one
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float x = v[e] - base;
      add(x < -FAR ? -FAR : x);
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) add(v[e] - base);
  }
}
__device__ __forceinline__ float highest(const float (&v)[VEC]) {
  float h = v[0];
#pragma unroll
  for (int e = 1; e < VEC; ++e) h = fmaxf(h, v[e]);
  return h;
}

// The vector at `at` of a row that ends at `end`, -inf behind it.
template <class T>
__device__ __forceinline__ Raw<T> fetch_upto(const T* z, int at, int end) {
  if (at + VEC <= end) return fetch(z + at);
  T e[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    e[i] = static_cast<T>(-INFINITY);
    if (at + i < end) e[i] = z[at + i];
  }
  Raw<T> raw;
  __builtin_memcpy(&raw, e, sizeof(raw));
  return raw;
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
constexpr uint32_t LOWEST = 0x007fffffu;   // of -inf

// Orders by value, and the lowest index first among equals.
__device__ __forceinline__ uint64_t entry_of(uint32_t order, int index) {
  return static_cast<uint64_t>(order) << 32 | static_cast<uint32_t>(~index);
}

// What the lanes of a wave have written to LDS is there for the others.
__device__ __forceinline__ void wave_settled() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave's candidates, in LDS. A vector brings at most 512; `top` and those fit.
constexpr int CANDIDATES = LOGPS_MAX_TOP + 64 * VEC;
constexpr int AT_ONCE = 8;   // entries of a list that are read together
constexpr int LAST = 256;    // entries that are left for the final order, hardly ever more than 2 top
struct Candidates {
  uint64_t list[CANDIDATES];
  uint64_t ordered[LOGPS_MAX_TOP];
  uint32_t best[64];   // greatest order of each lane
};

// Zeros behind a list's entries, up to where it is read.
__device__ __forceinline__ void pad(uint64_t* list, int count, int size) {
  const int lane = threadIdx.x & 63;
  if (lane < AT_ONCE && count + lane < size) list[count + lane] = 0;
  wave_settled();
}
// How many entries of a padded list stand before `mine`.
__device__ __forceinline__ int rank_in(const uint64_t* list, int count, uint64_t mine) {
  int rank = 0;
  for (int k = 0; k < count; k += AT_ONCE)
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) rank += list[k + i] > mine;
  return rank;
}

// A number that `top` of N orders a lane reach, near the greatest such: its upper 16
// bits, one a step.
template <int N>
__device__ __forceinline__ uint32_t reached_by(const uint32_t (&order)[N], int top) {
  uint32_t t = 0;
#pragma unroll
  for (int b = 31; b >= 16; --b) {
    const uint32_t more = t | 1u << b;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popcll(__ballot(order[i] >= more));
    t = n >= top ? more : t;
  }
  return t;
}

// What a wave knows: entries from order `from` on (value `from_value`) are
// candidates, `count` so far; best is the lane's greatest entry and, where more than MANY
// are wanted, second the greatest of its other vectors: the least of 64 lanes' greatest
// entries would let too many pass (4096 rows of 128000, top 64: 304 us, 652 without).
constexpr int MANY = 32;
struct Choice {
  uint32_t from;
  float from_value, best, second;
  int count;

  __device__ __forceinline__ void raise(uint32_t to) {
    from = max(from, to);
    from_value = value_of(from);   // (behind inf: NaN, which nothing reaches)
  }
};

// Leaves the `top` first candidates, in order. Every entry is another number, so
// ranks are distinct.
__device__ __forceinline__ void compact(Candidates& c, Choice& w, int top) {
  const int lane = threadIdx.x & 63;
  pad(c.list, w.count, CANDIDATES);
  for (int first = 0; first < w.count; first += 64) {
    const int i = first + lane;
    const uint64_t mine = i < w.count ? c.list[i] : 0;
    const int rank = rank_in(c.list, w.count, mine);
    if (i < w.count && rank < top) c.ordered[rank] = mine;
  }
  wave_settled();
  const int left = min(w.count, top);
  if (lane < left) c.list[lane] = c.ordered[lane];
  wave_settled();
  // indices rise from one vector of a wave to the next: an entry equal to the last of these is behind it
  if (w.count >= top) w.raise(static_cast<uint32_t>(c.list[top - 1] >> 32) + 1);
  w.count = left;
}

// Offers a step's entries. `high` is the greatest of each of the lane's vectors.
template <int THREADS, class T>
__device__ __forceinline__ void offer(const Raw<T> (&raw)[UNROLL], const float (&high)[UNROLL], int at, int end,
                                      int top, Candidates& c, Choice& w) {
  float most = high[0];
#pragma unroll
  for (int j = 1; j < UNROLL; ++j) most = fmaxf(most, high[j]);
  if (!__any(most >= w.from_value)) return;
  if (top <= MANY) {
    w.best = fmaxf(w.best, most);
    const uint32_t best[1] = {order_of(w.best)};
    w.raise(reached_by(best, top));
  } else {
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      const bool above = high[j] > w.best;   // (a NaN is not)
      w.second = above ? w.best : fmaxf(w.second, high[j]);
      w.best = above ? high[j] : w.best;
    }
    const uint32_t best[2] = {order_of(w.best), order_of(w.second)};
    w.raise(reached_by(best, top));
  }
#pragma unroll
  for (int j = 0; j < UNROLL; ++j) {
    const unsigned long long hits = __ballot(high[j] >= w.from_value);
    if (hits == 0) continue;
    if (w.count + VEC * __popcll(hits) > CANDIDATES) compact(c, w, top);
    float v[VEC];
    Raw<T> again = raw[j];   // widened once more: kept since the sums, the numbers would take 64 registers
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(again) / 16); ++i) asm("" : "+v"(again.q[i]));
    widen(again, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int index = at + j * THREADS * VEC + e;
      const bool in = v[e] >= w.from_value && index < end;
      const unsigned long long all = __ballot(in);
      if (all == 0) continue;
      const int before = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(all >> 32),
                                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(all), 0));
      if (in) c.list[w.count + before] = entry_of(order_of(v[e]), index);
      w.count += __popcll(all);
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
  __shared__ Candidates found[TOP ? WAVES : 1];
  __shared__ uint64_t last[TOP && WAVES > 1 ? LAST + AT_ONCE : 1];
  __shared__ int counts[WAVES], lasts;
  const int64_t row = blockIdx.x;
  const int64_t token = token_at(a, row);
  if (!counted(a, token)) {
    if (blockIdx.y == 0) write_nothing(a, o, row);
    return;
  }
  const int begin = blockIdx.y * sp.piece, end = min(a.vocab, begin + sp.piece);
  const T* z = static_cast<const T*>(a.logits) + offset_of(a, row, a.ld_seq, a.ld);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int col0 = threadIdx.x * VEC;
  const float token_logit = static_cast<float>(z[token]);
  Candidates& mine = found[TOP ? wave : 0];
  if (TOP && threadIdx.x == 0) lasts = 0;
  Sums r;
  Choice w = {LOWEST, -INFINITY, -INFINITY, -INFINITY, 0};
  for (int base = begin; base < end; base += STEP) {
    float high[UNROLL];
    Raw<T> raw[UNROLL];
    int there = UNROLL;
    if (base + STEP <= end) {
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) raw[j] = fetch(z + base + j * THREADS * VEC + col0);
    } else {
      there = (end - base + THREADS * VEC - 1) / (THREADS * VEC);
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) raw[j] = fetch_upto(z, base + j * THREADS * VEC + col0, end);
    }
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
      float v[VEC];
      widen(raw[j], v);
      high[j] = highest(v);
      if (j < there) take(v, high[j], r);
    }
    end_step(r);
    if constexpr (TOP) offer<THREADS>(raw, high, base + col0, end, a.top, mine, w);
  }
  if constexpr (TOP) {
    mine.best[lane] = order_of(w.best);
    if (lane == 0) counts[wave] = w.count;
    pad(mine.list, w.count, CANDIDATES);
  }
  const float wave_top = wave_max(r.m);
  if (lane == 0) red_m[wave] = wave_top;
  __syncthreads();
  float m = red_m[0];
#pragma unroll
  for (int u = 1; u < WAVES; ++u) m = fmaxf(m, red_m[u]);
  rebase(r, m);
  const double ws = wave_sum64(static_cast<double>(r.all_s)), wt = wave_sum64(static_cast<double>(r.all_t));
  if (lane == 0) {
    red_s[wave] = ws;
    red_t[wave] = wt;
  }
  if constexpr (TOP && WAVES > 1) {   // those of all waves that reach what `top` lanes have reached
    uint32_t best[WAVES];
#pragma unroll
    for (int u = 0; u < WAVES; ++u) best[u] = found[u].best[lane];
    const uint32_t from = reached_by(best, a.top);
    for (int i = lane; i < w.count; i += 64) {
      const uint64_t e = mine.list[i];
      if (static_cast<uint32_t>(e >> 32) >= from) {
        const int at = atomicAdd(&lasts, 1);
        if (at < LAST) last[at] = e;
      }
    }
  }
  __syncthreads();
  double s = 0.0, t = 0.0;
#pragma unroll
  for (int u = 0; u < WAVES; ++u) {
    s += red_s[u];
    t += red_t[u];
  }
  s += OF_E * t;   // (of t itself it is less than a step)
  const bool whole = sp.pieces == 1;
  const int64_t part = row * sp.pieces + blockIdx.y;
  if (threadIdx.x == 0) {
    if (whole) write_row(o, row, token_logit, m, s, t);
    else parts[part] = {m, s, t};
  }
  if constexpr (TOP) {
    const double log_s = whole ? log(s) : 0.0;
    auto put = [&](int rank, uint64_t e) {
      if (rank >= a.top) return;
      if (whole) write_entry(a, o, row, rank, e, m, log_s);
      else entries[part * a.top + rank] = e;
    };
    const int left = WAVES > 1 ? lasts : w.count;
    if (WAVES > 1 && left <= LAST) {
      if (wave == 0) pad(last, left, LAST + AT_ONCE);
      __syncthreads();
      for (int i = threadIdx.x; i < left; i += THREADS) put(rank_in(last, left, last[i]), last[i]);
    } else {   // one wave, or many equal entries: ranks among all candidates
      for (int i = lane; i < w.count; i += 64) {
        int rank = 0;
        for (int u = 0; u < WAVES; ++u) rank += rank_in(found[u].list, counts[u], mine.list[i]);
        put(rank, mine.list[i]);
      }
    }
    for (int rank = left + threadIdx.x; rank < a.top; rank += THREADS) put(rank, 0);   // short, or NaN
  }
}

// Makes one row of its pieces.
constexpr int JOIN_THREADS = 256;
template <class T>
__global__ __launch_bounds__(JOIN_THREADS) void join_kernel(LogpsArgs a, int pieces,
                                                            const LogpsPart* parts,
                                                            const uint64_t* entries, LogpsOut o) {
  __shared__ uint64_t list[LOGPS_JOIN + AT_ONCE];
  const int64_t row = blockIdx.x;
  const int64_t token = token_at(a, row);
  if (!counted(a, token)) return;   // written by the row's first piece
  const LogpsPart* p = parts + row * pieces;
  const int all = pieces * a.top;
  for (int i = threadIdx.x; i < all + AT_ONCE; i += JOIN_THREADS) list[i] = i < all ? entries[row * all + i] : 0;
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
    write_row(o, row, static_cast<float>(static_cast<const T*>(a.logits)[offset_of(a, row, a.ld_seq, a.ld) + token]), m, s, t);
  __syncthreads();
  const double log_s = log(s);
  for (int i = threadIdx.x; i < all; i += JOIN_THREADS) {
    const uint64_t mine = list[i];
    int rank = rank_in(list, all, mine);
    if (mine == 0)   // empty places are equal: they are told apart by where they stand
      for (int k = 0; k < i; ++k) rank += list[k] == 0;
    if (rank < a.top) write_entry(a, o, row, rank, mine, m, log_s);
  }
}

// --------------------------------------------------------------- gradient

// How many elements behind a boundary of N of them an address lies.
template <int N, class T>
__device__ __forceinline__ int behind_boundary(const T* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) / sizeof(T) % N);
}

// Workgroups take a step each, in the order of the addresses. A lane's vectors are 16
// bytes each, so that a wave stores whole lines in fp32 too (5913 rows of 21273: 183 us,
// 293 with 32 bytes a lane). In long 16-bit rows they begin where the row's gradient is
// 16-byte aligned (2048 rows of 128001: 196 us, 208 with vectors from the row's first element;
// 5913 of 21273 112 and 127; 16000 of 2001 32.1 and 31.8). The sums above are laid from a row's
// first element all the same: their order, and with it their last bits, would
// depend on where the logits lie.
constexpr int GRAD_UNROLL = 8, LONG = 4096;
template <class T>
constexpr int GRAD_VEC = 16 / sizeof(T);
template <class T>
constexpr int grad_step(int threads) {
  return threads * GRAD_VEC<T> * GRAD_UNROLL;
}
template <class T>
union Sixteen {
  Quad q;
  T e[GRAD_VEC<T>];
};
template <class T, int THREADS, bool ENTROPY>
__global__ __launch_bounds__(THREADS) void logps_grad_kernel(LogpsArgs a, const float* lse,
                                                             const float* entropy, const float* dlogps,
                                                             const float* dentropy, T* dlogits,
                                                             int64_t ld_dlogits, int64_t ld_dseq, int steps) {
  constexpr int N = GRAD_VEC<T>, U = GRAD_UNROLL;
  const int64_t all = static_cast<int64_t>(a.rows) * steps;
  for (int64_t block = blockIdx.x; block < all; block += gridDim.x) {
    const int row = static_cast<int>(block / steps);
    T* d = dlogits + offset_of(a, row, ld_dseq, ld_dlogits);
    const T* z = static_cast<const T*>(a.logits) + offset_of(a, row, a.ld_seq, a.ld);
    const int base = static_cast<int>(block - static_cast<int64_t>(row) * steps) * grad_step<T>(THREADS) -
                     (sizeof(T) == 2 && a.vocab >= LONG ? behind_boundary<N>(d) : 0);
    const int first = base + static_cast<int>(threadIdx.x) * N;
    const int64_t token = token_at(a, row);
    const bool counts = counted(a, token);
    Sixteen<T> x[U];
    if (counts) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (base + j * THREADS * N >= a.vocab) break;
        const int at = first + j * THREADS * N;
        if (at >= 0 && at + N <= a.vocab) {
          x[j].q = __builtin_nontemporal_load(reinterpret_cast<const Quad*>(z + at));
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) x[j].e[e] = at + e >= 0 && at + e < a.vocab ? z[at + e] : static_cast<T>(0.f);
        }
      }
    }
    const float l = counts ? lse[row] : 0.f, g = counts && dlogps ? dlogps[row] : 0.f;
    const float h = ENTROPY && counts ? dentropy[row] : 0.f, H = ENTROPY && counts ? entropy[row] : 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (base + j * THREADS * N >= a.vocab) break;
      const int at = first + j * THREADS * N;
      Sixteen<T> y;
      float v[N];
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = static_cast<float>(x[j].e[e]) - l;
      float low = v[0];
#pragma unroll
      for (int e = 1; e < N; ++e) low = fminf(low, v[e]);
      auto put = [&](int e, float v) {
        const float p = exp_exact(v), slope = ENTROPY ? fmaf(h, v + H, g) : g;
        y.e[e] = static_cast<T>(counts ? fmaf(-p, slope, at + e == token ? g : 0.f) : 0.f);
      };
      if (__any(low < -FAR)) {   // an entry at -inf has no share, and p log p goes to 0; a NaN stays one
#pragma unroll
        for (int e = 0; e < N; ++e) put(e, v[e] < -FAR ? -FAR : v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) put(e, v[e]);
      }
      if (at >= 0 && at + N <= a.vocab) {
        __builtin_nontemporal_store(y.q, reinterpret_cast<Quad*>(d + at));
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (at + e >= 0 && at + e < a.vocab) d[at + e] = y.e[e];
      }
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
  // Where many entries are wanted, pieces of about one length: nearly all of a short last one's
  // would be candidates (8 rows of 50021, top 64: 20 us, 43 with a piece of 869; top 20: 22.9 and 21.8).
  if (top > MANY && sp.pieces > 1) {
    const int unit = (vocab <= SHORT_VOCAB ? 64 : 256) * VEC;
    sp.piece = static_cast<int>(((vocab + sp.pieces - 1) / sp.pieces + unit - 1) / unit * unit);
    sp.pieces = static_cast<int>((vocab + sp.piece - 1) / sp.piece);
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
    hipError_t e = a.vocab <= one_wave_vocab(a.rows, a.top) ? shaped(std::integral_constant<int, 64>{})
                                          : shaped(std::integral_constant<int, 256>{});
    if (e != hipSuccess || sp.pieces == 1) return e;
    hipLaunchKernelGGL(join_kernel<T>, dim3(static_cast<unsigned>(a.rows)), dim3(JOIN_THREADS), 0, stream,
                       a, sp.pieces, parts, entries, o);
    return hipGetLastError();
  });
}

hipError_t launch_token_logps_grad(const LogpsArgs& a, int type, const float* lse, const float* entropy,
                                   const float* dlogps, const float* dentropy, void* dlogits,
                                   int64_t ld_dlogits, int64_t ld_dseq, hipStream_t stream) {
  const int threads = a.vocab <= SHORT_VOCAB ? 64 : 256;
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    // (a row may begin up to a vector behind the first one's)
    const int step = grad_step<T>(threads), steps = (a.vocab + GRAD_VEC<T> - 1 + step - 1) / step;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(a.rows) * steps, 1 << 23)));
    auto go = [&](auto n, auto with) {
      constexpr int N = n();
      constexpr bool E = with();
      hipLaunchKernelGGL((logps_grad_kernel<T, N, E>), grid, dim3(N), 0, stream, a, lse, entropy, dlogps,
                         dentropy, static_cast<T*>(dlogits), ld_dlogits, ld_dseq, steps);
      return hipGetLastError();
    };
    auto shaped = [&](auto n) { return dentropy ? go(n, std::true_type{}) : go(n, std::false_type{}); };
    return threads == 64 ? shaped(std::integral_constant<int, 64>{})
                         : shaped(std::integral_constant<int, 256>{});
  });
}

}  // namespace nsmi
