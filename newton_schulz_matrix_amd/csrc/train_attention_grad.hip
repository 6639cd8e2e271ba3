// Gradient of causal attention over packed sequences with grouped heads.
//
//   P = exp(S - lse), S = scale q k^T;   delta = sum of dout out over a head's columns
//   dv = P^T dout,  dS = P (dout v^T - delta),  dq = scale dS k,  dk = scale dS^T q
//
// Bound by the matrix units, at 1.9 GHz of 2.4. Two launches: dq, where a workgroup keeps 128 queries and
// goes over the keys before them, and which leaves delta of its rows; dk and dv,
// where it keeps 128 keys of one key head and goes over the queries of its group's
// heads behind them. S and dout v^T are worked out in both (seven products instead of five): the
// alternative, adding to dq from every workgroup of keys, would need atomics, whose
// order changes the sums, or a place for every pair of tiles. Everything is laid out
// as in the forward pass: the weights of a lane are one row or column, and go on as
// the next product's operand.
//
// Measured, bf16, 32 heads of 128 that read 8, 16256 tokens of eight sequences of 0 to 5113:
// dq 690 us, dk and dv 890 (1.12 TFLOP that the gradient cannot do without, 1.57 with S and
// dout v^T again: 990 TFLOP/s; a library product of 8192 cubed reaches 1180).
//
// fp16: weights and dS of a long row lie among its subnormals. Weights are taken
// times 2^14, and dS times a power of two that keeps the largest one possible
// below 2^14; both are taken back from the sums in fp32. What a row's dS may reach is
// |dout| max |v| + |delta|, over the keys before its tile's end: dq's power of two is
// the row's own, that of dk the greatest of the rows behind the keys in their sequence
// and group of heads. No other sequence and no other group of heads has a part in it,
// and rows that are not finite have none (theirs are NaN whatever they are scaled by).
#include <algorithm>
#include <type_traits>

#include "attention_device.h"
#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int WAVES = 4, THREADS = 64 * WAVES;
constexpr int ROWS = 32 * WAVES;      // queries or keys that a workgroup keeps
constexpr int STEP = 64;              // rows of the tiles that it goes over
constexpr float LOG2E = 1.442695041f;

template <class T>
constexpr bool NARROW = false;        // whether the type needs the scaling
template <>
constexpr bool NARROW<_Float16> = true;
constexpr float LIFT = 14.f;

// What dS is multiplied by, for fp16, if it may reach `most`.
__device__ __forceinline__ float ds_scale(float most) {
  if (!(most > 0.f && most < INFINITY)) return 1.f;
  int e;
  frexpf(most, &e);
  return ldexpf(1.f, min(max(14 - e, -60), 60));
}

// Greatest finite of `lines` times n numbers, `apart` from one line to the next, for all of
// a workgroup (at least 0).
template <int WAVES_OF>
__device__ __forceinline__ float greatest(const float* p, int lines, int64_t apart, int n, float (&tops)[WAVES_OF]) {
  float top = 0.f;
  for (int line = 0; line < lines; ++line, p += apart)
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += 64 * WAVES_OF) top = p[i] < INFINITY ? fmaxf(top, p[i]) : top;
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES_OF; ++w) top = fmaxf(top, tops[w]);
  return top;
}

// fp16: the norms of v's rows, 16 lanes a row.
constexpr int NORM_THREADS = 256, NORM_ROWS = NORM_THREADS / 16, NORM_BLOCKS = 2048;
template <class T>
__global__ __launch_bounds__(NORM_THREADS) void norms_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 15;
  const int first = offset_at(a.offsets, 0, a.tokens), last = offset_at(a.offsets, a.sequences, a.tokens);
  const int64_t rows = static_cast<int64_t>(last - first) * a.k_heads;
  for (int64_t row = blockIdx.x * NORM_ROWS + threadIdx.x / 16; row - threadIdx.x / 16 < rows;
       row += static_cast<int64_t>(gridDim.x) * NORM_ROWS) {
    const int64_t token = first + row / a.k_heads;
    const int head = static_cast<int>(row % a.k_heads);
    float norm = 0.f;
    if (row < rows && 8 * lane < a.dim) {
      float x[VEC];
      load8(static_cast<const T*>(a.v.p) + token * a.v.token + head * a.v.head + 8 * lane, x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) norm = fmaf(x[e], x[e], norm);
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) norm += __shfl_xor(norm, off, 64);
    if (row < rows && lane == 0) a.v_norms[head * static_cast<int64_t>(a.tokens) + token] = sqrtf(norm);
  }
}

// Rows behind the last sequence: zeros.
template <class T>
__device__ __forceinline__ void clear_rows(const HeadsAt& to, int head, int dim, int first, int last) {
  const int threads = blockDim.x;
  T* p = static_cast<T*>(to.p) + head * to.head;
  const int chunks = dim / 8, n = (last - first) * chunks;
  const U32x4 zero = {0, 0, 0, 0};
  for (int i = threadIdx.x; i < n; i += threads)
    *reinterpret_cast<U32x4*>(p + (first + i / chunks) * to.token + i % chunks * 8) = zero;
}

// ------------------------------------------------------------------------ dq

// 32 queries a wave. With two SIDES eight waves share 128 queries, each half of every
// tile's keys, and add up at the end: for launches that leave most of a CU empty. The
// rows' delta, lse log2(e) and what their dS may reach are left for the kernel below.
template <class T, int DP, int SIDES>
__global__ __launch_bounds__(THREADS * SIDES, 2) void dq_kernel(AttnArgs a, int tiles, int parts, float* sums) {
  typedef typename Eight<T>::type V8;
  constexpr int KC = DP / 16, DT = DP / 32;
  constexpr int TILE = STEP * Tile<DP>::ROW;
  __shared__ __attribute__((aligned(1024))) char smem[4 * TILE];   // keys, values, twice
  static_assert(4 * TILE >= ROWS * DP * 4, "the sums of one side fit in the tiles");
  __shared__ float tops[WAVES * SIDES];
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int side = wave / WAVES;
  const Share share = share_of(tiles * a.q_heads, parts);
  if (share.block < 0) return;
  const int part = share.part;
  const Work w = work_of(share.block, a.q_heads, a.k_heads);
  const Place at = place_of<ROWS, false>(a.offsets, a.sequences, a.tokens, tiles, w.tile);
  if (at.length == 0) return;
  if (at.rest) {
    if (a.clear_rest && part == 0)
      clear_rows<T>(a.dq, w.head, a.dim, at.begin + at.row, min(at.begin + at.row + ROWS, at.begin + at.length));
    return;
  }
  const int kv_head = w.head / (a.q_heads / a.k_heads);
  const T* k = static_cast<const T*>(a.k.p) + at.begin * a.k.token + kv_head * a.k.head;
  const T* v = static_cast<const T*>(a.v.p) + at.begin * a.v.token + kv_head * a.v.head;
  const uint32_t k_step = static_cast<uint32_t>(a.k.token * 2), v_step = static_cast<uint32_t>(a.v.token * 2);
  const Copier<DP, STEP, WAVES * SIDES> k_copy(wave, lane, k_step, a.dim), v_copy(wave, lane, v_step, a.dim);
  const uint32_t lds = lds_address(smem);
  const int keys = min(at.length, at.row + ROWS);
  const Range range = range_of((keys + STEP - 1) / STEP, part, parts);
  const int steps = range.last;
  auto fetch_tile = [&](int n) {
    const uint32_t to = lds + (n & 1) * 2 * TILE;
    const int first = n * STEP;
    k_copy.copy(k + first * a.k.token, at.length - first, k_step, a.dim, to);
    v_copy.copy(v + first * a.v.token, at.length - first, v_step, a.dim, to + TILE);
  };
  if (range.first < steps) fetch_tile(range.first);

  const int first_query = at.row + 32 * (wave % WAVES), query = first_query + (lane & 31);
  const bool there = query < at.length;
  const int last_query = first_query < at.length ? first_query + 31 : -1;   // none: it only brings tiles in
  const int64_t token = at.begin + query;
  V8 q[KC], g[KC];
  load_operands<T, DP>(there ? static_cast<const T*>(a.q.p) + token * a.q.token + w.head * a.q.head : nullptr,
                       a.dim, half, q);
  load_operands<T, DP>(there ? static_cast<const T*>(a.dout.p) + token * a.dout.token + w.head * a.dout.head : nullptr,
                       a.dim, half, g);
  float dot = 0.f, norm = 0.f;
  {
    V8 o[KC];
    load_operands<T, DP>(there ? static_cast<const T*>(a.out.p) + token * a.out.token + w.head * a.out.head : nullptr,
                         a.dim, half, o);
#pragma unroll
    for (int j = 0; j < KC; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dot = fmaf(static_cast<float>(g[j][e]), static_cast<float>(o[j][e]), dot);
        if (NARROW<T>) norm = fmaf(static_cast<float>(g[j][e]), static_cast<float>(g[j][e]), norm);
      }
  }
  float lower, upper;
  both_halves(dot, lower, upper);
  dot = lower + upper;
  float scaled = 1.f;   // each lane its query's
  if constexpr (NARROW<T>) {
    const float* norms = a.v_norms + kv_head * static_cast<int64_t>(a.tokens) + at.begin;
    both_halves(norm, lower, upper);
    norm = fmaf(sqrtf(lower + upper), greatest(norms, 1, 0, keys, tops), fabsf(dot));
    scaled = ds_scale(norm);
  }
  const int64_t stat = static_cast<int64_t>(w.head) * a.tokens + token;
  float lse2 = there ? a.lse[stat] * LOG2E : 0.f;
  if (there && half == 0 && side == 0 && part == 0) {
    a.delta[stat] = -dot;
    a.lse2[stat] = (NARROW<T> ? LIFT : 0.f) - lse2;
    if (NARROW<T>) a.reach[stat] = norm;
  }
  const float to_ds = NARROW<T> ? scaled * (1.f / 16384.f) : 1.f;
  const float delta = dot * to_ds;
  if (NARROW<T>) lse2 -= LIFT;
  const RowReader<DP> rows(lane);
  const ColumnReader<DP> columns(lane);
  const float c = a.scale * LOG2E;
  Acc dq[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) dq[t] = no_sum();

  for (int n = range.first; n < steps; ++n) {
    copies_done();
    __syncthreads();
    if (n + 1 < steps) fetch_tile(n + 1);
    // (one side: both halves of the tile, one after the other)
    const int key1 = n * STEP + 32 * side;
    const uint32_t tile = lds + (n & 1) * 2 * TILE + 32 * side * Tile<DP>::ROW;
    const auto kt = rows.in(tile);
    const auto kc = columns.in(tile);
#pragma unroll
    for (int i = 0; i < STEP / 32 / SIDES; ++i) {
      const int key0 = key1 + 32 * i, at_row = 32 * i * Tile<DP>::ROW;
      if (key0 > last_query) break;
      Acc s = no_sum(), dp = no_sum();
#pragma unroll
      for (int j = 0; j < KC; ++j) s = product(kt.template read<T>(j, at_row), q[j], s);
#pragma unroll
      for (int j = 0; j < KC; ++j) dp = product(kt.template read<T>(j, at_row + TILE), g[j], dp);
#pragma unroll
      for (int r = 0; r < 16; ++r)
        s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse2)) *
               (NARROW<T> ? fmaf(dp[r], to_ds, -delta) : dp[r] - delta);
      if (key0 + 31 > first_query) {   // some keys lie behind some queries
        const int hidden = query - key0 - 4 * half;   // rows above it are
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = 8 * (r / 4) + r % 4 > hidden ? 0.f : s[r];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const V8 ds = operand<T>(s, j);   // rounded to T, half a step each
#pragma unroll
        for (int t = 0; t < DT; ++t)
          dq[t] = product(kc.template read<T>(t, at_row + 16 * j * Tile<DP>::ROW), ds, dq[t]);
      }
    }
  }
  if constexpr (SIDES == 2) {
    __syncthreads();
    float* const shared = reinterpret_cast<float*>(smem) + wave % WAVES * 64 * DP / 2 + lane;
    if (side == 1) {
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) shared[64 * (16 * t + r)] = dq[t][r];
    }
    __syncthreads();
    if (side == 1) return;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) dq[t][r] += shared[64 * (16 * t + r)];
  }
  if (parts > 1) {
    const int64_t row = (static_cast<int64_t>(part) * a.q_heads + w.head) * a.tokens + token;
    store_sums<DP>(there ? sums + row * a.dim : nullptr, a.dim, half, dq, a.scale / scaled);
    return;
  }
  T* to = static_cast<T*>(a.dq.p) + token * a.dq.token + w.head * a.dq.head;
  store_columns<T, DP>(there ? to : nullptr, a.dim, half, dq, a.scale / scaled);
}

// ----------------------------------------------------------------- dk and dv

// Eight waves: four times 32 keys, and of every tile of queries each half. The two
// waves of the same keys add up their sums at the end: the longest workgroup, which
// keeps the first keys of the longest sequence, is done in half the time so.
constexpr int KV_WAVES = 8, KV_THREADS = 64 * KV_WAVES;
constexpr int KV_STEP = 128;          // queries of a tile

// The products come in the order they are written in, each operand read AHEAD, the
// weights' exponentials between those of dout v^T: left to itself the compiler puts every
// read right before its product, and the kernel takes 14% more cycles (5% more time: the
// clock falls with the work in each of them). The registers for it (two waves of 256 a
// SIMD) come from the second half of a wave's keys, which lies in LDS for heads above 64,
// and from addresses that are made where they are used.
constexpr int KEY_CHUNKS = 4;         // of 16 columns in registers
__device__ __forceinline__ float4 read4(const __attribute__((address_space(3))) float4* p) {
  typedef float F4 __attribute__((ext_vector_type(4)));
  const F4 v = *(const __attribute__((address_space(3))) F4*)p;
  return make_float4(v[0], v[1], v[2], v[3]);
}

// Where the keys alone would not fill the chip, `parts` workgroups share the
// queries of the same keys, and leave their sums in fp32 for a kernel that adds
// them up in order.
template <class T, int DP>
__global__ __launch_bounds__(KV_THREADS, 2) void dkv_kernel(AttnArgs a, int tiles, int parts, float* sums) {
  typedef typename Eight<T>::type V8;
  constexpr int KC = DP / 16, DT = DP / 32;
  constexpr int TILE = KV_STEP * Tile<DP>::ROW, STATS = 2 * KV_STEP * 4, STAGE = 2 * TILE + STATS;
  static_assert(KC == KEY_CHUNKS || 16 * (KC - KEY_CHUNKS) == 64, "the keys' second half is a tile of 64 columns");
  static_assert(2 * STAGE >= 2 * ROWS * DP * 4, "both sums of half the waves fit in the tiles");
  constexpr int KR = std::min(KC, KEY_CHUNKS), KL = KC - KR;   // key chunks in registers, in LDS
  // queries, dout, lse, delta, twice, and the keys' second half
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE + (KL ? ROWS * Tile<64>::ROW : 0)];
  __shared__ float tops[KV_WAVES];
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int side = wave / 4;           // of a tile's queries
  const Share share = share_of(tiles * a.k_heads, parts);
  if (share.block < 0) return;
  const int part = share.part;
  const Work w = work_of(share.block, a.k_heads, a.k_heads);
  const Place at = place_of<ROWS, true>(a.offsets, a.sequences, a.tokens, tiles, w.tile);
  if (at.length == 0) return;
  if (at.rest) {
    if (a.clear_rest && part == 0) {
      const int first = at.begin + at.row, last = min(first + ROWS, at.begin + at.length);
      clear_rows<T>(a.dk, w.head, a.dim, first, last);
      clear_rows<T>(a.dv, w.head, a.dim, first, last);
    }
    return;
  }
  const int group = a.q_heads / a.k_heads;
  const T* q = static_cast<const T*>(a.q.p) + at.begin * a.q.token + w.head * group * a.q.head;
  const T* g = static_cast<const T*>(a.dout.p) + at.begin * a.dout.token + w.head * group * a.dout.head;
  const int64_t stat0 = static_cast<int64_t>(w.head) * group * a.tokens + at.begin;
  const uint32_t q_step = static_cast<uint32_t>(a.q.token * 2), g_step = static_cast<uint32_t>(a.dout.token * 2);
  const Copier<DP, KV_STEP, KV_WAVES> q_copy(wave, lane, q_step, a.dim), g_copy(wave, lane, g_step, a.dim);
  const uint32_t lds = lds_address(smem);
  const int begin = at.row / KV_STEP;
  const int each = (at.length + KV_STEP - 1) / KV_STEP - begin;   // >= 1
  const Range range = range_of(static_cast<int64_t>(each) * group, part, parts);
  const int steps = range.last;
  auto fetch_tile = [&](int n) {
    const uint32_t to = lds + (n & 1) * STAGE;
    const int h = n / each, first = (begin + n - h * each) * KV_STEP, rows = at.length - first;
    q_copy.copy(q + h * a.q.head + first * a.q.token, rows, q_step, a.dim, to);
    g_copy.copy(g + h * a.dout.head + first * a.dout.token, rows, g_step, a.dim, to + TILE);
    if (wave < 4) {   // lse and delta of 64 rows each
      const int row = 64 * (wave & 1), left = min(rows - row, 64);
      const float* from = (wave < 2 ? a.lse2 : a.delta) + stat0 + static_cast<int64_t>(h) * a.tokens + first + row;
      copy4(descriptor(from, left > 0 ? 4 * left : 0), to + 2 * TILE + wave * 64 * 4, 4 * lane);
    }
  };
  if (range.first < steps) {
    fetch_tile(range.first);
    if constexpr (KL > 0) {
      const uint32_t k_step = static_cast<uint32_t>(a.k.token * 2);
      const int further = 16 * KR, left = a.dim - further;
      const Copier<64, ROWS, KV_WAVES> k_copy(wave, lane, k_step, left);
      k_copy.copy(static_cast<const T*>(a.k.p) + (at.begin + at.row) * a.k.token + w.head * a.k.head + further,
                  at.length - at.row, k_step, left, lds + 2 * STAGE);
    }
  }

  const int first_key = at.row + 32 * (wave & 3), key = first_key + (lane & 31);
  const bool there = key < at.length;
  const int64_t token = at.begin + key;
  V8 k[KR], v[KC];
  load_operands<T, 16 * KR>(there ? static_cast<const T*>(a.k.p) + token * a.k.token + w.head * a.k.head : nullptr,
                            min(a.dim, 16 * KR), half, k);
  load_operands<T, DP>(there ? static_cast<const T*>(a.v.p) + token * a.v.token + w.head * a.v.head : nullptr,
                       a.dim, half, v);
  float scaled = 1.f;
  if constexpr (NARROW<T>)
    scaled = ds_scale(greatest(a.reach + stat0 + at.row, group, a.tokens, at.length - at.row, tops));
  const float to_ds = NARROW<T> ? scaled * (1.f / 16384.f) : 1.f;
  const RowReader<DP> rows(lane);
  const auto k_rows = RowReader<64>(lane).in(lds + 2 * STAGE + 32 * (wave & 3) * Tile<64>::ROW);
  const ColumnReader<DP> columns(lane);
  const float c = a.scale * LOG2E;
  Acc dk[DT], dv[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) dk[t] = dv[t] = no_sum();

  for (int n = range.first; n < steps; ++n) {
    copies_done();
    __syncthreads();
    if (n + 1 < steps) fetch_tile(n + 1);
    const int first_query = (begin + n % each) * KV_STEP;
    const uint32_t qt = lds + (n & 1) * STAGE;
#pragma unroll 1
    for (int i = 0; i < KV_STEP / 64; ++i) {
      const int row0 = 64 * i + 32 * side, query0 = first_query + row0;
      if (query0 + 31 < first_key || max(query0, first_key) >= at.length) continue;
      const auto qr = rows.lean_in(qt + row0 * Tile<DP>::ROW);   // dout's tile lies TILE behind
      const auto qc = columns.lean_in(qt + row0 * Tile<DP>::ROW);
      const __attribute__((address_space(3))) float4* const stats =
          (const __attribute__((address_space(3))) float4*)(qt + 2 * TILE) + row0 / 4 + half;
      // The products in their order, and what each reads: S, dout v^T, then dv and dk
      // by halves of the queries and 32 columns.
      constexpr int ROW_READS = 2 * KC, READS = ROW_READS + 4 * DT;
      V8 read[READS], kl[KL > 0 ? KL : 1];
      auto fetch = [&](int n) {
        if (n >= READS) return;
        if (n < ROW_READS) {
          read[n] = qr.template read<T>(n % KC, n / KC * TILE);
          if (n >= KR && n < KC) kl[n - KR] = k_rows.template read<T>(n - KR, 0);
        } else {
          const int m = n - ROW_READS;
          read[n] = qc.template read<T>(m % DT, (m < 2 * DT ? TILE : 0) + 16 * (m / DT % 2) * Tile<DP>::ROW);
        }
      };
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) fetch(n);
      Acc s = no_sum(), dp;
      float4 lse;
      auto weights = [&](int g) {
        s[4 * g] = __builtin_amdgcn_exp2f(fmaf(s[4 * g], c, lse.x));
        s[4 * g + 1] = __builtin_amdgcn_exp2f(fmaf(s[4 * g + 1], c, lse.y));
        s[4 * g + 2] = __builtin_amdgcn_exp2f(fmaf(s[4 * g + 2], c, lse.z));
        s[4 * g + 3] = __builtin_amdgcn_exp2f(fmaf(s[4 * g + 3], c, lse.w));
      };
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 x = read4(stats + KV_STEP / 4 + 2 * g);   // -delta
        dp[4 * g] = x.x, dp[4 * g + 1] = x.y, dp[4 * g + 2] = x.z, dp[4 * g + 3] = x.w;
      }
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        fetch(j + AHEAD);
        in_order();
        s = product(read[j], j < KR ? k[j] : kl[j - KR], s);
        in_order();
      }
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        fetch(KC + j + AHEAD);
        in_order();
        dp = product(read[KC + j], v[j], dp);
        in_order();
        if (j * 4 % KC == 0) {   // weights of four rows meanwhile
          const int g = j * 4 / KC;
          if (g > 0) weights(g - 1);
          lse = read4(stats + 2 * g);   // LIFT - lse2
        }
      }
      weights(3);
#pragma unroll
      for (int r = 0; r < 16; ++r) dp[r] = NARROW<T> ? s[r] * (dp[r] * to_ds) : s[r] * dp[r];
      if (query0 < first_key + 31) {   // some keys lie behind some queries
        const int hidden = key - query0 - 4 * half;   // rows below it are
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[r] = 8 * (r / 4) + r % 4 < hidden ? 0.f : s[r];
          dp[r] = 8 * (r / 4) + r % 4 < hidden ? 0.f : dp[r];
        }
      }
      // rounded to T, half a step each
      const V8 p[2] = {operand<T>(s, 0), operand<T>(s, 1)}, ds[2] = {operand<T>(dp, 0), operand<T>(dp, 1)};
#pragma unroll
      for (int m = 0; m < 4 * DT; ++m) {
        const int j = m / DT % 2, t = m % DT;
        fetch(ROW_READS + m + AHEAD);
        in_order();
        if (m < 2 * DT) dv[t] = product(read[ROW_READS + m], p[j], dv[t]);
        else dk[t] = product(read[ROW_READS + m], ds[j], dk[t]);
        in_order();
      }
    }
  }

  // the first four waves finish dk, the others dv
  __syncthreads();
  float* const shared = reinterpret_cast<float*>(smem) + (wave & 3) * 64 * DP / 2 + lane;
  float* const give = shared + (side ? 0 : 2 * 64 * DP);
  float* const take = shared + (side ? 2 * 64 * DP : 0);
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) give[64 * (16 * t + r)] = side ? dk[t][r] : dv[t][r];
  __syncthreads();
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[t][r] = (side ? dv[t][r] : dk[t][r]) + take[64 * (16 * t + r)];
  const float by = side == 0 ? a.scale / scaled : NARROW<T> ? 1.f / 16384.f : 1.f;
  if (parts == 1) {
    const HeadsAt& to = side ? a.dv : a.dk;
    T* row = static_cast<T*>(to.p) + token * to.token + w.head * to.head;
    store_columns<T, DP>(there ? row : nullptr, a.dim, half, dk, by);
  } else {
    const int64_t row = ((static_cast<int64_t>(part) * 2 + side) * a.k_heads + w.head) * a.tokens + token;
    store_sums<DP>(there ? sums + row * a.dim : nullptr, a.dim, half, dk, by);
  }
}

// Adds up the parts' sums, of one tensor or of two one behind the other, eight columns a lane.
template <class T>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, HeadsAt first, HeadsAt second, int heads, int parts,
                                                   const float* sums) {
  const int chunks = a.dim / 8, head = blockIdx.y % heads;
  const int i = blockIdx.x * 256 + threadIdx.x, token = i / chunks, column = i % chunks * 8;
  if (token < offset_at(a.offsets, 0, a.tokens) || token >= offset_at(a.offsets, a.sequences, a.tokens)) return;
  const int64_t one = static_cast<int64_t>(gridDim.y) * a.tokens * a.dim;
  const float* from = sums + (static_cast<int64_t>(blockIdx.y) * a.tokens + token) * a.dim + column;
  float v[VEC];
  load8(from, v);
  for (int k = 1; k < parts; ++k) {
    float x[VEC];
    load8(from + k * one, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] += x[e];
  }
  const HeadsAt& to = static_cast<int>(blockIdx.y) < heads ? first : second;
  store8(static_cast<T*>(to.p) + token * to.token + head * to.head + column, v);
}

}  // namespace

hipError_t launch_attention_grad(const AttnArgs& a, int type, int q_parts, int k_parts, float* sums,
                                 hipStream_t stream) {
  const int64_t tiles = tiles_of(a.tokens, a.sequences, ROWS);
  auto on = [&](auto t, auto dp) {
    using T = decltype(t);
    constexpr int DP = dp();
    if constexpr (NARROW<T>) {
      const int64_t rows = static_cast<int64_t>(a.tokens) * a.k_heads;
      hipLaunchKernelGGL(norms_kernel<T>, dim3(std::min<int64_t>((rows + NORM_ROWS - 1) / NORM_ROWS, NORM_BLOCKS)),
                         dim3(NORM_THREADS), 0, stream, a);
    }
    auto join = [&](int tensors, const HeadsAt& first, const HeadsAt& second, int heads, int parts) {
      if (parts > 1)
        hipLaunchKernelGGL(join_kernel<T>, dim3((a.tokens * (a.dim / 8) + 255) / 256, tensors * heads), dim3(256), 0,
                           stream, a, first, second, heads, parts, sums);
    };
    auto queries = [&](auto sides) {
      constexpr int SIDES = sides();
      hipLaunchKernelGGL((dq_kernel<T, DP, SIDES>), dim3(shared_blocks(tiles * a.q_heads, q_parts)),
                         dim3(THREADS * SIDES), 0, stream, a, static_cast<int>(tiles), q_parts, sums);
    };
    if (two_sides(tiles * a.q_heads * q_parts, a.tokens, a.sequences)) queries(std::integral_constant<int, 2>{});
    else queries(std::integral_constant<int, 1>{});
    join(1, a.dq, a.dq, a.q_heads, q_parts);
    hipLaunchKernelGGL((dkv_kernel<T, DP>), dim3(shared_blocks(tiles * a.k_heads, k_parts)),
                       dim3(KV_THREADS), 0, stream, a, static_cast<int>(tiles), k_parts, sums);
    join(2, a.dk, a.dv, a.k_heads, k_parts);
    return hipGetLastError();
  };
  auto shaped = [&](auto t) {
    return a.dim <= 64 ? on(t, std::integral_constant<int, 64>{}) : on(t, std::integral_constant<int, 128>{});
  };
  return type == NS_DT_BF16 ? shaped(__bf16{}) : shaped(_Float16{});
}

}  // namespace nsmi
