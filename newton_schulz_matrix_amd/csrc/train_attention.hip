// Causal attention over packed sequences with grouped heads.
//
//   S = scale q k^T (keys up to the query's own position), out = softmax(S) v,
//   lse = log sum exp S
//
// Bound by the matrix units, and close behind them by the exponentials. A
// workgroup takes 128 queries of one head, 32 a wave, and goes over the keys up
// to its last query in tiles of 64, with the running maximum and sum of each row. Products are
// taken transposed (keys x queries, columns x queries): a lane then holds one
// query, a row's maximum and sum are its own registers and one exchange, and the
// weights are the next product's operand as they stand. Keys and values come
// into LDS directly, the next tile while this one is worked on.
#include <algorithm>
#include <type_traits>

#include "attention_device.h"
#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int WAVES = 4, THREADS = 64 * WAVES;
constexpr int QUERIES = 32 * WAVES;   // of a workgroup
constexpr int KEYS = 64;              // of a tile

// The weights of a row stand against a reference that trails its running maximum
// by up to 2^LAG: the sums are rescaled only where it falls further behind. For fp16
// the reference lies 2^7 lower, which keeps small weights out of its subnormals.
constexpr float LAG = 8.f;
template <class T>
constexpr float LIFT = 0.f;
template <>
constexpr float LIFT<_Float16> = 7.f;

// Rows behind the last sequence: zeros.
template <class T>
__device__ __forceinline__ void clear_rows(const AttnArgs& a, int head, int first, int last) {
  T* out = static_cast<T*>(a.out.p) + head * a.out.head;
  const int threads = blockDim.x;
  const int chunks = a.dim / 8, n = (last - first) * chunks;
  const U32x4 zero = {0, 0, 0, 0};
  for (int i = threadIdx.x; i < n; i += threads)
    *reinterpret_cast<U32x4*>(out + (first + i / chunks) * a.out.token + i % chunks * 8) = zero;
  for (int r = first + threadIdx.x; r < last; r += threads) a.lse[static_cast<int64_t>(head) * a.tokens + r] = 0.f;
}

// With two SIDES eight waves share 128 queries, each half of every tile's keys, and
// bring their sums together at the end: for launches that leave most of a CU empty.
template <class T, int DP, int SIDES>
__global__ __launch_bounds__(THREADS * SIDES, 2) void attention_kernel(AttnArgs a, int tiles, int parts, float* sums,
                                                                       float2* known_to) {
  typedef typename Eight<T>::type V8;
  constexpr int KC = DP / 16, DT = DP / 32, SUB = KEYS / 32 / SIDES;   // 32 keys a time, SUB of them a tile
  constexpr int TILE = KEYS * Tile<DP>::ROW;
  __shared__ __attribute__((aligned(1024))) char smem[4 * TILE];   // keys, values, twice
  __shared__ float2 known[SIDES == 2 ? WAVES * 64 : 1];            // reference and sum of the second side
  static_assert(4 * TILE >= QUERIES * DP * 4, "the sums of one side fit in the tiles");
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int side = wave / WAVES;
  const unsigned blocks = gridDim.x / parts;
  const int part = blockIdx.x / blocks;
  const Work w = work_of(blockIdx.x - part * blocks, a.q_heads, a.k_heads);
  const Place at = place_of<QUERIES, false>(a.offsets, a.sequences, a.tokens, tiles, w.tile);
  if (at.length == 0) return;
  if (at.rest) {
    if (a.clear_rest && part == 0)
      clear_rows<T>(a, w.head, at.begin + at.row, min(at.begin + at.row + QUERIES, at.begin + at.length));
    return;
  }
  const int kv_head = w.head / (a.q_heads / a.k_heads);
  const T* k = static_cast<const T*>(a.k.p) + at.begin * a.k.token + kv_head * a.k.head;
  const T* v = static_cast<const T*>(a.v.p) + at.begin * a.v.token + kv_head * a.v.head;
  const uint32_t k_step = static_cast<uint32_t>(a.k.token * 2), v_step = static_cast<uint32_t>(a.v.token * 2);
  const Copier<DP, KEYS, WAVES * SIDES> k_copy(wave, lane, k_step, a.dim), v_copy(wave, lane, v_step, a.dim);
  const uint32_t lds = lds_address(smem);
  const int keys = min(at.length, at.row + QUERIES);   // that any query here sees
  const Range range = range_of((keys + KEYS - 1) / KEYS, part, parts);
  const int steps = range.last;

  auto fetch_tile = [&](int n) {
    const uint32_t to = lds + (n & 1) * 2 * TILE;
    const int first = n * KEYS;
    k_copy.copy(k + first * a.k.token, at.length - first, k_step, a.dim, to);
    v_copy.copy(v + first * a.v.token, at.length - first, v_step, a.dim, to + TILE);
  };
  if (range.first < steps) fetch_tile(range.first);

  const int first_query = at.row + 32 * (wave % WAVES), query = first_query + (lane & 31);
  const bool there = query < at.length;
  V8 q[KC];
  load_operands<T, DP>(there ? static_cast<const T*>(a.q.p) + (at.begin + query) * a.q.token + w.head * a.q.head
                             : nullptr,
                       a.dim, half, q);
  const RowReader<DP> rows(lane);
  const ColumnReader<DP> columns(lane);
  const float c = a.scale * 1.442695041f;   // weights as powers of two
  Acc o[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) o[t] = no_sum();
  float ref = -INFINITY, sum = 0.f;

  for (int n = range.first; n < steps; ++n) {
    copies_done();
    __syncthreads();   // tile n is there, and nobody reads the place of tile n + 1
    if (n + 1 < steps) fetch_tile(n + 1);
    const int first_key = n * KEYS + 32 * side;
    if (first_key > first_query + 31) continue;
    const uint32_t tile = lds + (n & 1) * 2 * TILE + 32 * side * Tile<DP>::ROW;
    const auto kt = rows.in(tile);
    const auto vt = columns.in(tile + TILE);
    Acc s[SUB];
#pragma unroll
    for (int i = 0; i < SUB; ++i) {
      s[i] = no_sum();
#pragma unroll
      for (int j = 0; j < KC; ++j) s[i] = product(kt.template read<T>(j, 32 * i * Tile<DP>::ROW), q[j], s[i]);
    }
    if (first_key + 32 * SUB - 1 > first_query) {   // some keys lie behind some queries
#pragma unroll
      for (int i = 0; i < SUB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int key = first_key + 32 * i + 8 * (r / 4) + 4 * half + r % 4;
          s[i][r] = key > query ? -INFINITY : s[i][r];
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int i = 0; i < SUB; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[i][r]);
    float lower, upper;
    both_halves(top, lower, upper);
    top = fmaxf(lower, upper) * c;
    if (__any(top > ref + LAG + LIFT<T>)) {
      const float to = fmaxf(ref, top - LIFT<T>);
      // (a row of another side or part may not have met a key yet: its sums stay 0)
      const float by = to == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ref - to);
      ref = to;
      sum *= by;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[t][r] *= by;
    }
    const float base = ref == -INFINITY ? 0.f : ref;
#pragma unroll
    for (int i = 0; i < SUB; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[i][r] = __builtin_amdgcn_exp2f(fmaf(s[i][r], c, -base));
        sum += s[i][r];
      }
#pragma unroll
    for (int j = 0; j < 2 * SUB; ++j) {
      const V8 p = operand<T>(s[j / 2], j % 2);   // weights of at most 2^15, rounded to T: half a step each
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] = product(vt.template read<T>(t, 16 * j * Tile<DP>::ROW), p, o[t]);
    }
  }

  float lower, upper;
  both_halves(sum, lower, upper);
  sum = lower + upper;
  if constexpr (SIDES == 2) {
    __syncthreads();
    float* const shared = reinterpret_cast<float*>(smem) + wave % WAVES * 64 * DP / 2 + lane;
    if (side == 1) {
      known[wave % WAVES * 64 + lane] = make_float2(ref, sum);
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) shared[64 * (16 * t + r)] = o[t][r];
    }
    __syncthreads();
    if (side == 1) return;
    const float2 other = known[wave * 64 + lane];
    const float to = fmaxf(ref, other.x), base = to == -INFINITY ? 0.f : to;
    const float mine = __builtin_amdgcn_exp2f(ref - base), theirs = __builtin_amdgcn_exp2f(other.x - base);
    ref = to;
    sum = sum * mine + other.y * theirs;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[t][r] = o[t][r] * mine + shared[64 * (16 * t + r)] * theirs;
  }
  if (parts > 1) {
    const int64_t row = (static_cast<int64_t>(part) * a.q_heads + w.head) * a.tokens + at.begin + query;
    store_sums<DP>(there ? sums + row * a.dim : nullptr, a.dim, half, o, 1.f);
    if (there && half == 0) known_to[row] = make_float2(ref, sum);
    return;
  }
  T* out = static_cast<T*>(a.out.p) + (at.begin + query) * a.out.token + w.head * a.out.head;
  store_columns<T, DP>(there ? out : nullptr, a.dim, half, o, 1.f / sum);
  if (there && half == 0)
    a.lse[static_cast<int64_t>(w.head) * a.tokens + at.begin + query] =
        0.693147182f * (ref + __builtin_amdgcn_logf(sum));
}

// Brings the parts' sums of a row together, eight columns a lane.
template <class T>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int parts, const float* sums,
                                                             const float2* known) {
  const int chunks = a.dim / 8, head = blockIdx.y;
  const int i = blockIdx.x * 256 + threadIdx.x, token = i / chunks, column = i % chunks * 8;
  if (token < offset_at(a.offsets, 0, a.tokens) || token >= offset_at(a.offsets, a.sequences, a.tokens)) return;
  const int64_t row = static_cast<int64_t>(head) * a.tokens + token, one = static_cast<int64_t>(a.q_heads) * a.tokens;
  float to = -INFINITY;
  for (int k = 0; k < parts; ++k) to = fmaxf(to, known[row + k * one].x);
  const float base = to == -INFINITY ? 0.f : to;
  float v[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  for (int k = 0; k < parts; ++k) {
    const float2 of = known[row + k * one];
    const float by = __builtin_amdgcn_exp2f(of.x - base);
    float x[VEC];
    load8(sums + (row + k * one) * a.dim + column, x);
    sum = fmaf(of.y, by, sum);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = fmaf(x[e], by, v[e]);
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] /= sum;
  store8(static_cast<T*>(a.out.p) + token * a.out.token + head * a.out.head + column, v);
  if (column == 0) a.lse[row] = 0.693147182f * (to + __builtin_amdgcn_logf(sum));
}

}  // namespace

// Up to eight parts, of 512 rows or more, where there are few workgroups: as many as
// make three of them for a CU. Two of the keys where there are less than three for a CU
// and the sequences are long: all are on the chip at once then, and those of the ends take twice the
// average. Forward (and whole gradient) of bf16 heads of 128, us in one part and so: 16384
// tokens of 1 head 313 and 130 (733, 367); 4096 of 4 heads 71 and 48 (194, 144); 1500 of 8
// heads that read 2 24 and 22 (134, 52); 8192 of 8 that read 2 203 and 161; of 12 that read 4,
// where it is one part, two take 241 instead of 228.
int attention_parts(int64_t tokens, int64_t sequences, int64_t heads, int64_t rows, bool keys) {
  const int64_t blocks = tiles_of(tokens, sequences, QUERIES) * heads;
  const int64_t few = std::min<int64_t>({8, 3 * CUS / blocks, rows / 512});
  if (few >= 2) return static_cast<int>(few);
  return keys && blocks < 3 * CUS && tokens / std::max<int64_t>(1, sequences) >= 4096 ? 2 : 1;
}

hipError_t launch_attention(const AttnArgs& a, int type, int parts, float* sums, float2* known, hipStream_t stream) {
  const int64_t tiles = tiles_of(a.tokens, a.sequences, QUERIES);
  auto on = [&](auto t, auto dp, auto sides) {
    using T = decltype(t);
    constexpr int DP = dp(), SIDES = sides();
    hipLaunchKernelGGL((attention_kernel<T, DP, SIDES>), dim3(static_cast<unsigned>(tiles * a.q_heads * parts)),
                       dim3(THREADS * SIDES), 0, stream, a, static_cast<int>(tiles), parts, sums, known);
    if (parts > 1)
      hipLaunchKernelGGL(attention_join_kernel<T>, dim3((a.tokens * (a.dim / 8) + 255) / 256, a.q_heads), dim3(256),
                         0, stream, a, parts, sums, known);
    return hipGetLastError();
  };
  auto sided = [&](auto t, auto dp) {
    return two_sides(tiles * a.q_heads * parts) ? on(t, dp, std::integral_constant<int, 2>{})
                                                : on(t, dp, std::integral_constant<int, 1>{});
  };
  auto shaped = [&](auto t) {
    return a.dim <= 64 ? sided(t, std::integral_constant<int, 64>{}) : sided(t, std::integral_constant<int, 128>{});
  };
  return type == NS_DT_BF16 ? shaped(__bf16{}) : shaped(_Float16{});
}

}  // namespace nsmi
