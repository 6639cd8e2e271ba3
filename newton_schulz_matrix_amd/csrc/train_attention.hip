// Causal attention over packed sequences with grouped heads.
//
//   S = scale q k^T (keys up to the query's own position), out = softmax(S) v,
//   lse = log sum exp S
//
// Bound by the matrix units, at a clock that falls with what is done in each cycle
// (2.4 GHz at most, 1.9 here): fewer reads of LDS are worth more than a denser order of
// instructions. A workgroup takes 128 or 256 queries of one head, 32 or 64 a wave, and
// goes over the keys up to its last query in tiles of 64 (or 32), with the running maximum and
// sum of each row. Products are taken transposed (keys x queries, columns x queries): a
// lane then holds one query (or two), a row's maximum and sum are its own registers and
// one exchange, and the weights are the next product's operand as they stand. Keys and
// values come into LDS directly, the next tile while this one is worked on.
//
// Measured, bf16, 32 heads of 128 that read 8: 16384 tokens of one sequence 1925 us
// (1142 TFLOP/s of what a query sees; a library product of 8192 cubed reaches 1180), 16256
// tokens of eight sequences of 0 to 5113 460 us (980).
#include <algorithm>
#include <type_traits>

#include "attention_device.h"
#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int WAVES = 4, THREADS = 64 * WAVES;

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
//
// With two GROUPS a wave has 64 queries, so that an operand from LDS serves two
// products: half the reads, and half the copies of tiles. It takes 32 keys at once then and
// reads operands AHEAD, in the order written, to stay within 256 registers.
//
// Tiles of 32 KEYS instead of 64 leave registers and LDS for three workgroups a CU instead of two.
template <class T, int DP, int SIDES, int GROUPS, int KEYS>
__global__ __launch_bounds__(THREADS * SIDES, KEYS == 32 ? 3 : 2) void attention_kernel(
    AttnArgs a, int tiles, int parts, float* sums, float2* known_to) {
  typedef typename Eight<T>::type V8;
  constexpr int KC = DP / 16, DT = DP / 32;
  constexpr int SUB = GROUPS == 2 ? 1 : KEYS / 32 / SIDES;   // times 32 keys at once
  constexpr int QUERIES = 128 * GROUPS;
  constexpr bool WIDE = GROUPS == 2;
  constexpr int EARLIER = WIDE ? AHEAD : 0;
  constexpr int TILE = KEYS * Tile<DP>::ROW;
  __shared__ __attribute__((aligned(1024))) char smem[4 * TILE];   // keys, values, twice
  __shared__ float2 known[SIDES == 2 ? WAVES * 64 : 1];            // reference and sum of the second side
  static_assert(SIDES == 1 || GROUPS == 1, "the sums of two groups do not fit in the tiles");
  static_assert(SIDES == 1 || 4 * TILE >= QUERIES * DP * 4, "the sums of one side fit in the tiles");
  const int lane = threadIdx.x & 63, half = lane >> 5;
  auto own_lane = [&] { return WIDE ? lane_anew() : lane; };
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int side = wave / WAVES;
  const Share share = share_of(tiles * a.q_heads, parts);
  if (share.block < 0) return;
  const int part = share.part;
  const Work w = work_of(share.block, a.q_heads, a.k_heads);
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
  const uint32_t lds = lds_address(smem);
  const int keys = min(at.length, at.row + QUERIES);   // that any query here sees
  const Range range = range_of((keys + KEYS - 1) / KEYS, part, parts);
  const int steps = range.last;

  auto fetch_tile = [&](int n) {
    const uint32_t to = lds + (n & 1) * 2 * TILE;
    const int first = n * KEYS, l = own_lane();
    const Copier<DP, KEYS, WAVES * SIDES> k_copy(wave, l, k_step, a.dim), v_copy(wave, l, v_step, a.dim);
    k_copy.copy(k + first * a.k.token, at.length - first, k_step, a.dim, to);
    v_copy.copy(v + first * a.v.token, at.length - first, v_step, a.dim, to + TILE);
  };
  if (range.first < steps) fetch_tile(range.first);

  // (the wave's queries, 32 a group; a lane has one of each)
  const int first_query = at.row + 32 * GROUPS * (wave % WAVES), query = first_query + (lane & 31);
  // (a wave without rows only brings tiles in: one row behind the last full tile would cost a tile's time)
  const int last_query = first_query < at.length ? first_query + 32 * GROUPS - 1 : -1;
  V8 q[GROUPS][KC];
#pragma unroll
  for (int g = 0; g < GROUPS; ++g)
    load_operands<T, DP>(query + 32 * g < at.length ? static_cast<const T*>(a.q.p) +
                                                          (at.begin + query + 32 * g) * a.q.token + w.head * a.q.head
                                                    : nullptr,
                         a.dim, half, q[g]);
  const RowReader<DP> rows(lane);
  const ColumnReader<DP> columns(lane);
  const float c = a.scale * 1.442695041f;   // weights as powers of two
  Acc o[GROUPS][DT];
  float ref[GROUPS], sum[GROUPS];
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
#pragma unroll
    for (int t = 0; t < DT; ++t) o[g][t] = no_sum();
    ref[g] = -INFINITY, sum[g] = 0.f;
  }

  for (int n = range.first; n < steps; ++n) {
    copies_done();
    __syncthreads();   // tile n is there, and nobody reads the place of tile n + 1
    if (n + 1 < steps) fetch_tile(n + 1);
#pragma unroll 1
    for (int u = 0; u < KEYS / 32 / SIDES / SUB; ++u) {
      const int row0 = 32 * side + 32 * SUB * u, first_key = n * KEYS + row0;
      if (first_key > last_query) break;
      const uint32_t tile = lds + (n & 1) * 2 * TILE + row0 * Tile<DP>::ROW;
      const auto kt = lean_or_all<WIDE>(rows, tile);
      const auto vt = lean_or_all<WIDE>(columns, tile);   // TILE behind
      constexpr int ROW_READS = SUB * KC, READS = ROW_READS + 2 * SUB * DT;
      V8 read[READS];
      auto fetch = [&](int m) {
        if (m >= READS) return;
        if (m < ROW_READS)
          read[m] = kt.template read<T>(m / SUB, m % SUB * 32 * Tile<DP>::ROW);
        else
          read[m] = vt.template read<T>((m - ROW_READS) % DT, TILE + (m - ROW_READS) / DT * 16 * Tile<DP>::ROW);
      };
#pragma unroll
      for (int m = 0; m < EARLIER; ++m) fetch(m);
      Acc s[GROUPS][SUB];
#pragma unroll
      for (int m = 0; m < ROW_READS; ++m) {
        fetch(m + EARLIER);
        in_order<WIDE>();
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
          s[g][m % SUB] = product(read[m], q[g][m / SUB], m < SUB ? no_sum() : s[g][m % SUB]);
        in_order<WIDE>();
      }
      V8 p[GROUPS][2 * SUB];
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        if (first_key + 32 * SUB - 1 > first_query + 32 * g) {   // some keys lie behind some queries
          const int l = own_lane(), hidden = first_query + 32 * g + (l & 31) - first_key - 4 * (l >> 5);
#pragma unroll
          for (int i = 0; i < SUB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              s[g][i][r] = 32 * i + 8 * (r / 4) + r % 4 > hidden ? -INFINITY : s[g][i][r];
        }
        float top = s[g][0][0];
#pragma unroll
        for (int i = 0; i < SUB; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) top = fmaxf(top, s[g][i][r]);
        float lower, upper;
        both_halves(top, lower, upper);
        top = fmaxf(lower, upper) * c;
        if (__any(top > ref[g] + LAG + LIFT<T>)) {
          const float to = fmaxf(ref[g], top - LIFT<T>);
          // (a row of another side or part may not have met a key yet: its sums stay 0)
          const float by = to == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ref[g] - to);
          ref[g] = to;
          sum[g] *= by;
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[g][t][r] *= by;
        }
        const float base = ref[g] == -INFINITY ? 0.f : ref[g];
        // (by themselves first: beside a row's whole sum the small ones would be lost, always to one
        // side; lse of 16384 keys of scores of deviation 4 would be 123 half steps of 1 too low)
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < SUB; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            s[g][i][r] = __builtin_amdgcn_exp2f(fmaf(s[g][i][r], c, -base));
            add += s[g][i][r];
          }
        sum[g] += add;
        // weights of at most 2^15, rounded to T: half a step each
#pragma unroll
        for (int j = 0; j < 2 * SUB; ++j) p[g][j] = operand<T>(s[g][j / 2], j % 2);
      }
#pragma unroll
      for (int m = 0; m < 2 * SUB * DT; ++m) {
        fetch(ROW_READS + m + EARLIER);
        in_order<WIDE>();
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) o[g][m % DT] = product(read[ROW_READS + m], p[g][m / DT], o[g][m % DT]);
        in_order<WIDE>();
      }
    }
  }

#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    float lower, upper;
    both_halves(sum[g], lower, upper);
    sum[g] = lower + upper;
  }
  if constexpr (SIDES == 2) {
    __syncthreads();
    float* const shared = reinterpret_cast<float*>(smem) + wave % WAVES * 64 * DP / 2 + lane;
    if (side == 1) {
      known[wave % WAVES * 64 + lane] = make_float2(ref[0], sum[0]);
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) shared[64 * (16 * t + r)] = o[0][t][r];
    }
    __syncthreads();
    if (side == 1) return;
    const float2 other = known[wave * 64 + lane];
    const float to = fmaxf(ref[0], other.x), base = to == -INFINITY ? 0.f : to;
    const float mine = __builtin_amdgcn_exp2f(ref[0] - base), theirs = __builtin_amdgcn_exp2f(other.x - base);
    ref[0] = to;
    sum[0] = sum[0] * mine + other.y * theirs;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[0][t][r] = o[0][t][r] * mine + shared[64 * (16 * t + r)] * theirs;
  }
  const int l = own_lane();
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    const int query = first_query + 32 * g + (l & 31), half = l >> 5;
    const bool there = query < at.length;
    const int64_t token = at.begin + query;
    if (parts > 1) {
      const int64_t row = (static_cast<int64_t>(part) * a.q_heads + w.head) * a.tokens + token;
      store_sums<DP>(there ? sums + row * a.dim : nullptr, a.dim, half, o[g], 1.f);
      if (there && half == 0) known_to[row] = make_float2(ref[g], sum[g]);
      continue;
    }
    T* out = static_cast<T*>(a.out.p) + token * a.out.token + w.head * a.out.head;
    store_columns<T, DP>(there ? out : nullptr, a.dim, half, o[g], 1.f / sum[g]);
    if (there && half == 0)
      a.lse[static_cast<int64_t>(w.head) * a.tokens + token] =
          0.693147182f * (ref[g] + __builtin_amdgcn_logf(sum[g]));
  }
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
// make three of them for a CU, or two and a half where they are those of keys, of which a CU
// holds one. Two of the keys where there are less than three for a CU and the sequences are
// long: all are on the chip at once then, and those of the ends take twice the average.
// Forward and whole gradient of bf16 heads of 128, us in one part and so: 16384 tokens of 1
// head 313 and 94 (733, 286); 4096 of 4 heads 71 and 41 (194, 116); 1500 of 8 heads that read 2 24
// and 22 (134, 68); 8192 of 8 that read 2 203 and 161; of 12 that read 4, where it is one part,
// two take 241 instead of 228. Three parts of the keys for a CU: 302, 129 and 68 for the first
// three gradients; two: 295, 113 and, 2048 tokens of 16 that read 4, 120 instead of 118.
int attention_parts(int64_t tokens, int64_t sequences, int64_t heads, int64_t rows, bool keys) {
  const int64_t blocks = tiles_of(tokens, sequences, 32 * WAVES) * heads;
  const int64_t few = std::min<int64_t>({8, (keys ? 6 : 5) * CUS / (2 * blocks), rows / 512});
  if (few >= 2) return static_cast<int>(few);
  return keys && blocks < 3 * CUS && tokens / std::max<int64_t>(1, sequences) >= 4096 ? 2 : 1;
}

// Whether a wave takes 64 queries, for heads above 64: where the rows of all heads are 2304 times
// 128 or more, and 512 or more a sequence. Us with 32 and 64 a wave (bf16, heads of 128): 4096
// times 128, 16384 tokens of one sequence, 2076 and 1925; 2560, 1305 and 1238; 2048, 1042 and
// 1052; 1024, 152 and 173: the chip is full of the wide ones at 512, and the longest of them are not
// done when the others are. 32 sequences of 512, 135 and 134; 40 of 200, 55 and 60. Heads of
// 64, whose four waves a SIMD hide more: 4096, 600 and 618.
bool many_queries(const AttnArgs& a) {
  const int64_t tokens = a.tokens;
  return tokens * a.q_heads >= 9 * CUS * 128 && tokens / 512 >= a.sequences;
}

// Whether tiles of 32 keys pay, for heads above 64: at 512 workgroups or more of sequences of less
// than 512 on average, else at 1024. Us with 64 and 32 (bf16, 32 heads of 128 unless said): 128
// sequences of 64, 51 and 42; 64 of 128, 49 and 41; 40 of 200, 56 and 49; 16 of 512, 66 and 64;
// 4096 tokens of one, 156 and 148; 16384 of 8 heads 581 and 563, of 16 heads 1062 and 1075;
// 4096 of 24 heads, 792 workgroups, 118 and 130.
bool short_tiles(const AttnArgs& a, int64_t tiles) {
  return tiles * a.q_heads >= (a.tokens / 512 < a.sequences ? 2 * CUS : 4 * CUS);
}

hipError_t launch_attention(const AttnArgs& a, int type, int parts, float* sums, float2* known, hipStream_t stream) {
  const int64_t tiles = tiles_of(a.tokens, a.sequences, 32 * WAVES);
  auto on = [&](auto t, auto dp, auto sides, auto groups, auto keys) {
    using T = decltype(t);
    constexpr int DP = dp(), SIDES = sides(), GROUPS = groups(), KEYS = keys();
    const int64_t n = tiles_of(a.tokens, a.sequences, 32 * WAVES * GROUPS);
    hipLaunchKernelGGL((attention_kernel<T, DP, SIDES, GROUPS, KEYS>), dim3(shared_blocks(n * a.q_heads, parts)),
                       dim3(THREADS * SIDES), 0, stream, a, static_cast<int>(n), parts, sums, known);
    if (parts > 1)
      hipLaunchKernelGGL(attention_join_kernel<T>, dim3((a.tokens * (a.dim / 8) + 255) / 256, a.q_heads), dim3(256),
                         0, stream, a, parts, sums, known);
    return hipGetLastError();
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  using Short = std::integral_constant<int, 32>;
  using Long = std::integral_constant<int, 64>;
  auto sided = [&](auto t, auto dp) {
    if constexpr (dp() == 128) {
      if (parts == 1 && many_queries(a)) return on(t, dp, One{}, Two{}, Long{});
      if (parts == 1 && short_tiles(a, tiles)) return on(t, dp, One{}, One{}, Short{});
    }
    return two_sides(tiles * a.q_heads * parts, a.tokens, a.sequences) ? on(t, dp, Two{}, One{}, Long{})
                                                                       : on(t, dp, One{}, One{}, Long{});
  };
  auto shaped = [&](auto t) {
    return a.dim <= 64 ? sided(t, std::integral_constant<int, 64>{}) : sided(t, std::integral_constant<int, 128>{});
  };
  return type == NS_DT_BF16 ? shaped(__bf16{}) : shaped(_Float16{});
}

}  // namespace nsmi
