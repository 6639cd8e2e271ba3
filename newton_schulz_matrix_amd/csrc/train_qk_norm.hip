// RMS norm of each query's and key's head, with the rotation of its position in
// the same pass, and the gradient of both.
//
//   rstd = 1 / sqrt(mean(x^2) + eps),  u = x rstd w
//   (y_a, y_b) = (u_a cos t - u_b sin t, u_b cos t + u_a sin t),   t = position inv_freq
//   gradient: g = dy turned back, n = x rstd:  dw = sum g n,
//   dx = rstd (g w - n mean(g w n))
//
// Bound by memory. A head is the work of a team of lanes, each with two vectors of
// W elements that hold W whole pairs: W from each half of the rotated part (or 2 W
// in a row where pairs are neighbours), and two of the rest for the lanes behind.
// A wave takes one token, several heads at a time, so that its lanes keep the
// same pairs and the angles are worked out once for all heads of a token.
//
// Measured, bf16, heads of 128, 32 of queries and 8 of keys: 16384 tokens 66 us (336 MB:
// 5.1 TB/s), the gradient 104 + 5 us (503 MB: 4.8), where a library copy of 1 GB runs at 5.0. With
// few small heads the angles (a reduction in 64 bits and a sine a pair and token) bound
// it: 65536 tokens of 8 heads of 80, 53 us (3.2 TB/s).
#include <algorithm>
#include <type_traits>

#include "heads_internal.h"
#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int THREADS = 256, WAVES = THREADS / 64;
constexpr int MAX_PAIRS = QK_MAX_DIM / 2;

// W elements as loaded, from any element's address.
typedef uint32_t Duo __attribute__((ext_vector_type(2), aligned(2), may_alias));
typedef uint32_t Uno __attribute__((aligned(2), may_alias));
template <int BYTES>
struct Access {
  typedef Quad type;
};
template <>
struct Access<8> {
  typedef Duo type;
};
template <>
struct Access<4> {
  typedef Uno type;
};
template <class T, int W>
struct Part {
  static constexpr int BYTES = sizeof(T) * W;
  typedef typename Access<BYTES>::type A;
  static constexpr int N = BYTES / sizeof(A);
  A q[N];

  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = reinterpret_cast<const A*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<A*>(p)[i] = q[i];
  }
  __device__ __forceinline__ void widen(float (&v)[W]) const {
    if constexpr (std::is_same_v<T, __bf16>) {   // one step each, from the words
      uint32_t words[W / 2];
      __builtin_memcpy(words, q, sizeof(words));
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        v[2 * i] = __builtin_bit_cast(float, words[i] << 16);
        v[2 * i + 1] = __builtin_bit_cast(float, words[i] & 0xffff0000u);
      }
      return;
    }
    T r[W];
    __builtin_memcpy(r, q, sizeof(r));
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = static_cast<float>(r[e]);
  }
  __device__ __forceinline__ void narrow(const float (&v)[W]) {
    T r[W];
#pragma unroll
    for (int e = 0; e < W; ++e) r[e] = static_cast<T>(v[e]);
    __builtin_memcpy(q, r, sizeof(r));
  }
};

// What a lane is within its team: the columns of its two vectors, and whether
// they hold pairs that turn.
template <int W>
struct Lane {
  int a, b, pair;      // first columns, first pair
  bool turns, there;   // else the vectors pass, or there are none
  __device__ __forceinline__ Lane(const QkArgs& q, int j) {
    const int turning = q.rotary / (2 * W);
    turns = j < turning;
    there = j < q.dim / (2 * W);
    pair = turns ? W * j : 0;
    if (turns && !q.interleaved) {
      a = W * j;
      b = q.rotary / 2 + W * j;
    } else {
      a = there ? 2 * W * j : 0;   // (rotary is 2 W times the lanes that turn)
      b = a + W;
    }
  }
};

// sin and cos of a token's angles, one pair a lane, into LDS. The angle is
// taken in turns and in 64 bits before its whole turns are dropped: at position
// 10^6 an angle in 32 bits would be off by 0.03.
template <class I>
__device__ __forceinline__ void angles(const QkArgs& a, int64_t token, int lane, float2* table) {
  const I* positions = static_cast<const I*>(a.positions);
  for (int p = lane; p < a.rotary / 2; p += 64) {
    int axis = 0;
#pragma unroll
    for (int k = 1; k < QK_AXES; ++k) axis += p >= a.first[k];
    const double position = static_cast<double>(positions[axis * a.ld_positions + token]);
    const double turns = position * static_cast<double>(a.inv_freq[p]) * 0.15915494309189533577;
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    table[p] = make_float2(c, s);
  }
}
__device__ __forceinline__ void angles_of(const QkArgs& a, int64_t token, int lane, float2* table) {
  if (a.positions64) angles<int64_t>(a, token, lane, table);
  else angles<int32_t>(a, token, lane, table);
}

// What the lanes of a wave have written to LDS is there for the others.
__device__ __forceinline__ void wave_settled() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int W>
__device__ __forceinline__ void read_angles(const Lane<W>& l, const float2* table, float (&c)[W],
                                            float (&s)[W]) {
#pragma unroll
  for (int e = 0; e < W; ++e) {
    const float2 t = table[l.pair + e];
    c[e] = l.turns ? t.x : 1.f;
    s[e] = l.turns ? t.y : 0.f;
  }
}

// Turns the pairs of two vectors by (c, sign s).
template <int W>
__device__ __forceinline__ void turn(bool neighbours, float sign, const float (&c)[W],
                                     const float (&s)[W], float (&a)[W], float (&b)[W]) {
  if (neighbours) {
#pragma unroll
    for (int e = 0; e < W / 2; ++e) {
      const float x = a[2 * e], y = a[2 * e + 1], u = b[2 * e], v = b[2 * e + 1];
      const float sx = sign * s[e], su = sign * s[W / 2 + e];
      a[2 * e] = x * c[e] - y * sx;
      a[2 * e + 1] = y * c[e] + x * sx;
      b[2 * e] = u * c[W / 2 + e] - v * su;
      b[2 * e + 1] = v * c[W / 2 + e] + u * su;
    }
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const float x = a[e], y = b[e], t = sign * s[e];
      a[e] = x * c[e] - y * t;
      b[e] = y * c[e] + x * t;
    }
  }
}

// Sum over the lanes of a team (a power of two of them), each step one instruction
// on the lanes of a row: neighbours, pairs, then mirrored halves, whose lanes all
// hold the same by then.
template <int CONTROL>
__device__ __forceinline__ float moved(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CONTROL, 0xf, 0xf,
                                                               false));
}
__device__ __forceinline__ float team_sum(float v, int team) {
  constexpr int XOR1 = 0xb1, XOR2 = 0x4e, HALF_MIRROR = 0x141, MIRROR = 0x140;
  if (team > 1) v += moved<XOR1>(v);
  if (team > 2) v += moved<XOR2>(v);
  if (team > 4) v += moved<HALF_MIRROR>(v);
  if (team > 8) v += moved<MIRROR>(v);
  if (team > 16) v += __shfl_xor(v, 16, 64);
  if (team > 32) v += __shfl_xor(v, 32, 64);
  return v;
}

// The weights of queries and keys into LDS, as fp32.
template <class T>
__device__ __forceinline__ void share_weights(const QkArgs& a, float (*to)[QK_MAX_DIM]) {
  for (int i = threadIdx.x; i < 2 * a.dim; i += THREADS) {
    const int k = i >= a.dim, col = i - k * a.dim;
    const void* w = a.part[k].weight;
    to[k][col] = a.weight32 ? static_cast<const float*>(w)[col] : static_cast<float>(static_cast<const T*>(w)[col]);
  }
}
template <int W>
__device__ __forceinline__ void read_weights(const float* w, int at, float (&v)[W]) {
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] = w[at + e];
}

// The head that a team takes in round r of a wave's: queries first, then keys.
struct Slot {
  bool key, mine;
  int head;
  __device__ __forceinline__ Slot(const QkArgs& a, int slot, bool there) {
    key = slot >= a.part[0].heads;
    head = slot - (key ? a.part[0].heads : 0);
    mine = there && slot < a.part[0].heads + a.part[1].heads;
  }
  template <class T>
  __device__ __forceinline__ T* in(const QkArgs& a, T* queries, T* keys, int64_t token, int64_t q_token,
                                   int64_t q_head, int64_t k_token, int64_t k_head) const {
    return (key ? keys : queries) + token * (key ? k_token : q_token) + head * (key ? k_head : q_head);
  }
};

// Waves take tokens, or chunks of `rounds` rounds of a token's heads, in turn. The
// loads of U rounds are in flight before the angles are worked out.
template <class T, int W>
__global__ __launch_bounds__(THREADS) void qk_norm_kernel(QkArgs a, int team, int rounds, int chunks) {
  constexpr int U = sizeof(T) == 2 ? 4 : 2;
  __shared__ float2 tables[WAVES][MAX_PAIRS];
  __shared__ float weights[2][QK_MAX_DIM];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool norm = a.part[0].weight != nullptr;
  const Lane<W> l(a, lane & (team - 1));
  const int each = 64 / team;
  float2* table = tables[wave];
  if (norm) share_weights<T>(a, weights);
  __syncthreads();
  const int64_t units = static_cast<int64_t>(a.tokens) * chunks;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * WAVES + wave; unit < units;
       unit += static_cast<int64_t>(gridDim.x) * WAVES) {
    const int64_t token = unit / chunks;
    const int slot0 = static_cast<int>(unit - token * chunks) * rounds * each + lane / team;
    float c[W], s[W];
    for (int r0 = 0; r0 < rounds; r0 += U) {
      Part<T, W> ra[U], rb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Slot at(a, slot0 + (r0 + u) * each, l.there && r0 + u < rounds);
        ra[u] = {};
        rb[u] = {};
        if (at.mine) {
          const T* x = at.in(a, static_cast<const T*>(a.part[0].x), static_cast<const T*>(a.part[1].x), token,
                             a.part[0].x_token, a.part[0].x_head, a.part[1].x_token, a.part[1].x_head);
          ra[u].load(x + l.a);
          rb[u].load(x + l.b);
        }
      }
      if (r0 == 0) {
        wave_settled();   // the last token's angles have been read
        angles_of(a, token, lane, table);
        wave_settled();
        read_angles<W>(l, table, c, s);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r0 + u >= rounds) break;
        const Slot at(a, slot0 + (r0 + u) * each, l.there);
        float va[W], vb[W];
        ra[u].widen(va);
        rb[u].widen(vb);
        if (norm) {
          float sum = 0.f, wa[W], wb[W];
#pragma unroll
          for (int e = 0; e < W; ++e) sum = fmaf(va[e], va[e], fmaf(vb[e], vb[e], sum));
          const float rstd = rsqrtf(team_sum(sum, team) / static_cast<float>(a.dim) + a.eps);
          read_weights<W>(weights[at.key], l.a, wa);
          read_weights<W>(weights[at.key], l.b, wb);
#pragma unroll
          for (int e = 0; e < W; ++e) {
            va[e] *= rstd * wa[e];
            vb[e] *= rstd * wb[e];
          }
        }
        turn<W>(a.interleaved, 1.f, c, s, va, vb);
        if (at.mine) {
          T* y = at.in(a, static_cast<T*>(a.part[0].out), static_cast<T*>(a.part[1].out), token, a.part[0].out_token,
                       a.part[0].out_head, a.part[1].out_token, a.part[1].out_head);
          Part<T, W> o;
          o.narrow(va);
          o.store(y + l.a);
          o.narrow(vb);
          o.store(y + l.b);
        }
      }
    }
  }
}

// The gradient: waves take tokens in turn and keep their share of the weights'
// gradients in registers; a workgroup adds its waves' shares at the end.
template <class T, int W>
__global__ __launch_bounds__(THREADS, W == 8 ? 3 : 4) void qk_grad_kernel(QkArgs a, int team, int rounds,
                                                          float* partial) {
  constexpr int U = sizeof(T) == 2 ? 2 : 1;
  __shared__ float2 tables[WAVES][MAX_PAIRS];
  __shared__ float weights[2][QK_MAX_DIM];
  __shared__ float shares[WAVES][4 * W][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool norm = a.part[0].weight != nullptr;
  const Lane<W> l(a, lane & (team - 1));
  const int each = 64 / team, q_heads = a.part[0].heads;
  float2* table = tables[wave];
  if (norm) share_weights<T>(a, weights);
  __syncthreads();
  float dw[2][2][W];   // queries and keys, the two vectors
#pragma unroll
  for (int i = 0; i < 4 * W; ++i) dw[i / (2 * W)][i / W % 2][i % W] = 0.f;
  for (int64_t token = static_cast<int64_t>(blockIdx.x) * WAVES + wave; token < a.tokens;
       token += static_cast<int64_t>(gridDim.x) * WAVES) {
    float c[W], s[W];
    for (int r0 = 0; r0 < rounds; r0 += U) {
      Part<T, W> ga[U], gb[U], xa[U], xb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Slot at(a, (r0 + u) * each + lane / team, l.there);
        ga[u] = gb[u] = xa[u] = xb[u] = {};
        if (at.mine) {
          const T* dy = at.in(a, static_cast<const T*>(a.part[0].dy), static_cast<const T*>(a.part[1].dy), token,
                              a.part[0].dy_token, a.part[0].dy_head, a.part[1].dy_token, a.part[1].dy_head);
          ga[u].load(dy + l.a);
          gb[u].load(dy + l.b);
          if (norm) {
            const T* x = at.in(a, static_cast<const T*>(a.part[0].x), static_cast<const T*>(a.part[1].x), token,
                               a.part[0].x_token, a.part[0].x_head, a.part[1].x_token, a.part[1].x_head);
            xa[u].load(x + l.a);
            xb[u].load(x + l.b);
          }
        }
      }
      if (r0 == 0) {
        wave_settled();   // the last token's angles have been read
        angles_of(a, token, lane, table);
        wave_settled();
        read_angles<W>(l, table, c, s);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r0 + u >= rounds) break;
        const int first = (r0 + u) * each;
        const Slot at(a, first + lane / team, l.there);
        float va[W], vb[W];
        ga[u].widen(va);
        gb[u].widen(vb);
        turn<W>(a.interleaved, -1.f, c, s, va, vb);
        if (norm) {
          float na[W], nb[W], wa[W], wb[W], sum = 0.f, dot = 0.f;
          xa[u].widen(na);
          xb[u].widen(nb);
          read_weights<W>(weights[at.key], l.a, wa);
          read_weights<W>(weights[at.key], l.b, wb);
#pragma unroll
          for (int e = 0; e < W; ++e) sum = fmaf(na[e], na[e], fmaf(nb[e], nb[e], sum));
          sum = team_sum(sum, team) / static_cast<float>(a.dim) + a.eps;
          const float rstd = at.mine ? rsqrtf(sum) : 0.f;   // (idle lanes hold zeros, also where eps is 0)
#pragma unroll
          for (int e = 0; e < W; ++e) {
            na[e] *= rstd;
            nb[e] *= rstd;
          }
          if (first + each <= q_heads) {   // all of them queries, or keys
#pragma unroll
            for (int e = 0; e < W; ++e) {
              dw[0][0][e] = fmaf(va[e], na[e], dw[0][0][e]);
              dw[0][1][e] = fmaf(vb[e], nb[e], dw[0][1][e]);
            }
          } else if (first >= q_heads) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
              dw[1][0][e] = fmaf(va[e], na[e], dw[1][0][e]);
              dw[1][1][e] = fmaf(vb[e], nb[e], dw[1][1][e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < W; ++e) {
              const float da = va[e] * na[e], db = vb[e] * nb[e];
              dw[0][0][e] += at.key ? 0.f : da;
              dw[0][1][e] += at.key ? 0.f : db;
              dw[1][0][e] += at.key ? da : 0.f;
              dw[1][1][e] += at.key ? db : 0.f;
            }
          }
#pragma unroll
          for (int e = 0; e < W; ++e) {
            va[e] *= wa[e];
            vb[e] *= wb[e];
            dot = fmaf(va[e], na[e], fmaf(vb[e], nb[e], dot));
          }
          const float mean = team_sum(dot, team) / static_cast<float>(a.dim);
#pragma unroll
          for (int e = 0; e < W; ++e) {
            va[e] = rstd * fmaf(-na[e], mean, va[e]);
            vb[e] = rstd * fmaf(-nb[e], mean, vb[e]);
          }
        }
        if (at.mine) {
          T* dx = at.in(a, static_cast<T*>(a.part[0].out), static_cast<T*>(a.part[1].out), token,
                        a.part[0].out_token, a.part[0].out_head, a.part[1].out_token, a.part[1].out_head);
          Part<T, W> o;
          o.narrow(va);
          o.store(dx + l.a);
          o.narrow(vb);
          o.store(dx + l.b);
        }
      }
    }
  }
  if (!norm) return;
#pragma unroll
  for (int i = 0; i < 4 * W; ++i) shares[wave][i][lane] = dw[i / (2 * W)][i / W % 2][i % W];
  __syncthreads();
  // a thread a column: the lane of a team and the value that hold it, of all teams and waves
  for (int i = threadIdx.x; i < 2 * a.dim; i += THREADS) {
    const int k = i >= a.dim, col = i - k * a.dim;
    int j = col / (2 * W), value = col % (2 * W);
    if (!a.interleaved && col < a.rotary) {
      const int second = col >= a.rotary / 2, at = col - second * (a.rotary / 2);
      j = at / W;
      value = at % W + second * W;
    }
    float v = 0.f;
    for (int w = 0; w < WAVES; ++w)
#pragma unroll 4
      for (int t = j; t < 64; t += team) v += shares[w][2 * W * k + value][t];
    partial[static_cast<int64_t>(blockIdx.x) * 2 * a.dim + i] = v;
  }
}

// dweight[c] = sum over the workgroups' shares, in 64 bits: 16 columns by 64 groups
// of shares in a workgroup.
constexpr int DW_COLS = 16, DW_GROUPS = 64;
template <class TO>
__global__ __launch_bounds__(DW_COLS * DW_GROUPS) void qk_dweight_kernel(const float* partial,
                                                                         int blocks, int dim,
                                                                         TO* dq, TO* dk) {
  __shared__ double sums[DW_GROUPS][DW_COLS + 1];
  const int tx = threadIdx.x % DW_COLS, ty = threadIdx.x / DW_COLS;
  const int col = blockIdx.x * DW_COLS + tx;
  double s = 0.0;
  if (col < 2 * dim) {
#pragma unroll 8
    for (int b = ty; b < blocks; b += DW_GROUPS) s += partial[static_cast<int64_t>(b) * 2 * dim + col];
  }
  sums[ty][tx] = s;
  __syncthreads();
  if (ty != 0 || col >= 2 * dim) return;
  for (int k = 1; k < DW_GROUPS; ++k) s += sums[k][tx];
  TO* to = col < dim ? dq : dk;
  if (to) to[col < dim ? col : col - dim] = static_cast<TO>(static_cast<float>(s));
}

// Calls f with the widest vectors that the sizes allow, up to MOST, as a type.
template <int MOST, class F>
hipError_t by_vector(const QkArgs& a, F f) {
  if constexpr (MOST == 8)
    if (a.dim % 16 == 0 && a.rotary % 16 == 0) return f(std::integral_constant<int, 8>{});
  if (a.dim % 8 == 0 && a.rotary % 8 == 0) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 2>{});
}
int team_of(int dim, int w) {
  int team = 1;
  while (team * 2 * w < dim) team *= 2;
  return team;
}

}  // namespace

// fp32 has vectors of 4 (16 bytes; 30000 tokens of 8 heads of 80: 25.6 us, 29 with vectors
// of 8; 8192 of 40 heads of 128 65 and 67; the gradient is no faster with them, 108 and 105).
//
// Workgroups that take many tokens bring the weights to LDS once for all of them (65536
// tokens of 8 heads of 80: 52.8 us, 61 with a workgroup for each four).
constexpr int NORM_BLOCKS = 4096;

hipError_t launch_qk_norm_rope(const QkArgs& a, int type, hipStream_t stream) {
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    return by_vector<sizeof(T) == 4 ? 4 : 8>(a, [&](auto w) {
      constexpr int W = w();
      const int team = team_of(a.dim, W), each = 64 / team;
      const int all = (a.part[0].heads + a.part[1].heads + each - 1) / each;
      // few tokens: one round a wave; else all heads of a token, whose angles are shared
      const int rounds = a.tokens < 2048 ? 1 : all;
      const int chunks = (all + rounds - 1) / rounds;
      const int64_t units = static_cast<int64_t>(a.tokens) * chunks;
      hipLaunchKernelGGL((qk_norm_kernel<T, W>), dim3(std::min<int64_t>((units + WAVES - 1) / WAVES, NORM_BLOCKS)),
                         dim3(THREADS), 0, stream, a, team, rounds, chunks);
      return hipGetLastError();
    });
  });
}

// As many workgroups as the chip holds at a time: three a CU where vectors are of 8,
// whose registers allow no more (16384 tokens of 40 heads of 128: 115 us; 129 with 1024
// workgroups, a third of which come in a second round), else four.
int qk_grad_blocks(int64_t tokens, int64_t dim) {
  return static_cast<int>(std::min<int64_t>((tokens + WAVES - 1) / WAVES, dim % 16 == 0 ? 768 : 1024));
}

hipError_t launch_qk_norm_rope_grad(const QkArgs& a, int type, float* partial, void* dq_weight,
                                    void* dk_weight, int dweight_type, hipStream_t stream) {
  const int blocks = a.tokens > 0 ? qk_grad_blocks(a.tokens, a.dim) : 0;
  if (blocks > 0) {
    const hipError_t e = by_type(type, [&](auto t) {
      using T = decltype(t);
      return by_vector<8>(a, [&](auto w) {
        constexpr int W = w();
        const int team = team_of(a.dim, W), each = 64 / team;
        const int rounds = (a.part[0].heads + a.part[1].heads + each - 1) / each;
        hipLaunchKernelGGL((qk_grad_kernel<T, W>), dim3(blocks), dim3(THREADS), 0, stream, a, team,
                           rounds, partial);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  if (!dq_weight && !dk_weight) return hipSuccess;
  return by_type(dweight_type, [&](auto t) {
    using TO = decltype(t);
    hipLaunchKernelGGL(qk_dweight_kernel<TO>, dim3((2 * a.dim + DW_COLS - 1) / DW_COLS),
                       dim3(DW_COLS * DW_GROUPS), 0, stream, partial, blocks, a.dim,
                       static_cast<TO*>(dq_weight), static_cast<TO*>(dk_weight));
    return hipGetLastError();
  });
}

}  // namespace nsmi
