// RMS norm with the residual's addition, and its gradient.
//
//   h = x + r;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h * rstd * w
//   dx = rstd * (g - u * mean(g * u)) + dh,  u = h * rstd, g = dy * w
//   dw = sum over rows of dy * u
//
// Bound by memory: every input is read once and every output written once. A
// row stays in the registers of its team of TEAM threads (V vectors of eight
// columns each) between the sum and the scaling. Teams of one wave need no
// barrier and share a workgroup by fours; wider rows take a workgroup.
//
// 16384 rows of 4096 in bf16 with a residual: to e4m3 in 77 us (470 MB, 6.1
// TB/s), the gradient in 87 and 5 for the sum of dw (537 MB, 6.2 TB/s). What
// it took: the loads of a row's operands all in flight before the first
// conversion (97 -> 85 us for the forward kernel), the next row's with them
// (-> 78), and no run-time type or width between a load and its use.
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

constexpr int block_of(int team) { return team < 256 ? 256 : team; }

// Sum (or maximum) over a team, in a fixed order. `red` has a place for each
// wave of the workgroup and is used in alternation by the caller, so that one
// barrier a call is enough.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* red) {
  v = wave_sum(v);
  if (TEAM == 64) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < TEAM / 64; ++w) t += red[w];
  return t;
}
template <int TEAM>
__device__ __forceinline__ float team_max(float v, float* red) {
  v = wave_max(v);
  if (TEAM == 64) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = red[0];
#pragma unroll
  for (int w = 1; w < TEAM / 64; ++w) t = fmaxf(t, red[w]);
  return t;
}

// Eight e4m3 codes, rounded to nearest even.
__device__ __forceinline__ uint2 to_e4m3(const float (&v)[VEC]) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  return make_uint2(lo, hi);
}

constexpr float E4M3_MAX = 448.f;
constexpr float SCALE_MIN = 0x1p-126f;   // its reciprocal is finite

// What a kernel knows of the row width: a multiple of a vector, any other of
// at least a vector, or less. Decided at compile time, so that no branch
// stands between a row's loads and their uses.
enum class Width { EVEN, RAGGED, NARROW };

template <Width S, Use U, int V, class T>
__device__ __forceinline__ void fetch_vecs(const T* row, int dim, int col, int stride,
                                           Raw<T> (&raw)[V]) {
  if constexpr (S == Width::NARROW) return;
#pragma unroll
  for (int j = 0; j < V; ++j) raw[j] = fetch_at<U>(row, dim, col + j * stride);
}
template <Width S, int V, class T>
__device__ __forceinline__ void widen_vecs(const Raw<T> (&raw)[V], const T* row, int dim, int col,
                                           int stride, float (&v)[V][VEC]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if constexpr (S == Width::EVEN) widen(raw[j], v[j]);
    else if constexpr (S == Width::RAGGED) widen_ragged(raw[j], dim, col + j * stride, v[j]);
    else widen_narrow(row, dim, col + j * stride, v[j]);
  }
}
template <Width S, Use U = Use::AGAIN, class T>
__device__ __forceinline__ void store_vec(T* row, int dim, int col, const float (&v)[VEC]) {
  if constexpr (S == Width::EVEN) {
    if (col < dim) store8<U>(row + col, v);
  } else {
    store8_upto<U>(row + col, dim - col, v);
  }
}

// Eight columns (or those left of the row) that this thread stored itself.
template <class T>
__device__ __forceinline__ void widen_own(const T* row, int dim, int col, float (&v)[VEC]) {
  if (col + VEC <= dim) {
    load8(row + col, v);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = col + e < dim ? static_cast<float>(row[col + e]) : 0.f;
  }
}

// The two are kept apart: merged, as the compiler would, they lose the hint.
template <Width S, class T>
__device__ __forceinline__ void store_either(bool once, T* row, int dim, int col,
                                             const float (&v)[VEC]) {
  if (once) {
    store_vec<S, Use::ONCE>(row, dim, col, v);
    asm volatile("" ::: "memory");
  } else {
    store_vec<S>(row, dim, col, v);
  }
}

// The weights of a thread's columns, of type T or fp32.
template <Width S, class T, int V>
__device__ __forceinline__ void load_weight(const void* weight, bool f32, int dim, int col,
                                            int stride, float (&w)[V][VEC]) {
  if (f32) {
    Raw<float> r[V];
    fetch_vecs<S, Use::AGAIN>(static_cast<const float*>(weight), dim, col, stride, r);
    widen_vecs<S>(r, static_cast<const float*>(weight), dim, col, stride, w);
  } else {
    Raw<T> r[V];
    fetch_vecs<S, Use::AGAIN>(static_cast<const T*>(weight), dim, col, stride, r);
    widen_vecs<S>(r, static_cast<const T*>(weight), dim, col, stride, w);
  }
}

// Eight columns of y: the values, or their codes.
template <Width S>
__device__ __forceinline__ void store_y(const RmsArgs& a, int y_type, int row, int col,
                                        const float (&v)[VEC]) {
  const int64_t at = row * a.ldy;
  if (y_type == OUT_F32) {
    store_vec<S>(static_cast<float*>(a.y) + at, a.dim, col, v);
  } else if (y_type == OUT_BF16) {
    store_either<S>(a.stream, static_cast<__bf16*>(a.y) + at, a.dim, col, v);
  } else if (y_type == OUT_F16) {
    store_either<S>(a.stream, static_cast<_Float16*>(a.y) + at, a.dim, col, v);
  } else {
    const uint2 q = to_e4m3(v);
    uint8_t* y = static_cast<uint8_t*>(a.y) + at + col;
    const int left = a.dim - col;
    if (left >= VEC) {
      __builtin_memcpy(y, &q, sizeof(q));
    } else if constexpr (S != Width::EVEN) {
      uint8_t b[VEC];
      __builtin_memcpy(b, &q, sizeof(q));
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e < left) y[e] = b[e];
    }
  }
}

// A row's scale for its largest |y|. The codes are those of y times its rounded
// reciprocal, which makes the largest 448, by three roundings more at most: that
// still rounds to the code of 448, no clamp. A quotient within a rounding of fp32 of
// the middle between two codes may take either; dividing instead decides 2886 of
// 67 million codes otherwise, no nearer to 64 bits (2.6e-2 both), in 82 us, not 78.
__device__ __forceinline__ float scale_of(float top) {
  return top > 0.f ? fmaxf(top / E4M3_MAX, SCALE_MIN) : 1.f;
}

// A workgroup goes round the rows (by teams) and has the next row's loads in
// flight while it reduces and writes the present one; the weights stay in
// registers (V is 1 or 2).
template <Width S, class T, class H, int TEAM, int V>
__global__ __launch_bounds__(block_of(TEAM)) void rms_norm_kernel(RmsArgs a, int y_type, bool w32) {
  constexpr int TEAMS = block_of(TEAM) / TEAM, STRIDE = TEAM * VEC;
  __shared__ float red_sum[2][block_of(TEAM) / 64], red_max[block_of(TEAM) / 64];
  const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM, col0 = t * VEC;
  const int step = gridDim.x * TEAMS;
  int row = blockIdx.x * TEAMS + team;
  if (TEAM == 64 && row >= a.rows) return;   // (a workgroup of one team has a row)
  auto x_of = [&](int r) { return static_cast<const T*>(a.x) + r * a.ldx; };
  auto res_of = [&](int r) { return static_cast<const H*>(a.residual) + r * a.ld_residual; };
  Raw<T> rx[V];
  Raw<H> rr[V];
  fetch_vecs<S, Use::ONCE>(x_of(row), a.dim, col0, STRIDE, rx);
  if (a.residual) fetch_vecs<S, Use::ONCE>(res_of(row), a.dim, col0, STRIDE, rr);
  float w[V][VEC];
  load_weight<S, T>(a.weight, w32, a.dim, col0, STRIDE, w);
  int turn = 0;
  for (; row < a.rows; row += step, turn ^= 1) {
    float v[V][VEC];
    widen_vecs<S>(rx, x_of(row), a.dim, col0, STRIDE, v);
    if (a.residual) {
      float r[V][VEC];
      widen_vecs<S>(rr, res_of(row), a.dim, col0, STRIDE, r);
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j][e] = rounded<H>(v[j][e] + r[j][e]);
    }
    if (row + step < a.rows) {
      fetch_vecs<S, Use::ONCE>(x_of(row + step), a.dim, col0, STRIDE, rx);
      if (a.residual) fetch_vecs<S, Use::ONCE>(res_of(row + step), a.dim, col0, STRIDE, rr);
    }
    if (a.residual) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        H* h = static_cast<H*>(a.h) + row * a.ldh;
        store_either<S>(sizeof(H) == 2 && a.stream && y_type == OUT_E4M3, h, a.dim, j * STRIDE + col0,
                        v[j]);
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) part = fmaf(v[j][e], v[j][e], part);
      ss += (j * TEAM + t) * VEC < a.dim ? part : 0.f;
    }
    const float rstd = 1.f / sqrtf(team_sum<TEAM>(ss, red_sum[turn]) / a.dim + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[j][e] = v[j][e] * rstd * w[j][e];
    if (y_type == OUT_E4M3) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float part = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) part = fmaxf(part, fabsf(v[j][e]));
        top = fmaxf(top, (j * TEAM + t) * VEC < a.dim ? part : 0.f);
      }
      top = team_max<TEAM>(top, red_max);
      const float scale = scale_of(top), inv = 1.f / scale;
      if (t == 0) a.scales[row] = scale;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j][e] *= inv;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) store_y<S>(a, y_type, row, j * STRIDE + col0, v[j]);
  }
}

// Rows too wide for the registers of a workgroup: the sum, the largest |y|
// (for codes) and the output are passes over the row, the later ones from the
// caches; with a residual they read back the h that the first one stored.
constexpr int WIDE = 1024;
template <class T, class H>
__global__ __launch_bounds__(WIDE) void rms_norm_wide_kernel(RmsArgs a, int y_type, bool w32) {
  constexpr Width S = Width::RAGGED;
  __shared__ float red_sum[2][WIDE / 64], red_max[WIDE / 64];
  const int step = WIDE * VEC;
  int turn = 0;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const H* res = static_cast<const H*>(a.residual) + row * a.ld_residual;
    H* h = static_cast<H*>(a.h) + row * a.ldh;
    float ss = 0.f;
    for (int col = threadIdx.x * VEC; col < a.dim; col += step) {
      float v[1][VEC], r[1][VEC];
      Raw<T> rx[1];
      Raw<H> rr[1];
      fetch_vecs<S, Use::AGAIN>(x, a.dim, col, 0, rx);
      if (a.residual) fetch_vecs<S, Use::ONCE>(res, a.dim, col, 0, rr);
      widen_vecs<S>(rx, x, a.dim, col, 0, v);
      if (a.residual) {
        widen_vecs<S>(rr, res, a.dim, col, 0, r);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[0][e] = rounded<H>(v[0][e] + r[0][e]);
        store_vec<S>(h, a.dim, col, v[0]);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(v[0][e], v[0][e], ss);
    }
    const float rstd = 1.f / sqrtf(team_sum<WIDE>(ss, red_sum[turn]) / a.dim + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    // y of eight columns, before any scale; a thread reads back only what it stored
    auto y_of = [&](int col, float (&v)[1][VEC]) {
      float w[1][VEC];
      if (a.residual) {
        // the vector that crosses the row's end would begin among the
        // neighbouring thread's columns
        widen_own(h, a.dim, col, v[0]);
      } else {
        Raw<T> rx[1];
        fetch_vecs<S, Use::AGAIN>(x, a.dim, col, 0, rx);
        widen_vecs<S>(rx, x, a.dim, col, 0, v);
      }
      load_weight<S, T>(a.weight, w32, a.dim, col, 0, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[0][e] = v[0][e] * rstd * w[0][e];
    };
    float inv = 1.f;
    if (y_type == OUT_E4M3) {
      float top = 0.f;
      for (int col = threadIdx.x * VEC; col < a.dim; col += step) {
        float v[1][VEC];
        y_of(col, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) top = fmaxf(top, fabsf(v[0][e]));
      }
      const float scale = scale_of(team_max<WIDE>(top, red_max));
      if (threadIdx.x == 0) a.scales[row] = scale;
      inv = 1.f / scale;
    }
    for (int col = threadIdx.x * VEC; col < a.dim; col += step) {
      float v[1][VEC];
      y_of(col, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[0][e] *= inv;
      store_y<S>(a, y_type, row, col, v[0]);
    }
  }
}

// --------------------------------------------------------------- gradient

// A workgroup takes every gridDim.x-th row (by teams) and keeps its share of
// dw in registers; the shares are added up by dweight_kernel.
template <Width S, class T, class H, class D, int TEAM, int V>
__global__ __launch_bounds__(block_of(TEAM)) void rms_grad_kernel(RmsGradArgs a, bool w32) {
  constexpr int TEAMS = block_of(TEAM) / TEAM, STRIDE = TEAM * VEC;
  __shared__ float red[2][block_of(TEAM) / 64];
  __shared__ float share[TEAMS > 1 ? TEAM * V * VEC : 1];
  const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM, col0 = t * VEC;
  const int step = gridDim.x * TEAMS;
  auto dy_of = [&](int r) { return static_cast<const T*>(a.dy) + r * a.lddy; };
  auto h_of = [&](int r) { return static_cast<const H*>(a.h) + r * a.ldh; };
  auto past_of = [&](int r) { return static_cast<const D*>(a.dh) + r * a.lddh; };
  Raw<T> rg[V];
  Raw<H> ru[V];
  Raw<D> rp[V];
  float next_rstd = 0.f;
  auto begin = [&](int r) {   // the loads of a row
    next_rstd = a.rstd[r];
    fetch_vecs<S, Use::ONCE>(dy_of(r), a.dim, col0, STRIDE, rg);
    fetch_vecs<S, Use::ONCE>(h_of(r), a.dim, col0, STRIDE, ru);
    if (a.dh) fetch_vecs<S, Use::ONCE>(past_of(r), a.dim, col0, STRIDE, rp);
  };
  int row = blockIdx.x * TEAMS + team;
  if (row < a.rows) begin(row);
  float w[V][VEC], dw[V][VEC];
  load_weight<S, T>(a.weight, w32, a.dim, col0, STRIDE, w);
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[j][e] = 0.f;
  int turn = 0;
  for (; row < a.rows; row += step, turn ^= 1) {
    float g[V][VEC], u[V][VEC], past[V][VEC];
    const float rstd = next_rstd;
    widen_vecs<S>(rg, dy_of(row), a.dim, col0, STRIDE, g);
    widen_vecs<S>(ru, h_of(row), a.dim, col0, STRIDE, u);
    if (a.dh) widen_vecs<S>(rp, past_of(row), a.dim, col0, STRIDE, past);
    if (row + step < a.rows) begin(row + step);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        u[j][e] *= rstd;
        dw[j][e] = fmaf(g[j][e], u[j][e], dw[j][e]);
        g[j][e] *= w[j][e];
        part = fmaf(g[j][e], u[j][e], part);
      }
      dot += (j * TEAM + t) * VEC < a.dim ? part : 0.f;
    }
    const float mean = team_sum<TEAM>(dot, red[turn]) / a.dim;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float d[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        d[e] = rstd * fmaf(-u[j][e], mean, g[j][e]);
        if (a.dh) d[e] += past[j][e];
      }
      store_vec<S>(static_cast<D*>(a.dx) + row * a.lddx, a.dim, j * STRIDE + col0, d);
    }
  }
  if (!a.dweight) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * a.dim;
  if (TEAMS > 1) {   // add the teams' shares one after the other
    for (int k = 0; k < TEAMS; ++k) {
      if (team == k)
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float& s = share[(j * VEC + e) * TEAM + t];
            dw[j][e] = k == 0 ? dw[j][e] : s + dw[j][e];
            s = dw[j][e];
          }
      __syncthreads();
    }
    if (team != TEAMS - 1) return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    store_vec<S>(out, a.dim, j * STRIDE + col0, dw[j]);
  }
}

// Rows too wide for the registers of a workgroup: two passes over each row
// (the second from the caches), dw's share kept in the workgroup's own row
// of `partial`, whose columns each belong to one thread.
template <class T, class H, class D>
__global__ __launch_bounds__(WIDE) void rms_grad_wide_kernel(RmsGradArgs a, bool w32) {
  constexpr Width S = Width::RAGGED;
  __shared__ float red[2][WIDE / 64];
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * a.dim;
  const int step = WIDE * VEC;
  int turn = 0;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const H* h = static_cast<const H*>(a.h) + row * a.ldh;
    const D* dh = static_cast<const D*>(a.dh) + row * a.lddh;
    const float rstd = a.rstd[row];
    float dot = 0.f;
    for (int col = threadIdx.x * VEC; col < a.dim; col += step) {
      float g[1][VEC], u[1][VEC], w[1][VEC];
      Raw<T> rg[1];
      Raw<H> ru[1];
      fetch_vecs<S, Use::AGAIN>(dy, a.dim, col, 0, rg);
      fetch_vecs<S, Use::AGAIN>(h, a.dim, col, 0, ru);
      load_weight<S, T>(a.weight, w32, a.dim, col, 0, w);
      widen_vecs<S>(rg, dy, a.dim, col, 0, g);
      widen_vecs<S>(ru, h, a.dim, col, 0, u);
#pragma unroll
      for (int e = 0; e < VEC; ++e) dot = fmaf(g[0][e] * w[0][e], u[0][e] * rstd, dot);
    }
    const float mean = team_sum<WIDE>(dot, red[turn]) / a.dim;
    for (int col = threadIdx.x * VEC; col < a.dim; col += step) {
      float g[1][VEC], u[1][VEC], w[1][VEC], past[1][VEC], s[1][VEC], d[VEC];
      Raw<T> rg[1];
      Raw<H> ru[1];
      Raw<D> rp[1];
      Raw<float> rs[1];
      const bool more = a.dweight && row != static_cast<int>(blockIdx.x);
      fetch_vecs<S, Use::AGAIN>(dy, a.dim, col, 0, rg);
      fetch_vecs<S, Use::AGAIN>(h, a.dim, col, 0, ru);
      if (a.dh) fetch_vecs<S, Use::ONCE>(dh, a.dim, col, 0, rp);
      if (more) fetch_vecs<S, Use::AGAIN>(static_cast<const float*>(out), a.dim, col, 0, rs);
      load_weight<S, T>(a.weight, w32, a.dim, col, 0, w);
      widen_vecs<S>(rg, dy, a.dim, col, 0, g);
      widen_vecs<S>(ru, h, a.dim, col, 0, u);
      if (a.dh) widen_vecs<S>(rp, dh, a.dim, col, 0, past);
      if (more) widen_vecs<S>(rs, static_cast<const float*>(out), a.dim, col, 0, s);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        u[0][e] *= rstd;
        s[0][e] = fmaf(g[0][e], u[0][e], more ? s[0][e] : 0.f);
        d[e] = rstd * fmaf(-u[0][e], mean, g[0][e] * w[0][e]);
        if (a.dh) d[e] += past[0][e];
      }
      if (a.dweight) store_vec<S>(out, a.dim, col, s[0]);
      store_vec<S>(static_cast<D*>(a.dx) + row * a.lddx, a.dim, col, d);
    }
  }
}

// dweight[c] = sum over the workgroups' shares: 32 columns by 32 groups of
// shares in a workgroup, the groups' sums joined in order. In 64 bits: rounded to
// fp32 at every share, the sum of 1031 rows was three times as far off as its
// terms, and the kernel's time is that of its loads.
constexpr int DW_COLS = 32, DW_GROUPS = 32;
template <class TO>
__global__ __launch_bounds__(DW_COLS * DW_GROUPS) void dweight_kernel(const float* partial,
                                                                      int blocks, int dim,
                                                                      TO* dweight) {
  __shared__ double sums[DW_GROUPS][DW_COLS + 1];
  const int tx = threadIdx.x % DW_COLS, ty = threadIdx.x / DW_COLS;
  const int col = blockIdx.x * DW_COLS + tx;
  double s = 0.0;
  if (col < dim) {
#pragma unroll 4
    for (int b = ty; b < blocks; b += DW_GROUPS) s += partial[static_cast<int64_t>(b) * dim + col];
  }
  sums[ty][tx] = s;
  __syncthreads();
  if (ty != 0 || col >= dim) return;
  for (int k = 1; k < DW_GROUPS; ++k) s += sums[k][tx];
  dweight[col] = static_cast<TO>(static_cast<float>(s));
}

// Calls f(team, vectors, width) for a row width, each as a type. Rows of up
// to 1024 columns are one wave's, wider ones, up to 8192, a workgroup's. The
// forward kernel is fastest with two vectors a thread (16384 rows of 4096 in
// 79 us; 84 with one, in a team twice as large), the gradient, which holds
// five operands of each, with one (93 us; 101 with two).
template <int FULL, class F>
hipError_t by_width(int dim, F f) {
  using std::integral_constant;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  const integral_constant<int, FULL> full;
  auto shaped = [&](auto team, auto v) {
    if (dim % VEC == 0) return f(team, v, integral_constant<Width, Width::EVEN>{});
    return f(team, v, integral_constant<Width, Width::RAGGED>{});
  };
  if (dim < VEC) return f(integral_constant<int, 64>{}, one, integral_constant<Width, Width::NARROW>{});
  if (dim <= 64 * VEC) return shaped(integral_constant<int, 64>{}, one);
  if (dim <= 128 * VEC) return shaped(integral_constant<int, 64>{}, two);
  if (dim <= 256 * VEC) return shaped(integral_constant<int, 256>{}, one);
  if (dim <= 512 * VEC) return shaped(integral_constant<int, 512 / FULL>{}, full);
  if (dim <= 768 * VEC) return shaped(integral_constant<int, 768 / FULL>{}, full);
  return shaped(integral_constant<int, 1024 / FULL>{}, full);
}

// Workgroups of a kernel: as many as the chip holds at a time; for the
// gradient half of that, which halves what their shares of dw cost and leaves
// the loads as they were (93 us instead of 95).
constexpr int CHIP_THREADS = 256 * 2048;

template <class T, class H>
hipError_t rms_norm_on(const RmsArgs& a, int y_type, bool w32, hipStream_t stream) {
  auto go = [&](auto team, auto v, auto width) {
    constexpr int TEAM = team(), V = v(), TEAMS = block_of(TEAM) / TEAM;
    constexpr Width S = width();
    const int blocks = std::min((a.rows + TEAMS - 1) / TEAMS, CHIP_THREADS / block_of(TEAM));
    hipLaunchKernelGGL((rms_norm_kernel<S, T, H, TEAM, V>), dim3(blocks), dim3(block_of(TEAM)), 0,
                       stream, a, y_type, w32);
    return hipGetLastError();
  };
  if (a.dim <= WIDE * VEC) return by_width<2>(a.dim, go);
  hipLaunchKernelGGL((rms_norm_wide_kernel<T, H>), dim3(std::min(a.rows, CHIP_THREADS / WIDE)),
                     dim3(WIDE), 0, stream, a, y_type, w32);
  return hipGetLastError();
}

template <class T, class H, class D>
hipError_t rms_grad_on(const RmsGradArgs& a, bool w32, hipStream_t stream) {
  if (a.dim > WIDE * VEC) {
    hipLaunchKernelGGL((rms_grad_wide_kernel<T, H, D>), dim3(a.blocks), dim3(WIDE), 0, stream, a, w32);
    return hipGetLastError();
  }
  return by_width<1>(a.dim, [&](auto team, auto v, auto width) {
    constexpr int TEAM = team(), V = v();
    constexpr Width S = width();
    hipLaunchKernelGGL((rms_grad_kernel<S, T, H, D, TEAM, V>), dim3(a.blocks),
                       dim3(block_of(TEAM)), 0, stream, a, w32);
    return hipGetLastError();
  });
}

// Calls f(T{}, H{}): H is T or fp32.
template <class F>
hipError_t by_types(int type, int h_type, F f) {
  return by_type(type, [&](auto t) {
    if (type != h_type) return f(t, float{});
    return f(t, t);
  });
}

}  // namespace

// Elements from which on a call with a residual stores one of its two outputs
// non-temporally, a 16-bit y or, beside e4m3 codes, a 16-bit h: two large outputs
// push the inputs and each other through the caches. 16384 rows of 4096 in bf16
// take 83 us so (both non-temporal 98, none 101), with codes 78 (none 92).
// Without a residual it costs (49 us instead of 45), and in fp32, where a wave's
// store is not whole lines (8192 rows with codes: 86 us, 81 without).
constexpr int64_t STREAM_ELEMS = int64_t{1} << 23;

hipError_t launch_rms_norm(RmsArgs a, int x_type, int h_type, int weight_type, int y_type,
                           hipStream_t stream) {
  if (a.rows <= 0) return hipSuccess;
  a.stream = a.residual && static_cast<int64_t>(a.rows) * a.dim >= STREAM_ELEMS;
  return by_types(x_type, h_type, [&](auto t, auto h) {
    return rms_norm_on<decltype(t), decltype(h)>(a, y_type, weight_type == OUT_F32, stream);
  });
}

int rms_grad_blocks(int64_t rows, int64_t dim) {
  const int64_t teams = dim <= 128 * VEC ? 4 : 1;
  const int64_t threads = dim <= 256 * VEC ? 256 : dim <= 512 * VEC ? 512
                          : dim <= 768 * VEC ? 768 : 1024;
  return static_cast<int>(std::min<int64_t>((rows + teams - 1) / teams, CHIP_THREADS / 2 / threads));
}

hipError_t launch_rms_norm_grad(const RmsGradArgs& a, int dy_type, int h_type, int weight_type,
                                int dx_type, int dweight_type, hipStream_t stream) {
  if (a.rows > 0) {
    const hipError_t e = by_types(dy_type, h_type, [&](auto t, auto h) {
      using T = decltype(t);
      using H = decltype(h);
      const bool w32 = weight_type == OUT_F32;
      if (dx_type == dy_type) return rms_grad_on<T, H, T>(a, w32, stream);
      return rms_grad_on<T, H, float>(a, w32, stream);
    });
    if (e != hipSuccess) return e;
  }
  if (!a.dweight) return hipSuccess;
  return by_type(dweight_type, [&](auto t) {
    using TO = decltype(t);
    hipLaunchKernelGGL(dweight_kernel<TO>, dim3((a.dim + DW_COLS - 1) / DW_COLS),
                       dim3(DW_COLS * DW_GROUPS), 0, stream, a.partial, a.rows > 0 ? a.blocks : 0,
                       a.dim, static_cast<TO*>(a.dweight));
    return hipGetLastError();
  });
}

}  // namespace nsmi
