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

template <class T>
__device__ __forceinline__ void load_weight(const RmsArgs& a, bool w32, int col, float (&w)[VEC]) {
  if (w32) load8_upto(static_cast<const float*>(a.weight) + col, a.dim - col, w);
  else load8_upto(static_cast<const T*>(a.weight) + col, a.dim - col, w);
}

template <class T, class H, int TEAM, int V>
__global__ __launch_bounds__(block_of(TEAM)) void rms_norm_kernel(RmsArgs a, int y_type, bool w32) {
  constexpr int TEAMS = block_of(TEAM) / TEAM;
  // the weights stay in registers over the rows of a workgroup where they fit
  constexpr bool KEEP = V <= 4;
  __shared__ float red_sum[2][block_of(TEAM) / 64], red_max[block_of(TEAM) / 64];
  const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  float w[KEEP ? V : 1][VEC];
  if (KEEP)
#pragma unroll
    for (int j = 0; j < V; ++j) load_weight<T>(a, w32, (j * TEAM + t) * VEC, w[KEEP ? j : 0]);
  int turn = 0;
  for (int row = blockIdx.x * TEAMS + team; row < a.rows; row += gridDim.x * TEAMS, turn ^= 1) {
    float v[V][VEC];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * TEAM + t) * VEC;
      load8_upto(static_cast<const T*>(a.x) + row * a.ldx + col, a.dim - col, v[j]);
    }
    if (a.residual) {
      float r[V][VEC];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * TEAM + t) * VEC;
        load8_upto(static_cast<const H*>(a.residual) + row * a.ld_residual + col, a.dim - col, r[j]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * TEAM + t) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j][e] = rounded<H>(v[j][e] + r[j][e]);
        store8_upto(static_cast<H*>(a.h) + row * a.ldh + col, a.dim - col, v[j]);
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(v[j][e], v[j][e], ss);
    const float rstd = 1.f / sqrtf(team_sum<TEAM>(ss, red_sum[turn]) / a.dim + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float late[VEC];
      if (!KEEP) load_weight<T>(a, w32, (j * TEAM + t) * VEC, late);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[j][e] = v[j][e] * rstd * (KEEP ? w[KEEP ? j : 0][e] : late[e]);
    }
    if (y_type == OUT_E4M3) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) top = fmaxf(top, fabsf(v[j][e]));
      top = team_max<TEAM>(top, red_max);
      const float scale = top > 0.f ? fmaxf(top / E4M3_MAX, SCALE_MIN) : 1.f;
      const float inv = 1.f / scale;
      if (t == 0) a.scales[row] = scale;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * TEAM + t) * VEC, left = a.dim - col;
        // no clamp: |v * inv| exceeds 448 by two roundings at most, which
        // still rounds to the code of 448
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j][e] *= inv;
        const uint2 q = to_e4m3(v[j]);
        uint8_t* y = static_cast<uint8_t*>(a.y) + row * a.ldy + col;
        if (left >= VEC) {
          __builtin_memcpy(y, &q, sizeof(q));
        } else {
          uint8_t b[VEC];
          __builtin_memcpy(b, &q, sizeof(q));
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (e < left) y[e] = b[e];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * TEAM + t) * VEC, left = a.dim - col;
        const int64_t at = row * a.ldy + col;
        if (y_type == OUT_F32) store8_upto(static_cast<float*>(a.y) + at, left, v[j]);
        else if (y_type == OUT_BF16) store8_upto(static_cast<__bf16*>(a.y) + at, left, v[j]);
        else store8_upto(static_cast<_Float16*>(a.y) + at, left, v[j]);
      }
    }
  }
}

// --------------------------------------------------------------- gradient

struct GradRow {   // eight columns of one row
  float g[VEC], u[VEC], dwu[VEC];
};

template <class T>
__device__ __forceinline__ void load_weight(const RmsGradArgs& a, bool w32, int col,
                                            float (&w)[VEC]) {
  if (w32) load8_upto(static_cast<const float*>(a.weight) + col, a.dim - col, w);
  else load8_upto(static_cast<const T*>(a.weight) + col, a.dim - col, w);
}

// dx of eight columns, with the gradient that comes past the norm.
template <class T>
__device__ __forceinline__ void store_dx(const RmsGradArgs& a, bool dx32, int row, int col,
                                         float (&d)[VEC]) {
  const int left = a.dim - col;
  if (a.dh) {
    float p[VEC];
    const int64_t at = row * a.lddh + col;
    if (dx32) load8_upto(static_cast<const float*>(a.dh) + at, left, p);
    else load8_upto(static_cast<const T*>(a.dh) + at, left, p);
#pragma unroll
    for (int e = 0; e < VEC; ++e) d[e] += p[e];
  }
  const int64_t at = row * a.lddx + col;
  if (dx32) store8_upto(static_cast<float*>(a.dx) + at, left, d);
  else store8_upto(static_cast<T*>(a.dx) + at, left, d);
}

// A workgroup takes every gridDim.x-th row (by teams) and keeps its share of
// dw in registers; the shares are added up by dweight_kernel.
template <class T, class H, int TEAM, int V>
__global__ __launch_bounds__(block_of(TEAM)) void rms_grad_kernel(RmsGradArgs a, bool w32,
                                                                  bool dx32) {
  constexpr int TEAMS = block_of(TEAM) / TEAM;
  __shared__ float red[2][block_of(TEAM) / 64];
  __shared__ float share[TEAMS > 1 ? TEAM * V * VEC : 1];
  const int t = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  float w[V][VEC], dw[V][VEC];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    load_weight<T>(a, w32, (j * TEAM + t) * VEC, w[j]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[j][e] = 0.f;
  }
  int turn = 0;
  for (int row = blockIdx.x * TEAMS + team; row < a.rows; row += gridDim.x * TEAMS, turn ^= 1) {
    float g[V][VEC], u[V][VEC];
    const float rstd = a.rstd[row];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * TEAM + t) * VEC;
      load8_upto(static_cast<const T*>(a.dy) + row * a.lddy + col, a.dim - col, g[j]);
      load8_upto(static_cast<const H*>(a.h) + row * a.ldh + col, a.dim - col, u[j]);
    }
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        u[j][e] *= rstd;
        dw[j][e] = fmaf(g[j][e], u[j][e], dw[j][e]);
        g[j][e] *= w[j][e];
        dot = fmaf(g[j][e], u[j][e], dot);
      }
    const float mean = team_sum<TEAM>(dot, red[turn]) / a.dim;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float d[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) d[e] = rstd * fmaf(-u[j][e], mean, g[j][e]);
      store_dx<T>(a, dx32, row, (j * TEAM + t) * VEC, d);
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
    const int col = (j * TEAM + t) * VEC;
    store8_upto(out + col, a.dim - col, dw[j]);
  }
}

// Rows too wide for the registers of a workgroup: two passes over each row
// (the second from the caches), dw's share kept in the workgroup's own row
// of `partial`, whose columns each belong to one thread.
constexpr int WIDE = 1024;
template <class T, class H>
__global__ __launch_bounds__(WIDE) void rms_grad_wide_kernel(RmsGradArgs a, bool w32, bool dx32) {
  __shared__ float red[2][WIDE / 64];
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * a.dim;
  const int step = WIDE * VEC;
  int turn = 0;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const H* h = static_cast<const H*>(a.h) + row * a.ldh;
    const float rstd = a.rstd[row];
    float dot = 0.f;
    for (int col = threadIdx.x * VEC; col < a.dim; col += step) {
      float g[VEC], u[VEC], w[VEC];
      load8_upto(dy + col, a.dim - col, g);
      load8_upto(h + col, a.dim - col, u);
      load_weight<T>(a, w32, col, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) dot = fmaf(g[e] * w[e], u[e] * rstd, dot);
    }
    const float mean = team_sum<WIDE>(dot, red[turn]) / a.dim;
    for (int col = threadIdx.x * VEC; col < a.dim; col += step) {
      float g[VEC], u[VEC], w[VEC], d[VEC], s[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      load8_upto(dy + col, a.dim - col, g);
      load8_upto(h + col, a.dim - col, u);
      load_weight<T>(a, w32, col, w);
      if (a.dweight && row != static_cast<int>(blockIdx.x)) load8_upto(out + col, a.dim - col, s);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        u[e] *= rstd;
        s[e] = fmaf(g[e], u[e], s[e]);
        d[e] = rstd * fmaf(-u[e], mean, g[e] * w[e]);
      }
      if (a.dweight) store8_upto(out + col, a.dim - col, s);
      store_dx<T>(a, dx32, row, col, d);
    }
  }
}

// dweight[c] = sum over the workgroups' shares: 32 columns by 32 groups of
// shares in a workgroup, the groups' sums joined in order.
constexpr int DW_COLS = 32, DW_GROUPS = 32;
template <class TO>
__global__ __launch_bounds__(DW_COLS * DW_GROUPS) void dweight_kernel(const float* partial,
                                                                      int blocks, int dim,
                                                                      TO* dweight) {
  __shared__ float sums[DW_GROUPS][DW_COLS + 1];
  const int tx = threadIdx.x % DW_COLS, ty = threadIdx.x / DW_COLS;
  const int col = blockIdx.x * DW_COLS + tx;
  float s = 0.f;
  if (col < dim) {
#pragma unroll 4
    for (int b = ty; b < blocks; b += DW_GROUPS) s += partial[static_cast<int64_t>(b) * dim + col];
  }
  sums[ty][tx] = s;
  __syncthreads();
  if (ty != 0 || col >= dim) return;
  for (int k = 1; k < DW_GROUPS; ++k) s += sums[k][tx];
  dweight[col] = static_cast<TO>(s);
}

// The team and vector count of a row width: calls f<TEAM, V>().
template <class F>
hipError_t by_width(int dim, F f) {
  if (dim <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (dim <= 1024) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (dim <= 2048) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  if (dim <= 4096) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (dim <= 8192) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}
constexpr int REGISTER_DIM = 1024 * 2 * VEC;   // widest row of by_width

constexpr int MAX_BLOCKS = 1 << 16;   // of the forward kernel; further rows go round

template <class T, class H>
hipError_t rms_norm_on(const RmsArgs& a, int y_type, bool w32, hipStream_t stream) {
  auto go = [&](auto team, auto v) {
    constexpr int TEAM = team(), V = v(), TEAMS = block_of(TEAM) / TEAM;
    const int blocks = std::min((a.rows + TEAMS - 1) / TEAMS, MAX_BLOCKS);
    hipLaunchKernelGGL((rms_norm_kernel<T, H, TEAM, V>), dim3(blocks), dim3(block_of(TEAM)), 0,
                       stream, a, y_type, w32);
    return hipGetLastError();
  };
  if (a.dim <= REGISTER_DIM) return by_width(a.dim, go);
  if (a.dim <= 2 * REGISTER_DIM)
    return go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
  return go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
}

template <class T, class H>
hipError_t rms_grad_on(const RmsGradArgs& a, bool w32, bool dx32, hipStream_t stream) {
  if (a.dim > REGISTER_DIM) {
    hipLaunchKernelGGL((rms_grad_wide_kernel<T, H>), dim3(a.blocks), dim3(WIDE), 0, stream, a, w32,
                       dx32);
    return hipGetLastError();
  }
  return by_width(a.dim, [&](auto team, auto v) {
    constexpr int TEAM = team(), V = v();
    hipLaunchKernelGGL((rms_grad_kernel<T, H, TEAM, V>), dim3(a.blocks), dim3(block_of(TEAM)), 0,
                       stream, a, w32, dx32);
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

hipError_t launch_rms_norm(const RmsArgs& a, int x_type, int h_type, int weight_type, int y_type,
                           hipStream_t stream) {
  if (a.rows <= 0) return hipSuccess;
  return by_types(x_type, h_type, [&](auto t, auto h) {
    return rms_norm_on<decltype(t), decltype(h)>(a, y_type, weight_type == OUT_F32, stream);
  });
}

int rms_grad_blocks(int64_t rows, int64_t dim) {
  const int teams = dim <= 2048 ? 4 : 1;
  return static_cast<int>(std::min<int64_t>((rows + teams - 1) / teams, 1024));
}

hipError_t launch_rms_norm_grad(const RmsGradArgs& a, int dy_type, int h_type, int weight_type,
                                int dx_type, int dweight_type, hipStream_t stream) {
  if (a.rows > 0) {
    const hipError_t e = by_types(dy_type, h_type, [&](auto t, auto h) {
      return rms_grad_on<decltype(t), decltype(h)>(a, weight_type == OUT_F32, dx_type == OUT_F32,
                                                   stream);
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
