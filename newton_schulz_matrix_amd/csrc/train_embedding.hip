// Embedding lookup with scaling and its gradient.
//
// out[i] = scale * table[ids[i]];  grad[v] = scale * sum_{i: ids[i] = v} grad_out[i].
//
// Both are bound by memory: the lookup moves count x dim elements in and out,
// the gradient reads count x dim and writes the rows x dim table once. A
// thread owns eight columns; TX threads (a power of two) lie along a row and
// 256 / TX rows share a workgroup, so narrow tables fill the lanes too.
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

// ---------------------------------------------------------------- lookup

template <class TI, class TO, class I, int R>
__global__ __launch_bounds__(256) void embedding_kernel(EmbedArgs a, int tx_log2) {
  const int tx = threadIdx.x & ((1 << tx_log2) - 1);
  const int ty = threadIdx.x >> tx_log2, teams = 256 >> tx_log2;
  const int col = ((blockIdx.y << tx_log2) + tx) * VEC;
  if (col >= a.dim) return;
  const int first = blockIdx.x * (R * teams) + ty;
  int64_t id[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = first + r * teams;
    id[r] = i < a.count ? static_cast<int64_t>(static_cast<const I*>(a.ids)[i]) : -1;
  }
  float v[R][VEC];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[r][e] = 0.f;
    if (id[r] >= 0 && id[r] < a.rows)
      load8_upto(static_cast<const TI*>(a.table) + id[r] * a.ld_table + col, a.dim - col, v[r]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = first + r * teams;
    if (i >= a.count) break;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[r][e] *= a.scale;
    store8_upto(static_cast<TO*>(a.out) + i * a.ld_out + col, a.dim - col, v[r]);
  }
}

// ------------------------------------------------------------- id sorting

constexpr int SORT_THREADS = 1024;
constexpr int SORT_WAVES = SORT_THREADS / 64;
constexpr int SORT_RANGE = 512;    // most slots of a group: 32 KB of counters
constexpr int SORT_BATCH = 4;      // windows of 64 ids loaded ahead

// A stable counting sort in one launch. Workgroup g takes the ids whose low
// bits are g. It counts them per slot, and how many ids belong to groups
// before it, so it knows where its part of `order` begins without hearing
// from another workgroup; then it goes over the ids again and puts each
// position in its place. Every workgroup reads all ids (twice): they are a
// thousandth of the gradient's bytes and come from the caches. Each wave takes a contiguous part of the ids
// and keeps its own counters, so positions of one row stay in order.
template <class I>
__global__ __launch_bounds__(SORT_THREADS) void sort_kernel(EmbedGradArgs a) {
  extern __shared__ int counters[];            // (SORT_WAVES, range)
  __shared__ int wave_total[SORT_WAVES], wave_below[SORT_WAVES];
  const int range = a.sort.range, gl = a.sort.groups_log2;
  const int group = blockIdx.x, mask = (1 << gl) - 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* mine = counters + wave * range;
  for (int i = threadIdx.x; i < SORT_WAVES * range; i += SORT_THREADS) counters[i] = 0;
  __syncthreads();

  const I* ids = static_cast<const I*>(a.ids);
  const int per = ((a.count + SORT_WAVES * 64 - 1) / (SORT_WAVES * 64)) * 64;
  const int begin = min(a.count, wave * per), end = min(a.count, begin + per);
  // id at position i, -1 where it does not count
  auto id_at = [&](int i) -> int {
    if (i >= end) return -1;
    const int64_t id = static_cast<int64_t>(ids[i]);
    return id >= 0 && id < a.rows && id != a.padding_id ? static_cast<int>(id) : -1;
  };

  int below = 0;
  for (int base = begin; base < end; base += 64 * SORT_BATCH) {
    int id[SORT_BATCH];
#pragma unroll
    for (int u = 0; u < SORT_BATCH; ++u) id[u] = id_at(base + u * 64 + lane);
#pragma unroll
    for (int u = 0; u < SORT_BATCH; ++u) {
      if (id[u] < 0) continue;
      const int g = id[u] & mask;
      below += g < group;
      if (g == group) atomicAdd(&mine[id[u] >> gl], 1);
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) below += __shfl_xor(below, off, 64);
  if (lane == 0) wave_below[wave] = below;
  __syncthreads();

  // slot r's ids: the total over the waves, then an exclusive scan over the slots
  const int r = threadIdx.x;
  int total = 0;
  if (r < range)
    for (int w = 0; w < SORT_WAVES; ++w) {
      const int n = counters[w * range + r];
      counters[w * range + r] = total;
      total += n;
    }
  int upto = total;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int x = __shfl_up(upto, off, 64);
    if (lane >= off) upto += x;
  }
  if (lane == 63) wave_total[wave] = upto;
  __syncthreads();
  int at = upto - total;
  for (int w = 0; w < SORT_WAVES; ++w) {
    at += wave_below[w];
    if (w < wave) at += wave_total[w];
  }
  if (r < range) {
    a.start[group * range + r] = at;
    for (int w = 0; w < SORT_WAVES; ++w) counters[w * range + r] += at;
    if (group == mask && r == range - 1) a.start[a.sort.slots] = at + total;
  }
  __syncthreads();

  const uint64_t before = (uint64_t{1} << lane) - 1;
  for (int base = begin; base < end; base += 64 * SORT_BATCH) {
    int id[SORT_BATCH];
#pragma unroll
    for (int u = 0; u < SORT_BATCH; ++u) id[u] = id_at(base + u * 64 + lane);
#pragma unroll
    for (int u = 0; u < SORT_BATCH; ++u) {
      const bool own = id[u] >= 0 && (id[u] & mask) == group;
      uint64_t todo = __ballot(own);
      while (todo) {   // one distinct id at a time; few share a group
        const int leader = __ffsll(static_cast<unsigned long long>(todo)) - 1;
        const int which = __shfl(id[u], leader, 64);
        const bool same = own && id[u] == which;
        const uint64_t peers = __ballot(same);
        int first = 0;
        if (lane == leader) first = atomicAdd(&mine[which >> gl], __popcll(peers));
        first = __shfl(first, leader, 64);
        if (same) a.order[first + __popcll(peers & before)] = base + u * 64 + lane;
        todo &= ~peers;
      }
    }
  }
}

// --------------------------------------------------------------- gradient

// Adds the gradients of sorted places [from, to), in order, to sum.
template <class T>
__device__ __forceinline__ void add_terms(const EmbedGradArgs& a, int from, int to, int col,
                                          float (&sum)[VEC]) {
  constexpr int U = 4;
  const T* g = static_cast<const T*>(a.grad_out) + col;
  int k = from;
  for (; k + U <= to; k += U) {
    int i[U];
    float v[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) i[u] = a.order[k + u];
#pragma unroll
    for (int u = 0; u < U; ++u) load8_upto(g + i[u] * a.ld_grad_out, a.dim - col, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[e] += v[u][e];
  }
  for (; k < to; ++k) {
    float v[VEC];
    load8_upto(g + a.order[k] * a.ld_grad_out, a.dim - col, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] += v[e];
  }
}

// Sums of the windows of `window` sorted places that belong to one row
// altogether: a row that a large share of the ids name is summed by many
// workgroups. Other windows are left alone.
template <class T, class I>
__global__ __launch_bounds__(256) void window_kernel(EmbedGradArgs a, int tx_log2) {
  const int tx = threadIdx.x & ((1 << tx_log2) - 1);
  const int w = blockIdx.x * (256 >> tx_log2) + (threadIdx.x >> tx_log2);
  const int col = ((blockIdx.y << tx_log2) + tx) * VEC;
  if (col >= a.dim || w >= a.sort.windows) return;
  const int from = w * a.sort.window, to = from + a.sort.window;
  if (to > a.start[a.sort.slots]) return;
  const I* ids = static_cast<const I*>(a.ids);
  if (ids[a.order[from]] != ids[a.order[to - 1]]) return;
  float sum[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  add_terms<T>(a, from, to, col, sum);
  store8_upto(a.partial + static_cast<int64_t>(w) * a.dim + col, a.dim - col, sum);
}

// Every row of the table's gradient: its terms up to the first whole window,
// the whole windows' sums, the terms after the last.
template <class T, class TO>
__global__ __launch_bounds__(256) void rows_kernel(EmbedGradArgs a, int tx_log2) {
  const int tx = threadIdx.x & ((1 << tx_log2) - 1);
  const int teams = 256 >> tx_log2;
  const int col = ((blockIdx.y << tx_log2) + tx) * VEC;
  if (col >= a.dim) return;
  const int left = a.dim - col, S = a.sort.window;
  for (int v = blockIdx.x * teams + (threadIdx.x >> tx_log2); v < a.rows; v += gridDim.x * teams) {
    const int p = sorted_slot(v, a.sort);
    const int s = a.start[p], e = a.start[p + 1];
    TO* out = static_cast<TO*>(a.grad) + v * a.ld_grad + col;
    float sum[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (s == e) {
      if (!a.accumulate) store8_upto(out, left, sum);
      continue;
    }
    const int w0 = (s + S - 1) / S, w1 = e / S;
    if (w0 < w1) {
      add_terms<T>(a, s, w0 * S, col, sum);
      for (int w = w0; w < w1; ++w) {
        float part[VEC];
        load8_upto(a.partial + static_cast<int64_t>(w) * a.dim + col, left, part);
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += part[i];
      }
      add_terms<T>(a, w1 * S, e, col, sum);
    } else {
      add_terms<T>(a, s, e, col, sum);
    }
    float old[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.accumulate) load8_upto(static_cast<const TO*>(out), left, old);
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum[i] = fmaf(a.scale, sum[i], old[i]);
    store8_upto(out, left, sum);
  }
}

// Threads along a row (log2) and workgroups along it.
struct Across { int tx_log2; unsigned blocks; };
Across across(int dim) {
  const int vecs = (dim + VEC - 1) / VEC;
  int lg = 0;
  while (lg < 8 && (1 << lg) < vecs) ++lg;
  return {lg, static_cast<unsigned>((vecs + (1 << lg) - 1) >> lg)};
}
unsigned ceil_div(int64_t a, int64_t b) { return static_cast<unsigned>((a + b - 1) / b); }

template <class TI, class TO, class I>
void embedding_on(const EmbedArgs& a, hipStream_t stream) {
  const Across x = across(a.dim);
  const int teams = 256 >> x.tx_log2;
  if (a.count >= 4096 * teams)
    hipLaunchKernelGGL((embedding_kernel<TI, TO, I, 4>), dim3(ceil_div(a.count, 4 * teams), x.blocks),
                       dim3(256), 0, stream, a, x.tx_log2);
  else
    hipLaunchKernelGGL((embedding_kernel<TI, TO, I, 1>), dim3(ceil_div(a.count, teams), x.blocks),
                       dim3(256), 0, stream, a, x.tx_log2);
}

}  // namespace

hipError_t launch_embedding(const EmbedArgs& a, int table_type, bool ids64, int out_type,
                            hipStream_t stream) {
  if (a.count <= 0) return hipSuccess;
  return by_type(table_type, [&](auto ti) {
    return by_type(out_type, [&](auto to) {
      if (ids64) embedding_on<decltype(ti), decltype(to), int64_t>(a, stream);
      else embedding_on<decltype(ti), decltype(to), int32_t>(a, stream);
      return hipGetLastError();
    });
  });
}

EmbedSort embed_sort_plan(int64_t rows, int64_t count) {
  EmbedSort s;
  s.groups_log2 = 8;
  while (((rows - 1) >> s.groups_log2) + 1 > SORT_RANGE) ++s.groups_log2;
  while (s.groups_log2 > 0 && (int64_t{1} << s.groups_log2) > rows) --s.groups_log2;
  s.range = static_cast<int>(((rows - 1) >> s.groups_log2) + 1);
  s.slots = s.range << s.groups_log2;
  // a row of c terms takes up to 2 window + c / window steps: about sqrt(count) of each
  s.window = 32;
  while (4 * int64_t{s.window} * s.window < count) s.window *= 2;
  s.windows = static_cast<int>(count / s.window);
  return s;
}

hipError_t launch_embedding_grad(const EmbedGradArgs& a, int grad_out_type, bool ids64,
                                 int grad_type, hipStream_t stream) {
  const EmbedSort& s = a.sort;
  const dim3 groups(1u << s.groups_log2), threads(SORT_THREADS);
  const size_t lds = sizeof(int) * SORT_WAVES * s.range;
  if (ids64) hipLaunchKernelGGL(sort_kernel<int64_t>, groups, threads, lds, stream, a);
  else hipLaunchKernelGGL(sort_kernel<int32_t>, groups, threads, lds, stream, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const Across x = across(a.dim);
  const int teams = 256 >> x.tx_log2;
  return by_type(grad_out_type, [&](auto t) {
    using T = decltype(t);
    if (s.windows > 0) {
      const dim3 grid(ceil_div(s.windows, teams), x.blocks);
      if (ids64) hipLaunchKernelGGL((window_kernel<T, int64_t>), grid, dim3(256), 0, stream, a, x.tx_log2);
      else hipLaunchKernelGGL((window_kernel<T, int32_t>), grid, dim3(256), 0, stream, a, x.tx_log2);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return by_type(grad_type, [&](auto to) {
      const unsigned blocks = std::min(ceil_div(a.rows, teams), 1u << 16);
      hipLaunchKernelGGL((rows_kernel<T, decltype(to)>), dim3(blocks, x.blocks), dim3(256), 0,
                         stream, a, x.tx_log2);
      return hipGetLastError();
    });
  });
}

}  // namespace nsmi
