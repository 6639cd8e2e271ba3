// Embedding lookup with scaling and its gradient.
//
// out[i] = scale * table[ids[i]];  grad[v] = scale * sum_{i: ids[i] = v} grad_out[i].
//
// Both are bound by memory: the lookup moves count x dim elements in and out,
// the gradient reads count x dim and writes rows x dim, most of them zeros. A
// thread owns eight columns; TX threads (a power of two) lie along a row and
// the other threads of a workgroup take further rows, so narrow tables fill
// the lanes too.
//
// The gradient is three launches. One sorts the ids. One sums, in windows of
// the sorted places, what belongs to runs (the places of one id) that cross a
// window's border, and, in further workgroups, clears the table. One adds up
// each run, from its terms or from its windows' sums, and writes its row. The
// rows that some id names are written twice: a clearing workgroup that first
// looked up whether its row is named would wait for that longer than the
// row's zeros take.
//
// 16384 tokens of 4096 columns in bf16, 128000 rows: the lookup takes 34 us
// (each row of the table is read once and found in the caches after that:
// 6.4 TB/s), the gradient 235 to 240 us for 1.18 GB: 9 to 12 for the sort, 160
// to 190 for the clearing (1.05 GB at 5.5 to 6.6 TB/s), 36 to 55 for the runs.
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace nsmi {
namespace {

// Eight columns of R rows of a table, all in flight together (row numbers must
// be valid).
template <int R, class T>
__device__ __forceinline__ void fetch_rows(const T* table, int64_t ld, const int (&rows)[R],
                                           int dim, int col, Raw<T> (&raw)[R]) {
  if (dim < VEC) return;
#pragma unroll
  for (int r = 0; r < R; ++r) raw[r] = fetch_at(table + rows[r] * ld, dim, col);
}
// ---------------------------------------------------------------- lookup

template <class TI, class TO, class I, int R>
__global__ __launch_bounds__(256) void embedding_kernel(EmbedArgs a, int tx_log2) {
  const int tx = threadIdx.x & ((1 << tx_log2) - 1);
  const int ty = threadIdx.x >> tx_log2, teams = 256 >> tx_log2;
  const int col = ((blockIdx.y << tx_log2) + tx) * VEC;
  if (col >= a.dim) return;
  const int first = blockIdx.x * (R * teams) + ty;
  int64_t id[R];
  int row[R];
  bool used[R];
#pragma unroll
  for (int r = 0; r < R; ++r) id[r] = static_cast<const I*>(a.ids)[min(first + r * teams, a.count - 1)];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    used[r] = id[r] >= 0 && id[r] < a.rows;
    row[r] = used[r] ? static_cast<int>(id[r]) : 0;
  }
  const TI* table = static_cast<const TI*>(a.table);
  Raw<TI> raw[R];
  fetch_rows(table, a.ld_table, row, a.dim, col, raw);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = first + r * teams;
    if (i >= a.count) break;
    float v[VEC];
    widen_at(raw[r], table + row[r] * a.ld_table, a.dim, col, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = used[r] ? v[e] * a.scale : 0.f;
    // a large output (R > 1) does not stay in the L2 caches anyway: 16384 rows of
    // 4096 take 34 us so in bf16 (37 cached) and 80 in fp32 (90)
    store8_upto<R == 1 ? Use::AGAIN : Use::ONCE>(static_cast<TO*>(a.out) + i * a.ld_out + col,
                                                 a.dim - col, v);
  }
}

// ------------------------------------------------------------- id sorting

constexpr int SORT_THREADS = 1024;
constexpr int SORT_WAVES = SORT_THREADS / 64;
constexpr int SORT_RANGE = 512;    // most slots of a group: 32 KB of counters
constexpr int SORT_BATCH = 16;     // windows of 64 ids loaded together

// A stable counting sort in one launch. Workgroup g takes the ids whose low
// bits are g. It counts them per slot, and how many ids belong to groups
// before it, so it knows where its part of `sorted` begins without hearing
// from another workgroup; then it goes over the ids again and puts each
// position in its place. Each wave takes a contiguous part of the ids and
// keeps its own counters, so positions of one id stay in order.
//
// Every workgroup reads all ids, from the caches, once up to 16384 of them
// (they stay in registers in between) and twice above. Groups grow with the
// table, from 256 up to 131072 rows to 16384 at 2^23, so the time goes as rows
// times ids: made for batches of up to some 65536 ids, whose rows of hundreds of
// columns and more take longer. 128000 rows: 16384 ids 9 to 12 us, most of it the
// latency of a launch, two rounds of loads and three barriers, 65536 ids 29 to
// 36, 2^20 ids 353. 2^18 rows, 2^20 ids: 629; 2^23 rows: 2^18 ids 4.4 ms, 2^20 17,
// 2^23 135.
template <class I>
__global__ __launch_bounds__(SORT_THREADS) void sort_kernel(EmbedGradArgs a) {
  extern __shared__ int counters[];            // (SORT_WAVES, range)
  __shared__ int wave_total[SORT_WAVES], wave_below[SORT_WAVES], counted;
  const int range = a.sort.range, gl = a.sort.groups_log2;
  const int group = blockIdx.x, mask = (1 << gl) - 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* mine = counters + wave * range;
  for (int i = threadIdx.x; i < SORT_WAVES * range; i += SORT_THREADS) counters[i] = 0;
  __syncthreads();

  const I* ids = static_cast<const I*>(a.ids);
  const int per = ((a.count + SORT_WAVES * 64 - 1) / (SORT_WAVES * 64)) * 64;
  const int begin = min(a.count, wave * per), end = min(a.count, begin + per);
  // id at position i, -1 where it does not count (no branch before the load:
  // a batch's loads are in flight together)
  const uint32_t rows = a.rows, padding = a.padding_id >= 0 && a.padding_id < a.rows
                                              ? static_cast<uint32_t>(a.padding_id) : rows;
  auto id_at = [&](int i) -> int {
    const int64_t id = static_cast<int64_t>(ids[min(i, end - 1)]);
    const uint32_t low = static_cast<uint32_t>(id);   // all of an id that counts
    const bool high = static_cast<uint32_t>(static_cast<uint64_t>(id) >> 32) != 0;
    return i < end && !high && low < rows && low != padding ? static_cast<int>(low) : -1;
  };

  int below = 0;
  int id[SORT_BATCH];
  for (int base = begin; base < end; base += 64 * SORT_BATCH) {
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
    if (group == mask && r == range - 1) {
      a.start[a.sort.slots] = at + total;
      counted = at + total;
    }
  }
  __syncthreads();
  if (group == mask)   // the places behind the last counted id
    for (int k = counted + threadIdx.x; k < a.count; k += SORT_THREADS)
      a.sorted[k] = make_int2(0, -1);

  const uint64_t before = (uint64_t{1} << lane) - 1;
  for (int base = begin; base < end; base += 64 * SORT_BATCH) {
    if (per > 64 * SORT_BATCH)
#pragma unroll
      for (int u = 0; u < SORT_BATCH; ++u) id[u] = id_at(base + u * 64 + lane);
#pragma unroll
    for (int u = 0; u < SORT_BATCH; ++u) {
      const bool own = id[u] >= 0 && (id[u] & mask) == group;
      uint64_t todo = __ballot(own);
      while (todo) {   // one distinct id at a time; few share a group
        const int leader = __ffsll(static_cast<unsigned long long>(todo)) - 1;
        const int which = __builtin_amdgcn_readlane(id[u], leader);   // (leader is uniform)
        const bool same = own && id[u] == which;
        const uint64_t peers = __ballot(same);
        int first = 0;
        if (lane == leader) first = atomicAdd(&mine[which >> gl], __popcll(peers));
        first = __builtin_amdgcn_readlane(first, leader);
        if (same) a.sorted[first + __popcll(peers & before)] = make_int2(base + u * 64 + lane, which);
        todo &= ~peers;
      }
    }
  }
}

// --------------------------------------------------------------- gradient

// Adds rows of `from`, at index(k) for k in [k0, k1), to sum, in order. A
// batch's rows are in flight together, the next batch's indices with them;
// the places past k1 in the last batch repeat its last row (which is then at
// hand) and do not count.
template <class T, class F>
__device__ __forceinline__ void add_rows(const T* from, int64_t ld, int dim, int col, int k0, int k1,
                                         F index, float (&sum)[VEC]) {
  constexpr int U = 8;
  int next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) next[u] = k0 < k1 ? index(min(k0 + u, k1 - 1)) : 0;
  for (int k = k0; k < k1; k += U) {
    int row[U];
    Raw<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) row[u] = next[u];
    fetch_rows(from, ld, row, dim, col, raw);
    if (k + U < k1)
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = index(min(k + U + u, k1 - 1));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[VEC];
      widen_at(raw[u], from + row[u] * ld, dim, col, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[e] += k + u < k1 ? v[e] : 0.f;
    }
  }
}

// Adds the gradients of sorted places [k0, k1).
template <class T>
__device__ __forceinline__ void add_terms(const EmbedGradArgs& a, int k0, int k1, int col,
                                          float (&sum)[VEC]) {
  add_rows(static_cast<const T*>(a.grad_out), a.ld_grad_out, a.dim, col, k0, k1,
           [&](int k) { return a.sorted[k].x; }, sum);
}

// What there is to clear: `rows` of `cols` elements; a dense table is one row.
struct Clear {
  int64_t rows, cols, across;   // across: workgroups along a row
};
constexpr int CLEAR_STEP = 256 * VEC * 4;   // elements of a workgroup

// How a table's gradient is stored. Non-temporal in 16 bits, where a wave's
// store is whole lines (160 to 190 us for the zeros of 1.05 GB). In fp32 a lane's
// eight elements are two stores, each of every second 16 bytes of its lines: past
// the caches those take 449 us for the same bytes, through them, which join the
// halves, 182; 64000 rows of 4096 with 8192 tokens are 498 us in all and 240.
template <class T>
constexpr Use TABLE = sizeof(T) == 2 ? Use::ONCE : Use::AGAIN;

template <class T>
__device__ __forceinline__ void clear_rows(T* table, int64_t ld, const Clear& c, int64_t block,
                                           int64_t blocks) {
  const float zero[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (; block < c.rows * c.across; block += blocks) {
    const int64_t row = c.rows == 1 ? 0 : block / c.across;
    const int64_t from = (block - row * c.across) * CLEAR_STEP;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t col = from + (j * 256 + threadIdx.x) * VEC;
      if (col + VEC <= c.cols) store8<TABLE<T>>(table + row * ld + col, zero);
      else if (col < c.cols) store8_upto(table + row * ld + col, static_cast<int>(c.cols - col), zero);
    }
  }
}

// The first `summing` workgroups take a window of the sorted places each (by
// teams) and sum what in it belongs to a run that came in from the window
// before (row 2 w of `partial`) and to one that begins here and goes on in the
// window after (row 2 w + 1). A run is then the sum of its windows' rows: an id
// that a tenth of the places name is summed by many workgroups, with no serial
// remainder. The other workgroups clear the table in the order of the
// addresses: 1.05 GB is written at 5.5 to 6.6 TB/s so, 1 GB at 5.4 by fewer
// workgroups that go round.
template <class T, class TO>
__global__ __launch_bounds__(256) void window_clear_kernel(EmbedGradArgs a, int tx_log2,
                                                           unsigned summing, Clear clear) {
  if (blockIdx.x >= summing) {
    clear_rows(static_cast<TO*>(a.grad), a.ld_grad, clear, blockIdx.x - summing,
               gridDim.x - summing);
    return;
  }
  const int tx = threadIdx.x & ((1 << tx_log2) - 1), ty = threadIdx.x >> tx_log2;
  const int teams = 256 >> tx_log2, across = (a.dim + (VEC << tx_log2) - 1) / (VEC << tx_log2);
  const int w = static_cast<int>(blockIdx.x / across) * teams + ty;
  const int col = (static_cast<int>(blockIdx.x % across) * (1 << tx_log2) + tx) * VEC;
  if (col >= a.dim || w >= a.sort.windows) return;
  const int from = w * a.sort.window, to = min(from + a.sort.window, a.count);
  const int head = a.sorted[from].y, tail = a.sorted[to - 1].y;
  const int before = from > 0 ? a.sorted[from - 1].y : -1;
  const int after = to < a.count ? a.sorted[to].y : -1;
  float* out = a.partial + static_cast<int64_t>(2 * w) * a.dim + col;
  int rest = from;   // first place behind the run that came in
  if (head >= 0 && head == before) {
    rest = min(to, a.start[sorted_slot(head, a.sort) + 1]);
    float sum[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    add_terms<T>(a, from, rest, col, sum);
    store8_upto(out, a.dim - col, sum);
  }
  if (tail >= 0 && tail == after && rest < to) {
    float sum[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    add_terms<T>(a, max(from, a.start[sorted_slot(tail, a.sort)]), to, col, sum);
    store8_upto(out + a.dim, a.dim - col, sum);
  }
}

// A team takes PLACES sorted places and the runs (places of one id) that
// begin there: all its rows are read at once and summed run by run. A run that
// goes on past the team's places is followed to its end, if that lies in the
// same window, and otherwise taken from its windows' sums.
template <class T, class TO, bool ADD>
__global__ __launch_bounds__(256) void runs_kernel(EmbedGradArgs a, int tx_log2) {
  constexpr int PLACES = ADD || sizeof(T) == 4 ? 4 : 8;
  const int tx = threadIdx.x & ((1 << tx_log2) - 1);
  const int first = (blockIdx.x * (256 >> tx_log2) + (threadIdx.x >> tx_log2)) * PLACES;
  const int col = ((blockIdx.y << tx_log2) + tx) * VEC;
  if (col >= a.dim || first >= a.count) return;
  const int left = a.dim - col, last = a.count - 1;
  int2 place[PLACES];
#pragma unroll
  for (int u = 0; u < PLACES; ++u) place[u] = a.sorted[min(first + u, last)];
  const int before = first > 0 ? a.sorted[first - 1].y : -1;
  const int after = first + PLACES <= last ? a.sorted[first + PLACES].y : -1;
  // id of the run each place belongs to, if that run begins here
  int id[PLACES], row[PLACES], head[PLACES];
  bool used[PLACES], heads[PLACES];
  bool any = false;
#pragma unroll
  for (int u = 0; u < PLACES; ++u) {
    id[u] = first + u <= last ? place[u].y : -1;
    const int previous = u == 0 ? before : place[u - 1].y;
    heads[u] = id[u] >= 0 && id[u] != previous;
    used[u] = id[u] >= 0 && (heads[u] || (u > 0 && used[u - 1]));
    row[u] = used[u] ? place[u].x : 0;
    head[u] = heads[u] ? id[u] : 0;
    any = any || used[u];
  }
  if (!any) return;
  const T* from = static_cast<const T*>(a.grad_out);
  const TO* into = static_cast<const TO*>(a.grad);
  Raw<T> raw[PLACES];
  Raw<TO> old[PLACES];
  fetch_rows(from, a.ld_grad_out, row, a.dim, col, raw);
  if constexpr (ADD) fetch_rows(into, a.ld_grad, head, a.dim, col, old);
  float sum[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, base[VEC];
  auto write = [&](int which) {
    float out[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[i] = fmaf(a.scale, sum[i], ADD ? base[i] : 0.f);
    store8_upto<TABLE<TO>>(static_cast<TO*>(a.grad) + which * a.ld_grad + col, left, out);
  };
#pragma unroll
  for (int u = 0; u < PLACES; ++u) {
    float v[VEC];
    widen_at(raw[u], from + row[u] * a.ld_grad_out, a.dim, col, v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum[i] = heads[u] ? v[i] : sum[i] + v[i];
    if constexpr (ADD) {
      float o[VEC];
      widen_at(old[u], into + head[u] * a.ld_grad, a.dim, col, o);
#pragma unroll
      for (int i = 0; i < VEC; ++i) base[i] = heads[u] ? o[i] : base[i];
    }
    if (u + 1 < PLACES && used[u] && id[u + 1] != id[u]) write(id[u]);
  }
  const int open = id[PLACES - 1];
  if (!used[PLACES - 1]) return;
  if (after == open) {
    const int S = a.sort.window, w = first / S;
    const int end = a.start[sorted_slot(open, a.sort) + 1];
    if (end <= (w + 1) * S) {
      add_terms<T>(a, first + PLACES, end, col, sum);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
      add_rows(a.partial, a.dim, a.dim, col, w, (end - 1) / S + 1,
               [&](int k) { return k == w ? 2 * w + 1 : 2 * k; }, sum);
    }
  }
  write(open);
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

constexpr unsigned CLEAR_BLOCKS = 1u << 23;   // at most, of one launch; more take turns

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
  // a run of c places takes up to window + c / window steps; the most frequent
  // token of a text is about every tenth
  s.window = 16;
  while (16 * int64_t{s.window} * s.window < count) s.window *= 2;
  s.windows = static_cast<int>((count + s.window - 1) / s.window);
  return s;
}

hipError_t launch_embedding_grad(const EmbedGradArgs& a, int grad_out_type, bool ids64,
                                 int grad_type, hipStream_t stream) {
  const EmbedSort& s = a.sort;
  const dim3 groups(1u << s.groups_log2), threads(SORT_THREADS);
  const size_t lds = sizeof(int) * SORT_WAVES * s.range;
  if (ids64) hipLaunchKernelGGL(sort_kernel<int64_t>, groups, threads, lds, stream, a);
  else hipLaunchKernelGGL(sort_kernel<int32_t>, groups, threads, lds, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const Across x = across(a.dim);
  const int teams = 256 >> x.tx_log2;
  const unsigned summing = ceil_div(s.windows, teams) * x.blocks;
  Clear c{a.rows, a.dim, 0};
  if (a.ld_grad == a.dim) c = {1, static_cast<int64_t>(a.rows) * a.dim, 0};
  c.across = (c.cols + CLEAR_STEP - 1) / CLEAR_STEP;
  const unsigned clearing =
      a.accumulate ? 0 : static_cast<unsigned>(std::min<int64_t>(c.rows * c.across, CLEAR_BLOCKS));
  return by_type(grad_out_type, [&](auto t) {
    return by_type(grad_type, [&](auto to) {
      using T = decltype(t);
      using TO = decltype(to);
      if (summing + clearing > 0) {
        hipLaunchKernelGGL((window_clear_kernel<T, TO>), dim3(summing + clearing), dim3(256), 0,
                           stream, a, x.tx_log2, summing, c);
        e = hipGetLastError();
        if (e != hipSuccess || a.count == 0) return e;
      }
      const int places = a.accumulate || sizeof(T) == 4 ? 4 : 8;
      const dim3 grid(ceil_div(a.count, places * teams), x.blocks);
      if (a.accumulate) hipLaunchKernelGGL((runs_kernel<T, TO, true>), grid, dim3(256), 0, stream, a, x.tx_log2);
      else hipLaunchKernelGGL((runs_kernel<T, TO, false>), grid, dim3(256), 0, stream, a, x.tx_log2);
      return hipGetLastError();
    });
  });
}

}  // namespace nsmi
