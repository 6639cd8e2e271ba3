// Device helpers of attention and its gradient: tiles of rows in LDS, matrix
// instructions on them, and where a workgroup's tile lies in the sequences.
//
// Matrix instructions are 32 x 32 x 16. Lane l holds of A the row l % 32 and of B
// the column l % 32, each at k = 8 (l / 32) .. + 7, and of the result column
// l % 32 in register r the row 8 (r / 4) + 4 (l / 32) + r % 4. A result that goes
// on as the B operand of a next product therefore needs no exchange between lanes:
// registers 8 c .. 8 c + 7 are its k chunk c, if the A operand brings its k in the
// same order, which is four rows from 16 c + 4 (l / 32) and four from 8 further on.
//
// A tile is ROWS rows of DP 16-bit values, DP 64 or 128; columns past the head's
// own are zeros. Its 16-byte chunk c of row r lies at chunk c ^ swizzle(r) of the
// row, which spreads both ways of reading over all banks: 16 rows of one chunk,
// and (transposed) four rows of four chunks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "heads_internal.h"

namespace nsmi {

constexpr int CUS = 256;

typedef float Acc __attribute__((ext_vector_type(16)));
typedef uint32_t U32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t U32x4 __attribute__((ext_vector_type(4)));
typedef int I32x4 __attribute__((ext_vector_type(4)));
typedef short S16x4 __attribute__((ext_vector_type(4)));

template <class T>
struct Eight {
  typedef T type __attribute__((ext_vector_type(8)));
};
typedef Eight<_Float16>::type Half8;
typedef Eight<__bf16>::type Brain8;

__device__ __forceinline__ Acc product(Half8 a, Half8 b, Acc c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ Acc product(Brain8 a, Brain8 b, Acc c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ Acc no_sum() {
  Acc a;
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = 0.f;
  return a;
}

// Registers 8 c .. 8 c + 7 of a result as the operand of a next product.
template <class T>
__device__ __forceinline__ typename Eight<T>::type operand(const Acc& a, int c) {
  typename Eight<T>::type v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<T>(a[8 * c + i]);
  return v;
}

// Value of the other half of the wave (lane l ^ 32) beside one's own.
__device__ __forceinline__ void both_halves(float v, float& lower, float& upper) {
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  const uint32_t low = r[0], high = r[1];   // (a cast of an element itself takes the first)
  lower = __builtin_bit_cast(float, low);
  upper = __builtin_bit_cast(float, high);
}

// ------------------------------------------------------------------ tiles

template <int DP>
struct Tile {
  static constexpr int CHUNKS = DP / 8;        // of a row
  static constexpr int ROW = DP * 2;           // bytes
  static constexpr int ROWS_A_COPY = 64 / CHUNKS;   // rows of one wave's copy instruction

  __device__ static __forceinline__ int swizzle(int row) {
    if (DP == 128) return (row & 3) << 2 | (row >> 2 & 3);
    return (row >> 1 & 1) << 2 | (row >> 2 & 3);
  }
};

// Buffer descriptor: reads past `bytes` return zeros. Every word is wave-uniform.
__device__ __forceinline__ I32x4 descriptor(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  I32x4 r = {__builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(a))),
             __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(a >> 32) & 0xffff)),
             __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000};
  return r;
}

// Copies 16 (4) bytes a lane from memory to LDS: lane i's land at `lds` + 16 i (4 i).
// In inline assembly, so that the only waits for them are copies_done()'s: the
// compiler would wait for every copy in flight before any LDS read. Between writing
// m0 and the copy that reads it stands one wait state: the hardware does not wait by
// itself, and the compiler looks for such pairs outside of inline assembly only.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16(I32x4 from, uint32_t lds, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(at), "s"(from) : "memory", "m0");
}
__device__ __forceinline__ void copy4(I32x4 from, uint32_t lds, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(lds), "v"(at), "s"(from) : "memory", "m0");
}
#pragma clang diagnostic pop
// The builtin tells the compiler that its own loads are there too: at the first use of
// one within a loop it would otherwise wait in every round, and so for the copies of
// the next tile.
__device__ __forceinline__ void copies_done() {
  __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt 0, the others as they are
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)p));
}

// A workgroup's copy of ROWS rows of a head into a tile: WAVES waves, each with
// every WAVES-th copy instruction.
template <int DP, int ROWS, int WAVES>
struct Copier {
  static constexpr int EACH = Tile<DP>::ROWS_A_COPY * WAVES;   // rows of an instruction of all waves
  static constexpr int N = ROWS / EACH;                        // instructions of a wave
  static_assert(EACH % 16 == 0 && N * EACH == ROWS, "the swizzle repeats with 16 rows");
  uint32_t at;         // this lane's byte offset from the tile's first row, in the first instruction
  uint32_t lds;        // of the wave's first instruction, from the tile

  // `step`: bytes from one row to the next, at most 2^24; dim: the head's own columns.
  __device__ __forceinline__ Copier(int wave, int lane, uint32_t step, int dim) {
    constexpr int C = Tile<DP>::CHUNKS;
    const int row = wave * Tile<DP>::ROWS_A_COPY + lane / C;
    const int chunk = (lane % C) ^ Tile<DP>::swizzle(row);
    at = 8 * chunk < dim ? row * step + 16 * chunk : 0x80000000u;   // past every descriptor
    lds = __builtin_amdgcn_readfirstlane(wave * 1024);
  }
  // `rows`: how many of the tile's rows there are.
  __device__ __forceinline__ void copy(const void* first, int rows, uint32_t step, int dim,
                                       uint32_t tile) const {
    // (a descriptor for each instruction: a distance added to `at` would stay in a register)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int n = min(rows - i * EACH, EACH);
      const char* const from = static_cast<const char*>(first) + static_cast<int64_t>(i * EACH) * step;
      copy16(descriptor(from, n > 0 ? (n - 1) * step + 2 * dim : 0), tile + lds + i * WAVES * 1024, at);
    }
  }
};

// For kernels that have no registers to spare: reads and products in the order written, the
// operand of a product read AHEAD products before it, and numbers that are made where they
// are used instead of being kept (a constant that the compiler does not know, the lane).
constexpr int AHEAD = 2;
template <bool ON = true>
__device__ __forceinline__ void in_order() {
  if (ON) __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ uint32_t anew(uint32_t x) {
  asm volatile("" : "+s"(x));
  return x;
}
__device__ __forceinline__ int lane_anew() {
  return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, anew(0)));
}

// Reading rows: A (or B) operand of 32 rows at columns 16 k .. + 15, a chunk for each
// lane. Tiles begin at multiples of a row, so that the chunk is told by the
// address' bits above 4 alone: the lane's addresses in a tile are one number with
// k in those bits, and rows further on, or tiles behind it, are at fixed distances.
template <int DP>
struct RowReader {
  uint32_t at;
  __device__ __forceinline__ explicit RowReader(int lane) {
    const int row = lane & 31, half = lane >> 5;
    at = row * Tile<DP>::ROW + ((half ^ Tile<DP>::swizzle(row)) << 4);
  }
  // One address, the others made where they are used.
  struct Lean {
    uint32_t at;
    template <class T>
    __device__ __forceinline__ typename Eight<T>::type read(int k, int further) const {
      const U32x4 v = *(const __attribute__((address_space(3))) U32x4*)((at ^ anew(k << 5)) + further);
      return __builtin_bit_cast(typename Eight<T>::type, v);
    }
  };
  __device__ __forceinline__ Lean lean_in(uint32_t tile) const { return {tile + at}; }
  struct In {
    uint32_t at[DP / 16];
    template <class T>
    __device__ __forceinline__ typename Eight<T>::type read(int k, int further) const {
      const U32x4 v = *(const __attribute__((address_space(3))) U32x4*)(at[k] + further);
      return __builtin_bit_cast(typename Eight<T>::type, v);
    }
  };
  __device__ __forceinline__ In in(uint32_t tile) const {
    In r;
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) r.at[k] = (tile + at) ^ (k << 5);
    return r;
  }
};

// The same for reading transposed: A operand whose rows are columns 32 t .. + 31 and
// whose k are 16 rows, in the order of a result's registers.
// ds_read_b64_tr_b16: within each 16 lanes, lane j supplies the address of four
// consecutive values M[j][0..3]; lane i receives M[4 q + i / 4][i % 4] in slot q.
template <int DP>
struct ColumnReader {
  uint32_t at;
  __device__ __forceinline__ explicit ColumnReader(int lane) {
    const int j = lane & 15, group = lane >> 4;
    const int row = 4 * (group >> 1) + (j >> 2), column = 16 * (group & 1) + 4 * (j & 3);
    at = row * Tile<DP>::ROW + (((column >> 3) ^ Tile<DP>::swizzle(row)) << 4) + (column & 4) * 2;
  }
  template <class T>
  __device__ static __forceinline__ typename Eight<T>::type read_at(uint32_t first, uint32_t eighth) {
    const S16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) S16x4*)first);
    const S16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) S16x4*)eighth);
    const U32x2 a = __builtin_bit_cast(U32x2, x), b = __builtin_bit_cast(U32x2, y);
    const U32x4 v = {a[0], a[1], b[0], b[1]};
    return __builtin_bit_cast(typename Eight<T>::type, v);
  }
  struct In {
    uint32_t at[DP / 32][2];   // four rows, and four from the eighth on
    template <class T>
    __device__ __forceinline__ typename Eight<T>::type read(int t, int further) const {
      return read_at<T>(at[t][0] + further, at[t][1] + (further + 8 * Tile<DP>::ROW));
    }
  };
  struct Lean {
    uint32_t at;
    template <class T>
    __device__ __forceinline__ typename Eight<T>::type read(int t, int further) const {
      return read_at<T>((at ^ anew(t << 6)) + further,
                        (at ^ anew(t << 6 ^ Tile<DP>::swizzle(8) << 4)) + (further + 8 * Tile<DP>::ROW));
    }
  };
  __device__ __forceinline__ Lean lean_in(uint32_t tile) const { return {tile + at}; }
  __device__ __forceinline__ In in(uint32_t tile) const {
    In r;
#pragma unroll
    for (int t = 0; t < DP / 32; ++t) {
      r.at[t][0] = (tile + at) ^ (t << 6);
      r.at[t][1] = r.at[t][0] ^ (Tile<DP>::swizzle(8) << 4);
    }
    return r;
  }
};

template <bool LEAN, class Reader>
__device__ __forceinline__ auto lean_or_all(const Reader& r, uint32_t tile) {
  if constexpr (LEAN) return r.lean_in(tile);
  else return r.in(tile);
}

// This lane's B operands of 32 rows of a head from memory (row: the lane's own, null
// where there is none): k chunk k holds its columns 16 k + 8 (l / 32) .. + 7.
template <class T, int DP>
__device__ __forceinline__ void load_operands(const T* row, int dim, int half,
                                              typename Eight<T>::type (&v)[DP / 16]) {
#pragma unroll
  for (int k = 0; k < DP / 16; ++k) {
    const int column = 16 * k + 8 * half;
    U32x4 x = {0, 0, 0, 0};
    if (row && column < dim) x = *reinterpret_cast<const U32x4*>(row + column);
    v[k] = __builtin_bit_cast(typename Eight<T>::type, x);
  }
}

// Stores a result whose columns are rows of a head (row: the lane's own, null where
// there is none) and whose rows are the head's columns, times `by`. The halves of the
// wave exchange four values each, so that every store is 16 bytes.
template <class T, int DP>
__device__ __forceinline__ void store_columns(T* row, int dim, int half, const Acc (&a)[DP / 32], float by) {
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      T x[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = static_cast<T>(a[t][4 * g + e] * by);
        y[e] = static_cast<T>(a[t][4 * g + 4 + e] * by);
      }
      U32x2 p, q;
      __builtin_memcpy(&p, x, 8);
      __builtin_memcpy(&q, y, 8);
      const auto r0 = __builtin_amdgcn_permlane32_swap(p[0], q[0], false, false);
      const auto r1 = __builtin_amdgcn_permlane32_swap(p[1], q[1], false, false);
      const U32x4 v = {r0[0], r1[0], r0[1], r1[1]};
      const int column = 32 * t + 8 * (g + half);
      if (row && column < dim) *reinterpret_cast<U32x4*>(row + column) = v;
    }
}

// --------------------------------------------------------------- sequences

// Offsets as they may be used whatever they hold: within the tokens.
__device__ __forceinline__ int offset_at(const int* offsets, int b, int tokens) {
  return min(max(offsets[b], 0), tokens);
}

// Where a workgroup's tile of ROWS rows lies.
struct Place {
  int begin, length, row;   // of the sequence; the tile's first row in it
  bool rest;                // behind the last sequence
};

// Tiles of sequence b begin at number offsets[b] / ROWS + b, which leaves room for each
// sequence's own without a count of them; b == sequences stands for the rows behind
// the last. The lanes of a wave look through 64 places at a time. Numbers without
// rows have length 0.
template <int ROWS>
__device__ __forceinline__ Place place_in_order(const int* offsets, int sequences, int tokens, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = sequences + 1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64, b = lo + lane * step;
    const bool before = b < hi && offset_at(offsets, b, tokens) / ROWS + b <= t;
    const int n = max(1, __popcll(__ballot(before)));
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  Place p;
  p.begin = offset_at(offsets, lo, tokens);
  const int end = lo < sequences ? offset_at(offsets, lo + 1, tokens) : tokens;
  p.row = (t - p.begin / ROWS - lo) * ROWS;
  p.rest = lo == sequences;
  p.length = p.row >= 0 && p.row < end - p.begin ? end - p.begin : 0;
  return p;
}

// Sum over a wave, in a scalar register: within rows of 16 lanes by shifts (lanes
// shifted in from outside are 0), then the rows' last lanes.
__device__ __forceinline__ int wave_total(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  return __builtin_amdgcn_readlane(v, 15) + __builtin_amdgcn_readlane(v, 31) + __builtin_amdgcn_readlane(v, 47) +
         __builtin_amdgcn_readlane(v, 63);
}

// The same tiles in the order of their work, the longest first: a tile's work is its
// number in its sequence counted from the end where the work of a tile is what lies
// behind it (BEHIND: keys, seen by the queries behind them), else from the beginning.
// A lane holds a sequence; the work w of the n-th tile is the greatest of which
// more than n tiles have at least as much, sum over the sequences of
// max(0, tiles - w + 1). For up to 64 sequences; without it the last of a batch's
// sequences begin when the others end, and 17% of the CUs' time is lost to that at
// 8 sequences of 1 to 5113 rows.
template <int ROWS, bool BEHIND>
__device__ __forceinline__ Place place_by_work(const int* offsets, int sequences, int tokens, int n) {
  const int lane = threadIdx.x & 63;
  const int begin = offset_at(offsets, min(lane, sequences), tokens);
  const int end = offset_at(offsets, min(lane + 1, sequences), tokens);
  const int mine = lane < sequences && end > begin ? (end - begin + ROWS - 1) / ROWS : 0;
  int lo = 0, hi = tokens / ROWS + 2;   // w is in [lo, hi); no tile has work hi
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (wave_total(max(0, mine - mid + 1)) > n) lo = mid;
    else hi = mid;
  }
  Place p;
  if (lo == 0) {   // behind all tiles of sequences
    p.begin = offset_at(offsets, sequences, tokens);
    p.row = (n - wave_total(mine)) * ROWS;
    p.rest = true;
    p.length = p.row >= 0 && p.row < tokens - p.begin ? tokens - p.begin : 0;
    return p;
  }
  unsigned long long have = __ballot(mine >= lo);
  for (int skip = n - wave_total(max(0, mine - lo)); skip > 0 && (have & (have - 1)) != 0; --skip) have &= have - 1;
  const int b = __builtin_amdgcn_readfirstlane(__ffsll(have) - 1);
  p.begin = __builtin_amdgcn_readlane(begin, b);
  p.length = __builtin_amdgcn_readlane(end, b) - p.begin;
  p.row = (BEHIND ? __builtin_amdgcn_readlane(mine, b) - lo : lo - 1) * ROWS;
  p.rest = false;
  return p;
}

// Place of the n-th of tiles_of() tiles.
template <int ROWS, bool BEHIND>
__device__ __forceinline__ Place place_of(const int* offsets, int sequences, int tokens, int tiles, int n) {
  if (sequences > 1 && sequences <= 64) return place_by_work<ROWS, BEHIND>(offsets, sequences, tokens, n);
  return place_in_order<ROWS>(offsets, sequences, tokens, BEHIND ? n : tiles - 1 - n);
}
inline int64_t tiles_of(int64_t tokens, int64_t sequences, int rows) {
  return tokens / rows + sequences + 1;
}

// The work of one of `parts` workgroups of a tile.
struct Range {
  int first, last;
};
__device__ __forceinline__ Range range_of(int64_t steps, int part, int parts) {
  return {static_cast<int>(steps * part / parts), static_cast<int>(steps * (part + 1) / parts)};
}

// Which part of which tile's work a workgroup has (block < 0: none). The parts of eight
// tiles come one behind the other, so that the longest tiles' parts are all begun
// first, and a tile's keys stay on the XCD that work_of() has in mind.
struct Share {
  int block, part;
};
__device__ __forceinline__ Share share_of(int blocks, int parts) {
  const int n = blockIdx.x / 8, block = n / parts * 8 + blockIdx.x % 8;
  return {block < blocks ? block : -1, n % parts};
}
inline unsigned shared_blocks(int64_t blocks, int parts) {
  return static_cast<unsigned>((blocks + 7) / 8 * 8 * parts);
}

// A part's result in memory as fp32: rows of a head by columns of the lane, as for
// store_columns.
template <int DP>
__device__ __forceinline__ void store_sums(float* row, int dim, int half, const Acc (&a)[DP / 32], float by) {
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int column = 32 * t + 8 * g + 4 * half;
      if (row && column < dim)
        *reinterpret_cast<float4*>(row + column) = make_float4(a[t][4 * g] * by, a[t][4 * g + 1] * by,
                                                               a[t][4 * g + 2] * by, a[t][4 * g + 3] * by);
    }
}

// Whether workgroups of eight waves share the keys of 128 queries: where there is no
// more than one for a CU, and sequences are longer than 384 on average. Us with four waves and
// with eight, forward and whole gradient, one sequence: bf16, 32 heads of 128, 23 tokens 5.1
// and 6.1 (18.1, 19.1), 128 7.0 and 8.6 (30.6, 33.2), 256 9.6 and 10.8 (40.0, 41.6), 384 12.1 and
// 12.9 (46.5, 46.8), 512 14.7 and 15.3 (54.3, 53.2); 8 heads, 384 11.5 and 12.2 (42.3, 42.3), 900
// 21.1 and 20.3 (63.2, 58.2); fp16, 6 heads of 80, 256 8.7 and 9.0 (40.3, 39.6), 512 13.3 and 12.8
// (45.7, 42.7), 900 20.9 and 18.8 (61.5, 54.8).
inline bool two_sides(int64_t workgroups, int64_t tokens, int64_t sequences) {
  return workgroups <= CUS && tokens > 384 * sequences;
}

// Which head and tile a workgroup takes. Workgroups go to the eight XCDs in turn,
// each with an L2 of its own: heads that read the same keys and values go to one
// XCD, one behind the other, where the number of key heads allows it.
struct Work {
  int head, tile;
};
__device__ __forceinline__ Work work_of(unsigned block, int q_heads, int k_heads) {
  const unsigned group = q_heads / k_heads;
  if (k_heads % 8 == 0) {
    unsigned n = block / 8;
    const unsigned g = n % group;
    n /= group;
    const unsigned kh = block % 8 + 8 * (n % (k_heads / 8));
    return {static_cast<int>(kh * group + g), static_cast<int>(n / (k_heads / 8))};
  }
  return {static_cast<int>(block % q_heads), static_cast<int>(block / q_heads)};
}

}  // namespace nsmi
