// Launch interfaces of the operators around the matrix update (train_*.hip),
// shared by their C ABI (train_api.hip) and their kernels. Not part of the
// C ABI. Element types are OutType codes; E4M3 is accepted where said.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ns.h"
#include "ns_internal.h"

namespace nsmi {

// NS_OK where the current device is a gfx950 (defined in ns_api.hip).
ns_status device_status() noexcept;

constexpr int OUT_E4M3 = 3;

// ----------------------------------------------------------- embedding

struct EmbedArgs {
  const void* table;
  const void* ids;
  void* out;
  int64_t ld_table, ld_out;
  int64_t rows;
  int count, dim;
  float scale;
};
hipError_t launch_embedding(const EmbedArgs& a, int table_type, bool ids64, int out_type,
                            hipStream_t stream);

// Sorted ids of one gradient call, in the workspace:
//   sorted[k]   position and id of the k-th place in sorted order; the places
//               of ids that do not count come last, with id -1 (count pairs);
//   start[p]    first k of table row v, with p = sorted_slot(v); the row's
//               places end at start[p + 1] (slots + 1 ints).
// Rows are dealt to `groups` sorting workgroups by their low bits, `range`
// consecutive slots to a workgroup, so that the most frequent ids (small ones,
// in most vocabularies) do not meet in one workgroup.
struct EmbedSort {
  int groups_log2;     // groups = 1 << groups_log2
  int range;           // slots of a group
  int slots;           // groups * range >= rows
  int window;          // places of one window (a multiple of 8)
  int windows;
};
__host__ __device__ inline int sorted_slot(int v, const EmbedSort& s) {
  return (v & ((1 << s.groups_log2) - 1)) * s.range + (v >> s.groups_log2);
}
EmbedSort embed_sort_plan(int64_t rows, int64_t count);

struct EmbedGradArgs {
  const void* grad_out;
  const void* ids;
  void* grad;
  int2* sorted;
  int* start;
  float* partial;      // (2 windows, dim)
  int64_t ld_grad_out, ld_grad;
  int64_t padding_id;
  int rows, count, dim;
  int accumulate;
  float scale;
  EmbedSort sort;
};
hipError_t launch_embedding_grad(const EmbedGradArgs& a, int grad_out_type, bool ids64,
                                 int grad_type, hipStream_t stream);

// ------------------------------------------------------------ RMS norm

struct RmsArgs {
  const void* x;
  const void* residual;
  void* h;
  const void* weight;
  void* y;
  float* scales;
  float* rstd;
  int64_t ldx, ld_residual, ldh, ldy;
  int rows, dim;
  float eps;
  bool stream;         // set by the launch: a 16-bit y, or h beside codes, is stored past the caches
};
// x_type, h_type (x_type or fp32), weight_type (x_type or fp32), y_type (any, or OUT_E4M3)
hipError_t launch_rms_norm(RmsArgs a, int x_type, int h_type, int weight_type, int y_type,
                           hipStream_t stream);

struct RmsGradArgs {
  const void* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dh;
  void* dx;
  void* dweight;
  float* partial;      // (blocks, dim): each workgroup's share of dweight
  int64_t lddy, ldh, lddh, lddx;
  int rows, dim;
  int blocks;
};
int rms_grad_blocks(int64_t rows, int64_t dim);
// dy_type, h_type (dy_type or fp32), weight_type (dy_type or fp32),
// dx_type (dy_type or fp32), dweight_type any
hipError_t launch_rms_norm_grad(const RmsGradArgs& a, int dy_type, int h_type, int weight_type,
                                int dx_type, int dweight_type, hipStream_t stream);

// ----------------------------------------------------- preference loss

struct PrefArgs {
  const void* logits;
  const void* labels;
  int64_t ld, ld_seq;  // from one position, one sequence to the next
  int pairs, length, vocab;
  float beta, smoothing;
};
// Pieces one row is cut into, and the length of each (the last is shorter).
struct PrefSplit {
  int pieces;
  int piece;
};
PrefSplit pref_split(int64_t rows, int64_t vocab);
hipError_t launch_preference_loss(const PrefArgs& a, int type, bool labels64, const PrefSplit& sp,
                                  double2* parts, const float* ref_logps, float* losses,
                                  float* margins, float* logps, float* lse, hipStream_t stream);
hipError_t launch_preference_grad(const PrefArgs& a, int type, bool labels64,
                                  const float* margins, const float* lse, const float* dlosses,
                                  void* dlogits, int64_t ld_dlogits, int64_t ld_dseq,
                                  hipStream_t stream);

// ------------------------------------------------- token log probabilities

constexpr int LOGPS_MAX_TOP = NS_MAX_TOP;
constexpr int LOGPS_JOIN = 1024;      // entries of a row's pieces, all together, where they are asked for
struct LogpsArgs {
  const void* logits;
  const void* tokens;
  int64_t ld, ld_seq;  // from one row of a sequence, one sequence to the next
  int rows, length, vocab, top;
  bool tokens64;
};
struct LogpsOut {
  float* logps;
  float* lse;
  float* entropy;
  float* top_logps;    // (rows, top)
  void* top_ids;       // (rows, top), of the tokens' type
};
// Maximum and sums of a piece of a row.
struct LogpsPart {
  double m, s, t;
};
PrefSplit logps_split(int64_t rows, int64_t vocab, int top);
// entries: (rows, pieces, top)
hipError_t launch_token_logps(const LogpsArgs& a, int type, const PrefSplit& sp, LogpsPart* parts,
                              uint64_t* entries, const LogpsOut& o, hipStream_t stream);
hipError_t launch_token_logps_grad(const LogpsArgs& a, int type, const float* lse, const float* entropy,
                                   const float* dlogps, const float* dentropy, void* dlogits,
                                   int64_t ld_dlogits, int64_t ld_dseq, hipStream_t stream);

// -------------------------------------------------------------- AdamW

constexpr int ADAMW_TENSORS = 32;     // tensors of one launch (its table is a kernel argument)
struct AdamwTensor {
  void* param;
  const void* grad;
  void* exp_avg;
  void* exp_avg_sq;
  float* master;
  int64_t elems;
  int param_type, grad_type, exp_avg_type, exp_avg_sq_type;
  float decay;         // lr * weight_decay
};
struct AdamwArgs {
  AdamwTensor t[ADAMW_TENSORS];
  unsigned begin[ADAMW_TENSORS];      // first workgroup of each tensor
  int count;
  float beta1, rest1, beta2, rest2;   // rest = 1 - beta, from 64 bits
  float step_size;                    // lr / (1 - beta1^step)
  float root_scale;                   // 1 / sqrt(1 - beta2^step)
  float eps;
};
unsigned adamw_blocks(int64_t elems);
hipError_t launch_adamw(const AdamwArgs& a, unsigned blocks, hipStream_t stream);

}  // namespace nsmi
