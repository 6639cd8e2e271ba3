// Launch interfaces of the operators on heads, (tokens, heads, dim) tensors:
// norm of queries and keys with their rotation (train_qk_norm.hip) and
// attention (train_attention.hip, train_attention_grad.hip), shared by their
// C ABI (heads_api.hip) and their kernels. Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ns.h"

namespace nsmi {

// ------------------------------------- norm and rotation of queries and keys

constexpr int QK_MAX_DIM = 256;
constexpr int QK_AXES = 4;

// The queries' or the keys' part of a call.
struct QkPart {
  const void* x;
  const void* dy;      // gradient only
  void* out;           // y, or dx
  const void* weight;  // NULL: no norm
  int64_t x_token, x_head, dy_token, dy_head, out_token, out_head;
  int heads;
};
struct QkArgs {
  QkPart part[2];      // queries, keys
  const void* positions;       // (axes, tokens)
  const float* inv_freq;
  int64_t ld_positions;
  int first[QK_AXES];  // first pair that turns with each axis (pairs, where there is no such axis)
  int tokens, dim, rotary;
  bool positions64, interleaved, weight32;
  float eps;
};
hipError_t launch_qk_norm_rope(const QkArgs& a, int type, hipStream_t stream);
// partial: (blocks, 2, dim), each workgroup's share of the weights' gradients
int qk_grad_blocks(int64_t tokens, int64_t dim);
hipError_t launch_qk_norm_rope_grad(const QkArgs& a, int type, float* partial, void* dq_weight,
                                    void* dk_weight, int dweight_type, hipStream_t stream);

// -------------------------------------------------------------- attention

constexpr int ATTN_MAX_DIM = 128;

// A (tokens, heads, dim) tensor.
struct HeadsAt {
  void* p;
  int64_t token, head;
};
struct AttnArgs {
  HeadsAt q, k, v, out;
  HeadsAt dout, dq, dk, dv;    // gradient only
  float* lse;                  // (q_heads, tokens)
  float* lse2;                 // -lse log2(e) (fp16: + 14), gradient only
  float* delta;                // -delta, (q_heads, tokens), gradient only
  float* reach;                // what a row's dS may reach, (q_heads, tokens), gradient of fp16 only
  float* v_norms;              // (k_heads, tokens), gradient of fp16 only
  const int* offsets;          // (sequences + 1)
  int tokens, sequences, q_heads, k_heads, dim;
  bool clear_rest;
  float scale;
};
// Into how many parts the keys of a tile of queries (or the queries of a tile of keys)
// are cut, each a workgroup's: where the tiles alone would leave CUs without work, or
// with one long sequence's ends. From two parts on their sums go through memory:
//   forward  sums (parts, q_heads, tokens, dim) fp32 and known (parts, q_heads, tokens),
//            each row's reference and sum of weights;
//   dq       sums (parts, q_heads, tokens, dim);
//   dk, dv   sums (parts, 2, k_heads, tokens, dim).
// rows: those of all heads that one workgroup goes over at most; keys: whether they are keys.
int attention_parts(int64_t tokens, int64_t sequences, int64_t heads, int64_t rows, bool keys);
hipError_t launch_attention(const AttnArgs& a, int type, int parts, float* sums, float2* known, hipStream_t stream);

hipError_t launch_attention_grad(const AttnArgs& a, int type, int q_parts, int k_parts, float* sums,
                                 hipStream_t stream);

}  // namespace nsmi
