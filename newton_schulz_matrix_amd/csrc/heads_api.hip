// C ABI of the operators on heads, (tokens, heads, dim) tensors: argument checks
// and launches. See include/ns.h for the contract. Every check runs on the host
// before any device work; nothing is allocated, copied or printed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/ns.h"
#include "heads_internal.h"
#include "train_checks.h"
#include "train_internal.h"

using namespace nsmi;

namespace nsmi {
namespace {

// A tensor of heads as the checks see it.
struct View {
  uintptr_t at;
  int64_t tokens, heads, dim, ld_token, ld_head;
  int64_t es;

  Span extent() const {
    if (!at || tokens < 1) return {at, at};
    return {at, at + ((tokens - 1) * ld_token + (heads - 1) * ld_head + dim) * es};
  }
  int64_t row() const { return ((heads - 1) * ld_head + dim) * es; }   // bytes of a token's heads
};
View view(const ns_heads& h, int64_t tokens, int64_t heads, int64_t dim, size_t es) {
  return {reinterpret_cast<uintptr_t>(h.data), tokens, heads, dim, h.ld_token, h.ld_head,
          static_cast<int64_t>(es)};
}
bool readable(const View& v) {
  return (v.at || v.tokens == 0) && v.at % v.es == 0 && v.ld_token >= 0 && v.ld_token <= MAX_LD &&
         v.ld_head >= 0 && v.ld_head <= MAX_LD;
}
bool writable(const View& v) {
  if (!readable(v)) return false;
  const bool by_token = (v.heads == 1 || v.ld_head >= v.dim) &&
                        (v.tokens <= 1 || v.ld_token >= (v.heads - 1) * v.ld_head + v.dim);
  const bool by_head = (v.tokens <= 1 || v.ld_token >= v.dim) &&
                       (v.heads == 1 || v.ld_head >= (v.tokens - 1) * v.ld_token + v.dim);
  return by_token || by_head;
}
bool same(const View& a, const View& b) {
  return a.at == b.at && (a.tokens <= 1 || a.ld_token == b.ld_token) &&
         (a.heads == 1 || a.ld_head == b.ld_head);
}
// Whether two tensors may share a byte. Parts of the same rows (queries and keys
// in one buffer) do not.
bool meet(const View& a, const View& b) {
  const Span x = a.extent(), y = b.extent();
  if (!overlap(x, y)) return false;
  const int64_t step = a.ld_token * a.es;
  if (a.tokens > 1 && b.tokens > 1 && step == b.ld_token * b.es && a.row() <= step && b.row() <= step) {
    const int64_t off = a.at < b.at ? static_cast<int64_t>((b.at - a.at) % step)
                                    : (step - static_cast<int64_t>((a.at - b.at) % step)) % step;
    return off < a.row() || off + b.row() > step;
  }
  return true;
}
bool meet(const View& a, const Span& b) { return overlap(a.extent(), b); }

Span dense(const void* p, int64_t n, size_t es) { return span(p, 1, n, n, es); }

bool qk_sizes_ok(int64_t tokens, int64_t dim) {
  return rows_ok(tokens) && dim >= 4 && dim <= QK_MAX_DIM && dim % 4 == 0;
}

// Checks what both calls share and fills the kernels' arguments.
ns_status check_qk(const ns_qk_norm_rope_args* p, bool reads_x, QkArgs* a) {
  if (!p || !type_ok(p->dtype) || !ids_ok(p->position_type)) return NS_ERR_INVALID_ARG;
  if (!qk_sizes_ok(p->tokens, p->dim) || p->q_heads < 1 || p->q_heads > NS_MAX_HEADS ||
      p->k_heads < 1 || p->k_heads > NS_MAX_HEADS)
    return NS_ERR_INVALID_ARG;
  if (p->rotary < 0 || p->rotary > p->dim || p->rotary % 4 != 0 || p->axes < 1 || p->axes > QK_AXES)
    return NS_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return NS_ERR_INVALID_ARG;
  if ((p->q_weight != nullptr) != (p->k_weight != nullptr)) return NS_ERR_INVALID_ARG;
  if (p->q_weight) {
    if (!type_ok(p->weight_dtype) || !same_or_f32(p->weight_dtype, p->dtype)) return NS_ERR_INVALID_ARG;
    const size_t we = type_bytes(p->weight_dtype);
    if (!aligned(p->q_weight, we) || !aligned(p->k_weight, we)) return NS_ERR_INVALID_ARG;
  }
  const int64_t pairs = p->rotary / 2;
  int64_t next = 0;
  for (int k = 0; k < QK_AXES; ++k) {
    a->first[k] = static_cast<int>(k < p->axes ? next : pairs);
    if (k >= p->axes || p->axes == 1) continue;
    if (p->sections[k] < 0 || p->sections[k] > pairs) return NS_ERR_INVALID_ARG;
    next += p->sections[k];
  }
  if (p->axes > 1 && next != pairs) return NS_ERR_INVALID_ARG;
  const size_t es = type_bytes(p->dtype);
  if (reads_x && (!readable(view(p->q, p->tokens, p->q_heads, p->dim, es)) ||
                  !readable(view(p->k, p->tokens, p->k_heads, p->dim, es))))
    return NS_ERR_INVALID_ARG;
  if (p->tokens > 0 && p->rotary > 0) {
    if (!p->positions || !p->inv_freq || !aligned(p->inv_freq, 4) ||
        !aligned(p->positions, id_bytes(p->position_type)))
      return NS_ERR_INVALID_ARG;
    if (p->axes > 1 && (p->ld_positions < 0 || p->ld_positions > MAX_LD)) return NS_ERR_INVALID_ARG;
  }
  a->part[0].x = p->q.data;
  a->part[0].x_token = p->q.ld_token;
  a->part[0].x_head = p->q.ld_head;
  a->part[0].heads = static_cast<int>(p->q_heads);
  a->part[0].weight = p->q_weight;
  a->part[1].x = p->k.data;
  a->part[1].x_token = p->k.ld_token;
  a->part[1].x_head = p->k.ld_head;
  a->part[1].heads = static_cast<int>(p->k_heads);
  a->part[1].weight = p->k_weight;
  a->positions = p->positions;
  a->inv_freq = p->inv_freq;
  a->ld_positions = p->axes > 1 ? p->ld_positions : 0;
  a->tokens = static_cast<int>(p->tokens);
  a->dim = static_cast<int>(p->dim);
  a->rotary = static_cast<int>(p->rotary);
  a->positions64 = p->position_type == NS_IDS_I64;
  a->interleaved = p->interleaved != 0;
  a->weight32 = p->weight_dtype == NS_DT_F32;
  a->eps = p->eps;
  return NS_OK;
}
// Whether a written range of bytes meets what both calls read beside the heads.
bool meets_inputs(const ns_qk_norm_rope_args& p, const Span& s) {
  const size_t we = type_bytes(p.weight_dtype), ie = id_bytes(p.position_type);
  const Span in[] = {dense(p.q_weight, p.dim, we), dense(p.k_weight, p.dim, we),
                     span(p.positions, p.axes, p.tokens, p.axes > 1 ? p.ld_positions : 0, ie),
                     dense(p.inv_freq, p.rotary / 2, 4)};
  for (const Span& i : in)
    if (overlap(s, i)) return true;
  return false;
}

}  // namespace
}  // namespace nsmi

// ------------------------------------- norm and rotation of queries and keys

NS_API ns_status ns_qk_norm_rope(const ns_qk_norm_rope_args* p, ns_heads q_out, ns_heads k_out,
                                 void* stream) {
  QkArgs a{};
  ns_status s = check_qk(p, true, &a);
  if (s != NS_OK) return s;
  if (p->tokens == 0) return NS_OK;
  const size_t es = type_bytes(p->dtype);
  const View q = view(p->q, p->tokens, p->q_heads, p->dim, es), k = view(p->k, p->tokens, p->k_heads, p->dim, es);
  const View qo = view(q_out, p->tokens, p->q_heads, p->dim, es), ko = view(k_out, p->tokens, p->k_heads, p->dim, es);
  if (!writable(qo) || !writable(ko)) return NS_ERR_INVALID_ARG;
  if ((!same(qo, q) && meet(qo, q)) || (!same(ko, k) && meet(ko, k)) || meet(qo, k) || meet(ko, q) ||
      meet(qo, ko) || meets_inputs(*p, qo.extent()) || meets_inputs(*p, ko.extent()))
    return NS_ERR_INVALID_ARG;
  s = device_status();
  if (s != NS_OK) return s;
  a.part[0].out = q_out.data;
  a.part[0].out_token = q_out.ld_token;
  a.part[0].out_head = q_out.ld_head;
  a.part[1].out = k_out.data;
  a.part[1].out_token = k_out.ld_token;
  a.part[1].out_head = k_out.ld_head;
  return from_hip(launch_qk_norm_rope(a, p->dtype, static_cast<hipStream_t>(stream)));
}

NS_API ns_status ns_qk_norm_rope_grad_workspace_size(int64_t tokens, int64_t dim, size_t* bytes) {
  if (!bytes || !qk_sizes_ok(tokens, dim)) return NS_ERR_INVALID_ARG;
  *bytes = std::max(ALIGN, align_up(sizeof(float) * 2 * dim * qk_grad_blocks(tokens, dim)));
  return NS_OK;
}

NS_API ns_status ns_qk_norm_rope_grad(const ns_qk_norm_rope_args* p, ns_heads dq_out, ns_heads dk_out,
                                      ns_heads dq, ns_heads dk, void* dq_weight, void* dk_weight,
                                      ns_dtype dweight_dtype, void* ws, size_t ws_bytes, void* stream) {
  QkArgs a{};
  const bool norm = p && p->q_weight;
  ns_status s = check_qk(p, norm, &a);
  if (s != NS_OK) return s;
  if (!norm && (dq_weight || dk_weight)) return NS_ERR_INVALID_ARG;
  const size_t es = type_bytes(p->dtype);
  if (norm) {
    if (!type_ok(dweight_dtype)) return NS_ERR_INVALID_ARG;
    const size_t de = type_bytes(dweight_dtype);
    if (!aligned(dq_weight, de) || !aligned(dk_weight, de)) return NS_ERR_INVALID_ARG;
  }
  const View gq = view(dq_out, p->tokens, p->q_heads, p->dim, es), gk = view(dk_out, p->tokens, p->k_heads, p->dim, es);
  const View oq = view(dq, p->tokens, p->q_heads, p->dim, es), ok = view(dk, p->tokens, p->k_heads, p->dim, es);
  if (!readable(gq) || !readable(gk) || !writable(oq) || !writable(ok)) return NS_ERR_INVALID_ARG;
  const View none = {0, 0, 0, 0, 0, 0, 1};
  const View q = norm ? view(p->q, p->tokens, p->q_heads, p->dim, es) : none;
  const View k = norm ? view(p->k, p->tokens, p->k_heads, p->dim, es) : none;
  size_t need = 0;
  if (norm) ns_qk_norm_rope_grad_workspace_size(p->tokens, p->dim, &need);
  if ((!same(oq, gq) && meet(oq, gq)) || (!same(ok, gk) && meet(ok, gk)) || meet(oq, gk) ||
      meet(ok, gq) || meet(oq, ok) || meet(oq, q) || meet(oq, k) || meet(ok, q) || meet(ok, k) ||
      meets_inputs(*p, oq.extent()) || meets_inputs(*p, ok.extent()))
    return NS_ERR_INVALID_ARG;
  if (norm) {
    const size_t de = type_bytes(dweight_dtype);
    const Span small[] = {dense(dq_weight, p->dim, de), dense(dk_weight, p->dim, de), dense(ws, need, 1)};
    for (int i = 0; i < 3; ++i) {
      if (meets_inputs(*p, small[i])) return NS_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (overlap(small[i], small[j])) return NS_ERR_INVALID_ARG;
      for (const View* v : {&gq, &gk, &oq, &ok, &q, &k})
        if (meet(*v, small[i])) return NS_ERR_INVALID_ARG;
    }
  }
  if (p->tokens == 0 && !dq_weight && !dk_weight) return NS_OK;
  if (norm && !workspace_ok(ws, ws_bytes, need)) return NS_ERR_WORKSPACE;
  s = device_status();
  if (s != NS_OK) return s;
  a.part[0].dy = dq_out.data;
  a.part[0].dy_token = dq_out.ld_token;
  a.part[0].dy_head = dq_out.ld_head;
  a.part[1].dy = dk_out.data;
  a.part[1].dy_token = dk_out.ld_token;
  a.part[1].dy_head = dk_out.ld_head;
  a.part[0].out = dq.data;
  a.part[0].out_token = dq.ld_token;
  a.part[0].out_head = dq.ld_head;
  a.part[1].out = dk.data;
  a.part[1].out_token = dk.ld_token;
  a.part[1].out_head = dk.ld_head;
  return from_hip(launch_qk_norm_rope_grad(a, p->dtype, static_cast<float*>(ws), dq_weight, dk_weight,
                                           dweight_dtype, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- attention

namespace nsmi {
namespace {

// 16-byte accesses, and offsets within a tile of rows that stay below 2^31 bytes.
constexpr int64_t ATTN_MAX_LD = int64_t{1} << 23;
bool vectors_ok(const View& v) {
  if (!readable(v) || v.at % 16 != 0 || (v.heads > 1 && v.ld_head % 8 != 0)) return false;
  return v.tokens <= 1 || (v.ld_token % 8 == 0 && v.ld_token >= v.dim && v.ld_token <= ATTN_MAX_LD);
}
HeadsAt place(const ns_heads& h, const View& v) {
  // one token: its stride is not used, whatever it is
  return {h.data, v.tokens <= 1 ? v.dim : v.ld_token, v.heads <= 1 ? 0 : v.ld_head};
}
bool attention_sizes_ok(int64_t tokens, int64_t sequences, int64_t q_heads, int64_t k_heads, int64_t dim) {
  if (!rows_ok(tokens) || !rows_ok(sequences) || q_heads < 1 || q_heads > NS_MAX_HEADS || k_heads < 1 ||
      k_heads > q_heads || q_heads % k_heads != 0 || dim < 8 || dim > ATTN_MAX_DIM || dim % 8 != 0)
    return false;
  // a launch's workgroups, of which each has 128 rows of a head at most
  return tokens == 0 || (tokens / 128 + sequences + 1) * q_heads <= NS_MAX_HEAD_TILES;
}
struct AttnViews {
  View q, k, v;
};
ns_status check_attention(const ns_attention_args* p, AttnArgs* a, AttnViews* in) {
  if (!p || (p->dtype != NS_DT_BF16 && p->dtype != NS_DT_F16)) return NS_ERR_INVALID_ARG;
  if (!attention_sizes_ok(p->tokens, p->sequences, p->q_heads, p->k_heads, p->dim)) return NS_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale) || p->scale <= 0.f) return NS_ERR_INVALID_ARG;
  if (p->tokens == 0) return NS_OK;
  in->q = view(p->q, p->tokens, p->q_heads, p->dim, 2);
  in->k = view(p->k, p->tokens, p->k_heads, p->dim, 2);
  in->v = view(p->v, p->tokens, p->k_heads, p->dim, 2);
  if (!vectors_ok(in->q) || !vectors_ok(in->k) || !vectors_ok(in->v)) return NS_ERR_INVALID_ARG;
  if (!p->offsets || !aligned(p->offsets, 4)) return NS_ERR_INVALID_ARG;
  a->q = place(p->q, in->q);
  a->k = place(p->k, in->k);
  a->v = place(p->v, in->v);
  a->offsets = p->offsets;
  a->tokens = static_cast<int>(p->tokens);
  a->sequences = static_cast<int>(p->sequences);
  a->q_heads = static_cast<int>(p->q_heads);
  a->k_heads = static_cast<int>(p->k_heads);
  a->dim = static_cast<int>(p->dim);
  a->clear_rest = p->clear_rest != 0;
  a->scale = p->scale;
  return NS_OK;
}
struct AttnPlan {
  int parts;
  size_t known, total;   // byte offset, bytes
};
AttnPlan attention_plan(int64_t tokens, int64_t sequences, int64_t q_heads, int64_t dim) {
  AttnPlan p;
  p.parts = attention_parts(tokens, sequences, q_heads, tokens, true);
  const size_t rows = p.parts > 1 ? static_cast<size_t>(p.parts) * tokens * q_heads : 0;
  p.known = align_up(sizeof(float) * rows * dim);
  p.total = p.known + align_up(sizeof(float2) * rows);
  return p;
}
struct AttnGradPlan {
  int q_parts, k_parts;
  size_t delta, reach, norms, sums, total;   // byte offsets, bytes
};
AttnGradPlan attention_grad_plan(int64_t tokens, int64_t sequences, int64_t q_heads, int64_t k_heads, int64_t dim) {
  AttnGradPlan p;
  const size_t rows = align_up(sizeof(float) * static_cast<size_t>(tokens) * q_heads);
  p.q_parts = attention_parts(tokens, sequences, q_heads, tokens, true);
  p.k_parts = attention_parts(tokens, sequences, k_heads, tokens * (q_heads / k_heads), false);
  p.delta = rows;
  p.reach = 2 * rows;
  p.norms = 3 * rows;
  p.sums = p.norms + align_up(sizeof(float) * static_cast<size_t>(tokens) * k_heads);
  const int64_t most = std::max(p.q_parts > 1 ? p.q_parts * q_heads : 0, p.k_parts > 1 ? 2 * p.k_parts * k_heads : 0);
  p.total = p.sums + align_up(sizeof(float) * static_cast<size_t>(most) * tokens * dim);
  return p;
}

}  // namespace
}  // namespace nsmi

NS_API ns_status ns_attention_workspace_size(int64_t tokens, int64_t sequences, int64_t q_heads, int64_t k_heads,
                                             int64_t dim, size_t* bytes) {
  if (!bytes || !attention_sizes_ok(tokens, sequences, q_heads, k_heads, dim)) return NS_ERR_INVALID_ARG;
  *bytes = attention_plan(tokens, sequences, q_heads, dim).total;
  return NS_OK;
}

NS_API ns_status ns_attention(const ns_attention_args* p, ns_heads out, float* lse, void* ws, size_t ws_bytes,
                              void* stream) {
  AttnArgs a{};
  AttnViews in;
  ns_status s = check_attention(p, &a, &in);
  if (s != NS_OK) return s;
  if (p->tokens == 0) return NS_OK;
  const View o = view(out, p->tokens, p->q_heads, p->dim, 2);
  if (!vectors_ok(o) || !writable(o) || !lse || !aligned(lse, 4)) return NS_ERR_INVALID_ARG;
  const AttnPlan plan = attention_plan(p->tokens, p->sequences, p->q_heads, p->dim);
  const Span l = dense(lse, p->tokens * p->q_heads, 4), ends = dense(p->offsets, p->sequences + 1, 4);
  const Span work = dense(ws, plan.total, 1);
  if (meet(o, l) || meet(o, ends) || overlap(l, ends) || meet(o, work) || overlap(l, work) || overlap(ends, work))
    return NS_ERR_INVALID_ARG;
  for (const View* v : {&in.q, &in.k, &in.v})
    if (meet(o, *v) || meet(*v, l) || meet(*v, work)) return NS_ERR_INVALID_ARG;
  if (plan.total > 0 && !workspace_ok(ws, ws_bytes, plan.total)) return NS_ERR_WORKSPACE;
  s = device_status();
  if (s != NS_OK) return s;
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.out = place(out, o);
  a.lse = lse;
  return from_hip(launch_attention(a, p->dtype, plan.parts, reinterpret_cast<float*>(w),
                                   reinterpret_cast<float2*>(w + plan.known), static_cast<hipStream_t>(stream)));
}

NS_API ns_status ns_attention_grad_workspace_size(int64_t tokens, int64_t sequences, int64_t q_heads,
                                                  int64_t k_heads, int64_t dim, size_t* bytes) {
  if (!bytes || !attention_sizes_ok(tokens, sequences, q_heads, k_heads, dim)) return NS_ERR_INVALID_ARG;
  *bytes = attention_grad_plan(tokens, sequences, q_heads, k_heads, dim).total;
  return NS_OK;
}

NS_API ns_status ns_attention_grad(const ns_attention_args* p, ns_heads dout, ns_heads out,
                                   const float* lse, ns_heads dq, ns_heads dk, ns_heads dv, void* ws,
                                   size_t ws_bytes, void* stream) {
  AttnArgs a{};
  AttnViews in;
  ns_status s = check_attention(p, &a, &in);
  if (s != NS_OK) return s;
  if (p->tokens == 0) return NS_OK;
  View g = view(dout, p->tokens, p->q_heads, p->dim, 2), o = view(out, p->tokens, p->q_heads, p->dim, 2);
  const View written[] = {view(dq, p->tokens, p->q_heads, p->dim, 2),
                          view(dk, p->tokens, p->k_heads, p->dim, 2),
                          view(dv, p->tokens, p->k_heads, p->dim, 2)};
  if (!vectors_ok(g) || !vectors_ok(o) || !lse || !aligned(lse, 4)) return NS_ERR_INVALID_ARG;
  const AttnGradPlan plan = attention_grad_plan(p->tokens, p->sequences, p->q_heads, p->k_heads, p->dim);
  const Span l = dense(lse, p->tokens * p->q_heads, 4), ends = dense(p->offsets, p->sequences + 1, 4);
  const Span work = dense(ws, plan.total, 1);
  for (int i = 0; i < 3; ++i) {
    const View& x = written[i];
    if (!vectors_ok(x) || !writable(x) || meet(x, l) || meet(x, ends) || meet(x, work))
      return NS_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(x, written[j])) return NS_ERR_INVALID_ARG;
    for (const View* v : {&in.q, &in.k, &in.v, &g, &o})
      if (meet(x, *v)) return NS_ERR_INVALID_ARG;
  }
  if (overlap(work, l) || overlap(work, ends)) return NS_ERR_INVALID_ARG;
  for (const View* v : {&in.q, &in.k, &in.v, &g, &o})
    if (meet(*v, work)) return NS_ERR_INVALID_ARG;
  if (!workspace_ok(ws, ws_bytes, plan.total)) return NS_ERR_WORKSPACE;
  s = device_status();
  if (s != NS_OK) return s;
  unsigned char* w = static_cast<unsigned char*>(ws);
  a.out = place(out, o);
  a.dout = place(dout, g);
  a.dq = place(dq, written[0]);
  a.dk = place(dk, written[1]);
  a.dv = place(dv, written[2]);
  a.lse = const_cast<float*>(lse);
  a.lse2 = reinterpret_cast<float*>(w);
  a.delta = reinterpret_cast<float*>(w + plan.delta);
  a.reach = reinterpret_cast<float*>(w + plan.reach);
  a.v_norms = reinterpret_cast<float*>(w + plan.norms);
  return from_hip(launch_attention_grad(a, p->dtype, plan.q_parts, plan.k_parts,
                                        reinterpret_cast<float*>(w + plan.sums),
                                        static_cast<hipStream_t>(stream)));
}
