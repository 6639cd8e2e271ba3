// C ABI of the operators around the matrix update: argument checks and
// launches. See include/ns.h for the contract. Every check runs on the host
// before any device work; nothing is allocated, copied or printed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/ns.h"
#include "train_internal.h"

#define NS_API extern "C" __attribute__((visibility("default")))

namespace nsmi {
namespace {

constexpr size_t ALIGN = 256;
size_t align_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }

bool type_ok(int t) { return t == NS_DT_F32 || t == NS_DT_BF16 || t == NS_DT_F16; }
size_t type_bytes(int t) { return t == NS_DT_E4M3 ? 1 : t == NS_DT_F32 ? 4 : 2; }
bool ids_ok(int t) { return t == NS_IDS_I32 || t == NS_IDS_I64; }
size_t id_bytes(int t) { return t == NS_IDS_I64 ? 8 : 4; }

// Types that go with `type`: itself or fp32.
bool same_or_f32(int t, int type) { return t == type || t == NS_DT_F32; }

// A device buffer: (rows, cols) elements of `es` bytes, leading dimension ld.
struct Span {
  uintptr_t first, last;
};
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (!p || rows < 1 || cols < 1) return {a, a};
  return {a, a + (static_cast<uintptr_t>(rows - 1) * ld + cols) * es};
}
bool overlap(Span x, Span y) { return x.first < y.last && y.first < x.last; }

// Whether any of the written ranges meets a read one or another written one.
template <int W, int R>
bool clash(const Span (&out)[W], const Span (&in)[R]) {
  for (int i = 0; i < W; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
    for (int j = 0; j < R; ++j)
      if (overlap(out[i], in[j])) return true;
  }
  return false;
}

bool aligned(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es == 0; }
bool rows_ok(int64_t r) { return r >= 0 && r <= NS_MAX_ROWS; }
bool dim_ok(int64_t d) { return d >= 1 && d <= NS_MAX_DIM; }
// Leading dimensions up to this keep every byte offset of a call in 63 bits.
constexpr int64_t MAX_LD = int64_t{1} << 36;
bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= MAX_LD; }

ns_status from_hip(hipError_t e) { return e == hipSuccess ? NS_OK : NS_ERR_HIP; }

// Workspace given, large enough and aligned.
bool workspace_ok(const void* ws, size_t have, size_t need) {
  return ws && have >= need && reinterpret_cast<uintptr_t>(ws) % ALIGN == 0;
}

}  // namespace
}  // namespace nsmi

using namespace nsmi;

// ---------------------------------------------------------------- embedding

NS_API ns_status ns_embedding(const void* table, ns_dtype table_dtype, int64_t rows, int64_t dim,
                              int64_t ld_table, const void* ids, ns_id_type id_type,
                              int64_t count, float scale, void* out, ns_dtype out_dtype,
                              int64_t ld_out, void* stream) {
  if (!type_ok(table_dtype) || !type_ok(out_dtype) || !ids_ok(id_type)) return NS_ERR_INVALID_ARG;
  if (!rows_ok(rows) || rows < 1 || !rows_ok(count) || !dim_ok(dim)) return NS_ERR_INVALID_ARG;
  if (!ld_ok(ld_table, dim) || !ld_ok(ld_out, dim) || !std::isfinite(scale))
    return NS_ERR_INVALID_ARG;
  if (count == 0) return NS_OK;
  const size_t te = type_bytes(table_dtype), oe = type_bytes(out_dtype), ie = id_bytes(id_type);
  if (!table || !ids || !out || !aligned(table, te) || !aligned(ids, ie) || !aligned(out, oe))
    return NS_ERR_INVALID_ARG;
  const Span writes[] = {span(out, count, dim, ld_out, oe)};
  const Span reads[] = {span(table, rows, dim, ld_table, te), span(ids, 1, count, count, ie)};
  if (clash(writes, reads)) return NS_ERR_INVALID_ARG;
  const ns_status s = device_status();
  if (s != NS_OK) return s;
  EmbedArgs a{};
  a.table = table;
  a.ids = ids;
  a.out = out;
  a.ld_table = ld_table;
  a.ld_out = ld_out;
  a.rows = rows;
  a.count = static_cast<int>(count);
  a.dim = static_cast<int>(dim);
  a.scale = scale;
  return from_hip(launch_embedding(a, table_dtype, id_type == NS_IDS_I64, out_dtype,
                                   static_cast<hipStream_t>(stream)));
}

namespace nsmi {
namespace {
struct EmbedGradPlan {
  EmbedSort sort;
  size_t sorted, start, partial, total;   // byte offsets, bytes
};
EmbedGradPlan embed_grad_plan(int64_t rows, int64_t dim, int64_t count) {
  EmbedGradPlan p;
  p.sort = embed_sort_plan(rows, count);
  p.sorted = 0;
  p.start = align_up(sizeof(int2) * static_cast<size_t>(count));
  p.partial = align_up(p.start + sizeof(int) * (static_cast<size_t>(p.sort.slots) + 1));
  p.total = align_up(p.partial + sizeof(float) * 2 * static_cast<size_t>(p.sort.windows) * dim);
  return p;
}
}  // namespace
}  // namespace nsmi

NS_API ns_status ns_embedding_grad_workspace_size(int64_t rows, int64_t dim, int64_t count,
                                                  size_t* bytes) {
  if (!bytes || !rows_ok(rows) || rows < 1 || !rows_ok(count) || !dim_ok(dim))
    return NS_ERR_INVALID_ARG;
  *bytes = embed_grad_plan(rows, dim, count).total;
  return NS_OK;
}

NS_API ns_status ns_embedding_grad(const void* grad_out, ns_dtype grad_out_dtype,
                                   int64_t ld_grad_out, const void* ids, ns_id_type id_type,
                                   int64_t count, int64_t rows, int64_t dim, float scale,
                                   int64_t padding_id, int accumulate, void* grad,
                                   ns_dtype grad_dtype, int64_t ld_grad, void* ws,
                                   size_t ws_bytes, void* stream) {
  if (!type_ok(grad_out_dtype) || !type_ok(grad_dtype) || !ids_ok(id_type))
    return NS_ERR_INVALID_ARG;
  if (!rows_ok(rows) || rows < 1 || !rows_ok(count) || !dim_ok(dim)) return NS_ERR_INVALID_ARG;
  if (!ld_ok(ld_grad_out, dim) || !ld_ok(ld_grad, dim) || !std::isfinite(scale))
    return NS_ERR_INVALID_ARG;
  const size_t ge = type_bytes(grad_out_dtype), te = type_bytes(grad_dtype), ie = id_bytes(id_type);
  if (!grad || !aligned(grad, te)) return NS_ERR_INVALID_ARG;
  if (count > 0 && (!grad_out || !ids || !aligned(grad_out, ge) || !aligned(ids, ie)))
    return NS_ERR_INVALID_ARG;
  const EmbedGradPlan p = embed_grad_plan(rows, dim, count);
  const Span writes[] = {span(grad, rows, dim, ld_grad, te), span(ws, 1, p.total, p.total, 1)};
  const Span reads[] = {span(grad_out, count, dim, ld_grad_out, ge), span(ids, 1, count, count, ie)};
  if (clash(writes, reads)) return NS_ERR_INVALID_ARG;
  if (count == 0 && accumulate) return NS_OK;
  if (!workspace_ok(ws, ws_bytes, p.total)) return NS_ERR_WORKSPACE;
  const ns_status s = device_status();
  if (s != NS_OK) return s;
  unsigned char* w = static_cast<unsigned char*>(ws);
  EmbedGradArgs a{};
  a.grad_out = grad_out;
  a.ids = ids;
  a.grad = grad;
  a.sorted = reinterpret_cast<int2*>(w + p.sorted);
  a.start = reinterpret_cast<int*>(w + p.start);
  a.partial = reinterpret_cast<float*>(w + p.partial);
  a.ld_grad_out = ld_grad_out;
  a.ld_grad = ld_grad;
  a.padding_id = padding_id;
  a.rows = static_cast<int>(rows);
  a.count = static_cast<int>(count);
  a.dim = static_cast<int>(dim);
  a.accumulate = accumulate != 0;
  a.scale = scale;
  a.sort = p.sort;
  return from_hip(launch_embedding_grad(a, grad_out_dtype, id_type == NS_IDS_I64, grad_dtype,
                                        static_cast<hipStream_t>(stream)));
}

// ----------------------------------------------------------------- RMS norm

NS_API ns_status ns_rms_norm(const ns_rms_norm_args* p, void* stream) {
  if (!p) return NS_ERR_INVALID_ARG;
  if (!type_ok(p->x_dtype) || !same_or_f32(p->h_dtype, p->x_dtype) ||
      !same_or_f32(p->weight_dtype, p->x_dtype))
    return NS_ERR_INVALID_ARG;
  const bool coded = p->y_dtype == NS_DT_E4M3;
  if (!coded && !type_ok(p->y_dtype)) return NS_ERR_INVALID_ARG;
  if (!rows_ok(p->rows) || !dim_ok(p->dim) || !std::isfinite(p->eps) || p->eps < 0.f)
    return NS_ERR_INVALID_ARG;
  if (!ld_ok(p->ldx, p->dim) || !ld_ok(p->ldy, p->dim)) return NS_ERR_INVALID_ARG;
  if (p->rows == 0) return NS_OK;   // empty tensors may have no address
  const bool res = p->residual != nullptr;
  if (res != (p->h != nullptr) || (!res && p->h_dtype != p->x_dtype)) return NS_ERR_INVALID_ARG;
  if (res && (!ld_ok(p->ld_residual, p->dim) || !ld_ok(p->ldh, p->dim))) return NS_ERR_INVALID_ARG;
  const size_t xe = type_bytes(p->x_dtype), he = type_bytes(p->h_dtype);
  const size_t we = type_bytes(p->weight_dtype), ye = type_bytes(p->y_dtype);
  if (!p->x || !p->weight || !p->y || coded != (p->scales != nullptr)) return NS_ERR_INVALID_ARG;
  if (!aligned(p->x, xe) || !aligned(p->weight, we) || !aligned(p->y, ye) ||
      !aligned(p->residual, he) || !aligned(p->h, he) || !aligned(p->scales, 4) ||
      !aligned(p->rstd, 4))
    return NS_ERR_INVALID_ARG;
  // h in the place of the residual, or of x: each element is read and written by one thread
  const bool on_residual = res && p->h == p->residual && p->ldh == p->ld_residual;
  const bool on_x = res && p->h == p->x && p->ldh == p->ldx && p->h_dtype == p->x_dtype;
  const Span none = {0, 0};
  const Span x = span(p->x, p->rows, p->dim, p->ldx, xe);
  const Span r = span(p->residual, p->rows, p->dim, p->ld_residual, he);
  const Span h = span(p->h, p->rows, p->dim, p->ldh, he);
  const Span writes[] = {span(p->y, p->rows, p->dim, p->ldy, ye),
                         span(p->scales, 1, p->rows, p->rows, 4),
                         span(p->rstd, 1, p->rows, p->rows, 4)};
  const Span reads[] = {x, r, h, span(p->weight, 1, p->dim, p->dim, we)};
  if (clash(writes, reads)) return NS_ERR_INVALID_ARG;
  const Span h_writes[] = {h};
  const Span h_reads[] = {on_x ? none : x, on_residual ? none : r, reads[3]};
  if (clash(h_writes, h_reads)) return NS_ERR_INVALID_ARG;
  const ns_status s = device_status();
  if (s != NS_OK) return s;
  RmsArgs a{};
  a.x = p->x;
  a.residual = p->residual;
  a.h = p->h;
  a.weight = p->weight;
  a.y = p->y;
  a.scales = p->scales;
  a.rstd = p->rstd;
  a.ldx = p->ldx;
  a.ld_residual = p->ld_residual;
  a.ldh = p->ldh;
  a.ldy = p->ldy;
  a.rows = static_cast<int>(p->rows);
  a.dim = static_cast<int>(p->dim);
  a.eps = p->eps;
  return from_hip(launch_rms_norm(a, p->x_dtype, p->h_dtype, p->weight_dtype, p->y_dtype,
                                  static_cast<hipStream_t>(stream)));
}

NS_API ns_status ns_rms_norm_grad_workspace_size(int64_t rows, int64_t dim, size_t* bytes) {
  if (!bytes || !rows_ok(rows) || !dim_ok(dim)) return NS_ERR_INVALID_ARG;
  *bytes = std::max(ALIGN, align_up(sizeof(float) * static_cast<size_t>(rms_grad_blocks(rows, dim)) * dim));
  return NS_OK;
}

NS_API ns_status ns_rms_norm_grad(const ns_rms_norm_grad_args* p, void* ws, size_t ws_bytes,
                                  void* stream) {
  if (!p) return NS_ERR_INVALID_ARG;
  if (!type_ok(p->dy_dtype) || !same_or_f32(p->h_dtype, p->dy_dtype) ||
      !same_or_f32(p->weight_dtype, p->dy_dtype) || !same_or_f32(p->dx_dtype, p->dy_dtype) ||
      !type_ok(p->dweight_dtype))
    return NS_ERR_INVALID_ARG;
  if (!rows_ok(p->rows) || !dim_ok(p->dim)) return NS_ERR_INVALID_ARG;
  if (!ld_ok(p->lddy, p->dim) || !ld_ok(p->ldh, p->dim) || !ld_ok(p->lddx, p->dim) ||
      (p->dh && !ld_ok(p->lddh, p->dim)))
    return NS_ERR_INVALID_ARG;
  const size_t ye = type_bytes(p->dy_dtype), he = type_bytes(p->h_dtype);
  const size_t we = type_bytes(p->weight_dtype), xe = type_bytes(p->dx_dtype);
  const size_t de = type_bytes(p->dweight_dtype);
  if (p->rows > 0) {
    if (!p->dy || !p->h || !p->weight || !p->rstd || !p->dx) return NS_ERR_INVALID_ARG;
    if (!aligned(p->dy, ye) || !aligned(p->h, he) || !aligned(p->weight, we) ||
        !aligned(p->rstd, 4) || !aligned(p->dh, xe) || !aligned(p->dx, xe))
      return NS_ERR_INVALID_ARG;
  }
  if (!aligned(p->dweight, de)) return NS_ERR_INVALID_ARG;
  size_t need = 0;
  ns_rms_norm_grad_workspace_size(p->rows, p->dim, &need);
  const bool in_place = p->dh && p->dx == p->dh && p->lddx == p->lddh;
  const Span none = {0, 0};
  const Span writes[] = {span(p->dx, p->rows, p->dim, p->lddx, xe),
                         span(p->dweight, 1, p->dim, p->dim, de), span(ws, 1, need, need, 1)};
  const Span dh = span(p->dh, p->rows, p->dim, p->lddh, xe);
  const Span reads[] = {span(p->dy, p->rows, p->dim, p->lddy, ye),
                        span(p->h, p->rows, p->dim, p->ldh, he),
                        span(p->weight, 1, p->dim, p->dim, we),
                        span(p->rstd, 1, p->rows, p->rows, 4), in_place ? none : dh};
  if (clash(writes, reads)) return NS_ERR_INVALID_ARG;
  if (p->rows == 0 && !p->dweight) return NS_OK;
  if (!workspace_ok(ws, ws_bytes, need)) return NS_ERR_WORKSPACE;
  const ns_status s = device_status();
  if (s != NS_OK) return s;
  RmsGradArgs a{};
  a.dy = p->dy;
  a.h = p->h;
  a.weight = p->weight;
  a.rstd = p->rstd;
  a.dh = p->dh;
  a.dx = p->dx;
  a.dweight = p->dweight;
  a.partial = static_cast<float*>(ws);
  a.lddy = p->lddy;
  a.ldh = p->ldh;
  a.lddh = p->lddh;
  a.lddx = p->lddx;
  a.rows = static_cast<int>(p->rows);
  a.dim = static_cast<int>(p->dim);
  a.blocks = rms_grad_blocks(p->rows, p->dim);
  return from_hip(launch_rms_norm_grad(a, p->dy_dtype, p->h_dtype, p->weight_dtype, p->dx_dtype,
                                       p->dweight_dtype, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------- preference loss

namespace nsmi {
namespace {
bool pref_sizes_ok(int64_t pairs, int64_t length, int64_t vocab) {
  if (!rows_ok(pairs) || !rows_ok(length) || !rows_ok(vocab) || vocab < 1) return false;
  return rows_ok(2 * pairs) && rows_ok(2 * pairs * length);
}
size_t pref_workspace(int64_t pairs, int64_t length, int64_t vocab) {
  const int64_t rows = 2 * pairs * length;
  return std::max(ALIGN, align_up(sizeof(double2) * static_cast<size_t>(rows) *
                                  pref_split(rows, vocab).pieces));
}
// Sequences' bytes stay within 62 bits.
constexpr int64_t MAX_SEQUENCE = int64_t{1} << 60;
int64_t sequence_ld(const ns_preference_args& p) {
  return p.ld_sequence != 0 ? p.ld_sequence : p.length * p.ld;
}
// The logits' buffer (not empty).
Span logits_span(const ns_preference_args& p) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p.logits);
  if (p.pairs < 1 || p.length < 1) return {a, a};
  const int64_t last = (2 * p.pairs - 1) * sequence_ld(p) + (p.length - 1) * p.ld + p.vocab;
  return {a, a + static_cast<uintptr_t>(last) * type_bytes(p.dtype)};
}
ns_status check_pref(const ns_preference_args* p) {
  if (!p || !type_ok(p->dtype) || !ids_ok(p->label_type)) return NS_ERR_INVALID_ARG;
  if (!pref_sizes_ok(p->pairs, p->length, p->vocab) || !ld_ok(p->ld, p->vocab))
    return NS_ERR_INVALID_ARG;
  const int64_t seqs = 2 * p->pairs, seq = sequence_ld(*p);
  if (p->length > 0 && seqs > 1 &&
      (seq < (p->length - 1) * p->ld + p->vocab || seq > MAX_SEQUENCE / seqs))
    return NS_ERR_INVALID_ARG;
  if (!std::isfinite(p->beta) || !(p->label_smoothing >= 0.f && p->label_smoothing <= 1.f))
    return NS_ERR_INVALID_ARG;
  if (p->pairs > 0 && p->length > 0 &&
      (!p->logits || !p->labels || !aligned(p->logits, type_bytes(p->dtype)) ||
       !aligned(p->labels, id_bytes(p->label_type))))
    return NS_ERR_INVALID_ARG;
  return NS_OK;
}
PrefArgs pref_args(const ns_preference_args& p) {
  PrefArgs a{};
  a.logits = p.logits;
  a.labels = p.labels;
  a.ld = p.ld;
  a.ld_seq = sequence_ld(p);
  a.pairs = static_cast<int>(p.pairs);
  a.length = static_cast<int>(p.length);
  a.vocab = static_cast<int>(p.vocab);
  a.beta = p.beta;
  a.smoothing = p.label_smoothing;
  return a;
}
Span floats(const void* p, int64_t n) { return span(p, 1, n, n, 4); }
}  // namespace
}  // namespace nsmi

NS_API ns_status ns_preference_loss_workspace_size(int64_t pairs, int64_t length, int64_t vocab,
                                                   size_t* bytes) {
  if (!bytes || !pref_sizes_ok(pairs, length, vocab)) return NS_ERR_INVALID_ARG;
  *bytes = pref_workspace(pairs, length, vocab);
  return NS_OK;
}

NS_API ns_status ns_preference_loss(const ns_preference_args* p, const float* ref_logps,
                                    float* losses, float* margins, float* logps, float* lse,
                                    void* ws, size_t ws_bytes, void* stream) {
  ns_status s = check_pref(p);
  if (s != NS_OK) return s;
  if (p->pairs == 0) return NS_OK;
  if (!ref_logps || !losses || !margins || !logps || (p->length > 0 && !lse))
    return NS_ERR_INVALID_ARG;
  if (!aligned(ref_logps, 4) || !aligned(losses, 4) || !aligned(margins, 4) ||
      !aligned(logps, 4) || !aligned(lse, 4))
    return NS_ERR_INVALID_ARG;
  const int64_t rows = 2 * p->pairs * p->length;
  const size_t need = pref_workspace(p->pairs, p->length, p->vocab);
  const Span writes[] = {floats(losses, p->pairs), floats(margins, p->pairs),
                         floats(logps, 2 * p->pairs), floats(lse, rows),
                         span(ws, 1, need, need, 1)};
  const Span reads[] = {logits_span(*p),
                        span(p->labels, 1, rows, rows, id_bytes(p->label_type)),
                        floats(ref_logps, 2 * p->pairs)};
  if (clash(writes, reads)) return NS_ERR_INVALID_ARG;
  if (!workspace_ok(ws, ws_bytes, need)) return NS_ERR_WORKSPACE;
  s = device_status();
  if (s != NS_OK) return s;
  return from_hip(launch_preference_loss(pref_args(*p), p->dtype, p->label_type == NS_IDS_I64,
                                         pref_split(rows, p->vocab), static_cast<double2*>(ws),
                                         ref_logps, losses, margins, logps, lse,
                                         static_cast<hipStream_t>(stream)));
}

NS_API ns_status ns_preference_loss_grad(const ns_preference_args* p, const float* margins,
                                         const float* lse, const float* dlosses, void* dlogits,
                                         int64_t ld_dlogits, void* stream) {
  ns_status s = check_pref(p);
  if (s != NS_OK) return s;
  if (!ld_ok(ld_dlogits, p->vocab)) return NS_ERR_INVALID_ARG;
  if (p->pairs == 0 || p->length == 0) return NS_OK;
  if (!margins || !lse || !dlosses || !dlogits || !aligned(margins, 4) || !aligned(lse, 4) ||
      !aligned(dlosses, 4) || !aligned(dlogits, type_bytes(p->dtype)))
    return NS_ERR_INVALID_ARG;
  const int64_t rows = 2 * p->pairs * p->length;
  const size_t es = type_bytes(p->dtype);
  const bool in_place = dlogits == p->logits && ld_dlogits == p->ld;
  const Span none = {0, 0};
  const Span writes[] = {in_place ? logits_span(*p) : span(dlogits, rows, p->vocab, ld_dlogits, es)};
  const Span reads[] = {in_place ? none : logits_span(*p),
                        span(p->labels, 1, rows, rows, id_bytes(p->label_type)),
                        floats(margins, p->pairs), floats(lse, rows), floats(dlosses, p->pairs)};
  if (clash(writes, reads)) return NS_ERR_INVALID_ARG;
  s = device_status();
  if (s != NS_OK) return s;
  return from_hip(launch_preference_grad(pref_args(*p), p->dtype, p->label_type == NS_IDS_I64,
                                         margins, lse, dlosses, dlogits, ld_dlogits,
                                         in_place ? sequence_ld(*p) : p->length * ld_dlogits,
                                         static_cast<hipStream_t>(stream)));
}

// -------------------------------------------------------------------- AdamW

namespace nsmi {
namespace {
constexpr int64_t ADAMW_MAX_ELEMS = int64_t{1} << 33;   // of one tensor: ADAMW_MAX_BLOCKS of it
constexpr unsigned ADAMW_MAX_BLOCKS = 1u << 23;         // of one launch

ns_status check_adamw(const ns_adamw_tensor& t) {
  if (!type_ok(t.param_dtype) || !type_ok(t.grad_dtype) || !type_ok(t.exp_avg_dtype) ||
      !type_ok(t.exp_avg_sq_dtype) || t.exp_avg_sq_dtype == NS_DT_F16)
    return NS_ERR_INVALID_ARG;
  if (t.elems < 0 || t.elems > ADAMW_MAX_ELEMS || !std::isfinite(t.weight_decay) ||
      t.weight_decay < 0.f)
    return NS_ERR_INVALID_ARG;
  if (t.elems == 0) return NS_OK;
  const size_t pe = type_bytes(t.param_dtype), ge = type_bytes(t.grad_dtype);
  const size_t me = type_bytes(t.exp_avg_dtype), ve = type_bytes(t.exp_avg_sq_dtype);
  if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return NS_ERR_INVALID_ARG;
  if (!aligned(t.param, pe) || !aligned(t.grad, ge) || !aligned(t.exp_avg, me) ||
      !aligned(t.exp_avg_sq, ve) || !aligned(t.master, 4))
    return NS_ERR_INVALID_ARG;
  const int64_t n = t.elems;
  const Span writes[] = {span(t.param, 1, n, n, pe), span(t.exp_avg, 1, n, n, me),
                         span(t.exp_avg_sq, 1, n, n, ve), span(t.master, 1, n, n, 4)};
  const Span reads[] = {span(t.grad, 1, n, n, ge)};
  return clash(writes, reads) ? NS_ERR_INVALID_ARG : NS_OK;
}
bool in_unit(double b) { return b >= 0.0 && b < 1.0; }
bool finite_not_negative(double x) { return std::isfinite(x) && x >= 0.0; }
}  // namespace
}  // namespace nsmi

NS_API ns_status ns_adamw_step(const ns_adamw_tensor* tensors, int count, int64_t step, double lr,
                               double beta1, double beta2, double eps, void* stream) {
  if (count < 0 || (count > 0 && !tensors) || step < 1) return NS_ERR_INVALID_ARG;
  if (!in_unit(beta1) || !in_unit(beta2) || !finite_not_negative(lr) || !finite_not_negative(eps))
    return NS_ERR_INVALID_ARG;
  bool any = false;
  for (int i = 0; i < count; ++i) {
    const ns_status s = check_adamw(tensors[i]);
    if (s != NS_OK) return s;
    any = any || tensors[i].elems > 0;
  }
  if (!any) return NS_OK;
  const ns_status s = device_status();
  if (s != NS_OK) return s;
  AdamwArgs a{};
  a.beta1 = static_cast<float>(beta1);
  a.rest1 = static_cast<float>(1.0 - beta1);
  a.beta2 = static_cast<float>(beta2);
  a.rest2 = static_cast<float>(1.0 - beta2);
  a.step_size = static_cast<float>(lr / (1.0 - std::pow(beta1, static_cast<double>(step))));
  a.root_scale = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  a.eps = static_cast<float>(eps);
  unsigned blocks = 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  for (int i = 0; i < count; ++i) {
    const ns_adamw_tensor& t = tensors[i];
    if (t.elems == 0) continue;
    const unsigned more = adamw_blocks(t.elems);
    if (a.count == ADAMW_TENSORS || (a.count > 0 && blocks + more > ADAMW_MAX_BLOCKS)) {
      if (launch_adamw(a, blocks, st) != hipSuccess) return NS_ERR_HIP;
      a.count = 0;
      blocks = 0;
    }
    a.begin[a.count] = blocks;
    a.t[a.count++] = {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.master, t.elems,
                      t.param_dtype, t.grad_dtype, t.exp_avg_dtype, t.exp_avg_sq_dtype,
                      static_cast<float>(lr * t.weight_decay)};
    blocks += more;
  }
  return from_hip(launch_adamw(a, blocks, st));
}
