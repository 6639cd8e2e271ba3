// Argument checks that the C ABI of the operators around the matrix update
// shares (train_api.hip, heads_api.hip). Host code.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ns.h"
#include "train_internal.h"

#define NS_API extern "C" __attribute__((visibility("default")))

namespace nsmi {

constexpr size_t ALIGN = 256;
inline size_t align_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }

inline bool type_ok(int t) { return t == NS_DT_F32 || t == NS_DT_BF16 || t == NS_DT_F16; }
inline size_t type_bytes(int t) { return t == NS_DT_E4M3 ? 1 : t == NS_DT_F32 ? 4 : 2; }
inline bool ids_ok(int t) { return t == NS_IDS_I32 || t == NS_IDS_I64; }
inline size_t id_bytes(int t) { return t == NS_IDS_I64 ? 8 : 4; }

// Types that go with `type`: itself or fp32.
inline bool same_or_f32(int t, int type) { return t == type || t == NS_DT_F32; }

// A device buffer: (rows, cols) elements of `es` bytes, leading dimension ld.
struct Span {
  uintptr_t first, last;
};
inline Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (!p || rows < 1 || cols < 1) return {a, a};
  return {a, a + (static_cast<uintptr_t>(rows - 1) * ld + cols) * es};
}
inline bool overlap(Span x, Span y) { return x.first < y.last && y.first < x.last; }

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

inline bool aligned(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es == 0; }
inline bool rows_ok(int64_t r) { return r >= 0 && r <= NS_MAX_ROWS; }
inline bool dim_ok(int64_t d) { return d >= 1 && d <= NS_MAX_DIM; }
// Leading dimensions up to this keep every byte offset of a call in 63 bits.
constexpr int64_t MAX_LD = int64_t{1} << 36;
inline bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= MAX_LD; }

inline ns_status from_hip(hipError_t e) { return e == hipSuccess ? NS_OK : NS_ERR_HIP; }

// Workspace given, large enough and aligned.
inline bool workspace_ok(const void* ws, size_t have, size_t need) {
  return ws && have >= need && reinterpret_cast<uintptr_t>(ws) % ALIGN == 0;
}

}  // namespace nsmi
