// Host-side helpers shared by the C-ABI sources: the thread's error message,
// argument checks, and HIP status conversion.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "nt_internal.hpp"

namespace nt {
namespace host {

inline thread_local std::string g_last_error;

inline nt_status fail(nt_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

inline nt_status ok() {
  g_last_error.clear();
  return NT_OK;
}

// Largest cell count accepted: keeps every launch grid within 2^31 blocks
// (a 2^34-cell pair state is 256 GiB even at 8 bf16 features per cell).
constexpr int64_t kMaxCells = int64_t(1) << 34;

inline size_t esize(nt_dtype d) { return d == NT_BF16 ? 2 : 4; }

inline nt_status check_dtype(nt_dtype d) {
  if (d != NT_F32 && d != NT_BF16) return fail(NT_ERR_DTYPE, "unknown dtype %d", (int)d);
  return NT_OK;
}

inline nt_status check_width(const char* name, int32_t v, int max) {
  if (v <= 0 || v % 8 != 0 || v > max)
    return fail(NT_ERR_INVALID, "%s = %d must be a positive multiple of 8 and at most %d", name,
                (int)v, max);
  return NT_OK;
}

// A device array of `bytes` bytes: NULL only when empty, 16-byte aligned.
inline nt_status check_array(const char* name, const void* ptr, uint64_t bytes) {
  if (bytes == 0) return NT_OK;
  if (!ptr) return fail(NT_ERR_NULL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(ptr) % 16 != 0)
    return fail(NT_ERR_ALIGN, "%s is not 16-byte aligned", name);
  return NT_OK;
}

inline bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

inline nt_status check_partition(const nt_partition* p) {
  if (!p) return fail(NT_ERR_NULL, "partition is NULL");
  if (p->magic != nt::kPartitionMagic)
    return fail(NT_ERR_INVALID, "partition was not built by nt_make_partition");
  if (p->B < 0 || p->T < 0 || p->cells < 0 || p->cells > kMaxCells || p->T > INT32_MAX)
    return fail(NT_ERR_INVALID, "partition sizes are corrupt");
  if (p->T_cols < 0 || p->T_cols > INT32_MAX)
    return fail(NT_ERR_INVALID, "partition sizes are corrupt");
  if (!p->single_offsets || !p->pair_offsets || !p->row_splits || !p->item_offsets ||
      !p->col_offsets || (p->B > 0 && (!p->lengths || !p->col_lengths)) ||
      (p->T > 0 && !p->row_sample) || (p->cells > 0 && !p->tile_sample))
    return fail(NT_ERR_NULL, "partition arrays are NULL");
  return NT_OK;
}

inline nt_status hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess)
    return fail(NT_ERR_HIP, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
  return ok();
}

#define NT_TRY(expr)                      \
  do {                                    \
    const nt_status s_ = (expr);          \
    if (s_ != NT_OK) return s_;           \
  } while (0)

}  // namespace host
}  // namespace nt
