// C-ABI entry points of the operators between tokens and singles: host-side
// validation, then the launches. Every check runs before anything is enqueued.
#include <hip/hip_runtime_api.h>

#include <climits>
#include <cmath>

#include "nt_host.hpp"
#include "nt_internal.hpp"

namespace {

using namespace nt::host;

constexpr int64_t kMaxVocabulary = int64_t(1) << 26;

struct Array {
  const char* name;
  const void* ptr;
  uint64_t bytes;
};

// An array of single numbers of `size` bytes: the alignment of its type.
nt_status check_numbers(const Array& a, size_t size) {
  if (a.bytes == 0) return NT_OK;
  if (!a.ptr) return fail(NT_ERR_NULL, "%s is NULL", a.name);
  if (reinterpret_cast<uintptr_t>(a.ptr) % size != 0)
    return fail(NT_ERR_ALIGN, "%s is not aligned to %zu bytes", a.name, size);
  return NT_OK;
}

nt_status check(const Array& a) { return check_array(a.name, a.ptr, a.bytes); }

nt_status check_rows(const char* name, int64_t rows) {
  if (rows < 0 || rows > INT32_MAX)
    return fail(NT_ERR_INVALID, "%s = %lld must be in [0, INT32_MAX]", name, (long long)rows);
  return NT_OK;
}

nt_status check_sizes(int64_t T, int64_t V, int32_t C) {
  NT_TRY(check_rows("T", T));
  if (V < 1 || V > kMaxVocabulary)
    return fail(NT_ERR_INVALID, "V = %lld must be in [1, %lld]", (long long)V,
                (long long)kMaxVocabulary);
  return check_width("C", C, nt::kMaxCs);
}

nt_status check_flag(const char* name, int32_t v) {
  if (v != 0 && v != 1) return fail(NT_ERR_INVALID, "%s = %d must be 0 or 1", name, (int)v);
  return NT_OK;
}

nt_status check_eps(float eps) {
  if (!std::isfinite(eps) || eps < 0.0f)
    return fail(NT_ERR_INVALID, "eps must be finite and not negative");
  return NT_OK;
}

nt_status check_scale(float scale) {
  if (!std::isfinite(scale)) return fail(NT_ERR_INVALID, "scale must be finite");
  return NT_OK;
}

// The kernels take it times log2(e), which has to be finite as well.
nt_status check_logit_scale(float scale) {
  if (!(std::fabs(scale) <= 0x1p100f) || scale == 0.0f)
    return fail(NT_ERR_INVALID, "scale must not be zero, and at most 2^100 either way");
  return NT_OK;
}

nt_status check_workspace(const void* workspace, size_t have, size_t need) {
  if (have < need)
    return fail(NT_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return check_array("workspace", workspace, need);
}

// The written arrays against the read ones and each other; written[i] may be the
// same array as the inputs that the bits of same[i] name.
template <int W, int R>
nt_status check_apart(const Array (&written)[W], const Array (&read)[R], const int (&same)[W]) {
  for (int i = 0; i < W; ++i) {
    const Array& a = written[i];
    for (int j = 0; j < R; ++j) {
      const Array& b = read[j];
      if ((same[i] >> j & 1) && a.ptr == b.ptr && a.bytes == b.bytes) continue;
      if (overlaps(a.ptr, a.bytes, b.ptr, b.bytes))
        return fail(NT_ERR_INVALID, "%s overlaps %s", a.name, b.name);
    }
    for (int j = 0; j < i; ++j)
      if (overlaps(a.ptr, a.bytes, written[j].ptr, written[j].bytes))
        return fail(NT_ERR_INVALID, "%s overlaps %s", a.name, written[j].name);
  }
  return NT_OK;
}

nt_status check_loss(int64_t T, int64_t V, int32_t C, nt_dtype dtype) {
  NT_TRY(check_sizes(T, V, C));
  NT_TRY(check_dtype(dtype));
  return NT_OK;
}

// The norm's arrays, of either output.
nt_status check_norm(const void* x, const void* residual, const float* w, void* h, Array y,
                     Array scales, int64_t rows, int32_t C, float eps, nt_dtype dtype) {
  const uint64_t bytes = (uint64_t)rows * C * esize(dtype);
  const Array in[3] = {{"x", x, bytes},
                       {"residual", residual, residual ? bytes : 0},
                       {"w", w, w ? C * sizeof(float) : 0}};
  const Array out[3] = {{"h", h, residual ? bytes : 0}, y, scales};
  NT_TRY(check_eps(eps));
  for (const Array& a : in) NT_TRY(check(a));
  for (const Array& a : out) NT_TRY(check(a));
  return check_apart(out, in, {1 | 2, 1 | 2, 0});
}

}  // namespace

extern "C" {

nt_status nt_token_embedding(const void* table, const int32_t* tokens, void* out, int64_t T,
                             int64_t V, int32_t C, float scale, nt_dtype dtype, void* stream) {
  NT_TRY(check_dtype(dtype));
  NT_TRY(check_sizes(T, V, C));
  NT_TRY(check_scale(scale));
  const size_t es = esize(dtype);
  const Array in[2] = {{"table", table, (uint64_t)V * C * es},
                       {"tokens", tokens, T * sizeof(int32_t)}};
  const Array written[1] = {{"out", out, (uint64_t)T * C * es}};
  NT_TRY(check(in[0]));
  NT_TRY(check_numbers(in[1], sizeof(int32_t)));
  NT_TRY(check(written[0]));
  NT_TRY(check_apart(written, in, {0}));
  return hip_status(nt::launch_token_embedding(table, tokens, out, T, V, C, scale, dtype,
                                               static_cast<hipStream_t>(stream)),
                    "token embedding kernel");
}

nt_status nt_token_embedding_backward_workspace_bytes(int64_t T, int64_t V, int32_t C,
                                                      size_t* bytes) {
  NT_TRY(check_sizes(T, V, C));
  if (!bytes) return fail(NT_ERR_NULL, "bytes is NULL");
  *bytes = nt::token_embedding_backward_ws_bytes(T, V, C);
  return ok();
}

nt_status nt_token_embedding_backward(const int32_t* tokens, const void* g_out, float* g_table,
                                      int64_t T, int64_t V, int32_t C, float scale,
                                      int32_t accumulate, nt_dtype dtype, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  NT_TRY(check_dtype(dtype));
  NT_TRY(check_sizes(T, V, C));
  NT_TRY(check_scale(scale));
  NT_TRY(check_flag("accumulate", accumulate));
  const size_t need = nt::token_embedding_backward_ws_bytes(T, V, C);
  const Array in[2] = {{"tokens", tokens, T * sizeof(int32_t)},
                       {"g_out", g_out, (uint64_t)T * C * esize(dtype)}};
  const Array written[2] = {{"g_table", g_table, (uint64_t)V * C * sizeof(float)},
                            {"workspace", workspace, need}};
  NT_TRY(check_numbers(in[0], sizeof(int32_t)));
  NT_TRY(check(in[1]));
  NT_TRY(check(written[0]));
  NT_TRY(check_workspace(workspace, workspace_bytes, need));
  NT_TRY(check_apart(written, in, {0, 0}));
  return hip_status(
      nt::launch_token_embedding_backward(tokens, g_out, g_table, T, V, C, scale, accumulate != 0,
                                          dtype, workspace, static_cast<hipStream_t>(stream)),
      "token embedding gradient kernels");
}

nt_status nt_residual_norm(const void* x, const void* residual, const float* w, void* h, void* y,
                           int64_t rows, int32_t C, float eps, nt_dtype dtype, void* stream) {
  NT_TRY(check_dtype(dtype));
  NT_TRY(check_rows("rows", rows));
  NT_TRY(check_width("C", C, nt::kMaxCs));
  NT_TRY(check_norm(x, residual, w, h, {"y", y, (uint64_t)rows * C * esize(dtype)},
                    {"scales", nullptr, 0}, rows, C, eps, dtype));
  return hip_status(nt::launch_residual_norm(x, residual, w, h, y, nullptr, nullptr, rows, C, 0,
                                             eps, dtype, static_cast<hipStream_t>(stream)),
                    "residual norm kernel");
}

nt_status nt_residual_norm_8bit(const void* x, const void* residual, const float* w, void* h,
                                uint8_t* codes, float* scales, int64_t rows, int32_t C,
                                int32_t group, float eps, nt_dtype dtype, void* stream) {
  NT_TRY(check_dtype(dtype));
  NT_TRY(check_rows("rows", rows));
  NT_TRY(check_width("C", C, nt::kMaxCs));
  if (group != 0 && (group < 8 || group > 512 || (group & (group - 1)) != 0 || C % group != 0))
    return fail(NT_ERR_INVALID, "group = %d must be 0 or a power of two in [8, 512] that divides C",
                (int)group);
  const uint64_t count = (uint64_t)rows * (group ? C / group : 1);
  NT_TRY(check_norm(x, residual, w, h, {"codes", codes, (uint64_t)rows * C},
                    {"scales", scales, count * sizeof(float)}, rows, C, eps, dtype));
  return hip_status(nt::launch_residual_norm(x, residual, w, h, nullptr, codes, scales, rows, C,
                                             group, eps, dtype, static_cast<hipStream_t>(stream)),
                    "residual norm kernel");
}

nt_status nt_residual_norm_backward_workspace_bytes(int64_t rows, int32_t C, size_t* bytes) {
  NT_TRY(check_rows("rows", rows));
  NT_TRY(check_width("C", C, nt::kMaxCs));
  if (!bytes) return fail(NT_ERR_NULL, "bytes is NULL");
  *bytes = nt::residual_norm_backward_ws_bytes(rows, C);
  return ok();
}

nt_status nt_residual_norm_backward(const void* h, const void* g_y, const void* g_h,
                                    const float* w, void* g, float* g_w, int64_t rows, int32_t C,
                                    float eps, nt_dtype dtype, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  NT_TRY(check_dtype(dtype));
  NT_TRY(check_rows("rows", rows));
  NT_TRY(check_width("C", C, nt::kMaxCs));
  NT_TRY(check_eps(eps));
  const uint64_t bytes = (uint64_t)rows * C * esize(dtype), w_bytes = w ? C * sizeof(float) : 0;
  const size_t need = w ? nt::residual_norm_backward_ws_bytes(rows, C) : 0;
  const Array in[4] = {{"h", h, bytes},
                       {"g_y", g_y, bytes},
                       {"g_h", g_h, g_h ? bytes : 0},
                       {"w", w, w_bytes}};
  const Array written[3] = {{"g", g, bytes}, {"g_w", g_w, w_bytes}, {"workspace", workspace, need}};
  for (const Array& a : in) NT_TRY(check(a));
  NT_TRY(check(written[0]));
  NT_TRY(check(written[1]));
  NT_TRY(check_workspace(workspace, workspace_bytes, need));
  NT_TRY(check_apart(written, in, {2 | 4, 0, 0}));
  return hip_status(
      nt::launch_residual_norm_backward(h, g_y, g_h, w, g, g_w, rows, C, eps, dtype, workspace,
                                        static_cast<hipStream_t>(stream)),
      "residual norm gradient kernels");
}

nt_status nt_token_loss_workspace_bytes(int64_t T, int64_t V, int32_t C, nt_dtype dtype,
                                        size_t* bytes) {
  NT_TRY(check_loss(T, V, C, dtype));
  if (!bytes) return fail(NT_ERR_NULL, "bytes is NULL");
  *bytes = nt::token_loss_ws_bytes(T, V, C, dtype);
  return ok();
}

nt_status nt_token_loss(const void* x, const void* W, const int32_t* targets, float* nll,
                        float* lse, int64_t T, int64_t V, int32_t C, float scale, nt_dtype dtype,
                        void* workspace, size_t workspace_bytes, void* stream) {
  NT_TRY(check_loss(T, V, C, dtype));
  NT_TRY(check_logit_scale(scale));
  const size_t es = esize(dtype), need = nt::token_loss_ws_bytes(T, V, C, dtype);
  const uint64_t numbers = (uint64_t)T * sizeof(float);
  const Array in[3] = {{"x", x, (uint64_t)T * C * es},
                       {"W", W, (uint64_t)V * C * es},
                       {"targets", targets, numbers}};
  const Array written[3] = {{"nll", nll, numbers}, {"lse", lse, numbers},
                            {"workspace", workspace, need}};
  NT_TRY(check(in[0]));
  NT_TRY(check(in[1]));
  NT_TRY(check_numbers(in[2], sizeof(int32_t)));
  NT_TRY(check_numbers(written[0], sizeof(float)));
  NT_TRY(check_numbers(written[1], sizeof(float)));
  NT_TRY(check_workspace(workspace, workspace_bytes, need));
  NT_TRY(check_apart(written, in, {0, 0, 0}));
  return hip_status(nt::launch_token_loss(x, W, targets, nll, lse, T, V, C, scale, dtype, workspace,
                                          static_cast<hipStream_t>(stream)),
                    "token loss kernels");
}

nt_status nt_token_loss_backward_workspace_bytes(int64_t T, int64_t V, int32_t C, nt_dtype dtype,
                                                 size_t* bytes) {
  NT_TRY(check_loss(T, V, C, dtype));
  if (!bytes) return fail(NT_ERR_NULL, "bytes is NULL");
  *bytes = nt::token_loss_backward_ws_bytes(T, V, C, dtype);
  return ok();
}

nt_status nt_token_loss_backward(const void* x, const void* W, const int32_t* targets,
                                 const float* lse, const float* g_nll, const float* g_lse,
                                 void* g_x, float* g_W, int64_t T, int64_t V, int32_t C,
                                 float scale, int32_t accumulate, nt_dtype dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  NT_TRY(check_loss(T, V, C, dtype));
  NT_TRY(check_logit_scale(scale));
  NT_TRY(check_flag("accumulate", accumulate));
  const size_t es = esize(dtype), need = nt::token_loss_backward_ws_bytes(T, V, C, dtype);
  const uint64_t numbers = (uint64_t)T * sizeof(float);
  const Array in[6] = {{"x", x, (uint64_t)T * C * es},
                       {"W", W, (uint64_t)V * C * es},
                       {"targets", targets, numbers},
                       {"lse", lse, numbers},
                       {"g_nll", g_nll, numbers},
                       {"g_lse", g_lse, g_lse ? numbers : 0}};
  const Array written[3] = {{"g_x", g_x, g_x ? (uint64_t)T * C * es : 0},
                            {"g_W", g_W, g_W ? (uint64_t)V * C * sizeof(float) : 0},
                            {"workspace", workspace, need}};
  for (int i = 0; i < 2; ++i) NT_TRY(check(in[i]));
  for (int i = 2; i < 6; ++i) NT_TRY(check_numbers(in[i], sizeof(float)));
  for (int i = 0; i < 2; ++i) NT_TRY(check(written[i]));
  NT_TRY(check_workspace(workspace, workspace_bytes, need));
  NT_TRY(check_apart(written, in, {0, 0, 0}));
  return hip_status(
      nt::launch_token_loss_backward(x, W, targets, lse, g_nll, g_lse, g_x, g_W, T, V, C, scale,
                                     accumulate != 0, dtype, workspace,
                                     static_cast<hipStream_t>(stream)),
      "token loss gradient kernels");
}

}  // extern "C"
