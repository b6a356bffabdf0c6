// C-ABI entry points of the single attention operators and the optimizer's
// step: host-side validation, then the launches. Every check runs before
// anything is enqueued.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <new>
#include <vector>

#include "nt_host.hpp"
#include "nt_internal.hpp"

namespace {

using namespace nt::host;

constexpr int kMaxHeadDim = 128;
constexpr int kMaxHeads = 4096;
constexpr int64_t kMaxLd = int64_t(1) << 22;  // byte distances within a tile fit 32 bits

// An array of token rows: `width` elements every `ld`.
struct Rows {
  const char* name;
  const void* ptr;
  int64_t rows, ld, width;
};

uint64_t span(const Rows& a, size_t es) {
  return a.rows > 0 ? ((uint64_t)(a.rows - 1) * a.ld + a.width) * es : 0;
}

// Whether two arrays of rows share an element. Rows of one projected array
// (the same ld) interleave without meeting when their columns are apart.
bool rows_overlap(const Rows& a, const Rows& b, size_t es) {
  const uint64_t na = span(a, es), nb = span(b, es);
  if (!overlaps(a.ptr, na, b.ptr, nb)) return false;
  if (a.ld != b.ld) return true;
  const intptr_t x = reinterpret_cast<intptr_t>(a.ptr), y = reinterpret_cast<intptr_t>(b.ptr);
  const intptr_t pitch = (intptr_t)(a.ld * (int64_t)es);
  intptr_t off = (y - x) % pitch;
  if (off < 0) off += pitch;
  return off < (intptr_t)(a.width * (int64_t)es) || off + (intptr_t)(b.width * (int64_t)es) > pitch;
}

nt_status check_rows(const Rows& a, size_t es) {
  if (a.ld < a.width || a.ld % 8 != 0 || a.ld > kMaxLd)
    return fail(NT_ERR_INVALID, "ld of %s = %lld must be a multiple of 8 in [%lld, %lld]", a.name,
                (long long)a.ld, (long long)a.width, (long long)kMaxLd);
  return check_array(a.name, a.ptr, span(a, es));
}

nt_status check_heads(int32_t heads, int32_t kv_heads, int32_t head_dim, bool kv_none) {
  if (heads < 1 || heads > kMaxHeads)
    return fail(NT_ERR_INVALID, "heads = %d must be in [1, %d]", (int)heads, kMaxHeads);
  if (kv_heads < (kv_none ? 0 : 1) || kv_heads > kMaxHeads)
    return fail(NT_ERR_INVALID, "kv_heads = %d must be in [%d, %d]", (int)kv_heads,
                kv_none ? 0 : 1, kMaxHeads);
  return check_width("head_dim", head_dim, kMaxHeadDim);
}

int64_t ld_or(int64_t ld, int64_t packed) { return ld ? ld : packed; }

nt_status check_workspace(const void* workspace, size_t have, size_t need) {
  if (have < need)
    return fail(NT_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return check_array("workspace", workspace, need);
}

// The struct with its distances filled in.
nt_status check_norm(const nt_partition* p, const nt_norm_rotary* n, nt_dtype dtype,
                     nt_norm_rotary* out) {
  NT_TRY(check_partition(p));
  if (!n) return fail(NT_ERR_NULL, "the norm's description is NULL");
  NT_TRY(check_dtype(dtype));
  NT_TRY(check_heads(n->heads, n->kv_heads, n->head_dim, true));
  if (n->rot_dim < 0 || n->rot_dim > n->head_dim || n->rot_dim % 2 != 0)
    return fail(NT_ERR_INVALID, "rot_dim = %d must be even and in [0, head_dim = %d]",
                (int)n->rot_dim, (int)n->head_dim);
  if (n->interleaved != 0 && n->interleaved != 1)
    return fail(NT_ERR_INVALID, "interleaved = %d must be 0 or 1", (int)n->interleaved);
  if (!std::isfinite(n->eps) || n->eps < 0.0f)
    return fail(NT_ERR_INVALID, "eps must be finite and not negative");
  if (n->rot_dim && (n->positions < 1 || n->positions > INT32_MAX))
    return fail(NT_ERR_INVALID, "positions = %lld must be in [1, INT32_MAX]",
                (long long)n->positions);
  *out = *n;
  const int64_t q = (int64_t)n->heads * n->head_dim, k = (int64_t)n->kv_heads * n->head_dim;
  out->ld_q = ld_or(n->ld_q, q);
  out->ld_q_out = ld_or(n->ld_q_out, q);
  out->ld_k = ld_or(n->ld_k, k);
  out->ld_k_out = ld_or(n->ld_k_out, k);
  return NT_OK;
}

// Table, weights and positions; written: an array they must not overlap.
nt_status check_norm_inputs(const nt_partition& p, const nt_norm_rotary& n, const float* w_q,
                            const float* w_k, const float* table, const int32_t* positions_q,
                            const int32_t* positions_k, const Rows* written, int count,
                            size_t es) {
  const uint64_t nt_bytes = n.rot_dim ? (uint64_t)n.positions * n.rot_dim * sizeof(float) : 0;
  NT_TRY(check_array("table", table, nt_bytes));
  const uint64_t w_bytes = (uint64_t)n.head_dim * sizeof(float);
  if (w_q) NT_TRY(check_array("w_q", w_q, w_bytes));
  if (w_k) NT_TRY(check_array("w_k", w_k, w_bytes));
  if (positions_q) NT_TRY(check_array("positions_q", positions_q, p.T * sizeof(int32_t)));
  if (positions_k) NT_TRY(check_array("positions_k", positions_k, p.T_cols * sizeof(int32_t)));
  for (int i = 0; i < count; ++i) {
    const uint64_t bytes = span(written[i], es);
    if (overlaps(written[i].ptr, bytes, table, nt_bytes) ||
        overlaps(written[i].ptr, bytes, w_q, w_bytes) ||
        overlaps(written[i].ptr, bytes, w_k, w_bytes) ||
        overlaps(written[i].ptr, bytes, positions_q, p.T * sizeof(int32_t)) ||
        overlaps(written[i].ptr, bytes, positions_k, p.T_cols * sizeof(int32_t)))
      return fail(NT_ERR_INVALID, "%s overlaps the table, the weights or the positions",
                  written[i].name);
  }
  return NT_OK;
}

bool same_rows(const Rows& a, const Rows& b) { return a.ptr == b.ptr && a.ld == b.ld; }

nt_status check_attention(const nt_partition* p, const nt_attention* a, nt_dtype dtype,
                          nt_attention* out) {
  NT_TRY(check_partition(p));
  if (!a) return fail(NT_ERR_NULL, "the attention's description is NULL");
  NT_TRY(check_dtype(dtype));
  NT_TRY(check_heads(a->heads, a->kv_heads, a->head_dim, false));
  if (a->heads % a->kv_heads != 0)
    return fail(NT_ERR_INVALID, "heads = %d is not a multiple of kv_heads = %d", (int)a->heads,
                (int)a->kv_heads);
  if (a->causal != 0 && a->causal != 1)
    return fail(NT_ERR_INVALID, "causal = %d must be 0 or 1", (int)a->causal);
  if (!std::isfinite(a->scale)) return fail(NT_ERR_INVALID, "scale must be finite");
  *out = *a;
  out->ld_q = ld_or(a->ld_q, (int64_t)a->heads * a->head_dim);
  out->ld_k = ld_or(a->ld_k, (int64_t)a->kv_heads * a->head_dim);
  out->ld_v = ld_or(a->ld_v, (int64_t)a->kv_heads * a->head_dim);
  if (!nt::attention_fits(*p, *out))
    return fail(NT_ERR_OVERFLOW, "%lld rows of %d heads exceed one launch", (long long)p->T,
                (int)a->heads);
  return NT_OK;
}

struct Span {
  uintptr_t at, end;
  bool written;
  int tensor;
};

}  // namespace

extern "C" {

nt_status nt_rotary_table(const nt_rotary* r, float* table, int64_t positions, void* stream) {
  if (!r) return fail(NT_ERR_NULL, "the rotation's description is NULL");
  if (r->rot_dim < 2 || r->rot_dim > kMaxHeadDim || r->rot_dim % 2 != 0)
    return fail(NT_ERR_INVALID, "rot_dim = %d must be even and in [2, %d]", (int)r->rot_dim,
                kMaxHeadDim);
  if (!(r->base > 1.0) || !std::isfinite(r->base))
    return fail(NT_ERR_INVALID, "base must be finite and greater than 1");
  if (r->scaling != NT_ROTARY_NONE && r->scaling != NT_ROTARY_LINEAR &&
      r->scaling != NT_ROTARY_PARTS)
    return fail(NT_ERR_INVALID, "unknown scaling %d", (int)r->scaling);
  if (r->scaling != NT_ROTARY_NONE && (!(r->factor >= 1.0) || !std::isfinite(r->factor)))
    return fail(NT_ERR_INVALID, "factor must be finite and at least 1");
  if (r->scaling == NT_ROTARY_PARTS &&
      (!(r->original > 0.0) || !std::isfinite(r->original) || !(r->beta_slow >= 0.0) ||
       !(r->beta_fast > r->beta_slow) || !std::isfinite(r->beta_fast)))
    return fail(NT_ERR_INVALID, "scaling by parts needs original > 0 and beta_fast > beta_slow >= 0");
  if (!(r->magnitude > 0.0) || !std::isfinite(r->magnitude))
    return fail(NT_ERR_INVALID, "magnitude must be finite and greater than 0");
  if (positions < 0 || positions > INT32_MAX)
    return fail(NT_ERR_INVALID, "positions = %lld must be in [0, INT32_MAX]", (long long)positions);
  NT_TRY(check_array("table", table, (uint64_t)positions * r->rot_dim * sizeof(float)));
  return hip_status(nt::launch_rotary_table(*r, table, positions, static_cast<hipStream_t>(stream)),
                    "rotary table kernel");
}

nt_status nt_qk_norm_rotary(const nt_partition* p, const nt_norm_rotary* n, const void* q,
                            const void* k, const float* w_q, const float* w_k, const float* table,
                            const int32_t* positions_q, const int32_t* positions_k, void* q_out,
                            void* k_out, nt_dtype dtype, void* stream) {
  nt_norm_rotary x;
  NT_TRY(check_norm(p, n, dtype, &x));
  const size_t es = esize(dtype);
  const int64_t dq = (int64_t)x.heads * x.head_dim, dk = (int64_t)x.kv_heads * x.head_dim;
  const int64_t Tk = x.kv_heads ? p->T_cols : 0;
  const Rows in[2] = {{"q", q, p->T, x.ld_q, dq}, {"k", k, Tk, x.ld_k, dk}};
  const Rows out[2] = {{"q_out", q_out, p->T, x.ld_q_out, dq}, {"k_out", k_out, Tk, x.ld_k_out, dk}};
  for (int i = 0; i < 2; ++i) {
    NT_TRY(check_rows(in[i], es));
    NT_TRY(check_rows(out[i], es));
  }
  NT_TRY(check_norm_inputs(*p, x, w_q, w_k, table, positions_q, positions_k, out, 2, es));
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (!(i == j && same_rows(out[i], in[j])) && rows_overlap(out[i], in[j], es))
        return fail(NT_ERR_INVALID, "%s overlaps %s", out[i].name, in[j].name);
  if (rows_overlap(out[0], out[1], es)) return fail(NT_ERR_INVALID, "q_out overlaps k_out");
  return hip_status(nt::launch_norm_rotary(*p, x, q, k, w_q, w_k, table, positions_q, positions_k,
                                           q_out, k_out, dtype, static_cast<hipStream_t>(stream)),
                    "norm and rotation kernel");
}

nt_status nt_qk_norm_rotary_backward_workspace_bytes(const nt_partition* p,
                                                     const nt_norm_rotary* n, nt_dtype dtype,
                                                     size_t* bytes) {
  nt_norm_rotary x;
  NT_TRY(check_norm(p, n, dtype, &x));
  if (!bytes) return fail(NT_ERR_NULL, "bytes is NULL");
  *bytes = nt::norm_rotary_backward_ws_bytes(*p, x);
  return ok();
}

nt_status nt_qk_norm_rotary_backward(const nt_partition* p, const nt_norm_rotary* n,
                                     const void* q, const void* k, const void* g_q,
                                     const void* g_k, const float* w_q, const float* w_k,
                                     const float* table, const int32_t* positions_q,
                                     const int32_t* positions_k, void* g_q_in, void* g_k_in,
                                     float* g_w_q, float* g_w_k, nt_dtype dtype, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  nt_norm_rotary x;
  NT_TRY(check_norm(p, n, dtype, &x));
  const size_t es = esize(dtype);
  const int64_t dq = (int64_t)x.heads * x.head_dim, dk = (int64_t)x.kv_heads * x.head_dim;
  const int64_t Tk = x.kv_heads ? p->T_cols : 0;
  const Rows in[4] = {{"q", q, p->T, x.ld_q, dq},
                      {"k", k, Tk, x.ld_k, dk},
                      {"g_q", g_q, p->T, dq, dq},
                      {"g_k", g_k, Tk, dk, dk}};
  const Rows out[2] = {{"g_q_in", g_q_in, p->T, x.ld_q_out, dq},
                       {"g_k_in", g_k_in, Tk, x.ld_k_out, dk}};
  for (const Rows& a : in) NT_TRY(check_rows(a, es));
  for (const Rows& a : out) NT_TRY(check_rows(a, es));
  NT_TRY(check_norm_inputs(*p, x, w_q, w_k, table, positions_q, positions_k, out, 2, es));
  const uint64_t w_bytes = (uint64_t)x.head_dim * sizeof(float);
  if (w_q) NT_TRY(check_array("g_w_q", g_w_q, w_bytes));
  if (w_k) NT_TRY(check_array("g_w_k", g_w_k, w_bytes));
  const size_t need = w_q || w_k ? nt::norm_rotary_backward_ws_bytes(*p, x) : 0;
  NT_TRY(check_workspace(workspace, workspace_bytes, need));
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 4; ++j)
      if (!(i + 2 == j && same_rows(out[i], in[j])) && rows_overlap(out[i], in[j], es))
        return fail(NT_ERR_INVALID, "%s overlaps %s", out[i].name, in[j].name);
  if (rows_overlap(out[0], out[1], es)) return fail(NT_ERR_INVALID, "g_q_in overlaps g_k_in");
  // the small written arrays and the workspace against everything else
  const void* small[3] = {w_q ? g_w_q : nullptr, w_k ? g_w_k : nullptr, workspace};
  const uint64_t size[3] = {w_bytes, w_bytes, need};
  const uint64_t table_bytes = x.rot_dim ? (uint64_t)x.positions * x.rot_dim * sizeof(float) : 0;
  for (int i = 0; i < 3; ++i) {
    bool meets = false;
    for (const Rows& a : in) meets = meets || overlaps(small[i], size[i], a.ptr, span(a, es));
    for (const Rows& a : out) meets = meets || overlaps(small[i], size[i], a.ptr, span(a, es));
    meets = meets || overlaps(small[i], size[i], table, table_bytes) ||
            overlaps(small[i], size[i], w_q, w_bytes) || overlaps(small[i], size[i], w_k, w_bytes) ||
            overlaps(small[i], size[i], positions_q, p->T * sizeof(int32_t)) ||
            overlaps(small[i], size[i], positions_k, p->T_cols * sizeof(int32_t));
    for (int j = 0; j < i; ++j) meets = meets || overlaps(small[i], size[i], small[j], size[j]);
    if (meets)
      return fail(NT_ERR_INVALID, "g_w_q, g_w_k or the workspace overlaps another array");
  }
  return hip_status(
      nt::launch_norm_rotary_backward(*p, x, q, k, g_q, g_k, w_q, w_k, table, positions_q,
                                      positions_k, g_q_in, g_k_in, g_w_q, g_w_k, workspace, dtype,
                                      static_cast<hipStream_t>(stream)),
      "norm and rotation gradient kernels");
}

nt_status nt_attention_workspace_bytes(const nt_partition* p, const nt_attention* a,
                                       nt_dtype dtype, size_t* bytes) {
  nt_attention x;
  NT_TRY(check_attention(p, a, dtype, &x));
  if (!bytes) return fail(NT_ERR_NULL, "bytes is NULL");
  *bytes = nt::attention_ws_bytes(*p, x, dtype);
  return ok();
}

nt_status nt_single_attention(const nt_partition* p, const nt_attention* a, const void* q,
                              const void* k, const void* v, const void* bias, void* o, float* lse,
                              nt_dtype dtype, void* workspace, size_t workspace_bytes,
                              void* stream) {
  nt_attention x;
  NT_TRY(check_attention(p, a, dtype, &x));
  const size_t es = esize(dtype);
  const int64_t dq = (int64_t)x.heads * x.head_dim, dk = (int64_t)x.kv_heads * x.head_dim;
  const Rows in[3] = {{"q", q, p->T, x.ld_q, dq},
                      {"k", k, p->T_cols, x.ld_k, dk},
                      {"v", v, p->T_cols, x.ld_v, dk}};
  for (const Rows& r : in) NT_TRY(check_rows(r, es));
  const uint64_t bias_bytes = bias ? (uint64_t)p->cells * x.heads * es : 0;
  NT_TRY(check_array("bias", bias, bias_bytes));
  const uint64_t o_bytes = (uint64_t)p->T * dq * es;
  const uint64_t lse_bytes = (uint64_t)p->T * x.heads * sizeof(float);
  NT_TRY(check_array("o", o, o_bytes));
  NT_TRY(check_array("lse", lse, lse_bytes));
  const size_t need = nt::attention_ws_bytes(*p, x, dtype);
  NT_TRY(check_workspace(workspace, workspace_bytes, need));
  const void* out[3] = {o, lse, workspace};
  const uint64_t size[3] = {o_bytes, lse_bytes, need};
  for (int i = 0; i < 3; ++i) {
    bool meets = overlaps(out[i], size[i], bias, bias_bytes);
    for (const Rows& r : in) meets = meets || overlaps(out[i], size[i], r.ptr, span(r, es));
    for (int j = 0; j < i; ++j) meets = meets || overlaps(out[i], size[i], out[j], size[j]);
    if (meets) return fail(NT_ERR_INVALID, "o, lse or the workspace overlaps another array");
  }
  return hip_status(nt::launch_attention(*p, x, q, k, v, bias, o, lse, dtype, workspace,
                                         static_cast<hipStream_t>(stream)),
                    "attention kernels");
}

nt_status nt_attention_backward_workspace_bytes(const nt_partition* p, const nt_attention* a,
                                                nt_dtype dtype, size_t* bytes) {
  nt_attention x;
  NT_TRY(check_attention(p, a, dtype, &x));
  if (!bytes) return fail(NT_ERR_NULL, "bytes is NULL");
  *bytes = nt::attention_backward_ws_bytes(*p, x, dtype);
  return ok();
}

nt_status nt_single_attention_backward(const nt_partition* p, const nt_attention* a,
                                       const void* q, const void* k, const void* v,
                                       const void* bias, const void* o, const float* lse,
                                       const void* g_o, const nt_attention_grads* g,
                                       nt_dtype dtype, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  nt_attention x;
  NT_TRY(check_attention(p, a, dtype, &x));
  if (!g) return fail(NT_ERR_NULL, "grads is NULL");
  const size_t es = esize(dtype);
  const int64_t dq = (int64_t)x.heads * x.head_dim, dk = (int64_t)x.kv_heads * x.head_dim;
  nt_attention_grads y = *g;
  y.ld_q = ld_or(g->ld_q, dq);
  y.ld_k = ld_or(g->ld_k, dk);
  y.ld_v = ld_or(g->ld_v, dk);
  const Rows in[5] = {{"q", q, p->T, x.ld_q, dq},
                      {"k", k, p->T_cols, x.ld_k, dk},
                      {"v", v, p->T_cols, x.ld_v, dk},
                      {"o", o, p->T, dq, dq},
                      {"g_o", g_o, p->T, dq, dq}};
  const Rows out[3] = {{"g_q", y.q, p->T, y.ld_q, dq},
                       {"g_k", y.k, p->T_cols, y.ld_k, dk},
                       {"g_v", y.v, p->T_cols, y.ld_v, dk}};
  for (const Rows& r : in) NT_TRY(check_rows(r, es));
  for (const Rows& r : out) NT_TRY(check_rows(r, es));
  const uint64_t bias_bytes = (uint64_t)p->cells * x.heads * es;
  const uint64_t lse_bytes = (uint64_t)p->T * x.heads * sizeof(float);
  if (bias) NT_TRY(check_array("bias", bias, bias_bytes));
  if (y.bias) NT_TRY(check_array("g_bias", y.bias, bias_bytes));
  if (bias && p->T_cols >= int64_t(1) << 23)
    return fail(NT_ERR_OVERFLOW, "T_cols = %lld with a bias must be below 2^23",
                (long long)p->T_cols);
  if (y.bias && !bias) return fail(NT_ERR_NULL, "g_bias without a bias");
  NT_TRY(check_array("lse", lse, lse_bytes));
  const size_t need = nt::attention_backward_ws_bytes(*p, x, dtype);
  NT_TRY(check_workspace(workspace, workspace_bytes, need));
  for (int i = 0; i < 3; ++i) {
    for (const Rows& r : in)
      if (rows_overlap(out[i], r, es))
        return fail(NT_ERR_INVALID, "%s overlaps %s", out[i].name, r.name);
    for (int j = 0; j < i; ++j)
      if (rows_overlap(out[i], out[j], es))
        return fail(NT_ERR_INVALID, "%s overlaps %s", out[i].name, out[j].name);
    if (overlaps(out[i].ptr, span(out[i], es), bias, bias ? bias_bytes : 0) ||
        overlaps(out[i].ptr, span(out[i], es), lse, lse_bytes))
      return fail(NT_ERR_INVALID, "%s overlaps bias or lse", out[i].name);
  }
  const void* whole[2] = {y.bias, workspace};
  const uint64_t size[2] = {y.bias ? bias_bytes : 0, need};
  for (int i = 0; i < 2; ++i) {
    bool meets = overlaps(whole[i], size[i], bias, bias ? bias_bytes : 0) ||
                 overlaps(whole[i], size[i], lse, lse_bytes);
    for (const Rows& r : in) meets = meets || overlaps(whole[i], size[i], r.ptr, span(r, es));
    for (const Rows& r : out) meets = meets || overlaps(whole[i], size[i], r.ptr, span(r, es));
    if (i) meets = meets || overlaps(whole[0], size[0], whole[1], size[1]);
    if (meets) return fail(NT_ERR_INVALID, "g_bias or the workspace overlaps another array");
  }
  return hip_status(nt::launch_attention_backward(*p, x, q, k, v, bias, o, lse, g_o, y, dtype,
                                                  workspace, static_cast<hipStream_t>(stream)),
                    "attention gradient kernels");
}

nt_status nt_adamw_step(const nt_adamw_tensor* tensors, int32_t count, const nt_adamw* h,
                        nt_dtype dtype, void* stream) {
  if (!h) return fail(NT_ERR_NULL, "the step's description is NULL");
  NT_TRY(check_dtype(dtype));
  if (count < 0) return fail(NT_ERR_INVALID, "count = %d is negative", (int)count);
  if (count && !tensors) return fail(NT_ERR_NULL, "tensors is NULL");
  if (h->state_bits != 32 && h->state_bits != 8)
    return fail(NT_ERR_INVALID, "state_bits = %d must be 32 or 8", (int)h->state_bits);
  if (!(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0))
    return fail(NT_ERR_INVALID, "beta1 and beta2 must be in [0, 1)");
  if (!std::isfinite(h->lr) || !std::isfinite(h->weight_decay) || !std::isfinite(h->eps) ||
      h->eps < 0.0)
    return fail(NT_ERR_INVALID, "lr, weight_decay and eps must be finite and eps not negative");
  if (!h->step_device && h->step < 1)
    return fail(NT_ERR_INVALID, "step = %lld must be at least 1", (long long)h->step);
  if (reinterpret_cast<uintptr_t>(h->step_device) % 8 != 0 ||
      reinterpret_cast<uintptr_t>(h->lr_device) % 4 != 0)
    return fail(NT_ERR_ALIGN, "step_device or lr_device is not aligned to its type");
  try {
    std::vector<Span> spans;
    spans.reserve((size_t)count * 7 + 2);
    auto add = [&](const void* ptr, uint64_t bytes, bool written, int tensor) {
      if (ptr && bytes) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(ptr);
        spans.push_back({at, at + bytes, written, tensor});
      }
    };
    for (int32_t i = 0; i < count; ++i) {
      const nt_adamw_tensor& t = tensors[i];
      if (t.n < 0 || t.n > nt::kAdamwMostElements)
        return fail(NT_ERR_INVALID, "tensor %d has %lld elements", (int)i, (long long)t.n);
      const uint64_t n = (uint64_t)t.n;
      const uint64_t state = n * (h->state_bits == 8 ? 1 : sizeof(float));
      const uint64_t scale =
          h->state_bits == 8 ? (n + NT_ADAMW_BLOCK - 1) / NT_ADAMW_BLOCK * sizeof(float) : 0;
      NT_TRY(check_array("param", t.param, n * esize(dtype)));
      NT_TRY(check_array("grad", t.grad, n * sizeof(float)));
      if (t.master) NT_TRY(check_array("master", t.master, n * sizeof(float)));
      NT_TRY(check_array("m", t.m, state));
      NT_TRY(check_array("v", t.v, state));
      NT_TRY(check_array("m_scale", t.m_scale, scale));
      NT_TRY(check_array("v_scale", t.v_scale, scale));
      add(t.param, n * esize(dtype), true, i);
      add(t.grad, n * sizeof(float), false, i);
      add(t.master, n * sizeof(float), true, i);
      add(t.m, state, true, i);
      add(t.v, state, true, i);
      add(t.m_scale, scale, true, i);
      add(t.v_scale, scale, true, i);
    }
    add(h->step_device, sizeof(int64_t), false, -1);
    add(h->lr_device, sizeof(float), false, -1);
    std::sort(spans.begin(), spans.end(),
              [](const Span& a, const Span& b) { return a.at < b.at; });
    // the furthest ends so far, of all spans and of the written ones
    uintptr_t any = 0, written = 0;
    for (const Span& s : spans) {
      if (s.at < written || (s.written && s.at < any))
        return fail(NT_ERR_INVALID, "an array of tensor %d overlaps another one", s.tensor);
      any = std::max(any, s.end);
      if (s.written) written = std::max(written, s.end);
    }
  } catch (const std::bad_alloc&) {
    return fail(NT_ERR_INVALID, "no host memory to check %d tensors", (int)count);
  }
  return hip_status(nt::launch_adamw(tensors, count, *h, dtype, static_cast<hipStream_t>(stream)),
                    "AdamW kernel");
}

}  // extern "C"
