// C entry points of the expert layer (grouped products, gated activation) and of the global
// gradient norm: argument checks, then one launcher call on the caller's stream.
#include <cmath>

#include "capi_checks.h"

using namespace muon;

namespace {

static_assert(sizeof(TensorSpec) == sizeof(muon_tensor), "muon_tensor and TensorSpec must agree");

// What muon_grouped_mm and its workspace query both check.
muon_status check_mm(const GroupedMm& g) {
  EXPERT_TRY(check_dim(g.k, "k"));
  EXPERT_TRY(check_dim(g.n, "n"));
  EXPERT_TRY(check_pitch(g.ldx, g.k, "ldx"));
  EXPERT_TRY(check_pitch(g.ldw, g.trans ? g.k : g.n, "ldw"));
  EXPERT_TRY(check_pitch(g.ldy, g.n, "ldy"));
  if (g.n_experts > 1) EXPERT_TRY(check_pitch(g.w_stride, 1, "w_stride"));
  if (!grouped_mm_fits(g)) return fail(MUON_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles of y");
  if (g.rows > 0) {
    EXPERT_TRY(check_ptr(g.x, 2, "x"));
    EXPERT_TRY(check_ptr(g.w, 2, "w"));
  }
  return MUON_OK;
}

// Whether no two rows of dw share an element: experts one behind the other, rows of all experts
// side by side, or every distance between rows of two experts looked at.
bool rows_apart(const GroupedWgrad& g) {
  if (g.m - 1 <= (g.dw_stride - g.n) / g.lddw || g.n_experts - 1 <= (g.lddw - g.n) / g.dw_stride)
    return true;
  for (int64_t e = 1; e < g.n_experts; ++e) {
    const int64_t q = e * g.dw_stride / g.lddw, r = e * g.dw_stride - q * g.lddw;
    if ((q < g.m && r < g.n) || (q + 1 < g.m && g.lddw - r < g.n)) return false;
  }
  return true;
}

muon_status check_wgrad(const GroupedWgrad& g) {
  EXPERT_TRY(check_dim(g.m, "m"));
  EXPERT_TRY(check_dim(g.n, "n"));
  EXPERT_TRY(check_pitch(g.lda, g.m, "lda"));
  EXPERT_TRY(check_pitch(g.ldb, g.n, "ldb"));
  EXPERT_TRY(check_pitch(g.lddw, g.n, "lddw"));
  if (g.n_experts > 1) EXPERT_TRY(check_pitch(g.dw_stride, g.n, "dw_stride"));
  if (!grouped_wgrad_fits(g)) return fail(MUON_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles of dw");
  if (g.n_experts > 1 && !rows_apart(g))
    return fail(MUON_ERR_INVALID_ARG, "lddw=%lld and dw_stride=%lld: rows of dw overlap",
                (long long)g.lddw, (long long)g.dw_stride);
  if (g.rows > 0) {
    EXPERT_TRY(check_ptr(g.a, 2, "a"));
    EXPERT_TRY(check_ptr(g.b, 2, "b"));
  }
  return MUON_OK;
}

muon_status check_swiglu(const SwigluArgs& s, const char* const* names, const float* p, int64_t rows,
                         int32_t cols, int32_t dtype) {
  EXPERT_TRY(check_dtype(dtype, "dtype"));
  EXPERT_TRY(check_dim(cols, "cols"));
  if (rows < 0 || rows > INT32_MAX)
    return fail(MUON_ERR_INVALID_ARG, "rows=%lld outside 0..2^31-1", (long long)rows);
  for (int i = 0; i < s.n; ++i) {
    if (rows > 0) EXPERT_TRY(check_ptr(s.ptr[i], dtype_size(dtype), names[i]));
    EXPERT_TRY(check_pitch(s.ld[i], cols, names[i]));
  }
  if (p != nullptr) EXPERT_TRY(check_ptr(p, sizeof(float), "row_weight"));
  return MUON_OK;
}

// Lists of up to 2^45 elements (more than any device holds), so that their chunks and bytes count in
// 64 bits.
muon_status check_tensors(const muon_tensor* t, int32_t n, const char* name) {
  constexpr int64_t kMost = (int64_t)1 << 45;
  int64_t all = 0;
  if (n < 0) return fail(MUON_ERR_INVALID_ARG, "n=%d is negative", n);
  if (n > 0 && t == nullptr) return fail(MUON_ERR_INVALID_ARG, "%s is NULL", name);
  for (int32_t i = 0; i < n; ++i) {
    if (t[i].dtype < MUON_DTYPE_F32 || t[i].dtype > MUON_DTYPE_F16)
      return fail(MUON_ERR_INVALID_ARG, "%s[%d].dtype=%d is no muon_dtype", name, i, t[i].dtype);
    if (t[i].numel < 0)
      return fail(MUON_ERR_INVALID_ARG, "%s[%d].numel=%lld is negative", name, i,
                  (long long)t[i].numel);
    if (t[i].numel > kMost || (all += t[i].numel) > kMost)
      return fail(MUON_ERR_UNSUPPORTED, "%s: more elements than one call takes", name);
    if (t[i].numel == 0) continue;
    if (t[i].data == nullptr) return fail(MUON_ERR_INVALID_ARG, "%s[%d].data is NULL", name, i);
    if (reinterpret_cast<uintptr_t>(t[i].data) % dtype_size(t[i].dtype) != 0)
      return fail(MUON_ERR_ALIGNMENT, "%s[%d].data = %p is not aligned to its elements", name, i,
                  t[i].data);
  }
  return MUON_OK;
}

muon_status clip(const muon_tensor* grads, const muon_tensor* outs, bool scale, int32_t n,
                 float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                 cudaStream_t stream) {
  EXPERT_TRY(check_tensors(grads, n, "grads"));
  if (scale) {
    EXPERT_TRY(check_tensors(outs, n, "outs"));
    for (int32_t i = 0; i < n; ++i) {
      if (outs[i].numel != grads[i].numel)
        return fail(MUON_ERR_INVALID_ARG, "outs[%d] has %lld elements, grads[%d] %lld", i,
                    (long long)outs[i].numel, i, (long long)grads[i].numel);
      if (outs[i].dtype != grads[i].dtype && outs[i].dtype != MUON_DTYPE_F32)
        return fail(MUON_ERR_INVALID_ARG, "outs[%d].dtype=%d: grads[%d]'s (%d) or fp32", i,
                    outs[i].dtype, i, grads[i].dtype);
      if (outs[i].data == grads[i].data && outs[i].dtype != grads[i].dtype && outs[i].numel > 0)
        return fail(MUON_ERR_INVALID_ARG, "outs[%d] is grads[%d] in another type", i, i);
    }
  }
  if (!(max_norm >= 0.f) || !std::isfinite(max_norm))
    return fail(MUON_ERR_INVALID_ARG, "max_norm must be finite and not negative");
  EXPERT_TRY(check_ptr(norm, sizeof(float), "norm"));
  Device d;
  EXPERT_TRY(current_device(&d));
  const TensorSpec* g = reinterpret_cast<const TensorSpec*>(grads);
  if (clip_chunks(g, n) > INT32_MAX)
    return fail(MUON_ERR_UNSUPPORTED, "more elements than one call takes");
  const size_t need = clip_workspace_bytes(g, n, d.sms);
  if (workspace_bytes < need)
    return fail(MUON_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
  if (need > 0) EXPERT_TRY(check_ptr(workspace, sizeof(double), "workspace"));
  return done(launch_clip(g, scale ? reinterpret_cast<const TensorSpec*>(outs) : nullptr, n,
                          max_norm, norm, workspace, d.sms, stream),
              "gradient norm");
}

}  // namespace

extern "C" {

muon_status muon_grouped_mm_workspace_bytes(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                            int64_t w_stride, int64_t rows, int32_t n_experts,
                                            int32_t k, int32_t n, int32_t trans_w, size_t* bytes) {
  if (bytes == nullptr) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  EXPERT_TRY(check_groups(rows, n_experts));
  const GroupedMm g{x, w, nullptr, nullptr, ldx, ldw, w_stride, n, rows, n_experts, k, n,
                    trans_w ? 1 : 0, 0, 0, nullptr};
  EXPERT_TRY(check_mm(g));
  *bytes = grouped_mm_workspace(g);
  return done(cudaSuccess, "");
}

muon_status muon_grouped_mm(const void* x, int64_t ldx, const void* w, int64_t ldw,
                            int64_t w_stride, const int64_t* row_offsets, void* y, int64_t ldy,
                            int64_t rows, int32_t n_experts, int32_t k, int32_t n, int32_t trans_w,
                            int32_t dtype, int32_t out_dtype, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  EXPERT_TRY(check_groups(rows, n_experts));
  EXPERT_TRY(check_ptr(row_offsets, sizeof(int64_t), "row_offsets"));
  EXPERT_TRY(check_16bit(dtype, "dtype"));
  if (out_dtype != dtype && out_dtype != MUON_DTYPE_F32)
    return fail(MUON_ERR_INVALID_ARG, "out_dtype=%d: the inputs' type (%d) or fp32", out_dtype, dtype);
  GroupedMm g{x, w, y, row_offsets, ldx, ldw, w_stride, ldy, rows, n_experts, k, n,
              trans_w ? 1 : 0, dtype, out_dtype, nullptr};
  EXPERT_TRY(check_mm(g));
  if (rows > 0) EXPERT_TRY(check_ptr(y, dtype_size(out_dtype), "y"));
  EXPERT_TRY(check_workspace(workspace, workspace_bytes, grouped_mm_workspace(g)));
  Device d;
  EXPERT_TRY(current_device(&d));
  if (rows == 0) return done(cudaSuccess, "");
  g.err = d.err;
  return done(launch_grouped_mm(g, workspace, d.sms, stream), "grouped product");
}

muon_status muon_grouped_wgrad_workspace_bytes(const void* a, int64_t lda, const void* b,
                                               int64_t ldb, int64_t rows, int32_t m, int32_t n,
                                               size_t* bytes) {
  if (bytes == nullptr) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  EXPERT_TRY(check_groups(rows, 1));
  const GroupedWgrad g{a, b, nullptr, nullptr, lda, ldb, n, 0, rows, 1, m, n, 0, 0, nullptr};
  EXPERT_TRY(check_wgrad(g));
  *bytes = grouped_wgrad_workspace(g);
  return done(cudaSuccess, "");
}

muon_status muon_grouped_wgrad(const void* a, int64_t lda, const void* b, int64_t ldb,
                               const int64_t* row_offsets, float* dw, int64_t lddw,
                               int64_t dw_stride, int64_t rows, int32_t n_experts, int32_t m,
                               int32_t n, int32_t accumulate, int32_t dtype, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
  EXPERT_TRY(check_groups(rows, n_experts));
  EXPERT_TRY(check_ptr(row_offsets, sizeof(int64_t), "row_offsets"));
  EXPERT_TRY(check_16bit(dtype, "dtype"));
  GroupedWgrad g{a, b, dw, row_offsets, lda, ldb, lddw, dw_stride, rows, n_experts, m, n,
                 accumulate ? 1 : 0, dtype, nullptr};
  EXPERT_TRY(check_wgrad(g));
  EXPERT_TRY(check_ptr(dw, sizeof(float), "dw"));
  EXPERT_TRY(check_workspace(workspace, workspace_bytes, grouped_wgrad_workspace(g)));
  Device d;
  EXPERT_TRY(current_device(&d));
  g.err = d.err;
  return done(launch_grouped_wgrad(g, workspace, d.sms, stream), "grouped weight gradient");
}

muon_status muon_swiglu(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up,
                        const float* row_weight, void* out, int64_t ld_out, int64_t rows,
                        int32_t cols, int32_t dtype, cudaStream_t stream) {
  const SwigluArgs s{3, {const_cast<void*>(gate), const_cast<void*>(up), out},
                     {ld_gate, ld_up, ld_out}};
  static const char* const names[] = {"gate", "up", "out"};
  EXPERT_TRY(check_swiglu(s, names, row_weight, rows, cols, dtype));
  Device d;
  EXPERT_TRY(current_device(&d));
  if (rows == 0) return done(cudaSuccess, "");
  return done(launch_swiglu(s, dtype, row_weight, nullptr, rows, cols, d.sms, stream), "swiglu");
}

muon_status muon_swiglu_grad(const void* dout, int64_t ld_dout, const void* gate, int64_t ld_gate,
                             const void* up, int64_t ld_up, const float* row_weight, void* dgate,
                             int64_t ld_dgate, void* dup, int64_t ld_dup, float* d_row_weight,
                             int64_t rows, int32_t cols, int32_t dtype, cudaStream_t stream) {
  const SwigluArgs s{5,
                     {const_cast<void*>(dout), const_cast<void*>(gate), const_cast<void*>(up), dgate,
                      dup},
                     {ld_dout, ld_gate, ld_up, ld_dgate, ld_dup}};
  static const char* const names[] = {"dout", "gate", "up", "dgate", "dup"};
  EXPERT_TRY(check_swiglu(s, names, row_weight, rows, cols, dtype));
  if (d_row_weight != nullptr) EXPERT_TRY(check_ptr(d_row_weight, sizeof(float), "d_row_weight"));
  Device d;
  EXPERT_TRY(current_device(&d));
  if (rows == 0) return done(cudaSuccess, "");
  return done(launch_swiglu(s, dtype, row_weight, d_row_weight, rows, cols, d.sms, stream),
              "swiglu gradient");
}

muon_status muon_clip_workspace_bytes(const muon_tensor* grads, int32_t n, size_t* bytes) {
  if (bytes == nullptr) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  EXPERT_TRY(check_tensors(grads, n, "grads"));
  Device d;
  EXPERT_TRY(current_device(&d));
  *bytes = clip_workspace_bytes(reinterpret_cast<const TensorSpec*>(grads), n, d.sms);
  return done(cudaSuccess, "");
}

muon_status muon_grad_norm(const muon_tensor* grads, int32_t n, float max_norm, float* norm,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return clip(grads, nullptr, false, n, max_norm, norm, workspace, workspace_bytes, stream);
}

muon_status muon_clip_grads(const muon_tensor* grads, const muon_tensor* outs, int32_t n,
                            float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  return clip(grads, outs, true, n, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
