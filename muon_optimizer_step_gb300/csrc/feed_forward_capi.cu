// C entry points of the feed-forward operators around the expert layer: argument checks, then one
// launcher call on the caller's stream.
#include <cmath>

#include "capi_checks.h"

using namespace muon;

namespace {

muon_status check_rows(int64_t rows) {
  if (rows < 0 || rows > INT32_MAX)
    return fail(MUON_ERR_INVALID_ARG, "rows=%lld outside 0..2^31-1", (long long)rows);
  return MUON_OK;
}

// A float vector that may be NULL.
muon_status check_floats(const void* p, const char* name) {
  return p == nullptr ? MUON_OK : check_ptr(p, sizeof(float), name);
}

// One operand pair of a product: x (rows x k) and a weight for every expert.
muon_status check_operands(const GroupedMm& g, const void* x, int64_t ldx, const void* w, int64_t ldw,
                           int64_t w_stride, const char* const* names) {
  EXPERT_TRY(check_pitch(ldx, g.k, names[1]));
  EXPERT_TRY(check_pitch(ldw, g.trans ? g.k : g.n, names[3]));
  if (g.n_experts > 1) EXPERT_TRY(check_pitch(w_stride, 1, names[4]));
  if (g.rows > 0) {
    EXPERT_TRY(check_ptr(x, 2, names[0]));
    EXPERT_TRY(check_ptr(w, 2, names[2]));
  }
  return MUON_OK;
}

// What the products check before their operands.
muon_status check_product(const GroupedMm& g) {
  EXPERT_TRY(check_groups(g.rows, g.n_experts));
  EXPERT_TRY(check_16bit(g.dtype, "dtype"));
  EXPERT_TRY(check_dim(g.k, "k"));
  EXPERT_TRY(check_dim(g.n, "n"));
  if (!gated_mm_fits(g)) return fail(MUON_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles of the result");
  return MUON_OK;
}

muon_status check_offsets(const GroupedMm& g) {
  if (g.offsets != nullptr) return check_ptr(g.offsets, sizeof(int64_t), "row_offsets");
  if (g.n_experts != 1)
    return fail(MUON_ERR_INVALID_ARG, "row_offsets is NULL: n_experts=%d must be 1", g.n_experts);
  return MUON_OK;
}

// A matrix of rows x cols elements; NULL where `may` says so.
muon_status check_matrix(const void* p, int64_t ld, int64_t rows, int32_t cols, int32_t dtype, bool may,
                         const char* name) {
  if (p == nullptr && may) return MUON_OK;
  EXPERT_TRY(check_pitch(ld, cols, name));
  return rows > 0 ? check_ptr(p, dtype_size(dtype), name) : MUON_OK;
}

muon_status check_gated(const GatedMm& g) {
  static const char* const a[] = {"x", "ldx", "w_gate", "ldw_gate", "w_gate_stride"};
  static const char* const b[] = {"x", "ldx", "w_up", "ldw_up", "w_up_stride"};
  EXPERT_TRY(check_product(g));
  EXPERT_TRY(check_operands(g, g.x, g.ldx, g.w, g.ldw, g.w_stride, a));
  return check_operands(g, g.x, g.ldx, g.w2, g.ldw2, g.w2_stride, b);
}

muon_status check_gated_grad(const GatedGrad& g) {
  static const char* const a[] = {"dy", "lddy", "w", "ldw", "w_stride"};
  EXPERT_TRY(check_product(g));
  return check_operands(g, g.x, g.ldx, g.w, g.ldw, g.w_stride, a);
}

muon_status check_sum(const MmSum& g) {
  static const char* const a[] = {"x1", "ldx1", "w1", "ldw1", "w1_stride"};
  static const char* const b[] = {"x2", "ldx2", "w2", "ldw2", "w2_stride"};
  EXPERT_TRY(check_product(g));
  EXPERT_TRY(check_operands(g, g.x, g.ldx, g.w, g.ldw, g.w_stride, a));
  return check_operands(g, g.x2, g.ldx2, g.w2, g.ldw2, g.w2_stride, b);
}

void set_product(GroupedMm* g, const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t w_stride,
                 int64_t rows, int32_t n_experts, int32_t k, int32_t n, int32_t trans_w, int32_t dtype) {
  *g = GroupedMm{x, w, nullptr, nullptr, ldx, ldw, w_stride, n, rows, n_experts, k, n,
                 trans_w ? 1 : 0, dtype, dtype, nullptr};
}

}  // namespace

extern "C" {

muon_status muon_layer_norm(const void* x, int64_t ldx, const float* weight, const float* bias, void* y,
                            int64_t ldy, float* mean, float* rstd, int64_t rows, int32_t cols, float eps,
                            int32_t dtype, cudaStream_t stream) {
  EXPERT_TRY(check_dtype(dtype, "dtype"));
  EXPERT_TRY(check_rows(rows));
  EXPERT_TRY(check_dim(cols, "cols"));
  EXPERT_TRY(check_pitch(ldx, cols, "ldx"));
  EXPERT_TRY(check_pitch(ldy, cols, "ldy"));
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return fail(MUON_ERR_INVALID_ARG, "eps must be finite and not negative");
  EXPERT_TRY(check_floats(weight, "weight"));
  EXPERT_TRY(check_floats(bias, "bias"));
  EXPERT_TRY(check_floats(mean, "mean"));
  EXPERT_TRY(check_floats(rstd, "rstd"));
  if (rows > 0) {
    EXPERT_TRY(check_ptr(x, dtype_size(dtype), "x"));
    EXPERT_TRY(check_ptr(y, dtype_size(dtype), "y"));
  }
  Device d;
  EXPERT_TRY(current_device(&d));
  if (rows == 0) return done(cudaSuccess, "");
  NormArgs a{};
  a.x = x;
  a.out = y;
  a.w = weight;
  a.b = bias;
  a.mean = mean;
  a.rstd = rstd;
  a.ldx = ldx;
  a.ldo = ldy;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  return done(launch_layer_norm(a, dtype, d.sms, stream), "layer norm");
}

muon_status muon_layer_norm_grad_workspace_bytes(int64_t rows, int32_t cols, size_t* bytes) {
  if (bytes == nullptr) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  EXPERT_TRY(check_rows(rows));
  EXPERT_TRY(check_dim(cols, "cols"));
  *bytes = norm_grad_workspace(rows, cols);
  return done(cudaSuccess, "");
}

muon_status muon_layer_norm_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                 const float* weight, const float* mean, const float* rstd, void* dx,
                                 int64_t lddx, float* dweight, float* dbias, int64_t rows, int32_t cols,
                                 int32_t accumulate, int32_t dtype, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  EXPERT_TRY(check_dtype(dtype, "dtype"));
  EXPERT_TRY(check_rows(rows));
  EXPERT_TRY(check_dim(cols, "cols"));
  EXPERT_TRY(check_pitch(lddy, cols, "lddy"));
  EXPERT_TRY(check_pitch(ldx, cols, "ldx"));
  EXPERT_TRY(check_pitch(lddx, cols, "lddx"));
  EXPERT_TRY(check_floats(weight, "weight"));
  EXPERT_TRY(check_floats(dweight, "dweight"));
  EXPERT_TRY(check_floats(dbias, "dbias"));
  if (rows > 0) {
    EXPERT_TRY(check_ptr(dy, dtype_size(dtype), "dy"));
    EXPERT_TRY(check_ptr(x, dtype_size(dtype), "x"));
    EXPERT_TRY(check_ptr(dx, dtype_size(dtype), "dx"));
    EXPERT_TRY(check_ptr(mean, sizeof(float), "mean"));
    EXPERT_TRY(check_ptr(rstd, sizeof(float), "rstd"));
  }
  if (dweight != nullptr || dbias != nullptr) {
    const size_t need = norm_grad_workspace(rows, cols);
    if (workspace_bytes < need)
      return fail(MUON_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
    if (need > 0) EXPERT_TRY(check_ptr(workspace, 16, "workspace"));
  }
  Device d;
  EXPERT_TRY(current_device(&d));
  NormArgs a{};
  a.x = x;
  a.dy = dy;
  a.out = dx;
  a.w = weight;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.dw = dweight;
  a.db = dbias;
  a.part = static_cast<float*>(workspace);
  a.ldx = ldx;
  a.lddy = lddy;
  a.ldo = lddx;
  a.rows = rows;
  a.cols = cols;
  a.accumulate = accumulate ? 1 : 0;
  return done(launch_layer_norm_grad(a, dtype, d.sms, stream), "layer norm gradient");
}

muon_status muon_gated_mm_workspace_bytes(const void* x, int64_t ldx, const void* w_gate, int64_t ldw_gate,
                                          int64_t w_gate_stride, const void* w_up, int64_t ldw_up,
                                          int64_t w_up_stride, int64_t rows, int32_t n_experts, int32_t k,
                                          int32_t n, int32_t trans_w, size_t* bytes) {
  if (bytes == nullptr) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  GatedMm g{};
  set_product(&g, x, ldx, w_gate, ldw_gate, w_gate_stride, rows, n_experts, k, n, trans_w, kBf16);
  g.w2 = w_up;
  g.ldw2 = ldw_up;
  g.w2_stride = w_up_stride;
  EXPERT_TRY(check_gated(g));
  *bytes = gated_mm_workspace(g);
  return done(cudaSuccess, "");
}

muon_status muon_gated_mm(const void* x, int64_t ldx, const void* w_gate, int64_t ldw_gate,
                          int64_t w_gate_stride, const void* w_up, int64_t ldw_up, int64_t w_up_stride,
                          const int64_t* row_offsets, const float* row_weight, void* out, int64_t ld_out,
                          void* gate, int64_t ld_gate, void* up, int64_t ld_up, int64_t rows,
                          int32_t n_experts, int32_t k, int32_t n, int32_t trans_w, int32_t dtype,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  GatedMm g{};
  set_product(&g, x, ldx, w_gate, ldw_gate, w_gate_stride, rows, n_experts, k, n, trans_w, dtype);
  g.w2 = w_up;
  g.ldw2 = ldw_up;
  g.w2_stride = w_up_stride;
  g.offsets = row_offsets;
  g.p = row_weight;
  g.y = out;
  g.ldy = ld_out;
  g.gate = gate;
  g.ld_gate = ld_gate;
  g.up = up;
  g.ld_up = ld_up;
  EXPERT_TRY(check_gated(g));
  EXPERT_TRY(check_offsets(g));
  EXPERT_TRY(check_floats(row_weight, "row_weight"));
  EXPERT_TRY(check_matrix(out, ld_out, rows, n, dtype, false, "out"));
  EXPERT_TRY(check_matrix(gate, ld_gate, rows, n, dtype, true, "gate"));
  EXPERT_TRY(check_matrix(up, ld_up, rows, n, dtype, true, "up"));
  EXPERT_TRY(check_workspace(workspace, workspace_bytes, gated_mm_workspace(g)));
  Device d;
  EXPERT_TRY(current_device(&d));
  if (rows == 0) return done(cudaSuccess, "");
  g.err = d.err;
  return done(launch_gated_mm(g, workspace, d.sms, stream), "gated product");
}

muon_status muon_gated_mm_grad_workspace_bytes(const void* dy, int64_t lddy, const void* w, int64_t ldw,
                                               int64_t w_stride, int64_t rows, int32_t n_experts,
                                               int32_t k, int32_t n, int32_t trans_w,
                                               int32_t row_weight_grad, size_t* bytes) {
  if (bytes == nullptr) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  GatedGrad g{};
  set_product(&g, dy, lddy, w, ldw, w_stride, rows, n_experts, k, n, trans_w, kBf16);
  EXPERT_TRY(check_gated_grad(g));
  *bytes = gated_grad_workspace(g, row_weight_grad != 0);
  return done(cudaSuccess, "");
}

muon_status muon_gated_mm_grad(const void* dy, int64_t lddy, const void* w, int64_t ldw, int64_t w_stride,
                               const int64_t* row_offsets, const void* gate, int64_t ld_gate,
                               const void* up, int64_t ld_up, const float* row_weight, void* dgate,
                               int64_t ld_dgate, void* dup, int64_t ld_dup, void* out, int64_t ld_out,
                               float* d_row_weight, int64_t rows, int32_t n_experts, int32_t k, int32_t n,
                               int32_t trans_w, int32_t dtype, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  GatedGrad g{};
  set_product(&g, dy, lddy, w, ldw, w_stride, rows, n_experts, k, n, trans_w, dtype);
  g.offsets = row_offsets;
  g.gate = gate;
  g.ld_gate = ld_gate;
  g.up = up;
  g.ld_up = ld_up;
  g.p = row_weight;
  g.dgate = dgate;
  g.ld_dgate = ld_dgate;
  g.dup = dup;
  g.ld_dup = ld_dup;
  g.y = out;
  g.ldy = ld_out;
  g.dp = d_row_weight;
  EXPERT_TRY(check_gated_grad(g));
  EXPERT_TRY(check_offsets(g));
  EXPERT_TRY(check_matrix(gate, ld_gate, rows, n, dtype, false, "gate"));
  EXPERT_TRY(check_matrix(up, ld_up, rows, n, dtype, false, "up"));
  EXPERT_TRY(check_matrix(dgate, ld_dgate, rows, n, dtype, false, "dgate"));
  EXPERT_TRY(check_matrix(dup, ld_dup, rows, n, dtype, false, "dup"));
  EXPERT_TRY(check_matrix(out, ld_out, rows, n, dtype, true, "out"));
  EXPERT_TRY(check_floats(row_weight, "row_weight"));
  EXPERT_TRY(check_floats(d_row_weight, "d_row_weight"));
  EXPERT_TRY(check_workspace(workspace, workspace_bytes, gated_grad_workspace(g, d_row_weight != nullptr)));
  Device d;
  EXPERT_TRY(current_device(&d));
  if (rows == 0) return done(cudaSuccess, "");
  g.err = d.err;
  return done(launch_gated_grad(g, workspace, d.sms, stream), "gated product's gradient");
}

muon_status muon_grouped_mm_sum_workspace_bytes(const void* x1, int64_t ldx1, const void* w1, int64_t ldw1,
                                                int64_t w1_stride, const void* x2, int64_t ldx2,
                                                const void* w2, int64_t ldw2, int64_t w2_stride,
                                                int64_t rows, int32_t n_experts, int32_t k, int32_t n,
                                                int32_t trans_w, size_t* bytes) {
  if (bytes == nullptr) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
  MmSum g{};
  set_product(&g, x1, ldx1, w1, ldw1, w1_stride, rows, n_experts, k, n, trans_w, kBf16);
  g.x2 = x2;
  g.ldx2 = ldx2;
  g.w2 = w2;
  g.ldw2 = ldw2;
  g.w2_stride = w2_stride;
  EXPERT_TRY(check_sum(g));
  *bytes = mm_sum_workspace(g);
  return done(cudaSuccess, "");
}

muon_status muon_grouped_mm_sum(const void* x1, int64_t ldx1, const void* w1, int64_t ldw1,
                                int64_t w1_stride, const void* x2, int64_t ldx2, const void* w2,
                                int64_t ldw2, int64_t w2_stride, const int64_t* row_offsets, void* y,
                                int64_t ldy, int64_t rows, int32_t n_experts, int32_t k, int32_t n,
                                int32_t trans_w, int32_t dtype, int32_t out_dtype, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream) {
  MmSum g{};
  set_product(&g, x1, ldx1, w1, ldw1, w1_stride, rows, n_experts, k, n, trans_w, dtype);
  g.x2 = x2;
  g.ldx2 = ldx2;
  g.w2 = w2;
  g.ldw2 = ldw2;
  g.w2_stride = w2_stride;
  g.offsets = row_offsets;
  g.y = y;
  g.ldy = ldy;
  g.out_dtype = out_dtype;
  EXPERT_TRY(check_sum(g));
  EXPERT_TRY(check_offsets(g));
  if (out_dtype != dtype && out_dtype != MUON_DTYPE_F32)
    return fail(MUON_ERR_INVALID_ARG, "out_dtype=%d: the inputs' type (%d) or fp32", out_dtype, dtype);
  EXPERT_TRY(check_matrix(y, ldy, rows, n, out_dtype, false, "y"));
  EXPERT_TRY(check_workspace(workspace, workspace_bytes, mm_sum_workspace(g)));
  Device d;
  EXPERT_TRY(current_device(&d));
  if (rows == 0) return done(cudaSuccess, "");
  g.err = d.err;
  return done(launch_mm_sum(g, workspace, d.sms, stream), "sum of two grouped products");
}

muon_status muon_quantize_rows(const void* x, int64_t ldx, void* q, int64_t ldq, float* scale,
                               int64_t ld_scale, int64_t rows, int32_t cols, int32_t dtype,
                               cudaStream_t stream) {
  EXPERT_TRY(check_dtype(dtype, "dtype"));
  EXPERT_TRY(check_rows(rows));
  EXPERT_TRY(check_dim(cols, "cols"));
  EXPERT_TRY(check_matrix(x, ldx, rows, cols, dtype, false, "x"));
  EXPERT_TRY(check_pitch(ldq, cols, "ldq"));
  EXPERT_TRY(check_pitch(ld_scale, rows, "ld_scale"));
  if (rows > 0) {
    EXPERT_TRY(check_ptr(q, 1, "q"));
    EXPERT_TRY(check_ptr(scale, sizeof(float), "scale"));
  }
  Device d;
  EXPERT_TRY(current_device(&d));
  if (rows == 0) return done(cudaSuccess, "");
  const QuantizeRows a{x, static_cast<uint8_t*>(q), scale, ldx, ldq, ld_scale, rows, cols};
  return done(launch_quantize_rows(a, dtype, d.sms, stream), "quantization of rows");
}

muon_status muon_quantize_weights(const void* w, int64_t ldw, int64_t w_stride, void* q, int64_t ldq,
                                  int64_t q_stride, float* scale, int32_t n, int32_t rows, int32_t cols,
                                  int32_t transpose, int32_t dtype, cudaStream_t stream) {
  EXPERT_TRY(check_dtype(dtype, "dtype"));
  EXPERT_TRY(check_groups(0, n));
  EXPERT_TRY(check_dim(rows, "rows"));
  EXPERT_TRY(check_dim(cols, "cols"));
  EXPERT_TRY(check_matrix(w, ldw, rows, cols, dtype, false, "w"));
  const int64_t q_rows = transpose ? cols : rows, q_cols = transpose ? rows : cols;
  EXPERT_TRY(check_pitch(ldq, q_cols, "ldq"));
  if (n > 1) {
    EXPERT_TRY(check_pitch(w_stride, 1, "w_stride"));
    if (q_stride < q_cols || (q_stride - q_cols) / ldq < q_rows - 1 || q_stride >= (int64_t)1 << 52)
      return fail(MUON_ERR_INVALID_ARG, "q_stride=%lld: matrices of q overlap or lie too far apart",
                  (long long)q_stride);
  }
  EXPERT_TRY(check_ptr(q, 1, "q"));
  EXPERT_TRY(check_ptr(scale, sizeof(float), "scale"));
  Device d;
  EXPERT_TRY(current_device(&d));
  const QuantizeWeights a{w,        static_cast<uint8_t*>(q), scale, ldw,  w_stride, ldq,
                          q_stride, n,                        rows,  cols, transpose ? 1 : 0, false};
  return done(launch_quantize_weights(a, dtype, d.sms, stream), "quantization of weights");
}

muon_status muon_grouped_mm_fp8(const void* x, int64_t ldx, const float* x_scale, int64_t ld_x_scale,
                                const void* w, int64_t ldw, int64_t w_stride, const float* w_scale,
                                const int64_t* row_offsets, void* y, int64_t ldy, int64_t rows,
                                int32_t n_experts, int32_t k, int32_t n, int32_t out_dtype,
                                cudaStream_t stream) {
  Fp8Mm g{};
  set_product(&g, x, ldx, w, ldw, w_stride, rows, n_experts, k, n, 1, MUON_DTYPE_BF16);
  g.offsets = row_offsets;
  g.x_scale = x_scale;
  g.ld_x_scale = ld_x_scale;
  g.w_scale = w_scale;
  g.y = y;
  g.ldy = ldy;
  g.out_dtype = out_dtype;
  EXPERT_TRY(check_product(g));
  EXPERT_TRY(check_offsets(g));
  EXPERT_TRY(check_dtype(out_dtype, "out_dtype"));
  EXPERT_TRY(check_pitch(ldx, k, "ldx"));
  EXPERT_TRY(check_pitch(ldw, k, "ldw"));
  if (n_experts > 1) EXPERT_TRY(check_pitch(w_stride, 1, "w_stride"));
  EXPERT_TRY(check_pitch(ld_x_scale, rows, "ld_x_scale"));
  if ((rows > 1 && ldx % 16 != 0) || (n > 1 && ldw % 16 != 0) || (n_experts > 1 && w_stride % 16 != 0))
    return fail(MUON_ERR_ALIGNMENT, "ldx=%lld, ldw=%lld, w_stride=%lld: rows must start on 16 bytes",
                (long long)ldx, (long long)ldw, (long long)w_stride);
  EXPERT_TRY(check_matrix(y, ldy, rows, n, out_dtype, false, "y"));
  if (rows > 0) {
    EXPERT_TRY(check_ptr(x, 16, "x"));
    EXPERT_TRY(check_ptr(w, 16, "w"));
    EXPERT_TRY(check_ptr(x_scale, sizeof(float), "x_scale"));
    EXPERT_TRY(check_ptr(w_scale, sizeof(float), "w_scale"));
  }
  Device d;
  EXPERT_TRY(current_device(&d));
  if (rows == 0) return done(cudaSuccess, "");
  g.err = d.err;
  return done(launch_fp8_mm(g, d.sms, stream), "8-bit grouped product");
}

}  // extern "C"
