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

}  // extern "C"
