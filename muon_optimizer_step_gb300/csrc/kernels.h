// Host-side launchers of the kernels (one translation unit each) used by capi.cu.
#pragma once

#include <cuda_runtime.h>
#include <cuda.h>

#include <string>

#include "muon_internal.h"

namespace muon {

struct ShardPtrs;
struct ApplyArgs;
struct GroupParams;
struct DebugCtx;

// Tile shapes of the tcgen05 Newton-Schulz kernels (the values MUON_TC_KERNEL pins and
// muon_layout_ns_kernel reports).
constexpr int kShapeSingle = 1;  // one CTA per 128 x 256 tile, tcgen05 cta_group::1
constexpr int kShapePair = 2;    // 2-CTA cluster per 256 x 256 tile, tcgen05 cta_group::2
constexpr int kShapePairWide = 3;  // 2-CTA cluster per 256 x 512 tile: two cta_group::2
                                   // MMAs of N = 256 per k-step into one 512-column accumulator

// Device-resident tables of a layout (uploaded once per device).
struct DevTables {
  int device = -1;
  int n_sms = 0;
  ChunkDev* chunks = nullptr;
  MatDev* mats = nullptr;
  int* err = nullptr;           // device error word (MUON_ERR_TIMEOUT when a wait gave up)
  // fp32 path: one tile list per phase
  TileDev* tiles[3] = {nullptr, nullptr, nullptr};
  int32_t* cta_begin[3] = {nullptr, nullptr, nullptr};
  int64_t n_tiles[3] = {0, 0, 0};  // entries of each phase's tile list
  int grid[3] = {0, 0, 0};
  // Tensor-core paths: tc_lists tile lists back to back in tc_tiles; list l's offsets for
  // unit u are tc_begin[l * (tc_units + 1) + u] and the next entry.  One list per phase,
  // or, for a persistent launch, one per iteration and phase (q = 3 * it + phase), the
  // last iteration's lists serving any later one.
  TileDev* tc_tiles = nullptr;
  int32_t* tc_begin = nullptr;
  int tc_lists = 0;
  int64_t tc_n_tiles = 0;
  CUtensorMap* tmaps = nullptr; // kMapsPerMat per matrix (bf16 path)
  int tc_shape = kShapeSingle;  // bf16 path: tile shape (kShape*)
  bool tc_persistent = false;   // bf16 path: all phases in one launch
  bool fused_tail = false;      // tensor-core paths: the last Update applies W itself
  int tc_units = 0;             // tensor-core paths: CTAs (or pairs) of each launch
  const void* tmap_ws = nullptr;  // workspace the tensor maps were encoded for
};

// What the debug range checks of the kernels compare against (see DebugCtx).
DebugCtx make_debug_ctx(const Plan& plan, const DevTables& dt);

// Stage 1: momentum, orthogonalization input into X0, per-chunk sums of squares.
// grad_scale (may be null): device factor of every gradient.
cudaError_t launch_momentum_input(const Plan& plan, const DevTables& dt, const ShardPtrs& g,
                                  const ShardPtrs& m, void* ws, const GroupParams& gp,
                                  const float* grad_scale, cudaStream_t st);
// Full fp32 matrices -> X0 plus per-chunk sums of squares.
cudaError_t launch_full_input(const Plan& plan, const DevTables& dt, const float* full, void* ws,
                              cudaStream_t st);
// Per-matrix 1/||X||_F from the chunk sums (deterministic order).
cudaError_t launch_norm_finalize(const Plan& plan, const DevTables& dt, void* ws,
                                 cudaStream_t st);
// Stage 3: W <- W*decay - lr*scale*O, O read from the final X buffer.
cudaError_t launch_apply(const Plan& plan, const DevTables& dt, const ShardPtrs& w,
                         const void* ws, int final_buf, int pending_norm, const GroupParams& gp,
                         cudaStream_t st);
// Owner gather / scatter between shards and the fp32 full layout.
cudaError_t launch_gather(const Plan& plan, const DevTables& dt, const ShardPtrs& src,
                          float* full, cudaStream_t st);
cudaError_t launch_scatter(const Plan& plan, const DevTables& dt, const float* full,
                           const ShardPtrs& dst, cudaStream_t st);
// X buffer (0 or 1) -> fp32 full layout, times 1/||X|| when pending_norm.
cudaError_t launch_export(const Plan& plan, const DevTables& dt, const void* ws, int buf,
                          int pending_norm, float* full, cudaStream_t st);

// Stage 2, bf16 path: all ns_steps iterations of every matrix in one persistent tcgen05
// launch (with ap != nullptr the last Update also applies the step to the weights).
cudaError_t launch_ns_tc(const Plan& plan, const DevTables& dt, void* ws, int ns_steps,
                         long long budget, const ApplyArgs* ap, cudaStream_t st);
// Shared-memory opt-in of the tcgen05 kernels and how many CTA pairs / single CTAs can be
// resident at once.
cudaError_t prepare_ns_kernels(int* max_pairs, int* max_singles);
// Stage 2, fp32 path: one SIMT GEMM phase over every matrix.
cudaError_t launch_ns_phase_f32(const Plan& plan, const DevTables& dt, void* ws, int phase,
                                int x_in, int iter0, cudaStream_t st);
// Encodes the bf16 path's tensor maps for workspace `ws` into host memory.
bool encode_tensor_maps(const Plan& plan, const void* ws, std::vector<CUtensorMap>* maps,
                        std::string* err);
// One-block kernel that waits on an mbarrier nobody arrives on, with `budget` cycles.
cudaError_t launch_selftest_timeout(int* err, long long budget, cudaStream_t st);
// ---- expert layer (expert_capi.cu)
constexpr int kF32 = 0, kBf16 = 1, kF16 = 2;  // muon_dtype values
constexpr int kMaxExperts = 1024;             // MUON_MAX_EXPERTS
constexpr int kErrRowOffsets = 8;             // MUON_ERR_ROW_OFFSETS

struct GroupedMm {            // y = x W_e per expert (see muon_grouped_mm)
  const void* x;
  const void* w;
  void* y;
  const int64_t* offsets;
  int64_t ldx, ldw, w_stride, ldy, rows;
  int32_t n_experts, k, n, trans, dtype, out_dtype;
  int* err;
};
// Bytes for copies of operands whose rows do not start on 16 bytes.
size_t grouped_mm_workspace(const GroupedMm& g);
cudaError_t launch_grouped_mm(const GroupedMm& g, void* workspace, int sms, cudaStream_t st);

struct GroupedWgrad {         // dw_e (+)= a^T b per expert (see muon_grouped_wgrad)
  const void* a;
  const void* b;
  float* dw;
  const int64_t* offsets;
  int64_t lda, ldb, lddw, dw_stride, rows;
  int32_t n_experts, m, n, accumulate, dtype;
  int* err;
};
// Whether the product has few enough tiles for one launch.
bool grouped_mm_fits(const GroupedMm& g);
bool grouped_wgrad_fits(const GroupedWgrad& g);
size_t grouped_wgrad_workspace(const GroupedWgrad& g);
cudaError_t launch_grouped_wgrad(const GroupedWgrad& g, void* workspace, int sms, cudaStream_t st);

// Gated projections (see muon_gated_mm): x, w (the gate's), k and n of the products, y the result.
struct GatedMm : GroupedMm {
  const void* w2;             // the up projection's
  int64_t ldw2, w2_stride;
  void *gate, *up;            // may be null
  int64_t ld_gate, ld_up;
  const float* p;             // row weights, may be null
};
// What feeds the gated activation's gradient (see muon_gated_mm_grad): x = dy, w = w_down, y the
// activation (may be null).
struct GatedGrad : GroupedMm {
  const void *gate, *up;
  int64_t ld_gate, ld_up;
  void *dgate, *dup;
  int64_t ld_dgate, ld_dup;
  const float* p;             // may be null
  float *dp, *part;           // dp may be null; part: its sums over 32 columns
};
// y = x W_e + x2 W2_e.
struct MmSum : GroupedMm {
  const void *x2, *w2;
  int64_t ldx2, ldw2, w2_stride;
};
bool gated_mm_fits(const GroupedMm& g);
size_t gated_mm_workspace(const GatedMm& g);
cudaError_t launch_gated_mm(const GatedMm& g, void* workspace, int sms, cudaStream_t st);
size_t gated_grad_workspace(const GatedGrad& g, bool row_weight_grad);
cudaError_t launch_gated_grad(const GatedGrad& g, void* workspace, int sms, cudaStream_t st);
size_t mm_sum_workspace(const MmSum& g);
cudaError_t launch_mm_sum(const MmSum& g, void* workspace, int sms, cudaStream_t st);

// Quantization to e4m3 with a scale per block of 128 (see muon_quantize_rows, muon_quantize_weights).
struct QuantizeRows {
  const void* x;
  uint8_t* q;
  float* scale;
  int64_t ldx, ldq, ld_scale, rows;
  int32_t cols;
};
struct QuantizeWeights {
  const void* w;
  uint8_t* q;
  float* scale;
  int64_t ldw, w_stride, ldq, q_stride;
  int32_t n, rows, cols, transpose;
  bool wide_q;                // set by the launch: q's rows start on 8 bytes
};
cudaError_t launch_quantize_rows(const QuantizeRows& a, int dtype, int sms, cudaStream_t st);
cudaError_t launch_quantize_weights(const QuantizeWeights& a, int dtype, int sms, cudaStream_t st);

// The product of 8-bit operands (see muon_grouped_mm_fp8): x and w with their scales.
constexpr int kE4m3 = 3;      // an operand type of tensor maps, beside the muon_dtype values
struct Fp8Mm : GroupedMm {
  const float *x_scale, *w_scale;
  int64_t ld_x_scale;
};
cudaError_t launch_fp8_mm(const Fp8Mm& g, int sms, cudaStream_t st);

// n = 3: g, u, a (forward); n = 5: da, g, u, dg, du (gradient).
struct SwigluArgs {
  int n;
  void* ptr[5];
  int64_t ld[5];
};
cudaError_t launch_swiglu(const SwigluArgs& s, int dtype, const float* p, float* dp, int64_t rows,
                          int32_t cols, int sms, cudaStream_t st);

// Layer norm (out = y) and its gradient (out = dx); see muon_layer_norm.  Null weights count as 1,
// null biases as 0; null results are not wanted.
struct NormArgs {
  const void *x, *dy;
  void* out;
  const float *w, *b, *mean_in, *rstd_in;
  float *mean, *rstd, *dw, *db;
  float* part;                // the gradient's workspace
  int64_t ldx, lddy, ldo, rows;
  int32_t cols, accumulate;
  float eps;
};
cudaError_t launch_layer_norm(const NormArgs& a, int dtype, int sms, cudaStream_t st);
size_t norm_grad_workspace(int64_t rows, int32_t cols);
cudaError_t launch_layer_norm_grad(const NormArgs& a, int dtype, int sms, cudaStream_t st);

struct TensorSpec {           // same layout as muon_tensor
  void* data;
  int64_t numel;
  int32_t dtype;
  int32_t pad_;
};
// outs may be null (norm and coefficient only).
cudaError_t launch_clip(const TensorSpec* grads, const TensorSpec* outs, int n, float max_norm,
                        float* norm, void* ws, int sms, cudaStream_t st);
size_t clip_workspace_bytes(const TensorSpec* grads, int n, int sms);
// Work units of a list; at most 2^31 - 1 fit a launch.
int64_t clip_chunks(const TensorSpec* grads, int n);

// The word of device `dev` where kernels record errors (allocated and zeroed on first use).
cudaError_t device_error_word(int dev, int** out);
// Sets the message muon_last_error() returns on this thread.
void set_last_error(const std::string& msg);
// The allocation-free entry point's error word on device `dev` (inside its scratch
// array), or nullptr if that entry point has not run there.
int* noalloc_error_word(int dev);

}  // namespace muon
