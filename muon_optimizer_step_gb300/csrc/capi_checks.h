// Argument checks that the C entry points of the layers' operators share, and what a launch needs to
// know of the current device.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "../../include/muon.h"
#include "kernels.h"

namespace muon {

static_assert(kF32 == MUON_DTYPE_F32 && kBf16 == MUON_DTYPE_BF16 && kF16 == MUON_DTYPE_F16, "");
static_assert(kMaxExperts == MUON_MAX_EXPERTS && kErrRowOffsets == MUON_ERR_ROW_OFFSETS, "");

inline muon_status fail(muon_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  try {
    set_last_error(buf);
  } catch (...) {  // no memory for the message: the status still goes back
  }
  return s;
}

inline muon_status done(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return fail(MUON_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  set_last_error("");
  return MUON_OK;
}

#define EXPERT_TRY(expr)                  \
  do {                                    \
    const muon_status s_ = (expr);        \
    if (s_ != MUON_OK) return s_;         \
  } while (0)

// What the launches need to know of the current device, looked up once per device.
struct Device {
  int sms = 0;
  int* err = nullptr;
};

inline muon_status current_device(Device* out) {
  constexpr int kMaxDevices = 64;
  static Device known[kMaxDevices];
  static std::mutex mu;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(MUON_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(MUON_ERR_UNSUPPORTED, "device %d out of range", dev);
  std::lock_guard<std::mutex> g(mu);
  if (known[dev].err == nullptr) {
    int major = 0, minor = 0, sms = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (major != 10 || minor != 3)
      return fail(MUON_ERR_UNSUPPORTED, "libmuon is built for sm_103a; device %d is sm_%d%d", dev,
                  major, minor);
    int* err = nullptr;
    e = device_error_word(dev, &err);
    if (e != cudaSuccess) return fail(MUON_ERR_CUDA, "error word of device %d: %s", dev,
                                      cudaGetErrorString(e));
    known[dev].sms = sms;
    known[dev].err = err;
  }
  *out = known[dev];
  return MUON_OK;
}

inline muon_status check_ptr(const void* p, size_t align, const char* name) {
  if (p == nullptr) return fail(MUON_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return fail(MUON_ERR_ALIGNMENT, "%s = %p is not %zu-byte aligned", name, p, align);
  return MUON_OK;
}

// Pitches keep every offset well inside 64 bits (and a TMA stride inside its 40).
inline muon_status check_pitch(int64_t ld, int64_t len, const char* name) {
  if (ld < len || ld >= (int64_t)1 << 36)
    return fail(MUON_ERR_INVALID_ARG, "%s=%lld outside %lld..2^36-1", name, (long long)ld,
                (long long)len);
  return MUON_OK;
}

inline muon_status check_groups(int64_t rows, int32_t n_experts) {
  if (n_experts < 1 || n_experts > MUON_MAX_EXPERTS)
    return fail(MUON_ERR_INVALID_ARG, "n_experts=%d outside 1..%d", n_experts, MUON_MAX_EXPERTS);
  if (rows < 0 || rows > INT32_MAX)
    return fail(MUON_ERR_INVALID_ARG, "rows=%lld outside 0..2^31-1", (long long)rows);
  return MUON_OK;
}

inline muon_status check_16bit(int32_t dtype, const char* name) {
  if (dtype != MUON_DTYPE_BF16 && dtype != MUON_DTYPE_F16)
    return fail(MUON_ERR_INVALID_ARG, "%s=%d: the products take bf16 and fp16", name, dtype);
  return MUON_OK;
}

inline muon_status check_dim(int32_t v, const char* name) {
  if (v < 1) return fail(MUON_ERR_INVALID_ARG, "%s=%d must be at least 1", name, v);
  return MUON_OK;
}

inline size_t dtype_size(int32_t dtype) { return dtype == MUON_DTYPE_F32 ? 4 : 2; }

inline muon_status check_dtype(int32_t dtype, const char* name) {
  if (dtype < MUON_DTYPE_F32 || dtype > MUON_DTYPE_F16)
    return fail(MUON_ERR_INVALID_ARG, "%s=%d is no muon_dtype", name, dtype);
  return MUON_OK;
}

inline muon_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (bytes < need)
    return fail(MUON_ERR_INVALID_ARG, "workspace has %zu bytes, %zu needed", bytes, need);
  return need > 0 ? check_ptr(workspace, (size_t)kWsAlign, "workspace") : MUON_OK;
}

}  // namespace muon
