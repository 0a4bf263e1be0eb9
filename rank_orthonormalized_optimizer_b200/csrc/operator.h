// Host-side checks shared by the operators that give the step its gradients
// (k_act.cu, k_norm.cu, k_embed.cu, k_wgrad.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cmath>

#include "internal.h"

namespace dion {

// The current device must be an sm_100; *sms receives its SM count.  A device is asked once:
// what it is does not change while the process lives.
inline dion_status check_sm100(int* sms) {
  static std::atomic<int> known[64];  // SM count of a device found to be an sm_100
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return set_error(DION_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  const bool slot = dev >= 0 && dev < 64;
  if (slot && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return DION_OK;
  int major = 0, minor = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (major != 10 || minor != 0)
    return set_error(DION_ERR_DEVICE,
                     "device %d is sm_%d%d; this library is built for sm_100a (B200)", dev, major,
                     minor);
  *sms = 0;
  cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (*sms <= 0) *sms = 148;
  if (slot) known[dev].store(*sms, std::memory_order_relaxed);
  return DION_OK;
}

inline dion_status launch_status(const char* what, cudaError_t e = cudaGetLastError()) {
  return e == cudaSuccess ? DION_OK
                          : set_error(DION_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Launch a kernel that starts with grid_wait(): its CTAs are set up while the kernel before it
// on the stream still runs.  (After a kernel that calls grid_trigger() they may also wait on
// idle SMs; without it they come as that kernel's CTAs end.)
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                                cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool valid_dtype(int32_t t) { return t == DION_BF16 || t == DION_FP16 || t == DION_FP32; }
inline int64_t dtype_bytes(int32_t t) { return t == DION_FP32 ? 4 : 2; }

// Row of an item's index: a division by the items of a row.  In 32 bits (indexes below 2^31)
// by a multiplication with the rounded-up reciprocal, after Granlund and Montgomery, "Division
// by Invariant Integers using Multiplication": with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, i / d = (mulhi(m, i) + i) >> s.
template <typename I> struct RowDiv;
template <> struct RowDiv<uint32_t> {
  uint32_t m, s;
  explicit RowDiv(int64_t d) {
    s = 0;
    while ((int64_t(1) << s) < d) ++s;
    m = (uint32_t)(((uint64_t)((int64_t(1) << s) - d) << 32) / (uint64_t)d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t i) const { return (__umulhi(m, i) + i) >> s; }
};
template <> struct RowDiv<int64_t> {
  int64_t d;
  explicit RowDiv(int64_t n) : d(n) {}
  __device__ __forceinline__ int64_t operator()(int64_t i) const { return i / d; }
};

// Largest sizes taken: a grid's x dimension holds a row of each, and every offset
// tokens * ld stays far below 2^63.
constexpr int64_t kMaxTokens = INT32_MAX;
constexpr int64_t kMaxLd = int64_t(1) << 31;

inline dion_status check_tokens(int64_t tokens) {
  if (tokens < 0 || tokens > kMaxTokens)
    return set_error(DION_ERR_INVALID_ARG, "tokens %lld outside [0, 2^31)", (long long)tokens);
  return DION_OK;
}

// A row-major [tokens, features] array with rows ld elements apart.
inline dion_status check_rows(const char* name, const void* p, int64_t ld, int64_t features,
                              int64_t elem) {
  if (!p) return set_error(DION_ERR_INVALID_ARG, "%s is NULL", name);
  if (ld < features || ld > kMaxLd)
    return set_error(DION_ERR_INVALID_ARG, "%s: row stride %lld outside [features %lld, 2^31]", name,
                     (long long)ld, (long long)features);
  if (!aligned_to(p, (size_t)elem))
    return set_error(DION_ERR_MISALIGNED, "%s is not aligned to its %d-byte elements", name,
                     (int)elem);
  return DION_OK;
}

// Whether every row of the array starts on a 16-byte boundary.
inline bool rows_aligned16(const void* p, int64_t ld, int64_t elem) {
  return aligned_to(p, 16) && (ld * elem) % 16 == 0;
}

// Whether every row can be moved 8 elements at a time (rows.cuh): 16 bytes, 32 of fp32.
inline bool rows_vector(const void* p, int64_t ld, int64_t elem) {
  return aligned_to(p, 8 * (size_t)elem) && ld % 8 == 0;
}

// Rows of the 8-bit form: features rounded up to whole blocks.
inline int64_t kept_ld(int64_t features) { return (features + DION_ACT_BLOCK - 1) / DION_ACT_BLOCK * DION_ACT_BLOCK; }

inline dion_status check_kept(const dion_act_kept& k) {
  dion_status st = check_tokens(k.tokens);
  if (st != DION_OK) return st;
  if (k.features < 1 || k.features > kMaxLd - DION_ACT_BLOCK)
    return set_error(DION_ERR_INVALID_ARG, "features %lld outside [1, 2^31 - 32]", (long long)k.features);
  if (k.tokens == 0) return DION_OK;
  if (!k.q || !k.scale) return set_error(DION_ERR_INVALID_ARG, "the 8-bit rows: a NULL pointer");
  if (!aligned_to(k.q, 16))
    return set_error(DION_ERR_MISALIGNED, "the 8-bit rows are not 16-byte aligned");
  return DION_OK;
}

}  // namespace dion
