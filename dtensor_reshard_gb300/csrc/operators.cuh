// operators.cuh -- pieces shared by the operators that run beside a refit
// (fp8_quantize.cu, fp8_matmul.cu, sample.cu, balance.cu): element types,
// reductions and argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <string>

#include "internal.h"

namespace rs {
namespace op {

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float warp_max(float v) {
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The largest of N values (a NaN loses against any number).
template <int N>
__device__ __forceinline__ float largest_of(const float (&v)[N]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, v[i]);
  return m;
}
template <int N>
__device__ __forceinline__ float largest_of(const __nv_bfloat16 (&v)[N]) {
  __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(v);
#pragma unroll
  for (int i = 2; i < N; i += 2) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(v + i));
  return fmaxf(__low2float(m), __high2float(m));
}
template <int N>
__device__ __forceinline__ float largest_of(const __half (&v)[N]) {
  __half2 m = *reinterpret_cast<const __half2*>(v);
#pragma unroll
  for (int i = 2; i < N; i += 2) m = __hmax2(m, *reinterpret_cast<const __half2*>(v + i));
  return fmaxf(__low2float(m), __high2float(m));
}

inline int64_t cdiv(int64_t a, int64_t b) { return a / b + (a % b != 0); }
inline bool float_dtype(int32_t d) {
  return d == RESHARD_BF16 || d == RESHARD_FP16 || d == RESHARD_FP32;
}
inline bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
inline int64_t dtype_size(int32_t d) { return d == RESHARD_FP32 ? 4 : 2; }

// The status of the launch just made.
inline reshard_status_t launched(const char* what) {
  const cudaError_t ce = cudaGetLastError();
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(ce));
  return RESHARD_OK;
}

constexpr size_t kSmemMost = 227 * 1024;  // shared memory of a CTA

// Lets Kernel have MOST bytes of dynamic shared memory, the most that any call needs: the
// limit belongs to the kernel and the device, so no call may lower it under another thread's
// launch.  Set once a device.
template <auto Kernel, size_t MOST>
cudaError_t allow_smem(int dev) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (MOST <= 48 * 1024 || (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t ce =
      cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(MOST));
  if (ce == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return ce;
}

struct Launch {
  int64_t grid;
  int threads;
  size_t smem;
  int cluster;  // CTAs; 0: may start before the kernel in front of it has ended
  cudaStream_t stream;
};
template <auto Kernel, size_t MOST>
reshard_status_t launch(const char* what, int dev, const Launch& l, void** args) {
  cudaError_t ce = allow_smem<Kernel, MOST>(dev);
  if (ce == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(l.grid));
    cfg.blockDim = dim3(unsigned(l.threads));
    cfg.dynamicSmemBytes = l.smem;
    cfg.stream = l.stream;
    cudaLaunchAttribute attr[1];
    if (l.cluster == 0) {
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
    } else {
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim = {unsigned(l.cluster), 1, 1};
    }
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ce = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(Kernel), args);
  }
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(ce));
  return RESHARD_OK;
}

// f(T()) with T the element type of a floating dtype.
template <typename F>
reshard_status_t by_dtype(int32_t dtype, F&& f) {
  if (dtype == RESHARD_BF16) return f(__nv_bfloat16());
  if (dtype == RESHARD_FP16) return f(__half());
  return f(float());
}

}  // namespace op
}  // namespace rs
