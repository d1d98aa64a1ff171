// moe_device.cuh -- shared by route.cu, experts.cu and weighted.cu: element
// types, 16-byte vectors of them, launch chaining, host-side checks.
#pragma once

#include "a2av_handle.h"
#include "a2av_moe.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

namespace {

constexpr int kW = A2AV_MAX_RANKS;
constexpr unsigned kAll = 0xffffffffu;
constexpr long long kMaxCount = 0x7fffffffLL;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// Two elements in a 32-bit word, the first in its low half.
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t x, __nv_bfloat16) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
}
__device__ __forceinline__ float2 unpack2(uint32_t x, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// N elements that one load or store moves (16 bytes of them, or one).
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

// N elements as 32-bit words (or one element): unpacked and packed in pairs.
template <typename T, int N>
struct Piece {
  static constexpr int kWords = N * sizeof(T) / 4;
  struct alignas(4 * kWords) Raw {
    uint32_t w[kWords];
  };
  static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(r.w[i]);
      } else {
        const float2 v = unpack2(r.w[i], T());
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  }
  static __device__ __forceinline__ Raw pack(const float (&f)[N]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4)
        r.w[i] = __float_as_uint(f[i]);
      else
        r.w[i] = pack2(f[2 * i], f[2 * i + 1], T());
    }
    return r;
  }
};

template <typename T>
struct Piece<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[1]) { f[0] = to_float(r); }
  static __device__ __forceinline__ Raw pack(const float (&f)[1]) { return from_float<T>(f[0]); }
};

// Programmatic dependent launch, as in the exchange's kernels: let the next
// kernel of the stream be scheduled, then wait until the previous one is done
// and its writes are visible.  Both are no-ops in a plain launch.
__device__ __forceinline__ void chain() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void note_error(int* status, int code) { atomicCAS(status, 0, code); }

template <typename... Args, typename... Vals>
cudaError_t launch_chained(void (*kernel)(Args...), dim3 grid, int block, size_t smem,
                           cudaStream_t s, bool pdl, const Vals&... vals) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, vals...);
}

inline int current_device(const a2av_handle* h) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return A2AV_ERR_CUDA;
  return dev == h->device ? A2AV_OK : A2AV_ERR_INVALID_ARG;
}

inline int dtype_bytes(int dtype) {
  return dtype == A2AV_F32 ? 4 : dtype == A2AV_BF16 || dtype == A2AV_F16 ? 2 : 0;
}

inline bool aligned_to(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace
