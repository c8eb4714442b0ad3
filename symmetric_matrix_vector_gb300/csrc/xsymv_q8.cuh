// What the 8-bit linear-layer kernels share: the storage types, the rules of
// the 8-bit rounding, and block-wide reductions in a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/xsymv.h"
#include "xsymv_runtime.h"

namespace xsymv {

// float <-> T; every kernel computes in float and rounds to T once
template <class T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// The magnitude of v as bits: unsigned comparison orders finite values, then
// infinity, then NaN, so one integer maximum finds both the largest
// magnitude of a column and whether all of it is finite.
__device__ __forceinline__ uint32_t magnitude_bits(float v) {
  return __float_as_uint(v) & 0x7fffffffu;
}
constexpr uint32_t kInfBits = 0x7f800000u;

// How a column whose largest magnitude has the bits `top` is rounded to 8
// bits: q = rint(v * pre * inv).  pre is 1 except for columns so small
// that 127 / top would overflow (below 2^-60, taken 2^64 times larger).
// |v| <= top makes |q| <= 127 without a clamp: v * inv is at most
// 127 (1 + 2^-22) before it is rounded to an integer.
struct Rounding {
  float scale, pre, inv;
};
__device__ __forceinline__ Rounding rounding_of(uint32_t top) {
  Rounding r;
  const float a = __uint_as_float(top);
  if (top >= kInfBits) {   // an infinity or a NaN: reads back as NaN everywhere
    r.scale = __uint_as_float(0x7fc00000u);
    r.pre = r.inv = 0.f;
    return r;
  }
  r.scale = a / 127.f;
  r.pre = a < 0x1p-60f ? 0x1p64f : 1.f;
  r.inv = r.scale > 0.f ? 127.f / (a * r.pre) : 0.f;
  return r;
}
// inv = 0 (a column of zeros, or one that is not finite) gives 0 for every v
__device__ __forceinline__ int round_q8(float v, const Rounding& r) {
  return r.inv == 0.f ? 0 : __float2int_rn(v * r.pre * r.inv);
}

// Sum and maximum over a block of THREADS threads (a multiple of 32); every
// thread returns the result.  The order of the additions is fixed.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) s += buf[w];
  return s;
}
template <int THREADS>
__device__ __forceinline__ uint32_t block_max(uint32_t v, float* buf) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = __uint_as_float(v);
  __syncthreads();
  uint32_t s = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) s = max(s, __float_as_uint(buf[w]));
  return s;
}

// host: the status of a launch
inline int launched(cudaError_t e, int kernels) {
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return XSYMV_ERR_CUDA;
  }
  note_launches(kernels);
  return XSYMV_OK;
}

}  // namespace xsymv
