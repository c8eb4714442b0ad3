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

// How a column of largest magnitude a is rounded to 8 bits:
// q = rint(v * pre * inv).  pre is 1 except for columns so small
// that 127 / a would overflow (below 2^-60, taken 2^64 times larger).
// |v| <= a makes |q| <= 127 without a clamp: v * inv is at most
// 127 (1 + 2^-22) before it is rounded to an integer.
struct Rounding {
  float scale, pre, inv;
};
__device__ __forceinline__ Rounding rounding_of(float a) {
  Rounding r;
  if (magnitude_bits(a) >= kInfBits) {   // an infinity or a NaN: reads back as NaN everywhere
    r.scale = __uint_as_float(0x7fc00000u);
    r.pre = r.inv = 0.f;
    return r;
  }
  r.scale = a / 127.f;
  r.pre = a < 0x1p-60f ? 0x1p64f : 1.f;
  // inv = 0 (a column of zeros, or one that is not finite): Q is 0
  r.inv = r.scale > 0.f ? 127.f / (a * r.pre) : 0.f;
  return r;
}
// Every kernel of these operators may be launched while its predecessor on
// the stream still runs (programmatic dependent launch hides the launch's
// latency): await_predecessor comes before the first access to global memory,
// and only then is the successor allowed to do the same.
__device__ __forceinline__ void await_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... P, class... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// host: the end of a call that launched `kernels` kernels, none of which
// has a bounded wait.  Noting the call also tells a following SYMV call
// that its predecessor is not a SYMV finaliser it could overlap with.
inline int launched(cudaError_t e, int kernels, cudaStream_t st) {
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return XSYMV_ERR_CUDA;
  }
  note_launches(kernels);
  note_call_status(st, nullptr, 0);
  return XSYMV_OK;
}

inline bool short_ld(int ld, int rows) { return ld < (rows > 1 ? rows : 1); }

}  // namespace xsymv
