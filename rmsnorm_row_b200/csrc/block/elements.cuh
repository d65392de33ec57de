// 16-bit elements, widened to fp32 and rounded back, for the operators of include/block_ops.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../fused_norm_kernel.cuh"

namespace block_ops {

using fused_norm_impl::DivU32;
using fused_norm_impl::div_u32;

template <bool FP16>
__device__ __forceinline__ float2 widen16(uint32_t u) {
  if (FP16) {
    __half2 h;
    memcpy(&h, &u, 4);
    return __half22float2(h);
  }
  return make_float2(fused_norm_impl::lo_f(u), fused_norm_impl::hi_f(u));
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if (FP16) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
  }
  return fused_norm_impl::pack_rn(a, b);
}

template <bool FP16>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 e = widen16<FP16>(fused_norm_impl::word(v, i));
    f[2 * i] = e.x, f[2 * i + 1] = e.y;
  }
}

// The same value, which the compiler cannot trace: what depends on it is computed where it is
// used, and not earlier into registers that then wait (addresses of ten heads for all rows, or
// a row widened for its sum and kept for its output, took more registers than the row).
__device__ __forceinline__ uint4 here(uint4 v) {
  asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w));
  return v;
}
template <typename V>
__device__ __forceinline__ V here(V v) {
  if constexpr (sizeof(V) == 8) asm volatile("" : "+l"(v));
  else asm volatile("" : "+r"(v));
  return v;
}

}  // namespace block_ops
