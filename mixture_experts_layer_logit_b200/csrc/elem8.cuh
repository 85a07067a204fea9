// Eight elements of a row, held raw as they were loaded and converted to fp32
// when used.  The element type is a value, not a template parameter: the loads
// of several operands are issued before the first one is converted, and one
// kernel serves every combination of types.
#pragma once

#include "internal.cuh"

namespace moe {

__host__ __device__ inline int dtype_bytes(int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; }

// fp32: one element per word.  16-bit types: vector loads fill a.x..a.w with
// two elements each; scalar loads put one element in the low half of a word.
struct Raw8 {
  uint32_t w[8];
};

__device__ __forceinline__ uint32_t load_raw1(const void* p, int dt, size_t i) {
  if (dt == MOE_DTYPE_F32) return static_cast<const uint32_t*>(p)[i];
  return static_cast<const unsigned short*>(p)[i];
}

__device__ __forceinline__ float raw_to_float(uint32_t w, int dt) {
  if (dt == MOE_DTYPE_F32) return __uint_as_float(w);
  if (dt == MOE_DTYPE_BF16) return __uint_as_float(w << 16);
  return __half2float(__ushort_as_half((unsigned short)w));
}

__device__ __forceinline__ void store1(void* p, int dt, size_t i, float v) {
  if (dt == MOE_DTYPE_F32) static_cast<float*>(p)[i] = v;
  else if (dt == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// v rounded to the type dt and back
__device__ __forceinline__ float round_to(float v, int dt) {
  if (dt == MOE_DTYPE_F32) return v;
  if (dt == MOE_DTYPE_BF16) return __bfloat162float(__float2bfloat16_rn(v));
  return __half2float(__float2half_rn(v));
}

}  // namespace moe
