// Eight elements of a row, held raw as they were loaded and converted to fp32
// when used.  The element type is a value, not a template parameter: the loads
// of several operands are issued before the first one is converted, and one
// kernel serves every combination of types.
#pragma once

#include "internal.cuh"

namespace moe {

__host__ __device__ inline int dtype_bytes(int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; }

// fp32: one element per word.  16-bit types: a vector load fills w[0..3] with
// two elements each; scalar loads put one element in the low half of each word.
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

// 32 and 16 bytes at once, past L1: every operand of these kernels is used by one thread only
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void load16(const void* p, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Eight consecutive elements from i on, all there and aligned to their size (32 or 16 bytes).
__device__ __forceinline__ void load8(Raw8& r, const void* p, int dt, size_t i) {
  if (dt == MOE_DTYPE_F32) load32(static_cast<const float*>(p) + i, r.w);
  else load16(static_cast<const unsigned short*>(p) + i, r.w[0], r.w[1], r.w[2], r.w[3]);
}

__device__ __forceinline__ void to_float8(const Raw8& r, int dt, float (&v)[8]) {
  if (dt == MOE_DTYPE_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
  } else if (dt == MOE_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void store8(void* p, int dt, size_t i, const float (&v)[8]) {
  if (dt == MOE_DTYPE_F32) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[j]);
    store32(static_cast<float*>(p) + i, w);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (dt == MOE_DTYPE_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<unsigned short*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace moe
