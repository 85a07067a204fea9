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

// 16 bytes at once, past L1: every operand of these kernels is used by one thread only
__device__ __forceinline__ void load16(const void* p, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Words q * 4 .. (fp32) or q * 2 .. (16 bits) of r: four consecutive elements
// from i on, aligned to their size (16 or 8 bytes).
__device__ __forceinline__ void load4(Raw8& r, int q, const void* p, int dt, size_t i) {
  if (dt == MOE_DTYPE_F32)
    load16(static_cast<const float*>(p) + i, r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
  else
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
                 : "=r"(r.w[2 * q]), "=r"(r.w[2 * q + 1]) : "l"(static_cast<const unsigned short*>(p) + i));
}

__device__ __forceinline__ void load4_cached(Raw8& r, int q, const void* p, int dt, size_t i) {
  if (dt == MOE_DTYPE_F32) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i));
    r.w[4 * q] = v.x, r.w[4 * q + 1] = v.y, r.w[4 * q + 2] = v.z, r.w[4 * q + 3] = v.w;
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(p) + i));
    r.w[2 * q] = v.x, r.w[2 * q + 1] = v.y;
  }
}

// Asynchronous copies to shared memory, and reads of what they brought.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {   // until at most N of the thread's groups are under way
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void shared16(uint32_t at, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(at) : "memory");
}
__device__ __forceinline__ void shared4(uint32_t at, uint32_t& a) {
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a) : "r"(at) : "memory");
}
__device__ __forceinline__ void shared2(uint32_t at, uint32_t& a) {
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(a) : "r"(at) : "memory");
}
__device__ __forceinline__ void shared8(uint32_t at, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at) : "memory");
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

__device__ __forceinline__ void store4(void* p, int dt, size_t i, float a, float b, float c, float d) {
  if (dt == MOE_DTYPE_F32) {
    __stcs(reinterpret_cast<float4*>(static_cast<float*>(p) + i), make_float4(a, b, c, d));
    return;
  }
  uint2 w;
  if (dt == MOE_DTYPE_BF16) {
    const __nv_bfloat162 l = __floats2bfloat162_rn(a, b), h = __floats2bfloat162_rn(c, d);
    w = make_uint2(*reinterpret_cast<const uint32_t*>(&l), *reinterpret_cast<const uint32_t*>(&h));
  } else {
    const __half2 l = __floats2half2_rn(a, b), h = __floats2half2_rn(c, d);
    w = make_uint2(*reinterpret_cast<const uint32_t*>(&l), *reinterpret_cast<const uint32_t*>(&h));
  }
  __stcs(reinterpret_cast<uint2*>(static_cast<unsigned short*>(p) + i), w);
}

}  // namespace moe
