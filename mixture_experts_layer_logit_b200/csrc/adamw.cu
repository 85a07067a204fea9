// One AdamW step over many tensors at once.
//
// With gradient g (times grad_scale), step number t and c_i = 1 - beta_i^t:
//   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
//   p = p (1 - lr wd) - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps)
// m and v are fp32, or 8 bits each: blocks of 256 elements, an fp32 scale per
// block, E4M3 codes of m / scale and of sqrt(v) / scale with
// scale = max|.| / 448 (the root halves the range of exponents that v spans).
// The update uses the m and v of this step before they are rounded.  A root
// that is not zero keeps a code that is not zero: a denominator rounded down
// to zero would turn the next update into m / eps.  A value that is not finite
// gets the NaN code and leaves its block's scale alone.
//
// Ten operations per element against 12 to 30 bytes: bound by those bytes.  m
// and v are computed in separately rounded steps (no contraction), so that a
// code does not depend on how a compiler fuses them.
#include "elem8.cuh"

#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

namespace moe {
namespace {

constexpr int kBlock = MOE_ADAMW_BLOCK;
constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 3;
constexpr int kTile = kThreads / 32 * kBlock;   // elements a block of threads takes at a time: a block per warp
static_assert(kBlock == 256, "a warp holds a block, eight elements a lane");

// The tensors of one launch, in its parameters (at most 32764 bytes of them).
struct Entry {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* ms;
  float* vs;
  long long n;
  float decay;        // 1 - lr wd is formed on the device (lr may be there)
  unsigned tile0;     // first tile of the tensor
  unsigned char pdt, gdt, bits, vec, pad[4];
};
constexpr int kMaxEntries = 340;
struct Table {
  Entry e[kMaxEntries];
};
static_assert(sizeof(Table) + 128 <= 32764, "kernel parameters");

struct Hyper {
  float lr, beta1, omb1, beta2, omb2, lnb1, lnb2, eps, one;
  const float* lr_dev;
  const float* grad_scale;
  moe_adamw_state* state;
};

// What every element of a step shares.
struct Step {
  float beta1, omb1, beta2, omb2, eps, one, gs, alpha, rc2, keep;
};

// Two fp32 values in one instruction, each rounded on its own.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return r;
}
// a + b, rounded once: a product in a or b stays rounded, since `one` is not
// known to the compiler (add.rn.f32x2 after mul.rn.f32x2 was seen to fuse)
__device__ __forceinline__ float2 add2(float2 a, float2 b, float2 one) { return fma2(a, one, b); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 1 / v to about an ulp; v is a normal number here
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// max |v| over the warp's block as float bits
__device__ __forceinline__ unsigned block_top(const float (&v)[8]) {
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return __reduce_max_sync(0xffffffffu, top);
}

// Codes of the warp's block of eight values a lane, element i in byte i, and
// (returned) the scale.  The fast path takes a block of finite values, roots
// none of which is zero: they are lifted to the smallest code by a maximum.
template <bool ROOT>
__device__ __forceinline__ float encode(const float (&v)[8], uint2* codes) {
  unsigned top = block_top(v);
  bool odd = top >= 0x7f800000u;
  if (odd) {   // an inf or NaN: the largest of the others
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (isfinite(v[i])) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
  }
  const float most = fmaxf(__uint_as_float(top), 0x1p-100f);   // its reciprocal stays finite
  const float2 inv = both(__fmul_rn(__frcp_rn(most), 448.f));
  if (ROOT) {
    float least = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) least = fminf(least, v[i]);
    odd |= __any_sync(0xffffffffu, least == 0.f);
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 q = mul2(make_float2(v[2 * i], v[2 * i + 1]), inv);
    if (ROOT) q = make_float2(fmaxf(q.x, 0x1p-9f), fmaxf(q.y, 0x1p-9f));
    w[i] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
  }
  if (odd) {   // zeros and NaNs put right
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ROOT && v[2 * i] == 0.f) w[i] &= 0xff00u;
      if (ROOT && v[2 * i + 1] == 0.f) w[i] &= 0xffu;
      if (!isfinite(v[2 * i])) w[i] = (w[i] & 0xff00u) | 0x7fu;
      if (!isfinite(v[2 * i + 1])) w[i] = (w[i] & 0xffu) | 0x7f00u;
    }
  }
  *codes = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  return __fmul_rn(most, 1.f / 448.f);
}

__device__ __forceinline__ void decode(uint2 c, float scale, float (&v)[8]) {
  const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[i], __NV_E4M3);
    const float2 f = mul2(__half22float2(*reinterpret_cast<const __half2*>(&h)), both(scale));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint2 load_codes1(const unsigned char* p, int count, int lane) {
  uint32_t w[2] = {0u, 0u};
  for (int i = 0; i < 8; ++i)
    if (i * 32 + lane < count) w[i / 4] |= (uint32_t)p[i * 32 + lane] << (8 * (i % 4));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes1(unsigned char* p, int count, int lane, uint2 c) {
  for (int i = 0; i < 8; ++i)
    if (i * 32 + lane < count) p[i * 32 + lane] = (unsigned char)((i < 4 ? c.x : c.y) >> (8 * (i % 4)));
}

// One warp, one block of 256 elements from b0 on.  VEC: all there, every array
// aligned to eight of its elements, lane l holds elements 8 l .. 8 l + 7; else
// elements l, l + 32, ... below `count`, one by one.  Every load is issued
// before the first value is used.
template <bool VEC, int BITS>
__device__ __forceinline__ void update_block(const Entry& e, long long b0, int lane, const Step& s) {
  const int count = VEC ? kBlock : (int)min((long long)kBlock, e.n - b0);
  const long long at = VEC ? b0 + lane * 8 : b0 + lane;
  const bool has_master = e.master != nullptr;
  Raw8 rg, rp, rm, rv;
  uint2 cm, cv;
  float ms, vs;
  if constexpr (BITS == 8) {
    ms = e.ms[b0 / kBlock];
    vs = e.vs[b0 / kBlock];
  }
  const void* psrc = has_master ? e.master : e.param;
  const int psdt = has_master ? MOE_DTYPE_F32 : e.pdt;
  if constexpr (VEC) {
    load8(rg, e.grad, e.gdt, at);
    load8(rp, psrc, psdt, at);
    if constexpr (BITS == 8) {
      cm = __ldcs(reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(e.m) + at));
      cv = __ldcs(reinterpret_cast<const uint2*>(static_cast<const unsigned char*>(e.v) + at));
    } else {
      load8(rm, e.m, MOE_DTYPE_F32, at);
      load8(rv, e.v, MOE_DTYPE_F32, at);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      rg.w[i] = rp.w[i] = rm.w[i] = rv.w[i] = 0u;
      if (i * 32 + lane < count) {
        rg.w[i] = load_raw1(e.grad, e.gdt, at + i * 32);
        rp.w[i] = load_raw1(psrc, psdt, at + i * 32);
        if constexpr (BITS == 32) {
          rm.w[i] = load_raw1(e.m, MOE_DTYPE_F32, at + i * 32);
          rv.w[i] = load_raw1(e.v, MOE_DTYPE_F32, at + i * 32);
        }
      }
    }
    if constexpr (BITS == 8) {
      cm = load_codes1(static_cast<const unsigned char*>(e.m) + b0, count, lane);
      cv = load_codes1(static_cast<const unsigned char*>(e.v) + b0, count, lane);
    }
  }
  float g[8], p[8], m[8], v[8], root[8];
  if constexpr (VEC) {
    to_float8(rg, e.gdt, g);
    to_float8(rp, psdt, p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = raw_to_float(rg.w[i], e.gdt);
      p[i] = raw_to_float(rp.w[i], psdt);
    }
  }
  if constexpr (BITS == 8) {
    decode(cm, ms, m);
    decode(cv, vs, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
  } else {
    to_float8(rm, MOE_DTYPE_F32, m);
    to_float8(rv, MOE_DTYPE_F32, v);
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 gi = mul2(make_float2(g[i], g[i + 1]), both(s.gs));
    const float2 mi = add2(mul2(make_float2(m[i], m[i + 1]), both(s.beta1)), mul2(gi, both(s.omb1)), both(s.one));
    const float2 vi = add2(mul2(make_float2(v[i], v[i + 1]), both(s.beta2)), mul2(mul2(gi, gi), both(s.omb2)), both(s.one));
    const float2 ri = make_float2(sqrtf(vi.x), sqrtf(vi.y));
    const float2 den = fma2(ri, both(s.rc2), both(s.eps));
    const float2 upd = mul2(mul2(mi, both(s.alpha)), make_float2(reciprocal(den.x), reciprocal(den.y)));
    const float2 pi = fma2(make_float2(p[i], p[i + 1]), both(s.keep), upd);
    m[i] = mi.x, m[i + 1] = mi.y;
    v[i] = vi.x, v[i + 1] = vi.y;
    root[i] = ri.x, root[i + 1] = ri.y;
    p[i] = pi.x, p[i + 1] = pi.y;
  }
  if constexpr (VEC) {
    if (has_master) store8(e.master, MOE_DTYPE_F32, at, p);
    store8(e.param, e.pdt, at, p);
    if constexpr (BITS == 32) {
      store8(e.m, MOE_DTYPE_F32, at, m);
      store8(e.v, MOE_DTYPE_F32, at, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 32 + lane < count) {
        if (has_master) e.master[at + i * 32] = p[i];
        store1(e.param, e.pdt, at + i * 32, p[i]);
        if constexpr (BITS == 32) {
          static_cast<float*>(e.m)[at + i * 32] = m[i];
          static_cast<float*>(e.v)[at + i * 32] = v[i];
        }
      }
  }
  if constexpr (BITS == 8) {   // elements past the end are zeros throughout: they do not raise the maximum
    const float mscale = encode<false>(m, &cm), vscale = encode<true>(root, &cv);
    if (lane == 0) {
      e.ms[b0 / kBlock] = mscale;
      e.vs[b0 / kBlock] = vscale;
    }
    unsigned char* pm = static_cast<unsigned char*>(e.m);
    unsigned char* pv = static_cast<unsigned char*>(e.v);
    if constexpr (VEC) {
      *reinterpret_cast<uint2*>(pm + at) = cm;
      *reinterpret_cast<uint2*>(pv + at) = cv;
    } else {
      store_codes1(pm + b0, count, lane, cm);
      store_codes1(pv + b0, count, lane, cv);
    }
  }
}

// A block of threads takes a run of consecutive tiles: it looks its first
// tensor up and walks on from there.
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
adamw_kernel(const __grid_constant__ Table tab, int ntensors, unsigned ntiles, unsigned per_block, Hyper h,
             int last_launch) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int step = h.state->step + 1;
  const float t = (float)step;
  Step s;
  s.beta1 = h.beta1, s.omb1 = h.omb1, s.beta2 = h.beta2, s.omb2 = h.omb2, s.eps = h.eps, s.one = h.one;
  s.gs = h.grad_scale != nullptr ? *h.grad_scale : 1.f;
  const float lr = h.lr_dev != nullptr ? *h.lr_dev : h.lr;
  // 1 - beta^t = -expm1(t ln beta): exact to rounding also for the first steps
  s.alpha = lr / expm1f(t * h.lnb1);   // -lr / c1
  s.rc2 = 1.f / sqrtf(-expm1f(t * h.lnb2));
  const unsigned first = blockIdx.x * per_block, end = min(ntiles, first + per_block);
  int lo = 0;
  if (first < end) {
    int hi = ntensors - 1;   // the last tensor that starts at or before the tile
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.e[mid].tile0 <= first) lo = mid; else hi = mid - 1;
    }
  }
  for (unsigned tile = first; tile < end; ++tile) {
    while (lo + 1 < ntensors && tab.e[lo + 1].tile0 <= tile) ++lo;
    const Entry& e = tab.e[lo];
    const long long b0 = (long long)(tile - e.tile0) * kTile + warp * kBlock;   // the warp's block
    if (b0 >= e.n) continue;
    s.keep = 1.f - lr * e.decay;
    const bool vec = e.vec && b0 + kBlock <= e.n;
    if (e.bits == 8) {
      if (vec) update_block<true, 8>(e, b0, lane, s);
      else update_block<false, 8>(e, b0, lane, s);
    } else {
      if (vec) update_block<true, 32>(e, b0, lane, s);
      else update_block<false, 32>(e, b0, lane, s);
    }
  }
  if (!last_launch) return;
  // The last block to finish counts the step: by then every block has read it.
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicInc(&h.state->ticket, gridDim.x - 1) == gridDim.x - 1) h.state->step = step;
  }
}

// Every array of the tensor starts on a boundary of eight of its elements.
bool vector_aligned(const moe_adamw_tensor& t) {
  auto on = [](const void* p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
  const unsigned st = t.state_bits == 8 ? 8u : 32u;
  return on(t.param, 8u * dtype_bytes(t.param_dtype)) && on(t.grad, 8u * dtype_bytes(t.grad_dtype)) &&
         on(t.master, 32u) && on(t.m, st) && on(t.v, st);
}

}  // namespace

cudaError_t launch_adamw(const moe_adamw_tensor* t, int nt, const moe_adamw_hyper& hy, const float* lr_dev,
                         const float* grad_scale, moe_adamw_state* state, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  Hyper h{};
  h.lr = (float)hy.lr;
  h.beta1 = (float)hy.beta1;
  h.omb1 = (float)(1.0 - hy.beta1);
  h.beta2 = (float)hy.beta2;
  h.omb2 = (float)(1.0 - hy.beta2);
  h.lnb1 = (float)log(hy.beta1);
  h.lnb2 = (float)log(hy.beta2);
  h.eps = (float)hy.eps;
  h.one = 1.f;
  h.lr_dev = lr_dev;
  h.grad_scale = grad_scale;
  h.state = state;
  Table tab;
  int i = 0;
  do {   // at least one launch: a step over nothing counts, too
    int ne = 0;
    unsigned tiles = 0;
    for (; i < nt && ne < kMaxEntries; ++i) {
      if (t[i].n == 0) continue;
      const long long nt_i = (t[i].n + kTile - 1) / kTile;
      if (ne > 0 && (long long)tiles + nt_i > 0x7fffffffLL) break;
      Entry& e = tab.e[ne++];
      e = Entry{};
      e.param = t[i].param;
      e.grad = t[i].grad;
      e.master = t[i].master;
      e.m = t[i].m;
      e.v = t[i].v;
      e.ms = t[i].m_scale;
      e.vs = t[i].v_scale;
      e.n = t[i].n;
      e.decay = t[i].weight_decay;
      e.tile0 = tiles;
      e.pdt = (unsigned char)t[i].param_dtype;
      e.gdt = (unsigned char)t[i].grad_dtype;
      e.bits = (unsigned char)t[i].state_bits;
      e.vec = vector_aligned(t[i]) ? 1 : 0;
      tiles += (unsigned)nt_i;
    }
    const unsigned most = (unsigned)di.sms * kBlocksPerSm;
    const unsigned per = std::max(1u, (tiles + most - 1) / most), blocks = std::max(1u, (tiles + per - 1) / per);
    err = launch_pdl(adamw_kernel, dim3(blocks), dim3(kThreads), 0, s, tab, ne, tiles, per, h, i >= nt ? 1 : 0);
    if (err != cudaSuccess) return err;
  } while (i < nt);
  return cudaSuccess;
}

}  // namespace moe
