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
// 12 to 30 bytes an element are the floor.  32-bit states reach it (67 M
// elements with master copies: 326 us, 6.2 TB/s); with 8-bit states some 51
// instructions an element (two conversions each way, a root, a reciprocal, two
// maxima) take as long as the 12 bytes, and the kernel is bound by issue as
// much as by memory (0.55 G elements: 1185 us, 5.6 TB/s; 69 M in 5 tensors 153
// us, in 160 tensors 181, a quarter more instructions).  Hence few
// instructions: see root_in_range, the common path of encode, and the types
// taken out of the loop.  m and v are computed in separately rounded steps (no
// contraction), so that a code does not depend on how a compiler fuses them.
#include "adamw_access.cuh"
#include "elem8.cuh"

#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

constexpr int kBlock = MOE_ADAMW_BLOCK;
constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 2;   // with three the registers spill and the memory sees more streams: 4 % slower
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
  float decay;   // 1 - lr wd is formed on the device (lr may be there)
  unsigned char pdt, gdt, bits, vec;
};
constexpr int kMaxEntries = 340;
template <int CAP>
struct Table {
  Entry e[CAP];
  unsigned tile0[CAP + 1];   // first tile of each tensor, then the number of tiles
};
static_assert(sizeof(Table<kMaxEntries>) + 128 <= 32764, "kernel parameters");

struct Hyper {
  float lr, beta1, omb1, beta2, omb2, lnb1, lnb2, eps;
  const float* lr_dev;
  const float* grad_scale;
  moe_adamw_state* state;
};

// What every element of a step shares.
struct Step {
  float beta1, omb1, beta2, omb2, eps, gs, alpha, rc2, keep;
};

// 1 / v to about an ulp; v is a normal number here
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// sqrt(v) rounded to nearest for 2^-100 <= v < inf, without the library's
// branch for the other values: with y near 1 / sqrt(v) and s = v y, the residual
// v - s s is exact in one FMA and s + (v - s s) y / 2 rounds correctly
// (Markstein's correction step; tests/test_gpu_adamw_root.py compares the scales
// that come of it for every mantissa under an even and an odd exponent).
constexpr float kRootLow = 0x1p-100f;
__device__ __forceinline__ float root_in_range(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  const float s = __fmul_rn(v, y);
  return __fmaf_rn(__fmaf_rn(-s, s, v), __fmul_rn(y, 0.5f), s);
}

// Codes of the warp's block of eight values a lane, element i in byte i.  inv
// brings the block's largest finite |v| to 448.  ODD: some value is not finite
// or some root is zero.  Otherwise roots are lifted to the smallest code by a
// maximum, and the conversion's NaN code is the one wanted.
template <bool ROOT>
__device__ __forceinline__ uint2 encode(const float (&v)[8], float inv, bool odd) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = __fmul_rn(v[2 * i], inv), b = __fmul_rn(v[2 * i + 1], inv);
    if (ROOT) a = fmaxf(a, 0x1p-9f), b = fmaxf(b, 0x1p-9f);
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  }
  if (odd) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ROOT && v[2 * i] == 0.f) w[i] &= 0xff00u;
      if (ROOT && v[2 * i + 1] == 0.f) w[i] &= 0xffu;
      if (!isfinite(v[2 * i])) w[i] = (w[i] & 0xff00u) | 0x7fu;
      if (!isfinite(v[2 * i + 1])) w[i] = (w[i] & 0xffu) | 0x7f00u;
    }
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The largest finite |v| of the warp's block
__device__ __forceinline__ float finite_top(const float (&v)[8]) {
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (isfinite(v[i])) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}

__device__ __forceinline__ void decode(uint2 c, float scale, float (&v)[8]) {
  const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[i], __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = __fmul_rn(f.x, scale);
    v[2 * i + 1] = __fmul_rn(f.y, scale);
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

// A lane's share of a block of 256 elements as it was loaded.
template <int BITS>
struct Raw {
  Raw8 g, p, m, v;
};
template <>
struct Raw<8> {
  Raw8 g, p;
  uint2 m, v;
  float ms, vs;
};

// One warp, one block of 256 elements from b0 on.  Lane l holds elements l,
// l + 32, ... as far as the tensor goes, loaded one by one.
template <int BITS>
__device__ __forceinline__ void load_single(Raw<BITS>& r, const Entry& e, long long b0, int lane) {
  const void* psrc = e.master != nullptr ? e.master : e.param;
  const int psdt = e.master != nullptr ? MOE_DTYPE_F32 : e.pdt;
  const int count = (int)min((long long)kBlock, e.n - b0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long at = b0 + i * 32 + lane;
    const bool here = i * 32 + lane < count;
    r.g.w[i] = here ? load_raw1(e.grad, e.gdt, at) : 0u;
    r.p.w[i] = here ? load_raw1(psrc, psdt, at) : 0u;
    if constexpr (BITS == 32) {
      r.m.w[i] = here ? load_raw1(e.m, MOE_DTYPE_F32, at) : 0u;
      r.v.w[i] = here ? load_raw1(e.v, MOE_DTYPE_F32, at) : 0u;
    }
  }
  if constexpr (BITS == 8) {
    r.ms = e.ms[b0 / kBlock];
    r.vs = e.vs[b0 / kBlock];
    r.m = load_codes1(static_cast<const unsigned char*>(e.m) + b0, count, lane);
    r.v = load_codes1(static_cast<const unsigned char*>(e.v) + b0, count, lane);
  }
}

// A whole block, lane l with elements 8 l .. 8 l + 7.  With 32-bit states the
// bytes are many for the work: plain loads of 32 bytes keep the memory busy.
__device__ __forceinline__ void load8(Raw8& r, const void* p, int dt, long long i) {
  if (dt == MOE_DTYPE_F32)
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(static_cast<const float*>(p) + i));
  else
    load16(static_cast<const unsigned short*>(p) + i, r.w[0], r.w[1], r.w[2], r.w[3]);
}
__device__ __forceinline__ void load_whole(Raw<32>& r, const Entry& e, long long b0, int lane) {
  const long long at = b0 + lane * 8;
  load8(r.g, e.grad, e.gdt, at);
  if (e.master != nullptr) load8(r.p, e.master, MOE_DTYPE_F32, at);
  else load8(r.p, e.param, e.pdt, at);
  load8(r.m, e.m, MOE_DTYPE_F32, at);
  load8(r.v, e.v, MOE_DTYPE_F32, at);
}

// With 8-bit states the arithmetic weighs as much as the bytes, and a block's
// loads would have to wait for it: the warp copies its next block to shared
// memory, in whole lines, while it works on one.
constexpr int kStageG = 0, kStageP = 1024, kStageM = 2048, kStageV = 2304, kStageBytes = 2560;
constexpr int kStages = 2;

// 256 elements of type dt, 1024 or 512 bytes
__device__ __forceinline__ void copy_row(uint32_t to, const void* p, int dt, long long i, int lane) {
  const char* from = static_cast<const char*>(p) + i * (dt == MOE_DTYPE_F32 ? 4 : 2) + lane * 16;
  copy16(to + lane * 16, from);
  if (dt == MOE_DTYPE_F32) copy16(to + 512 + lane * 16, from + 512);
}
__device__ __forceinline__ void copy_block(uint32_t st, const Entry& e, long long b0, int lane) {
  copy_row(st + kStageG, e.grad, e.gdt, b0, lane);
  if (e.master != nullptr) copy_row(st + kStageP, e.master, MOE_DTYPE_F32, b0, lane);
  else copy_row(st + kStageP, e.param, e.pdt, b0, lane);
  // 16 lanes each for the codes of m and v, which lie one after the other
  copy16(st + kStageM + lane * 16, static_cast<const char*>(lane < 16 ? e.m : e.v) + b0 + (lane & 15) * 16);
}

__device__ __forceinline__ void shared_row(Raw8& r, uint32_t at, int dt, int lane) {
  at += lane * (dt == MOE_DTYPE_F32 ? 32 : 16);
  shared16(at, r.w[0], r.w[1], r.w[2], r.w[3]);
  if (dt == MOE_DTYPE_F32) shared16(at + 16, r.w[4], r.w[5], r.w[6], r.w[7]);
}
__device__ __forceinline__ void load_staged(Raw<8>& r, uint32_t st, const Entry& e, int lane) {
  shared_row(r.g, st + kStageG, e.gdt, lane);
  shared_row(r.p, st + kStageP, e.master != nullptr ? MOE_DTYPE_F32 : e.pdt, lane);
  shared8(st + kStageM + lane * 8, r.m.x, r.m.y);
  shared8(st + kStageV + lane * 8, r.v.x, r.v.y);
}

template <bool VEC, int BITS>
__device__ __forceinline__ void update_block(const Raw<BITS>& r, const Entry& e, long long b0, int lane,
                                             const Step& s) {
  const int count = VEC ? kBlock : (int)min((long long)kBlock, e.n - b0);
  const long long at = VEC ? b0 + lane * 8 : b0 + lane;
  const bool has_master = e.master != nullptr;
  const int psdt = has_master ? MOE_DTYPE_F32 : e.pdt;
  float g[8], p[8], m[8], v[8], root[8];
  if constexpr (VEC) {
    to_float8(r.g, e.gdt, g);
    to_float8(r.p, psdt, p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = raw_to_float(r.g.w[i], e.gdt);
      p[i] = raw_to_float(r.p.w[i], psdt);
    }
  }
  if constexpr (BITS == 8) {
    decode(r.m, r.ms, m);
    decode(r.v, r.vs, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
  } else {
    to_float8(r.m, MOE_DTYPE_F32, m);
    to_float8(r.v, MOE_DTYPE_F32, v);
  }
  // the bits of v >= 0 order like v, an inf's and a NaN's above all others
  unsigned low = ~0u, high = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = __fmul_rn(g[i], s.gs);
    m[i] = __fadd_rn(__fmul_rn(m[i], s.beta1), __fmul_rn(gi, s.omb1));
    v[i] = __fadd_rn(__fmul_rn(v[i], s.beta2), __fmul_rn(__fmul_rn(gi, gi), s.omb2));
    low = min(low, __float_as_uint(v[i]));
    high = max(high, __float_as_uint(v[i]));
  }
  high = __reduce_max_sync(0xffffffffu, high);
  // all zero: an expert that has not seen a token yet.  odd: some v out of the range of root_in_range
  const bool zero = high == 0u;
  const bool odd = !zero && (high >= 0x7f800000u || __any_sync(0xffffffffu, low < __float_as_uint(kRootLow)));
  if (zero) {
#pragma unroll
    for (int i = 0; i < 8; ++i) root[i] = 0.f;
  } else if (!odd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) root[i] = root_in_range(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) root[i] = sqrtf(v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    p[i] = fmaf(p[i], s.keep, m[i] * s.alpha * reciprocal(fmaf(root[i], s.rc2, s.eps)));
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
    float mt = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) mt = fmaxf(mt, fabsf(m[i]));   // leaves NaN out
    mt = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mt)));
    const bool inf = mt == INFINITY;
    if (inf) mt = finite_top(m);
    // the largest root is the root of the largest v
    float vt = zero ? 0.f : odd ? finite_top(root) : root_in_range(__uint_as_float(high));
    mt = fmaxf(mt, 0x1p-100f);   // the reciprocals stay finite
    vt = fmaxf(vt, 0x1p-100f);
    const uint2 cm = encode<false>(m, __fmul_rn(__frcp_rn(mt), 448.f), inf);
    const uint2 cv = zero ? make_uint2(0u, 0u) : encode<true>(root, __fmul_rn(__frcp_rn(vt), 448.f), odd);
    if (lane == 0) {
      e.ms[b0 / kBlock] = __fmul_rn(mt, 1.f / 448.f);
      e.vs[b0 / kBlock] = __fmul_rn(vt, 1.f / 448.f);
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

// A block whose copies are under way, and its scales.
struct Ahead {
  uint32_t stage;   // 0 or kStageBytes: where the next block to be worked on lies, or will
  float ms, vs;
};

__device__ __forceinline__ bool staged8(const Entry& e, long long b0) {
  return e.bits == 8 && e.vec && b0 + kBlock <= e.n;
}
__device__ __forceinline__ void start_copy(Ahead& a, const Entry& e, long long b0, uint32_t to, int lane) {
  copy_block(to, e, b0, lane);
  a.ms = e.ms[b0 / kBlock];
  a.vs = e.vs[b0 / kBlock];
}

// The warp's blocks of one tensor, from b0 on, `step` apart.  8-bit states:
// started says that the first one's copies are under way; next(to) starts those
// of the warp's first block in the tensor that it will see next.
template <int BITS, typename Next>
__device__ __forceinline__ void run_tensor(const Entry e, long long b0, long long step, uint32_t stages, int lane,
                                           const Step& s, Ahead& ahead, bool started, Next next) {
  if (e.vec) {
    if constexpr (BITS == 8) {
      if (!started && b0 + kBlock <= e.n) {
        start_copy(ahead, e, b0, stages + ahead.stage, lane);
        copy_commit();
      }
      while (b0 + kBlock <= e.n) {
        Raw<8> r;
        r.ms = ahead.ms;
        r.vs = ahead.vs;
        const uint32_t at = stages + ahead.stage;
        ahead.stage ^= kStageBytes;
        b0 += step;
        if (b0 + kBlock <= e.n) start_copy(ahead, e, b0, stages + ahead.stage, lane);
        else next(stages + ahead.stage);
        copy_commit();
        copy_wait<1>();
        __syncwarp();   // every lane's part of the block has arrived
        load_staged(r, at, e, lane);
        __syncwarp();   // and has been read: the stage may be filled again
        update_block<true, 8>(r, e, b0 - step, lane, s);
      }
    } else {
      for (; b0 + kBlock <= e.n; b0 += step) {
        Raw<32> r;
        load_whole(r, e, b0, lane);
        update_block<true, 32>(r, e, b0, lane, s);
      }
    }
  }
  for (; b0 < e.n; b0 += step) {
    Raw<BITS> r;
    load_single<BITS>(r, e, b0, lane);
    update_block<false, BITS>(r, e, b0, lane, s);
  }
}

// Tiles go round the blocks: all of them work on neighbouring lines (a run of
// its own for each block took 1450 us where this took 1200), and many small
// tensors are shared out.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
adamw_kernel(const __grid_constant__ Table<CAP> tab, int ntensors, unsigned ntiles, Hyper h, int last_launch) {
  extern __shared__ __align__(128) unsigned char staged[];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int step = h.state->step + 1;
  const float t = (float)step;
  Step s;
  s.beta1 = h.beta1, s.omb1 = h.omb1, s.beta2 = h.beta2, s.omb2 = h.omb2, s.eps = h.eps;
  s.gs = h.grad_scale != nullptr ? *h.grad_scale : 1.f;
  const float lr = h.lr_dev != nullptr ? *h.lr_dev : h.lr;
  // 1 - beta^t = -expm1(t ln beta): exact to rounding also for the first steps
  s.alpha = lr / expm1f(t * h.lnb1);   // -lr / c1
  s.rc2 = 1.f / sqrtf(-expm1f(t * h.lnb2));
  const uint32_t stages = (uint32_t)__cvta_generic_to_shared(staged) + warp * kStages * kStageBytes;
  // the tensor of a tile, looked for from `from` on: mostly one of the next few
  auto tensor_of = [&](unsigned tile, int from) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i, ++from)
      if (tab.tile0[from + 1] > tile) return from;   // tile < tile0[ntensors]
    int hi = ntensors - 1;
    while (from < hi) {
      const int mid = (from + hi + 1) >> 1;
      if (tab.tile0[mid] <= tile) from = mid; else hi = mid - 1;
    }
    return from;
  };
  const long long stride = (long long)gridDim.x * kTile;
  Ahead ahead{0, 0.f, 0.f};
  bool started = false;
  unsigned tile = blockIdx.x;
  int at = tile < ntiles ? tensor_of(tile, 0) : 0;
  while (tile < ntiles) {
    const Entry& e = tab.e[at];
    const unsigned stop = tab.tile0[at + 1];
    // the block's first tile of a later tensor
    const unsigned tile1 = tile + (stop - tile + gridDim.x - 1) / gridDim.x * gridDim.x;
    const int at1 = tile1 < ntiles ? tensor_of(tile1, at) : at;
    const long long b0 = (long long)(tile - tab.tile0[at]) * kTile + warp * kBlock;
    const long long b1 = (long long)(tile1 - tab.tile0[at1]) * kTile + warp * kBlock;
    bool started1 = false;
    s.keep = 1.f - lr * e.decay;
    auto next = [&](uint32_t to) {
      if (tile1 >= ntiles || !staged8(tab.e[at1], b1)) return;
      start_copy(ahead, tab.e[at1], b1, to, lane);
      started1 = true;
    };
    if (e.bits == 8) {
      // The arithmetic of 8-bit states is near the bytes' time: fp32 gradients (the layer's) of bf16 or fp16
      // weights without a master copy get code without decisions on types (0.55 G elements: 1186 us where it takes
      // 1305; 69 M in 160 tensors: 181 and 193).
      Entry f = e;
      const bool plain = e.gdt == MOE_DTYPE_F32 && e.master == nullptr;
      if (plain) f.gdt = MOE_DTYPE_F32, f.master = nullptr;
      if (plain && e.pdt == MOE_DTYPE_BF16) {
        f.pdt = MOE_DTYPE_BF16;
        run_tensor<8>(f, b0, stride, stages, lane, s, ahead, started, next);
      } else if (plain && e.pdt == MOE_DTYPE_F16) {
        f.pdt = MOE_DTYPE_F16;
        run_tensor<8>(f, b0, stride, stages, lane, s, ahead, started, next);
      } else {
        run_tensor<8>(e, b0, stride, stages, lane, s, ahead, started, next);
      }
    }
    else run_tensor<32>(e, b0, stride, stages, lane, s, ahead, false, next);
    started = started1;
    tile = tile1;
    at = at1;
  }
  if (!last_launch) return;
  // The last block to finish counts the step: by then every block has read it.
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicInc(&h.state->ticket, gridDim.x - 1) == gridDim.x - 1) h.state->step = step;
  }
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
  h.lr_dev = lr_dev;
  h.grad_scale = grad_scale;
  h.state = state;
  constexpr size_t kSmem = (size_t)kStages * kStageBytes * (kThreads / 32);
  static thread_local Table<kMaxEntries> tab, packed;   // 25 KB each: off the caller's stack
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
      tab.tile0[ne - 1] = tiles;
      e.pdt = (unsigned char)t[i].param_dtype;
      e.gdt = (unsigned char)t[i].grad_dtype;
      e.bits = (unsigned char)t[i].state_bits;
      e.vec = adamw_by_vectors(t[i]) ? 1 : 0;
      tiles += (unsigned)nt_i;
    }
    const unsigned most = (unsigned)di.sms * kBlocksPerSm;
    const unsigned per = std::max(1u, (tiles + most - 1) / most), blocks = std::max(1u, (tiles + per - 1) / per);
    tab.tile0[ne] = tiles;
    // the smallest parameter block that holds the tensors: a launch copies it whole
    auto go = [&](auto cap) {
      constexpr int CAP = decltype(cap)::value;
      const cudaError_t set = set_smem_once<adamw_kernel<CAP>>(kSmem);
      if (set != cudaSuccess) return set;
      Table<CAP>& t = *reinterpret_cast<Table<CAP>*>(&packed);
      std::copy(tab.e, tab.e + ne, t.e);
      std::copy(tab.tile0, tab.tile0 + ne + 1, t.tile0);
      return launch_pdl(adamw_kernel<CAP>, dim3(blocks), dim3(kThreads), kSmem, s, t, ne, tiles, h, i >= nt ? 1 : 0);
    };
    err = ne <= 8 ? go(std::integral_constant<int, 8>{})
                  : ne <= 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, kMaxEntries>{});
    if (err != cudaSuccess) return err;
  } while (i < nt);
  return cudaSuccess;
}

}  // namespace moe
