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
  unsigned char pdt, gdt, bits, pad[5];
};
constexpr int kMaxEntries = 340;
struct Table {
  Entry e[kMaxEntries];
};
static_assert(sizeof(Table) + 128 <= 32764, "kernel parameters");

struct Hyper {
  float lr, beta1, omb1, beta2, omb2, lnb1, lnb2, eps;
  const float* lr_dev;
  const float* grad_scale;
  moe_adamw_state* state;
};

__device__ __forceinline__ float quantised(float v, float inv, bool root, unsigned char* code) {
  float q = __fmul_rn(v, inv);
  q = fminf(fmaxf(q, -448.f), 448.f);
  unsigned char c = __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
  if (root && v > 0.f && c == 0) c = 1;
  *code = isfinite(v) ? c : 0x7f;
  return q;
}

__device__ __forceinline__ float from_code(unsigned char c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__global__ void __launch_bounds__(kThreads)
adamw_kernel(const __grid_constant__ Table tab, int ntensors, unsigned ntiles, Hyper h, int last_launch) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int step = h.state->step + 1;
  const float t = (float)step;
  // 1 - beta^t = -expm1(t ln beta): exact to rounding also for the first steps
  const float c1 = -expm1f(t * h.lnb1), rc2 = sqrtf(-expm1f(t * h.lnb2));
  const float lr = h.lr_dev != nullptr ? *h.lr_dev : h.lr;
  const float gs = h.grad_scale != nullptr ? *h.grad_scale : 1.f;
  const float alpha = lr / c1;
  for (unsigned tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
    int lo = 0, hi = ntensors - 1;   // the last tensor that starts at or before the tile
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.e[mid].tile0 <= tile) lo = mid; else hi = mid - 1;
    }
    const Entry& e = tab.e[lo];
    const long long b0 = (long long)(tile - e.tile0) * kTile + warp * kBlock;   // the warp's block
    if (b0 >= e.n) continue;
    const float keep = 1.f - lr * e.decay;
    const long long blk = b0 / kBlock;
    float ms = 0.f, vs = 0.f;
    if (e.bits == 8) {
      ms = e.ms[blk];
      vs = e.vs[blk];
    }
    float m[8], v[8], mmax = 0.f, vmax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long at = b0 + i * 32 + lane;
      m[i] = v[i] = 0.f;
      if (at >= e.n) continue;
      const float g = __fmul_rn(raw_to_float(load_raw1(e.grad, e.gdt, at), e.gdt), gs);
      if (e.bits == 8) {
        m[i] = __fmul_rn(from_code(static_cast<const unsigned char*>(e.m)[at]), ms);
        const float r = __fmul_rn(from_code(static_cast<const unsigned char*>(e.v)[at]), vs);
        v[i] = __fmul_rn(r, r);
      } else {
        m[i] = static_cast<const float*>(e.m)[at];
        v[i] = static_cast<const float*>(e.v)[at];
      }
      m[i] = __fadd_rn(__fmul_rn(m[i], h.beta1), __fmul_rn(g, h.omb1));
      v[i] = __fadd_rn(__fmul_rn(v[i], h.beta2), __fmul_rn(__fmul_rn(g, g), h.omb2));
      const float root = sqrtf(v[i]);
      float p = e.master != nullptr ? e.master[at] : raw_to_float(load_raw1(e.param, e.pdt, at), e.pdt);
      p = p * keep - alpha * m[i] / (root / rc2 + h.eps);
      if (e.master != nullptr) e.master[at] = p;
      store1(e.param, e.pdt, at, p);
      if (e.bits == 8) {
        v[i] = root;
        if (isfinite(m[i])) mmax = fmaxf(mmax, fabsf(m[i]));
        if (isfinite(root)) vmax = fmaxf(vmax, root);
      } else {
        static_cast<float*>(e.m)[at] = m[i];
        static_cast<float*>(e.v)[at] = v[i];
      }
    }
    if (e.bits != 8) continue;
    mmax = fmaxf(warp_max(mmax), 0x1p-100f);   // keeps the reciprocal finite
    vmax = fmaxf(warp_max(vmax), 0x1p-100f);
    const float mi = __fmul_rn(__frcp_rn(mmax), 448.f), vi = __fmul_rn(__frcp_rn(vmax), 448.f);
    if (lane == 0) {
      e.ms[blk] = __fmul_rn(mmax, 1.f / 448.f);
      e.vs[blk] = __fmul_rn(vmax, 1.f / 448.f);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long at = b0 + i * 32 + lane;
      if (at >= e.n) continue;
      quantised(m[i], mi, false, static_cast<unsigned char*>(e.m) + at);
      quantised(v[i], vi, true, static_cast<unsigned char*>(e.v) + at);
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
      tiles += (unsigned)nt_i;
    }
    const int blocks = (int)std::max<long long>(1, std::min<long long>(tiles, (long long)di.sms * 8));
    err = launch_pdl(adamw_kernel, dim3(blocks), dim3(kThreads), 0, s, tab, ne, tiles, h, i >= nt ? 1 : 0);
    if (err != cudaSuccess) return err;
  } while (i < nt);
  return cudaSuccess;
}

}  // namespace moe
