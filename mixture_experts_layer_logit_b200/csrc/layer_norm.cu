// Layer norm over the rows of the residual stream in front of the layer, with
// the residual addition fused in, and its backward with the weights' gradient.
//
//   h = x + add (rounded to x's type when add is given: what is stored as sum)
//   mu = mean h, var = mean (h - mu)^2, r = 1 / sqrt(var + eps)
//   y = (h - mu) r gamma + beta
// With xh = (h - mu) r and g = dy gamma:
//   dh = r (g - mean g - xh mean(g xh)) + dsum
//   dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
//
// Both directions do a few operations per element: they are bound by the bytes
// of their operands.  A row is held in the registers of a group of threads, so
// that every operand is read once; the variance is taken from the centred
// values (two passes over registers, not sums of squares, which cancel when
// the mean is large).  Sums are fp32.
#include "elem8.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kMaxWarps = 32;

// Columns of a thread, eight in each of its NC chunks; t of tpr threads own a
// row.  VEC (the width and every operand allow vector loads of eight elements):
// consecutive ones; else strided by tpr, loaded one by one.
template <bool VEC>
__device__ __forceinline__ int column(int j, int i, int t, int tpr) {
  return VEC ? (j * tpr + t) * 8 + i : (j * 8 + i) * tpr + t;
}

// The raw elements of chunk j of the row that starts at base (zeros past the width).
template <bool VEC>
__device__ __forceinline__ void load_chunk(Raw8& r, const void* p, int dt, size_t base, int j, int t, int tpr, int d) {
  if constexpr (VEC) {
    const int c = column<true>(j, 0, t, tpr);
    if (c < d) {
      load8(r, p, dt, base + c);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.w[i] = 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<false>(j, i, t, tpr);
      r.w[i] = c < d ? load_raw1(p, dt, base + c) : 0u;
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void chunk_to_float(const Raw8& r, int dt, float (&v)[8]) {
  if constexpr (VEC) {
    to_float8(r, dt, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = raw_to_float(r.w[i], dt);
  }
}
template <bool VEC>
__device__ __forceinline__ void store_chunk(void* p, int dt, size_t base, int j, int t, int tpr, int d,
                                            const float (&v)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(j, 0, t, tpr);
    if (c < d) store8(p, dt, base + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<false>(j, i, t, tpr);
      if (c < d) store1(p, dt, base + c, v[i]);
    }
  }
}

// Sum over the tpr threads of a row: lanes of a warp (a power of two up to 32)
// or whole warps (tpr a multiple of 32).  buf: one float2 per warp of the block.
__device__ __forceinline__ float2 row_sum(float2 v, int tpr, float2* buf) {
  const int width = tpr < 32 ? tpr : 32;
  for (int o = width / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (tpr > 32) {
    const int warp = threadIdx.x >> 5, wpr = tpr >> 5, first = warp / wpr * wpr;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
    for (int w = 0; w < wpr; ++w) {
      v.x += buf[first + w].x;
      v.y += buf[first + w].y;
    }
  }
  return v;
}

template <int NC, bool VEC>
__global__ void norm_fwd_kernel(const void* x, const void* add, const void* gamma, const void* beta, void* y,
                                void* sum, float* mean_out, float* rstd_out, int rows, int d, float eps, int xdt,
                                int ydt, int wdt, int adt, int tpr) {
  __shared__ float2 buf[2][kMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr;
  const int row = blockIdx.x * (blockDim.x / tpr) + g;
  const bool live = row < rows;
  const size_t base = (size_t)(live ? row : 0) * d;
  Raw8 rx[NC], ra[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) load_chunk<VEC>(rx[j], x, xdt, base, j, t, tpr, d);
  if (add != nullptr) {
#pragma unroll
    for (int j = 0; j < NC; ++j) load_chunk<VEC>(ra[j], add, adt, base, j, t, tpr, d);
  }
  float h[NC][8];
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    chunk_to_float<VEC>(rx[j], xdt, h[j]);
    if (add != nullptr) {
      float a[8];
      chunk_to_float<VEC>(ra[j], adt, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = round_to(h[j][i] + a[i], xdt);
      if (sum != nullptr && live) store_chunk<VEC>(sum, xdt, base, j, t, tpr, d, h[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s.x += h[j][i];   // columns past the width hold zeros
  }
  const float mu = row_sum(s, tpr, buf[0]).x / (float)d;
  s = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (column<VEC>(j, i, t, tpr) < d) {
        const float v = h[j][i] - mu;
        s.x += v * v;
      }
  const float rstd = 1.f / sqrtf(row_sum(s, tpr, buf[1]).x / (float)d + eps);
  if (!live) return;
  if (t == 0) {
    if (mean_out != nullptr) mean_out[row] = mu;
    if (rstd_out != nullptr) rstd_out[row] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    Raw8 r;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] = (h[j][i] - mu) * rstd;
    if (gamma != nullptr) {
      load_chunk<VEC>(r, gamma, wdt, 0, j, t, tpr, d);
      chunk_to_float<VEC>(r, wdt, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] *= w[i];
    }
    if (beta != nullptr) {
      load_chunk<VEC>(r, beta, wdt, 0, j, t, tpr, d);
      chunk_to_float<VEC>(r, wdt, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] += w[i];
    }
    store_chunk<VEC>(y, ydt, base, j, t, tpr, d, h[j]);
  }
}

// dx of a row at a time; the columns' sums over the block's rows stay with the
// thread that owns the column and end in part[block][2][d].
template <int NC, bool VEC>
__global__ void __launch_bounds__(512)
norm_bwd_kernel(const void* dy, const void* x, const float* __restrict__ mean, const float* __restrict__ rstd,
                const void* gamma, const void* dsum, void* dx, float* __restrict__ part, int rows, int d, int xdt,
                int wdt, int gdt, int odt, int tpr) {
  __shared__ float2 buf[2][kMaxWarps];
  extern __shared__ float cols[];   // [groups][2][d] when several rows share the block
  pdl_wait();
  pdl_launch_dependents();
  const int groups = blockDim.x / tpr;
  const int g = threadIdx.x / tpr, t = threadIdx.x - g * tpr;
  float dg[NC][8], db[NC][8];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[j][i] = db[j][i] = 0.f;
  int turn = 0;
  for (long long r0 = (long long)blockIdx.x * groups; r0 < rows; r0 += (long long)gridDim.x * groups, turn ^= 1) {
    const bool live = r0 + g < rows;
    const long long row = live ? r0 + g : 0;
    const size_t base = (size_t)row * d;
    Raw8 rx[NC], ry[NC], rs_[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      load_chunk<VEC>(ry[j], dy, gdt, base, j, t, tpr, d);
      load_chunk<VEC>(rx[j], x, xdt, base, j, t, tpr, d);
    }
    if (dsum != nullptr) {
#pragma unroll
      for (int j = 0; j < NC; ++j) load_chunk<VEC>(rs_[j], dsum, odt, base, j, t, tpr, d);
    }
    const float mu = mean[row], rs = rstd[row];
    float xh[NC][8], gy[NC][8];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      chunk_to_float<VEC>(rx[j], xdt, xh[j]);
      chunk_to_float<VEC>(ry[j], gdt, gy[j]);
      Raw8 r;
      float w[8];
      if (gamma != nullptr) {
        load_chunk<VEC>(r, gamma, wdt, 0, j, t, tpr, d);
        chunk_to_float<VEC>(r, wdt, w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[j][i] = (xh[j][i] - mu) * rs;   // of no use past the width, where dy is zero
        if (live) {
          dg[j][i] += gy[j][i] * xh[j][i];
          db[j][i] += gy[j][i];
        }
        if (gamma != nullptr) gy[j][i] *= w[i];
        s.x += gy[j][i];
        s.y += gy[j][i] * xh[j][i];
      }
    }
    s = row_sum(s, tpr, buf[turn]);
    const float a = s.x / (float)d, b = s.y / (float)d;
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float w[8];
      if (dsum != nullptr) chunk_to_float<VEC>(rs_[j], odt, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[j][i] = rs * (gy[j][i] - a - xh[j][i] * b);
        if (dsum != nullptr) xh[j][i] += w[i];
      }
      store_chunk<VEC>(dx, odt, base, j, t, tpr, d, xh[j]);
    }
  }
  if (part == nullptr) return;
  float* out = part + (size_t)blockIdx.x * 2 * d;
  float* mine = groups == 1 ? out : cols + (size_t)g * 2 * d;
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>(j, i, t, tpr);
      if (c < d) {
        mine[c] = dg[j][i];
        mine[d + c] = db[j][i];
      }
    }
  if (groups == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) {
    float v = 0.f;
    for (int q = 0; q < groups; ++q) v += cols[(size_t)q * 2 * d + c];
    out[c] = v;
  }
}

// dgamma and dbeta: the blocks' partial sums of each column.  A block takes 32
// columns; its eight warps each add a run of the parts, and the runs are added
// in order.
__global__ void __launch_bounds__(256)
norm_weights_kernel(const float* __restrict__ part, int nparts, int d, float* dgamma, float* dbeta) {
  __shared__ float runs[8][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int p0 = (int)((long long)nparts * warp / 8), p1 = (int)((long long)nparts * (warp + 1) / 8);
  float v = 0.f;
  if (c < 2 * d) {
#pragma unroll 8
    for (int p = p0; p < p1; ++p) v += part[(size_t)p * 2 * d + c];
  }
  runs[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || c >= 2 * d) return;
  v = 0.f;
  for (int w = 0; w < 8; ++w) v += runs[w][lane];
  if (c < d) {
    if (dgamma != nullptr) dgamma[c] = v;
  } else if (dbeta != nullptr) {
    dbeta[c - d] = v;
  }
}

// The width and a pointer allow vector accesses of eight elements.
bool vector_width(int d) { return d % 8 == 0; }
bool on_vector(const void* p, int dt) { return reinterpret_cast<uintptr_t>(p) % (8u * dtype_bytes(dt)) == 0; }

// Threads of a row, eight elements each or more: a power of two inside a warp, else whole warps up to `most`.
int threads_per_row(int d, int most) {
  const int chunks = (d + 7) / 8;
  if (chunks <= 32) {
    int t = 1;
    while (t < chunks) t *= 2;
    return t;
  }
  return std::min(most, (chunks + 31) / 32 * 32);
}

}  // namespace

// Blocks of the backward, each of which leaves one partial of the weights' gradient.
int norm_bwd_blocks(const moe_norm_config& c) {
  const int tpr = threads_per_row(c.d, 512), groups = std::max(1, 256 / tpr);
  return (int)std::max<long long>(1, std::min<long long>(((long long)c.rows + groups - 1) / groups, 2 * 148));
}

cudaError_t launch_norm_fwd(const moe_norm_config& c, const void* x, const void* add, const void* gamma,
                            const void* beta, void* y, void* sum, float* mean, float* rstd, cudaStream_t s) {
  const int tpr = threads_per_row(c.d, 512), nc = ((c.d + 7) / 8 + tpr - 1) / tpr;
  const int threads = std::max(tpr, 256 / tpr * tpr), groups = threads / tpr;
  const dim3 grid((unsigned)(((long long)c.rows + groups - 1) / groups));
  const bool vec = vector_width(c.d) && on_vector(x, c.x_dtype) && on_vector(add, c.add_dtype) &&
                   on_vector(gamma, c.w_dtype) && on_vector(beta, c.w_dtype) && on_vector(y, c.y_dtype) &&
                   on_vector(sum, c.x_dtype);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(threads), 0, s, x, add, gamma, beta, y, sum, mean, rstd, c.rows, c.d, c.eps,
                      c.x_dtype, c.y_dtype, c.w_dtype, c.add_dtype, tpr);
  };
  if (vec)
    return nc == 1 ? go(norm_fwd_kernel<1, true>) : nc == 2 ? go(norm_fwd_kernel<2, true>) : go(norm_fwd_kernel<4, true>);
  return nc == 1 ? go(norm_fwd_kernel<1, false>)
                 : nc == 2 ? go(norm_fwd_kernel<2, false>) : go(norm_fwd_kernel<4, false>);
}

cudaError_t launch_norm_bwd(const moe_norm_config& c, const void* dy, const void* x, const float* mean,
                            const float* rstd, const void* gamma, const void* dsum, void* dx, float* dgamma,
                            float* dbeta, float* part, cudaStream_t s) {
  const int tpr = threads_per_row(c.d, 512), nc = ((c.d + 7) / 8 + tpr - 1) / tpr;
  const int threads = std::max(tpr, 256 / tpr * tpr), groups = threads / tpr, blocks = norm_bwd_blocks(c);
  float* partials = dgamma != nullptr || dbeta != nullptr ? part : nullptr;
  // several groups have tpr <= 128 threads of one chunk: at most 16 KB
  const size_t smem = groups > 1 && partials != nullptr ? (size_t)groups * 2 * c.d * sizeof(float) : 0;
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(blocks), dim3(threads), smem, s, dy, x, mean, rstd, gamma, dsum, dx, partials,
                      c.rows, c.d, c.x_dtype, c.w_dtype, c.dy_dtype, c.dx_dtype, tpr);
  };
  const bool vec = vector_width(c.d) && on_vector(dy, c.dy_dtype) && on_vector(x, c.x_dtype) &&
                   on_vector(gamma, c.w_dtype) && on_vector(dsum, c.dx_dtype) && on_vector(dx, c.dx_dtype);
  cudaError_t e;
  if (vec)
    e = nc == 1 ? go(norm_bwd_kernel<1, true>) : nc == 2 ? go(norm_bwd_kernel<2, true>) : go(norm_bwd_kernel<4, true>);
  else
    e = nc == 1 ? go(norm_bwd_kernel<1, false>)
                : nc == 2 ? go(norm_bwd_kernel<2, false>) : go(norm_bwd_kernel<4, false>);
  if (e != cudaSuccess || partials == nullptr) return e;
  return launch_pdl(norm_weights_kernel, dim3((2 * c.d + 31) / 32), dim3(256), 0, s, (const float*)part, blocks,
                    c.d, dgamma, dbeta);
}

}  // namespace moe
