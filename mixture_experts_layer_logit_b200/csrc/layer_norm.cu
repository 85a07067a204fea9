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
// Both directions do a few operations per element: their floor is the bytes of
// their operands.  A row is held in the registers of a group of threads, so
// that every operand is read once; the variance is taken from the centred
// values (two passes over registers, not sums of squares, which cancel when
// the mean is large).  Sums are fp32.  16384 x 4096 with an fp32 stream: forward
// 140 us (940 MB, 6.7 TB/s), backward 172 us (1.07 GB, 6.2 TB/s).  With 16-bit
// operands the instructions of a row (more than 20 an element) take longer than its
// bytes: 8192 x 4096 in bf16 36.6 us forward (3.7 TB/s, 62 % of the issue slots).
#include "elem8.cuh"
#include "tc_ptx.cuh"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace moe {
namespace {

constexpr int kMaxWarps = 32;   // of a block
constexpr int kMaxStages = 4;   // of the backward's ring

// How a thread sees a row.  Its columns are eight in each of its NC chunks; t of
// tpr threads own a row.  kSingle: strided by tpr, one by one.  kVector (the
// width and every operand allow vectors of four elements): two runs of four,
// each a whole line over a warp.  kWhole: the same, and every column exists.
enum Mode { kSingle, kVector, kWhole };

struct Geometry {
  int rows, d, tpr, groups;   // groups of tpr threads in a block, a row each
  unsigned magic;             // ceil(2^16 / tpr): threadIdx / tpr without a division
  float fd, inv_d;
};

struct Place {
  int group, t;
  __device__ __forceinline__ explicit Place(const Geometry& G) {
    group = G.groups == 1 ? 0 : (int)((threadIdx.x * G.magic) >> 16);
    t = threadIdx.x - group * G.tpr;
  }
};

template <Mode M>
__device__ __forceinline__ int column(int j, int i, int t, int tpr) {
  return M != kSingle ? ((2 * j + i / 4) * tpr + t) * 4 + (i & 3) : (j * 8 + i) * tpr + t;
}
template <Mode M>
__device__ __forceinline__ bool inside(int c, int d) {
  return M == kWhole || c < d;
}

// The raw elements of chunk j of the row that starts at base (zeros past the
// width).  WEIGHTS: gamma or beta, which every row reads again and L1 keeps.
template <Mode M, bool WEIGHTS = false>
__device__ __forceinline__ void load_chunk(Raw8& r, const void* p, int dt, size_t base, int j, int t, int tpr, int d) {
  if constexpr (M != kWhole) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = 0u;
  }
  if constexpr (M != kSingle) {
    const int c = column<M>(j, 0, t, tpr), c2 = column<M>(j, 4, t, tpr);
    auto quad = [&](int q, int type, int col) {
      if constexpr (WEIGHTS) load4_cached(r, q, p, type, col);
      else load4(r, q, p, type, base + col);
    };
    if (dt == MOE_DTYPE_F32) {
      if (inside<M>(c, d)) quad(0, MOE_DTYPE_F32, c);
      if (inside<M>(c2, d)) quad(1, MOE_DTYPE_F32, c2);
    } else {
      if (inside<M>(c, d)) quad(0, MOE_DTYPE_BF16, c);
      if (inside<M>(c2, d)) quad(1, MOE_DTYPE_BF16, c2);
    }
  } else {
    if (dt == MOE_DTYPE_F32) {
      const uint32_t* f = static_cast<const uint32_t*>(p) + base;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (column<M>(j, i, t, tpr) < d) r.w[i] = f[column<M>(j, i, t, tpr)];
    } else {
      const unsigned short* f = static_cast<const unsigned short*>(p) + base;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (column<M>(j, i, t, tpr) < d) r.w[i] = f[column<M>(j, i, t, tpr)];
    }
  }
}
template <Mode M>
__device__ __forceinline__ void chunk_to_float(const Raw8& r, int dt, float (&v)[8]) {
  if constexpr (M != kSingle) {
    to_float8(r, dt, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = raw_to_float(r.w[i], dt);
  }
}
template <Mode M>
__device__ __forceinline__ void store_chunk(void* p, int dt, size_t base, int j, int t, int tpr, int d,
                                            const float (&v)[8]) {
  auto as = [&](int type) {
    if constexpr (M != kSingle) {
      const int c = column<M>(j, 0, t, tpr), c2 = column<M>(j, 4, t, tpr);
      if (inside<M>(c, d)) store4(p, type, base + c, v[0], v[1], v[2], v[3]);
      if (inside<M>(c2, d)) store4(p, type, base + c2, v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (column<M>(j, i, t, tpr) < d) store1(p, type, base + column<M>(j, i, t, tpr), v[i]);
    }
  };
  if (dt == MOE_DTYPE_F32) as(MOE_DTYPE_F32);
  else if (dt == MOE_DTYPE_BF16) as(MOE_DTYPE_BF16);
  else as(MOE_DTYPE_F16);
}

// Sums over the tpr threads of a row: lanes of a warp (a power of two up to 32)
// or up to 32 whole warps (tpr a multiple of 32), whose partials meet in buf
// (one entry per warp of the block) and are added by every warp for itself.
__device__ __forceinline__ float2 add(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float2 from_lane(float2 v, int o) {
  return make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o));
}
__device__ __forceinline__ float from_lane(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

template <typename T>
__device__ __forceinline__ T row_sum(T v, int tpr, int group, T* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < tpr) v = add(v, from_lane(v, o));
  if (tpr > 32) {
    const int lane = threadIdx.x & 31, wpr = tpr >> 5;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = T{};
    if (wpr > 16) {
      if (lane < wpr) v = buf[lane];
      v = add(v, from_lane(v, 16));
    } else if ((lane & 15) < wpr) {
      v = buf[group * wpr + (lane & 15)];
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = add(v, from_lane(v, o));
  }
  return v;
}

// s / d rounded to nearest, with inv = 1 / d: the quotient's exact residual
// corrects it (Markstein's correction step).  An infinite s has no residual and
// stays infinite.
__device__ __forceinline__ float over(float s, float d, float inv) {
  const float q = s * inv;
  return isinf(q) ? q : fmaf(fmaf(-q, d, s), inv, q);
}

// 1 / sqrt(v) to about an ulp: one Newton step on the approximation (which is
// 0 for an infinite v, and stays so).  The half goes with y, of which it is
// exact: v may be subnormal.
__device__ __forceinline__ float inverse_root(float v) {
  const float y = rsqrtf(v);
  return v == INFINITY ? y : y * fmaf(-0.5f * y * v, y, 1.5f);
}

struct NormFwd {
  Geometry G;
  const void* x;
  const void* add;
  const void* gamma;
  const void* beta;
  void* y;
  void* sum;
  float* mean;
  float* rstd;
  float eps;
  int xdt, ydt, wdt, adt;
};

// Chunk j of gamma and beta (1 and 0 without them).
template <Mode M>
__device__ __forceinline__ void load_affine(const NormFwd& a, int j, int t, float (&w)[8], float (&b)[8]) {
  Raw8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f, b[i] = 0.f;
  if (a.gamma != nullptr) {
    load_chunk<M, true>(r, a.gamma, a.wdt, 0, j, t, a.G.tpr, a.G.d);
    chunk_to_float<M>(r, a.wdt, w);
  }
  if (a.beta != nullptr) {
    load_chunk<M, true>(r, a.beta, a.wdt, 0, j, t, a.G.tpr, a.G.d);
    chunk_to_float<M>(r, a.wdt, b);
  }
}

template <int NC, Mode M>
__global__ void __launch_bounds__(NC == 1 ? 512 : 1024, NC == 1 ? 3 : 1) norm_fwd_kernel(const NormFwd a) {
  __shared__ float buf[2][kMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const Place at(a.G);
  const int tpr = a.G.tpr, d = a.G.d, t = at.t;
  const unsigned row = blockIdx.x * a.G.groups + at.group;   // up to 2^31 and a block's rows
  const bool live = row < (unsigned)a.G.rows;
  const size_t base = (size_t)(live ? row : 0) * d;
  Raw8 rx[NC], ra[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) load_chunk<M>(rx[j], a.x, a.xdt, base, j, t, tpr, d);
  if (a.add != nullptr) {
#pragma unroll
    for (int j = 0; j < NC; ++j) load_chunk<M>(ra[j], a.add, a.adt, base, j, t, tpr, d);
  }
  float h[NC][8], s = 0.f;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    chunk_to_float<M>(rx[j], a.xdt, h[j]);
    if (a.add != nullptr) {
      float v[8];
      chunk_to_float<M>(ra[j], a.adt, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] += v[i];
      if (a.xdt != MOE_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = round_to(h[j][i], a.xdt);
      }
      if (a.sum != nullptr && live) store_chunk<M>(a.sum, a.xdt, base, j, t, tpr, d, h[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s += h[j][i];   // columns past the width hold zeros
  }
  const float mu = over(row_sum(s, tpr, at.group, buf[0]), a.G.fd, a.G.inv_d);
  s = 0.f;
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[j][i] -= mu;
      if (inside<M>(column<M>(j, M == kSingle ? i : i & 4, t, tpr), d)) s += h[j][i] * h[j][i];
    }
  const float rstd = inverse_root(over(row_sum(s, tpr, at.group, buf[1]), a.G.fd, a.G.inv_d) + a.eps);
  if (!live) return;
  if (t == 0) {
    if (a.mean != nullptr) a.mean[row] = mu;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    float w[8], b[8];
    load_affine<M>(a, j, t, w, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] = fmaf(h[j][i] * rstd, w[i], b[i]);
    store_chunk<M>(a.y, a.ydt, base, j, t, tpr, d, h[j]);
  }
}

// Two rows to a group of threads, without an addend: their loads, reductions and
// barriers go together, and gamma and beta are read and converted once for both.
template <int NC, Mode M>
__global__ void __launch_bounds__(NC == 1 ? 512 : 256, NC == 1 ? 2 : 3) norm_fwd_pair_kernel(const NormFwd a) {
  __shared__ float2 buf[2][kMaxWarps];
  pdl_wait();
  pdl_launch_dependents();
  const Place at(a.G);
  const int tpr = a.G.tpr, d = a.G.d, t = at.t;
  const unsigned rows = a.G.rows, row = 2 * (blockIdx.x * a.G.groups + at.group);
  const bool live0 = row < rows, live1 = row + 1 < rows;
  const size_t base0 = (size_t)(live0 ? row : 0) * d, base1 = (size_t)(live1 ? row + 1 : 0) * d;
  Raw8 r0[NC], r1[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) load_chunk<M>(r0[j], a.x, a.xdt, base0, j, t, tpr, d);
#pragma unroll
  for (int j = 0; j < NC; ++j) load_chunk<M>(r1[j], a.x, a.xdt, base1, j, t, tpr, d);
  float h0[NC][8], h1[NC][8];
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    chunk_to_float<M>(r0[j], a.xdt, h0[j]);
    chunk_to_float<M>(r1[j], a.xdt, h1[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s.x += h0[j][i];
      s.y += h1[j][i];
    }
  }
  s = row_sum(s, tpr, at.group, buf[0]);
  const float mu0 = over(s.x, a.G.fd, a.G.inv_d), mu1 = over(s.y, a.G.fd, a.G.inv_d);
  s = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h0[j][i] -= mu0;
      h1[j][i] -= mu1;
      if (inside<M>(column<M>(j, M == kSingle ? i : i & 4, t, tpr), d)) {
        s.x += h0[j][i] * h0[j][i];
        s.y += h1[j][i] * h1[j][i];
      }
    }
  s = row_sum(s, tpr, at.group, buf[1]);
  const float rs0 = inverse_root(over(s.x, a.G.fd, a.G.inv_d) + a.eps);
  const float rs1 = inverse_root(over(s.y, a.G.fd, a.G.inv_d) + a.eps);
  if (!live0) return;
  if (t == 0) {
    if (a.mean != nullptr) a.mean[row] = mu0;
    if (a.rstd != nullptr) a.rstd[row] = rs0;
    if (a.mean != nullptr && live1) a.mean[row + 1] = mu1;
    if (a.rstd != nullptr && live1) a.rstd[row + 1] = rs1;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    float w[8], b[8];
    load_affine<M>(a, j, t, w, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h0[j][i] = fmaf(h0[j][i] * rs0, w[i], b[i]);
      h1[j][i] = fmaf(h1[j][i] * rs1, w[i], b[i]);
    }
    store_chunk<M>(a.y, a.ydt, base0, j, t, tpr, d, h0[j]);
    if (live1) store_chunk<M>(a.y, a.ydt, base1, j, t, tpr, d, h1[j]);
  }
}

// The block's column sums to part[block][2][d]: cols[groups][2][d] gathers them
// when several rows share the block.
template <int NC, Mode M>
__device__ __forceinline__ void write_columns(const float (&dg)[NC][8], const float (&db)[NC][8], float* cols,
                                              float* part, int d, int g, int groups, int t, int tpr) {
  float* out = part + (size_t)blockIdx.x * 2 * d;
  float* mine = groups == 1 ? out : cols + (size_t)g * 2 * d;
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<M>(j, i, t, tpr);
      if (inside<M>(c, d)) {
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

struct NormBwd {
  Geometry G;
  const void* dy;
  const void* x;
  const float* mean;
  const float* rstd;
  const void* gamma;
  const void* dsum;
  void* dx;
  float* part;
  int xdt, wdt, gdt, odt;
  uint32_t* status;
};

// Bytes of an operand in a stage: kSingle rows may begin inside a 16-byte piece
// and end inside another.
template <Mode M>
__host__ __device__ constexpr uint32_t stage_part(uint32_t bytes) {
  return M == kSingle ? (bytes + 15u) / 16u * 16u + 16u : bytes;
}

// dx of a row at a time; the columns' sums over the block's rows stay with the
// thread that owns the column.  The rows of the block's next rounds (one row
// for each of its groups, which lie one after the other) come by bulk copies
// of a whole row each, issued by one thread, into a ring of `stages`: the
// threads spend nothing on loads, and a stage is filled again as soon as every
// warp has read it.
template <int NC, Mode M>
__global__ void __launch_bounds__(512, NC == 1 ? 2 : 1)
norm_bwd_rows_kernel(const NormBwd a, int stages, unsigned copied, unsigned long long wait_ns) {
  __shared__ float2 buf[2][kMaxWarps];
  __shared__ unsigned long long full[kMaxStages], read[kMaxStages];
  __shared__ int abort_flag;
  extern __shared__ __align__(128) unsigned char dyn[];   // [stages][dy, x, dsum][groups][d]
  const Place place(a.G);
  const int tpr = a.G.tpr, d = a.G.d, groups = a.G.groups, g = place.group, t = place.t;
  const unsigned rows = a.G.rows;
  const uint32_t smem = tc::smem_u32(dyn), bars = tc::smem_u32(full), done = tc::smem_u32(read);
  const uint32_t row_y = d * (a.gdt == MOE_DTYPE_F32 ? 4 : 2), row_x = d * (a.xdt == MOE_DTYPE_F32 ? 4 : 2);
  const uint32_t row_s = a.dsum == nullptr ? 0 : d * (a.odt == MOE_DTYPE_F32 ? 4 : 2);
  const uint32_t part_y = stage_part<M>(groups * row_y), part_x = stage_part<M>(groups * row_x);
  const uint32_t stage = part_y + part_x + (row_s == 0 ? 0 : stage_part<M>(groups * row_s));
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      tc::mbar_init(bars + 8 * i, 1);
      tc::mbar_init(done + 8 * i, (blockDim.x + 31) / 32);
    }
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  // rows < 2^31, and a few steps of the grid more still fit 32 bits
  const unsigned step = gridDim.x * groups;
  // One thread: the rows from r0 on into stage `to`.  kSingle: rows begin anywhere,
  // and the whole 16-byte pieces that hold them are copied; the array's last
  // bytes, where they are no whole piece, are stored one by one ahead of the
  // arrival that makes them visible.
  auto fill = [&](int to, unsigned r0) {
    if (r0 >= copied) return;
    const uint32_t n = min((unsigned)groups, rows - r0), bar = bars + 8 * to;
    uint32_t at = smem + to * stage;
    if constexpr (M != kSingle) {
      tc::mbar_expect_tx(bar, n * (row_y + row_x + row_s));
      tc::bulk_load(at, static_cast<const char*>(a.dy) + (size_t)r0 * row_y, n * row_y, bar);
      at += part_y;
      tc::bulk_load(at, static_cast<const char*>(a.x) + (size_t)r0 * row_x, n * row_x, bar);
      at += part_x;
      if (row_s != 0) tc::bulk_load(at, static_cast<const char*>(a.dsum) + (size_t)r0 * row_s, n * row_s, bar);
    } else {
      struct Piece {
        const char* from;
        uint32_t bytes;
      };
      // the whole pieces that hold the rows; what is behind the last one goes to dst at once
      auto piece = [&](const void* p, uint32_t row_bytes, uint32_t dst) {
        const char* base = static_cast<const char*>(p);
        const long long total = (long long)rows * row_bytes, whole = total & ~15LL;
        const long long lo = ((long long)r0 * row_bytes) & ~15LL;
        const long long hi = min(whole, ((long long)(r0 + n) * row_bytes + 15) & ~15LL);
        if (r0 + n == rows)
          for (long long i = max(lo, whole); i < total; i += 2)
            *reinterpret_cast<unsigned short*>(dyn + (dst - smem) + (i - lo)) =
                *reinterpret_cast<const unsigned short*>(base + i);
        return Piece{base + lo, (uint32_t)max(0LL, hi - lo)};
      };
      Piece q[3];
      q[0] = piece(a.dy, row_y, at);
      q[1] = piece(a.x, row_x, at + part_y);
      q[2] = row_s != 0 ? piece(a.dsum, row_s, at + part_y + part_x) : Piece{nullptr, 0};
      tc::mbar_expect_tx(bar, q[0].bytes + q[1].bytes + q[2].bytes);
      if (q[0].bytes != 0) tc::bulk_load(at, q[0].from, q[0].bytes, bar);
      if (q[1].bytes != 0) tc::bulk_load(at + part_y, q[1].from, q[1].bytes, bar);
      if (q[2].bytes != 0) tc::bulk_load(at + part_y + part_x, q[2].from, q[2].bytes, bar);
    }
  };
  __syncthreads();
  unsigned r0 = blockIdx.x * groups;
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i) fill(i, r0 + i * step);
  // eight elements of the row that starts at `from`, chunk j
  auto fetch = [&](float (&v)[8], uint32_t from, int dt, int j) {
    Raw8 r;
    if constexpr (M != kWhole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.w[i] = 0u;
    }
    if constexpr (M == kSingle) {
      if (dt == MOE_DTYPE_F32) {
        from += (j * 8 * tpr + t) * 4;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (column<M>(j, i, t, tpr) < d) shared4(from + i * tpr * 4, r.w[i]);
      } else {
        from += (j * 8 * tpr + t) * 2;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (column<M>(j, i, t, tpr) < d) shared2(from + i * tpr * 2, r.w[i]);
      }
    } else {
      const int c = column<M>(j, 0, t, tpr), c2 = column<M>(j, 4, t, tpr);
      if (dt == MOE_DTYPE_F32) {
        if (inside<M>(c, d)) shared16(from + c * 4, r.w[0], r.w[1], r.w[2], r.w[3]);
        if (inside<M>(c2, d)) shared16(from + c2 * 4, r.w[4], r.w[5], r.w[6], r.w[7]);
      } else {
        if (inside<M>(c, d)) shared8(from + c * 2, r.w[0], r.w[1]);
        if (inside<M>(c2, d)) shared8(from + c2 * 2, r.w[2], r.w[3]);
      }
    }
    chunk_to_float<M>(r, dt, v);
  };
  // where the group's row begins in a part of the stage
  auto row_at = [&](uint32_t part, uint32_t row_bytes) {
    return part + g * row_bytes + (M == kSingle ? (r0 * row_bytes) & 15u : 0u);
  };
  float w[NC][8], dg[NC][8], db[NC][8];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if (a.gamma != nullptr) {
      Raw8 r;
      load_chunk<M, true>(r, a.gamma, a.wdt, 0, j, t, tpr, d);
      chunk_to_float<M>(r, a.wdt, w[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (a.gamma == nullptr) w[j][i] = 1.f;
      dg[j][i] = db[j][i] = 0.f;
    }
  }
  float mu = 0.f, rs = 0.f;
  if (r0 + g < rows) mu = a.mean[r0 + g], rs = a.rstd[r0 + g];
  int turn = 0, at = 0, drains = stages;
  uint32_t phase = 0;
  bool again = false;
  for (; r0 < rows; r0 += step, turn ^= 1, again = true) {
    const unsigned row = r0 + g;
    const bool live = row < rows;
    float mu_next = 0.f, rs_next = 0.f;
    if (row + step < rows) mu_next = a.mean[row + step], rs_next = a.rstd[row + step];
    // a wait that runs out: the status says so, no more copies are issued, those
    // under way are given a little longer, and the thread's share of this row and
    // all later ones (whose phases mean nothing any more) is NaN
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (tc::mbar_try_wait(bar, parity) || tc::mbar_wait(bar, parity, &abort_flag, wait_ns)) return true;
      abort_flag = 1;
      if (a.status != nullptr) atomicOr(a.status, MOE_DEV_TIMEOUT);
      if (drains-- > 0) tc::mbar_wait(bar, parity, nullptr, tc::kDrainNs);
      return false;
    };
    if (threadIdx.x == 0 && again) {   // the stage of the round before
      const int to = at == 0 ? stages - 1 : at - 1;
      if (wait(done + 8 * to, at == 0 ? phase ^ 1 : phase)) fill(to, r0 + (stages - 1) * step);
    }
    wait(bars + 8 * at, phase);
    if (drains != stages) mu = NAN;   // takes xh with it, and so dgamma and the row's sums
    const uint32_t from = row_at(smem + at * stage, row_y);
    const uint32_t from_x = row_at(smem + at * stage + part_y, row_x);
    float xh[NC][8], gy[NC][8];
    float2 s = make_float2(0.f, 0.f);
    if (live) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        fetch(gy[j], from, a.gdt, j);
        fetch(xh[j], from_x, a.xdt, j);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xh[j][i] = (xh[j][i] - mu) * rs;   // of no use past the width, where dy is zero
          dg[j][i] += gy[j][i] * xh[j][i];
          db[j][i] += gy[j][i];
          gy[j][i] *= w[j][i];
          s.x += gy[j][i];
          s.y += gy[j][i] * xh[j][i];
        }
      }
    }
    s = row_sum(s, tpr, g, buf[turn]);
    if (live) {
      const float r1 = -rs * s.x * a.G.inv_d, r2 = -rs * s.y * a.G.inv_d;
      const uint32_t from_s = row_at(smem + at * stage + part_y + part_x, row_s);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[j][i] = fmaf(xh[j][i], r2, fmaf(gy[j][i], rs, r1));
        if (a.dsum != nullptr) {
          float v[8];
          fetch(v, from_s, a.odt, j);
#pragma unroll
          for (int i = 0; i < 8; ++i) xh[j][i] += v[i];
        }
        store_chunk<M>(a.dx, a.odt, (size_t)row * d, j, t, tpr, d, xh[j]);
      }
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(done + 8 * at);
    mu = mu_next, rs = rs_next;
    if (++at == stages) at = 0, phase ^= 1;
  }
  if (a.part == nullptr) return;
  if (drains != stages) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) db[j][i] = NAN;
  }
  __syncthreads();   // the stages are free: the columns of the block's rows meet there
  write_columns<NC, M>(dg, db, reinterpret_cast<float*>(dyn), a.part, d, g, groups, t, tpr);
}

// Chunk j of the row at base: xh and dy; and gamma into dy.
template <Mode M>
__device__ __forceinline__ void read_chunk(const NormBwd& a, size_t base, float mu, float rs, int j, int t,
                                           float (&xh)[8], float (&gy)[8]) {
  Raw8 ry, rx;
  load_chunk<M>(ry, a.dy, a.gdt, base, j, t, a.G.tpr, a.G.d);
  load_chunk<M>(rx, a.x, a.xdt, base, j, t, a.G.tpr, a.G.d);
  chunk_to_float<M>(ry, a.gdt, gy);
  chunk_to_float<M>(rx, a.xdt, xh);
#pragma unroll
  for (int i = 0; i < 8; ++i) xh[i] = (xh[i] - mu) * rs;   // of no use past the width, where dy is zero
}
template <Mode M>
__device__ __forceinline__ void weigh_chunk(const NormBwd& a, int j, int t, float (&gy)[8]) {
  if (a.gamma == nullptr) return;
  Raw8 r;
  float w[8];
  load_chunk<M, true>(r, a.gamma, a.wdt, 0, j, t, a.G.tpr, a.G.d);
  chunk_to_float<M>(r, a.wdt, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) gy[i] *= w[i];
}

// Brings the whole 16-byte pieces of elements [base, base + d) into L2.
__device__ __forceinline__ void prefetch_row(const void* p, int dt, size_t base, int d) {
  const size_t es = dt == MOE_DTYPE_F32 ? 4 : 2;
  const uintptr_t lo = (reinterpret_cast<uintptr_t>(p) + base * es + 15) & ~(uintptr_t)15;
  const uintptr_t hi = (reinterpret_cast<uintptr_t>(p) + (base + d) * es) & ~(uintptr_t)15;
  if (hi > lo)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lo), "r"((uint32_t)(hi - lo)) : "memory");
}

// The same with plain loads, for operands that do not begin on 16 bytes.
template <int NC, Mode M>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormBwd a) {
  __shared__ float2 buf[2][kMaxWarps];
  extern __shared__ __align__(16) unsigned char dyn[];
  pdl_wait();
  pdl_launch_dependents();
  const Place place(a.G);
  const int tpr = a.G.tpr, d = a.G.d, rows = a.G.rows, groups = a.G.groups, g = place.group, t = place.t;
  float dg[NC][8], db[NC][8], xh[NC][8], gy[NC][8];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[j][i] = db[j][i] = 0.f;
  const float inv_d = a.G.inv_d;
  int turn = 0;
  for (long long r0 = (long long)blockIdx.x * groups; r0 < rows; r0 += (long long)gridDim.x * groups, turn ^= 1) {
    const bool live = r0 + g < rows;
    const long long row = live ? r0 + g : 0;
    const size_t base = (size_t)row * d;
    const float mu = a.mean[row], rs = a.rstd[row];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      read_chunk<M>(a, base, mu, rs, j, t, xh[j], gy[j]);
      if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dg[j][i] += gy[j][i] * xh[j][i];
          db[j][i] += gy[j][i];
        }
      }
      weigh_chunk<M>(a, j, t, gy[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s.x += gy[j][i];
        s.y += gy[j][i] * xh[j][i];
      }
    }
    s = row_sum(s, tpr, g, buf[turn]);
    const float m1 = s.x * inv_d, m2 = s.y * inv_d;
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) xh[j][i] = rs * (gy[j][i] - m1 - xh[j][i] * m2);
      if (a.dsum != nullptr) {
        Raw8 r;
        float v[8];
        load_chunk<M>(r, a.dsum, a.odt, base, j, t, tpr, d);
        chunk_to_float<M>(r, a.odt, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[j][i] += v[i];
      }
      store_chunk<M>(a.dx, a.odt, base, j, t, tpr, d, xh[j]);
    }
  }
  if (a.part == nullptr) return;
  write_columns<NC, M>(dg, db, reinterpret_cast<float*>(dyn), a.part, d, g, groups, t, tpr);
}

// Rows of more than 8192 columns, one to a block of up to 1024 threads with two
// chunks each.  The columns' sums lie in shared memory, every thread's own as
// float4s, which leaves the registers to the row; the next row is brought into
// L2 meanwhile (125 us without that).  2048 x 16384 in fp32: 118 us, 4.6 TB/s;
// 3727 x 9001: 219.  With one block an SM most of the waiting is for the row's
// loads (8.7 of some 22 cycles an issue; shared memory 3.2, the barrier 1.5).
// Sums in the registers of 512 threads with four chunks, and the row read
// twice, took 201 and 1100 us.
template <Mode M>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const NormBwd a) {
  constexpr int NC = 2;
  __shared__ float2 buf[2][kMaxWarps];
  extern __shared__ __align__(16) unsigned char dyn[];   // [dgamma, dbeta][2 NC][threads] of float4
  pdl_wait();
  pdl_launch_dependents();
  const int tpr = a.G.tpr, d = a.G.d, t = threadIdx.x;
  const unsigned rows = a.G.rows;
  float4* sums = reinterpret_cast<float4*>(dyn) + t;
  const bool weights = a.part != nullptr;
  if (weights) {
#pragma unroll
    for (int q = 0; q < 4 * NC; ++q) sums[q * tpr] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  int turn = 0;
  for (unsigned row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    const size_t base = (size_t)row * d;
    if (t == 0 && row + gridDim.x < rows) {
      const size_t next = base + (size_t)gridDim.x * d;
      prefetch_row(a.dy, a.gdt, next, d);
      prefetch_row(a.x, a.xdt, next, d);
      if (a.dsum != nullptr) prefetch_row(a.dsum, a.odt, next, d);
    }
    const float mu = a.mean[row], rs = a.rstd[row];
    float xh[NC][8], gy[NC][8];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      read_chunk<M>(a, base, mu, rs, j, t, xh[j], gy[j]);
      if (weights) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float *x4 = xh[j] + 4 * q, *g4 = gy[j] + 4 * q;
          float4 &dg = sums[(2 * j + q) * tpr], &db = sums[(2 * NC + 2 * j + q) * tpr];
          const float4 og = dg, ob = db;
          dg = make_float4(og.x + g4[0] * x4[0], og.y + g4[1] * x4[1], og.z + g4[2] * x4[2], og.w + g4[3] * x4[3]);
          db = make_float4(ob.x + g4[0], ob.y + g4[1], ob.z + g4[2], ob.w + g4[3]);
        }
      }
      weigh_chunk<M>(a, j, t, gy[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s.x += gy[j][i];
        s.y += gy[j][i] * xh[j][i];
      }
    }
    s = row_sum(s, tpr, 0, buf[turn]);
    const float r1 = -rs * s.x * a.G.inv_d, r2 = -rs * s.y * a.G.inv_d;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) xh[j][i] = fmaf(xh[j][i], r2, fmaf(gy[j][i], rs, r1));
      if (a.dsum != nullptr) {
        Raw8 r;
        float v[8];
        load_chunk<M>(r, a.dsum, a.odt, base, j, t, tpr, d);
        chunk_to_float<M>(r, a.odt, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[j][i] += v[i];
      }
      store_chunk<M>(a.dx, a.odt, base, j, t, tpr, d, xh[j]);
    }
  }
  if (!weights) return;
  float dg[NC][8], db[NC][8];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      *reinterpret_cast<float4*>(&dg[j][4 * q]) = sums[(2 * j + q) * tpr];
      *reinterpret_cast<float4*>(&db[j][4 * q]) = sums[(2 * NC + 2 * j + q) * tpr];
    }
  write_columns<NC, M>(dg, db, nullptr, a.part, d, 0, 1, t, tpr);
}

// dgamma and dbeta: the blocks' partial sums of each column.  A block takes 32
// columns; its 32 warps each add a run of the parts, and the runs are added
// in order.
__global__ void __launch_bounds__(1024)
norm_weights_kernel(const float* __restrict__ part, int nparts, int d, float* dgamma, float* dbeta) {
  __shared__ float runs[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int p0 = (int)((long long)nparts * warp / 32), p1 = (int)((long long)nparts * (warp + 1) / 32);
  float v = 0.f;
  if (c < 2 * d) {
#pragma unroll 8
    for (int p = p0; p < p1; ++p) v += part[(size_t)p * 2 * d + c];
  }
  runs[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || c >= 2 * d) return;
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) v += runs[w][lane];
  if (c < d) {
    if (dgamma != nullptr) dgamma[c] = v;
  } else if (dbeta != nullptr) {
    dbeta[c - d] = v;
  }
}

// The width and a pointer allow vector accesses of four elements.
bool vector_width(int d) { return d % 4 == 0; }
bool on_vector(const void* p, int dt) { return reinterpret_cast<uintptr_t>(p) % (4u * dtype_bytes(dt)) == 0; }

// How a row is spread over threads: tpr of them with nc chunks of eight columns
// each.  Up to 64 chunks stay inside a warp (no barrier); above, two chunks a
// thread (half the reductions of one: 181 against 256 us for the backward of
// 16384 x 4096), up to 1024 threads.  A width that is no multiple of four is read
// element by element, and one chunk leaves more threads to do it (165 against
// 226 us for 32357 x 1037).
struct Shape {
  int tpr, nc, threads, groups;
};
Shape shape_of(int d) {
  const int chunks = (d + 7) / 8;
  Shape s;
  if (chunks <= 32) {
    s.tpr = 1;
    while (s.tpr < chunks) s.tpr *= 2;
    s.nc = 1;
  } else if (chunks <= 64) {
    s.tpr = 32;
    s.nc = 2;
  } else {
    s.nc = chunks <= 512 && !vector_width(d) ? 1 : 2;
    s.tpr = ((chunks + s.nc - 1) / s.nc + 31) / 32 * 32;
  }
  s.groups = std::max(1, 256 / s.tpr);
  s.threads = s.groups * s.tpr;
  return s;
}

constexpr int kWide = 8192;   // columns of 512 threads with two chunks

Geometry geometry(const moe_norm_config& c, const Shape& s) {
  return Geometry{c.rows,   c.d, s.tpr, s.groups, (unsigned)((65536 + s.tpr - 1) / s.tpr),
                  (float)c.d, 1.f / (float)c.d};
}

template <typename F>
cudaError_t with_mode(bool vec, const Shape& s, int d, F&& f) {
  if (!vec) return f(std::integral_constant<Mode, kSingle>{});
  if (8 * s.nc * s.tpr == d) return f(std::integral_constant<Mode, kWhole>{});
  return f(std::integral_constant<Mode, kVector>{});
}

// Blocks of the backward that an SM holds at once: 64 registers a thread with
// one chunk, else 128.
int bwd_resident(const Shape& s) { return std::max(1, (s.nc == 1 ? 1024 : 512) / s.threads); }

// Blocks of the backward: at most what 148 SMs hold at once, as few as take the
// same number of rounds of rows (the last block fewer).  The blocks need not
// fill the SMs evenly: 8192 x 512 are 256 blocks of four rounds.
int bwd_blocks(const moe_norm_config& c, const Shape& s) {
  const long long rounds = std::max<long long>(1, ((long long)c.rows + s.groups - 1) / s.groups);
  const long long most = 148LL * bwd_resident(s);
  const long long per = (rounds + most - 1) / most;
  return (int)((rounds + per - 1) / per);
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Rows that are whole 16-byte pieces from a 16-byte boundary on.
bool whole_rows(const void* p, int dt, int d) { return on16(p) && (size_t)d * dtype_bytes(dt) % 16 == 0; }

std::atomic<unsigned long long> g_wait_ns{tc::kWaitNs};
std::atomic<int> g_kept_rounds{-1};

}  // namespace

void set_norm_test_hooks(unsigned long long wait_ns, int kept_rounds) {
  g_wait_ns.store(wait_ns != 0 ? wait_ns : tc::kWaitNs, std::memory_order_relaxed);
  g_kept_rounds.store(kept_rounds, std::memory_order_relaxed);
}

// Each block leaves one partial of the weights' gradient.
int norm_bwd_blocks(const moe_norm_config& c) { return bwd_blocks(c, shape_of(c.d)); }

cudaError_t launch_norm_fwd(const moe_norm_config& c, const void* x, const void* add, const void* gamma,
                            const void* beta, void* y, void* sum, float* mean, float* rstd, cudaStream_t s) {
  const Shape sh = shape_of(c.d);
  const bool vec = vector_width(c.d) && on_vector(x, c.x_dtype) && on_vector(add, c.add_dtype) &&
                   on_vector(gamma, c.w_dtype) && on_vector(beta, c.w_dtype) && on_vector(y, c.y_dtype) &&
                   on_vector(sum, c.x_dtype);
  const NormFwd a{geometry(c, sh), x,     add,       gamma,     beta,      y,
                  sum,             mean,  rstd,      c.eps,     c.x_dtype, c.y_dtype,
                  c.w_dtype,       c.add_dtype};
  // Two rows a group without an addend, from the rows on that fill the SMs either way: 12.5 against 13.6 us for
  // 2369 x 4096 in bf16, but 7.7 against 7.1 for 1185.  Groups of 512 threads do not have the registers.
  const bool pair = add == nullptr && (sh.nc == 1 || (sh.nc == 2 && sh.threads <= 256)) &&
                    c.rows >= 148LL * 12 * sh.groups;
  const long long each = pair ? 2LL * sh.groups : sh.groups;
  const dim3 grid((unsigned)(((long long)c.rows + each - 1) / each));
  return with_mode(vec, sh, c.d, [&](auto mode) {
    constexpr Mode M = decltype(mode)::value;
    if (pair)
      return launch_pdl(sh.nc == 1 ? norm_fwd_pair_kernel<1, M> : norm_fwd_pair_kernel<2, M>, grid, dim3(sh.threads), 0,
                        s, a);
    return launch_pdl(sh.nc == 1 ? norm_fwd_kernel<1, M> : norm_fwd_kernel<2, M>, grid, dim3(sh.threads), 0, s, a);
  });
}

cudaError_t launch_norm_bwd(const moe_norm_config& c, const void* dy, const void* x, const float* mean,
                            const float* rstd, const void* gamma, const void* dsum, void* dx, float* dgamma,
                            float* dbeta, moe_stats* stats, float* part, cudaStream_t s) {
  const Shape sh = shape_of(c.d);
  const bool weights = dgamma != nullptr || dbeta != nullptr;
  const int blocks = bwd_blocks(c, sh);
  const int kept = g_kept_rounds.load(std::memory_order_relaxed);
  const unsigned long long wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  const unsigned copied =   // rows before this one are copied: all of them, but in a test
      (unsigned)(kept < 0 ? c.rows : std::min<long long>(c.rows, (long long)kept * blocks * sh.groups));
  const NormBwd a{geometry(c, sh),          dy,        x,         mean,       rstd,       gamma, dsum, dx,
                  weights ? part : nullptr, c.x_dtype, c.w_dtype, c.dy_dtype, c.dx_dtype,
                  stats != nullptr ? &stats->status : nullptr};
  // the columns of several rows in a block: groups * d <= 256 * 16, at most 32 KB
  const size_t cols = sh.groups > 1 && weights ? (size_t)sh.groups * 2 * c.d * sizeof(float) : 0;
  const bool vec = vector_width(c.d) && on_vector(dy, c.dy_dtype) && on_vector(x, c.x_dtype) &&
                   on_vector(gamma, c.w_dtype) && on_vector(dsum, c.dx_dtype) && on_vector(dx, c.dx_dtype);
  const bool pieces = whole_rows(dy, c.dy_dtype, c.d) && whole_rows(x, c.x_dtype, c.d) &&
                      (dsum == nullptr || whole_rows(dsum, c.dx_dtype, c.d));
  const bool starts = on16(dy) && on16(x) && on16(dsum);
  const size_t share = (size_t)(220 << 10) / bwd_resident(sh) - (2 << 10);   // of an SM's shared memory
  const cudaError_t e = with_mode(vec, sh, c.d, [&](auto mode) {
    constexpr Mode M = decltype(mode)::value;
    // a ring of two to four rounds of rows
    auto part = [&](int dt) { return (size_t)stage_part<M>((uint32_t)(sh.groups * c.d * dtype_bytes(dt))); };
    const size_t round = part(c.dy_dtype) + part(c.x_dtype) + (dsum != nullptr ? part(c.dx_dtype) : 0);
    const int stages = (int)std::min<size_t>(kMaxStages, std::max<size_t>(1, share / round));
    const size_t smem = std::max(stages * round, cols);
    auto rows = [&](auto kernel, cudaError_t set) {
      if (set != cudaSuccess) return set;
      return launch_pdl(kernel, dim3(blocks), dim3(sh.threads), smem, s, a, stages, copied, wait_ns);
    };
    auto plain = [&](auto kernel) { return launch_pdl(kernel, dim3(blocks), dim3(sh.threads), cols, s, a); };
    const bool ring = M == kSingle ? starts : pieces;
    if (c.d > kWide) {
      const size_t sums = weights ? (size_t)sh.threads * 8 * sizeof(float4) : 0;
      const cudaError_t set = set_smem_once<norm_bwd_wide_kernel<M>>(1024 * 8 * sizeof(float4));
      return set != cudaSuccess ? set : launch_pdl(norm_bwd_wide_kernel<M>, dim3(blocks), dim3(sh.threads), sums, s, a);
    }
    if (sh.nc == 1)
      return ring ? rows(norm_bwd_rows_kernel<1, M>, set_smem_once<norm_bwd_rows_kernel<1, M>>(220 << 10))
                  : plain(norm_bwd_kernel<1, M>);
    return ring ? rows(norm_bwd_rows_kernel<2, M>, set_smem_once<norm_bwd_rows_kernel<2, M>>(220 << 10))
                : plain(norm_bwd_kernel<2, M>);
  });
  if (e != cudaSuccess || !weights) return e;
  return launch_pdl(norm_weights_kernel, dim3((2 * c.d + 31) / 32), dim3(1024), 0, s, (const float*)part, blocks,
                    c.d, dgamma, dbeta);
}

}  // namespace moe
