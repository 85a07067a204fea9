// The balance loss of a batch of sequences, per-expert counts and its gradient
// with respect to the router's scores.
//
// The Switch form E sum_e f_e P_e (Skywork slides, slide 4; Megatron-Core
// best-practice page, "MoE负载均衡的挑战与应对"), taken sequence by sequence
// over the tokens that the mask keeps:
//   c_se = assignments of sequence s to expert e, f_se = E c_se / sum_e c_se
//   p_t = softmax(z_t), or sigmoid(z_t) over its sum
//   loss = 1/G sum_s 1/n_s sum_{t in s} <f_s, p_t>
// (n_s tokens kept in s, G sequences with n_s > 0).  The counts carry no
// gradient, and the mean probabilities P never have to be formed: a token
// needs <f_s, p_t> for the gradient
//   dz_te = coef / (G n_s) p_te (f_se - <f_s, p_t>) [(1 - sigmoid(z_te))],
// and the loss is the weighted sum of the same products.  So the scores are
// read once and their gradient is written in the same pass, after a pass over
// the indices (k of them per token) that counts.
//
// The floor is the bytes of the scores and their gradient.  With few bytes per
// score (bf16) the exponentials, the reductions over a token's lanes and the
// bookkeeping of a token weigh as much: 16 experts to a lane spread the last two
// (131072 x 256: 62 us with 8, 46 with 16; 56 us in fp32, where the bytes alone
// take 43), and two blocks of 128 registers an SM beat three that spill (57 us).
#include "elem8.cuh"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLossBlocksPerSm = 2;   // by their registers: up to 128 with 16 experts a lane
constexpr int kMaxLossBlocks = 1024;
// One block does it all up to here: 4.2 to 6.9 us in a graph for 16 x 8 to 512 x 16 and 32 x 256, where three
// kernels take 6.4 to 7.7; calls in a row take 8 and 11.4.  Above, three kernels win in a graph: 256 x 64 8.9 and
// 7.8, 1024 x 16 11.4 and 6.8.
constexpr int kSmallScores = 8192, kSmallTokens = 512;

// Words at the start of the workspace; n_s of every sequence follows.
struct Head {
  unsigned groups;   // G
  unsigned ticket;   // blocks of the loss kernel that are done
};

// Sequence of token t among [lo, hi]: the last that begins at or before t.  Any
// contents of off give an index inside the range.
__device__ __forceinline__ int search(const int32_t* __restrict__ off, int lo, int hi, int t) {
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (off[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Zeros for the counters of the kernels that follow.
__global__ void __launch_bounds__(kThreads) balance_clear_kernel(int32_t* counts, size_t ncounts, int32_t* head,
                                                                 int nhead) {
  pdl_wait();
  pdl_launch_dependents();
  const size_t first = (size_t)blockIdx.x * kThreads + threadIdx.x, step = (size_t)gridDim.x * kThreads;
  for (size_t i = first; i < (size_t)nhead; i += step) head[i] = 0;
  for (size_t i = first; i < ncounts; i += step) counts[i] = 0;
}

// A block counts a tile of consecutive tokens, one to a thread, and writes each
// token's sequence (-1: none, or padded) for the loss.  Most tiles lie in one
// sequence or two: the first and the last sequence of the tile have a histogram
// each in shared memory, and only tokens of sequences between them go to global
// memory one by one.  Integer sums: their order does not matter.
struct Count {
  const int32_t* topk;
  const int32_t* off;
  const unsigned char* mask;
  int32_t* counts;
  int32_t* nkept;
  int32_t* seq_of;
  Head* head;
  moe_stats* stats;
  int T, E, k, S;
};

__device__ __forceinline__ void count_tile(const Count& a, int tile, int tiles) {
  constexpr int kDense = 16 * kThreads;   // up to so many sequences the whole table is looked through at once
  __shared__ int hist[2][kMaxExperts], kept[2], begin[2];
  const int32_t* __restrict__ topk = a.topk;
  const int32_t* __restrict__ off = a.off;
  const unsigned char* __restrict__ mask = a.mask;
  const int T = a.T, E = a.E, k = a.k, S = a.S;
  int32_t *counts = a.counts, *nkept = a.nkept, *seq_of = a.seq_of;
  Head* head = a.head;
  const int tid = threadIdx.x, t0 = tile * kThreads, t = t0 + tid, last = min(T, t0 + kThreads) - 1;
  bool bad = false;
  const bool kept_here = t < T && (mask == nullptr || mask[t] != 0);
  for (int e = tid; e < E; e += kThreads) hist[0][e] = hist[1][e] = 0;
  if (tid < 2) kept[tid] = begin[tid] = 0;
  // the first and the last token's sequences: how many sequences begin at or before them
  int lowest = 0, highest = 0;
  if (off != nullptr) {
    for (int s = tile * kThreads + tid; s < S; s += tiles * kThreads)
      bad |= off[s] < 0 || off[s + 1] < off[s] || off[s + 1] > T;
    if (S <= kDense) {
      int n0 = 0, n1 = 0;
      for (int s = tid; s < S; s += kThreads) {
        const int o = off[s];
        n0 += o <= t0;
        n1 += o <= last;
      }
      __syncthreads();
      n0 = __reduce_add_sync(0xffffffffu, n0);
      n1 = __reduce_add_sync(0xffffffffu, n1);
      if ((tid & 31) == 0) {
        atomicAdd(&begin[0], n0);
        atomicAdd(&begin[1], n1);
      }
      __syncthreads();
      lowest = max(begin[0] - 1, 0);
      highest = max(begin[1] - 1, lowest);
    } else {
      lowest = search(off, 0, S - 1, t0);
      highest = search(off, lowest, S - 1, last);
    }
  }
  __syncthreads();
  int s = -1;
  if (kept_here) {
    if (off == nullptr) s = 0;
    else if (t >= off[0] && t < off[S]) s = search(off, lowest, highest, t);
  }
  if (t < T) seq_of[t] = s;
  const unsigned in0 = __ballot_sync(0xffffffffu, s >= 0 && s == lowest);
  const unsigned in1 = __ballot_sync(0xffffffffu, s >= 0 && s == highest && s != lowest);
  if ((tid & 31) == 0) {
    if (in0 != 0) atomicAdd(&kept[0], __popc(in0));
    if (in1 != 0) atomicAdd(&kept[1], __popc(in1));
  }
  if (s >= 0) {
    int32_t* row = counts + (size_t)s * E;
    if (s != lowest && s != highest && atomicAdd(&nkept[s], 1) == 0) atomicAdd(&head->groups, 1u);
    if (topk != nullptr) {
      const int32_t* slots = topk + (size_t)t * k;
#pragma unroll 4
      for (int j = 0; j < k; ++j) {
        const int e = slots[j];
        if ((unsigned)e >= (unsigned)E) bad = true;
        else atomicAdd(s == lowest ? &hist[0][e] : s == highest ? &hist[1][e] : &row[e], 1);
      }
    }
  }
  __syncthreads();
  for (int h = 0; h < 2; ++h) {
    const int at = h == 0 ? lowest : highest, m = kept[h];
    if (m == 0) continue;
    if (tid == 0 && atomicAdd(&nkept[at], m) == 0) atomicAdd(&head->groups, 1u);
    if (topk != nullptr)
      for (int e = tid; e < E; e += kThreads)
        if (hist[h][e] != 0) atomicAdd(&counts[(size_t)at * E + e], hist[h][e]);
  }
  if (bad && a.stats != nullptr) atomicOr(&a.stats->status, MOE_DEV_BOUNDS);
}

__global__ void __launch_bounds__(kThreads) balance_count_kernel(const Count a) {
  pdl_wait();
  pdl_launch_dependents();
  count_tile(a, blockIdx.x, gridDim.x);
}

struct Loss {
  const void* scores;
  const int32_t* seq_of;
  const float* coef;
  const int32_t* counts;
  const int32_t* nkept;
  Head* head;
  double* part;
  float* loss;
  void* dscores;
  int T, E, lanes, per_warp;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFarBelow = 0x1p-28f;   // a sum of sigmoids

// How the experts of a token lie in its lanes, 4 N each: kSingle strided by the
// lanes, kVector in quads of consecutive ones, kWhole the same without a gap.
enum Mode { kSingle, kVector, kWhole };

// Tokens in runs of per_warp to a warp, `lanes` (a power of two) to a token.  The
// counts of a sequence stay in registers until the next one begins, and the
// next token's scores are loaded before the current ones are used.
//
// Softmax: e = exp(z - max).  Sigmoid: with x = exp(-|z|) and r = 1 / (1 + x),
// sigmoid = r or x r by z's sign and its slope sigmoid (1 - sigmoid) = x r r,
// without a maximum; where all scores are so far below zero that the small ones
// among them would leave fp32's range before their shares do, exp(z - max)
// again (sigmoid is exp there to 2^-28).  ex2.approx on z log2(e) adds a few units in the last place and
// |z| / 2^24, relative.
// DT: the scores' type, known here so that no element asks for it.
template <int N, Mode M, bool SIGMOID, int DT>
__device__ __forceinline__ float loss_of_run(const Loss& a, int run, int end) {
  const int lane = threadIdx.x & 31;
  const int L = a.lanes, sub = lane & (L - 1), E = a.E, per_pass = 32 / L;
  auto expert = [&](int q, int i) { return M != kSingle ? (q * L + sub) * 4 + i : (q * 4 + i) * L + sub; };
  auto there = [&](int q, int i) { return M == kWhole || expert(q, M == kSingle ? i : 0) < E; };
  auto over_lanes = [&](auto op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < L) op(o);
  };
  const float groups = (float)a.head->groups, coef = a.coef != nullptr ? *a.coef : 1.f;
  // 4 N scores of token t, as loaded; what is not there is -inf
  uint32_t raw[N][4];
  auto load = [&](int t) {
    const size_t row = (size_t)t * E;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      if constexpr (M != kSingle) {
        if (DT == MOE_DTYPE_F32) {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(a.scores) + row + expert(q, 0));
          const uint4 v = there(q, 0) ? __ldg(p) : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
          raw[q][0] = v.x, raw[q][1] = v.y, raw[q][2] = v.z, raw[q][3] = v.w;
        } else {
          const uint2* p =
              reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(a.scores) + row + expert(q, 0));
          const uint2 v = there(q, 0) ? __ldg(p) : make_uint2(0xff80ff80u, 0xff80ff80u);
          raw[q][0] = v.x, raw[q][1] = v.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          raw[q][i] = there(q, i) ? load_raw1(a.scores, DT, row + expert(q, i))
                                  : (DT == MOE_DTYPE_F32 ? 0xff800000u : 0xff80u);
      }
    }
  };
  // d[N][4] to the gradient's row
  auto store = [&](int t, const float (&d)[N][4]) {
    const size_t row = (size_t)t * E;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      if constexpr (M != kSingle) {
        if (there(q, 0)) store4(a.dscores, DT, row + expert(q, 0), d[q][0], d[q][1], d[q][2], d[q][3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (there(q, i)) store1(a.dscores, DT, row + expert(q, i), d[q][i]);
      }
    }
  };
  float f[N][4] = {}, scale = 0.f, weight = 0.f, acc = 0.f;   // f: the sequence's counts; f_se = scale f
  int seq = -1;
  int t = run + lane / L;
  auto sequence = [&](int i) { return i < end ? a.seq_of[i] : -1; };
  int now = sequence(t), next = sequence(t + per_pass);
  if (now >= 0) load(t);
  for (int p = run; p < end; p += per_pass, t += per_pass) {
    const int later = sequence(t + 2 * per_pass);
    const bool used = now >= 0, look = used && now != seq;
    if (__any_sync(0xffffffffu, look)) {   // some group's next sequence
      if (look) {
        seq = now;
        weight = 1.f / (groups * (float)a.nkept[seq]);
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[q][i] = expert(q, i) < E ? (float)a.counts[(size_t)seq * E + expert(q, i)] : 0.f;
      }
      float n = 0.f;
#pragma unroll
      for (int q = 0; q < N; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) n += f[q][i];
      over_lanes([&](int o) { n += __shfl_xor_sync(0xffffffffu, n, o); });
      scale = n > 0.f ? (float)E / n : 0.f;
    }
    float z[N][4], g[N][4];
    if (__any_sync(0xffffffffu, used)) {
#pragma unroll
      for (int q = 0; q < N; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (M != kSingle && DT != MOE_DTYPE_F32)
            z[q][i] = __uint_as_float(i & 1 ? raw[q][i / 2] & 0xffff0000u : raw[q][i / 2] << 16);
          else
            z[q][i] = raw_to_float(raw[q][i], DT);
        }
      if (next >= 0) load(t + per_pass);
      float sum = 0.f, dot = 0.f;
      auto sums_of = [&](float e, int q, int i) {
        sum += e;
        dot += e * f[q][i];
      };
      // exp(z - max) of every expert into g, zeros throughout where no score is above -inf
      auto shifted = [&]() {
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, z[q][i]);
        over_lanes([&](int o) { top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o)); });
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g[q][i] = exp2_approx((z[q][i] - base) * kLog2e);
            sums_of(g[q][i], q, i);
          }
      };
      if constexpr (SIGMOID) {
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = exp2_approx(-fabsf(z[q][i]) * kLog2e), r = reciprocal(1.f + x), w = x * r;
            sums_of(z[q][i] < 0.f ? w : r, q, i);
            g[q][i] = w * r;
          }
      } else {
        shifted();
      }
      over_lanes([&](int o) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      });
      if (SIGMOID && __any_sync(0xffffffffu, used && sum < kFarBelow)) {   // all scores of some token below -19
        const float sum0 = sum, dot0 = dot;
        float g0[N][4];
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) g0[q][i] = g[q][i];
        sum = dot = 0.f;
        shifted();
        over_lanes([&](int o) {
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        });
        if (!(sum0 < kFarBelow)) {   // this group's token was fine
          sum = sum0, dot = dot0;
#pragma unroll
          for (int q = 0; q < N; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) g[q][i] = g0[q][i];
        }
      }
      // a token whose scores are all -inf has no probabilities and counts as zeros
      const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
      dot *= inv * scale;
      if (used && sub == 0) acc += weight * dot;
      const float c = coef * weight * inv, cs = c * scale, cd = c * dot;
#pragma unroll
      for (int q = 0; q < N; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) g[q][i] *= fmaf(f[q][i], cs, -cd);
      if (!used) {
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) g[q][i] = 0.f;
      }
    } else {
      if (next >= 0) load(t + per_pass);
#pragma unroll
      for (int q = 0; q < N; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) g[q][i] = 0.f;
    }
    if (a.dscores != nullptr && t < end) store(t, g);
    now = next, next = later;
  }
  return acc;
}

// The warps' sums added in order; the result is thread 0's.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double sums[kWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < kWarps; ++i) v += sums[i];
  return v;
}

template <int N, Mode M, bool SIGMOID, int DT>
__global__ void __launch_bounds__(kThreads, kLossBlocksPerSm) balance_loss_kernel(const Loss a) {
  __shared__ bool last;
  pdl_wait();
  pdl_launch_dependents();
  // a block's warps lie far apart: padding, which costs little, is shared by all SMs
  const int run = (int)min((long long)a.T, ((long long)(threadIdx.x >> 5) * gridDim.x + blockIdx.x) * a.per_warp);
  const int end = (int)min((long long)a.T, (long long)run + a.per_warp);
  double v = block_sum((double)loss_of_run<N, M, SIGMOID, DT>(a, run, end));
  if (threadIdx.x == 0) {
    a.part[blockIdx.x] = v;
    __threadfence();
    last = atomicAdd(&a.head->ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (last && threadIdx.x < 32) {   // the blocks' sums, in a fixed order
    __threadfence();
    v = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += 32) v += __ldcg(a.part + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x == 0 && a.loss != nullptr) *a.loss = (float)v;
  }
}

// All of it in one block, for batches so small that three launches cost more
// than the work: the same steps with barriers between them.
template <int N, Mode M, bool SIGMOID, int DT>
__global__ void __launch_bounds__(kThreads) balance_small_kernel(const Count c, const Loss a, int nhead) {
  pdl_wait();
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < nhead; i += kThreads) reinterpret_cast<int32_t*>(c.head)[i] = 0;
  if (c.topk != nullptr)
    for (int i = threadIdx.x; i < c.S * c.E; i += kThreads) c.counts[i] = 0;
  __syncthreads();
  const int tiles = max(1, (c.T + kThreads - 1) / kThreads);
  for (int i = 0; i < tiles; ++i) {
    count_tile(c, i, tiles);
    __syncthreads();
  }
  if (a.loss == nullptr && a.dscores == nullptr) return;
  const int run = min(a.T, (int)(threadIdx.x >> 5) * a.per_warp);
  const double v = block_sum((double)loss_of_run<N, M, SIGMOID, DT>(a, run, min(a.T, run + a.per_warp)));
  if (threadIdx.x == 0 && a.loss != nullptr) *a.loss = (float)v;
}

}  // namespace

BalanceLayout balance_layout(const moe_balance_config& c) {
  BalanceLayout L{};
  L.nkept = align256(sizeof(Head));
  L.seq_of = align256(L.nkept + sizeof(int32_t) * (size_t)c.S);
  L.part = align256(L.seq_of + sizeof(int32_t) * (size_t)c.T);
  L.total = align256(L.part + sizeof(double) * kMaxLossBlocks);
  return L;
}

cudaError_t launch_balance(const moe_balance_config& c, const void* scores, const int32_t* topk, const int32_t* off,
                           const unsigned char* mask, const float* coef, int32_t* counts, float* loss, void* dscores,
                           moe_stats* stats, void* ws, cudaStream_t s) {
  const BalanceLayout L = balance_layout(c);
  char* base = static_cast<char*>(ws);
  Head* head = reinterpret_cast<Head*>(base);
  int32_t* nkept = reinterpret_cast<int32_t*>(base + L.nkept);
  int32_t* seq_of = reinterpret_cast<int32_t*>(base + L.seq_of);
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const Count count{topk, off, mask, counts, nkept, seq_of, head, stats, c.T, c.E, c.k, c.S};
  const int nhead = (int)(L.seq_of / 4);   // the head and n_s
  auto aligned = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  const bool vec =
      c.E % 4 == 0 && aligned(scores, 4 * dtype_bytes(c.dtype)) && aligned(dscores, 4 * dtype_bytes(c.dtype));
  const bool small = (long long)c.T * c.E <= kSmallScores && c.T <= kSmallTokens && c.S <= kSmallTokens;
  // Four quads of experts to a lane, so that a token costs few lanes' worth of
  // reductions and bookkeeping; fewer as long as warps would be without a token.
  const int quads = (c.E + 3) / 4;
  const long long warps = small ? kWarps : (long long)std::min(di.sms * kLossBlocksPerSm, kMaxLossBlocks) * kWarps;
  int lanes = 1;
  while (lanes * (small ? 2 : 4) < quads) lanes *= 2;
  while (lanes < 32 && lanes < quads && (long long)c.T * lanes / 32 < warps) lanes *= 2;
  const int n = (quads + lanes - 1) / lanes;
  // an even share of tokens for each warp, whole passes of the warp's token groups
  const int pass = 32 / lanes;
  const long long passes = std::max<long long>(1, ((long long)c.T + pass - 1) / pass);
  const int per_warp = (int)((passes + warps - 1) / warps) * pass;
  const Loss a{scores, seq_of,  coef, counts, nkept,   head,  reinterpret_cast<double*>(base + L.part),
               loss,   dscores, c.T,  c.E,    lanes, per_warp};
  // f(mode, type, sigmoid) with the three as types
  auto with_kind = [&](auto&& f) {
    auto typed = [&](auto mode) {
      using F32 = std::integral_constant<int, MOE_DTYPE_F32>;
      using BF16 = std::integral_constant<int, MOE_DTYPE_BF16>;
      if (c.dtype == MOE_DTYPE_F32)
        return c.score == MOE_SCORE_SIGMOID ? f(mode, F32{}, std::true_type{}) : f(mode, F32{}, std::false_type{});
      return c.score == MOE_SCORE_SIGMOID ? f(mode, BF16{}, std::true_type{}) : f(mode, BF16{}, std::false_type{});
    };
    if (!vec) return typed(std::integral_constant<Mode, kSingle>{});
    if (c.E == 4 * lanes * n) return typed(std::integral_constant<Mode, kWhole>{});
    return typed(std::integral_constant<Mode, kVector>{});
  };
  if (small)
    return with_kind([&](auto mode, auto type, auto sigmoid) {
      constexpr Mode M = decltype(mode)::value;
      constexpr int DT = decltype(type)::value;
      constexpr bool SIG = decltype(sigmoid)::value;
      return launch_pdl(n == 1 ? balance_small_kernel<1, M, SIG, DT> : balance_small_kernel<2, M, SIG, DT>, dim3(1),
                        dim3(kThreads), 0, s, count, a, nhead);
    });
  const size_t ncounts = topk != nullptr ? (size_t)c.S * c.E : 0, most = (size_t)di.sms * 4;
  const size_t words = std::max<size_t>(ncounts, nhead);
  e = launch_pdl(balance_clear_kernel, dim3((unsigned)std::min(most, (words + kThreads - 1) / kThreads)),
                 dim3(kThreads), 0, s, counts, ncounts, reinterpret_cast<int32_t*>(head), nhead);
  if (e != cudaSuccess) return e;
  const unsigned tiles = std::max(1, (c.T + kThreads - 1) / kThreads);
  if ((e = launch_pdl(balance_count_kernel, dim3(tiles), dim3(kThreads), 0, s, count)) != cudaSuccess) return e;
  if (loss == nullptr && dscores == nullptr) return cudaSuccess;
  const unsigned blocks =
      (unsigned)std::max<long long>(1, (((long long)c.T + per_warp - 1) / per_warp + kWarps - 1) / kWarps);
  return with_kind([&](auto mode, auto type, auto sigmoid) {
    constexpr Mode M = decltype(mode)::value;
    constexpr int DT = decltype(type)::value;
    constexpr bool SIG = decltype(sigmoid)::value;
    auto kernel = n == 1   ? balance_loss_kernel<1, M, SIG, DT>
                  : n == 2 ? balance_loss_kernel<2, M, SIG, DT>
                  : n == 3 ? balance_loss_kernel<3, M, SIG, DT> : balance_loss_kernel<4, M, SIG, DT>;
    return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, s, a);
  });
}

}  // namespace moe
