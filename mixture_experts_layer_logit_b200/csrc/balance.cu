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
// Bound by the bytes of the scores and their gradient.
#include "elem8.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kCountThreads = 256;
constexpr int kLossThreads = 256;
constexpr int kLossWarps = kLossThreads / 32;
constexpr int kMaxLossBlocks = 1024;

// Words at the start of the workspace, zeroed by the call: then n_s of every sequence.
struct Head {
  unsigned groups;   // G
  unsigned ticket;   // blocks of the loss kernel that are done
};

// Sequence of token t, or -1 behind the last or before the first one.  Any
// contents of off give an index inside [0, S).
__device__ __forceinline__ int sequence_of(const int32_t* off, int S, int t) {
  if (off == nullptr) return 0;
  if (t < off[0] || t >= off[S]) return -1;
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (off[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kCountThreads)
balance_count_kernel(const int32_t* topk, const int32_t* off, const unsigned char* mask, int T, int E, int k, int S,
                     int32_t* counts, int32_t* nkept, Head* head, moe_stats* stats) {
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;
  const int first = blockIdx.x * kCountThreads + threadIdx.x, step = gridDim.x * kCountThreads;
  if (off != nullptr)
    for (int s = first; s < S; s += step) bad |= off[s] < 0 || off[s + 1] < off[s] || off[s + 1] > T;
  for (long long t = first; t < T; t += step) {
    const int s = sequence_of(off, S, (int)t);
    if (s < 0 || (mask != nullptr && mask[t] == 0)) continue;
    if (atomicAdd(&nkept[s], 1) == 0) atomicAdd(&head->groups, 1u);
    if (topk == nullptr) continue;
    for (int j = 0; j < k; ++j) {
      const int e = topk[(size_t)t * k + j];
      if ((unsigned)e < (unsigned)E) atomicAdd(&counts[(size_t)s * E + e], 1);
      else bad = true;
    }
  }
  if (bad && stats != nullptr) atomicOr(&stats->status, MOE_DEV_BOUNDS);
}

// One warp per token, lanes hold experts lane + 32 i.
__global__ void __launch_bounds__(kLossThreads)
balance_loss_kernel(const void* scores, int dt, const int32_t* off, const unsigned char* mask, const float* coef,
                    const int32_t* counts, const int32_t* nkept, Head* head, double* part, int T, int E, int S,
                    int sigmoid, float* loss, void* dscores) {
  constexpr int PER = kMaxExperts / 32;
  __shared__ double sums[kLossWarps];
  __shared__ bool last;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float groups = (float)head->groups, c = coef != nullptr ? *coef : 1.f;
  double acc = 0.0;
  for (long long t = (long long)blockIdx.x * kLossWarps + warp; t < T; t += (long long)gridDim.x * kLossWarps) {
    const int s = sequence_of(off, S, (int)t);
    const size_t row = (size_t)t * E;
    if (s < 0 || (mask != nullptr && mask[t] == 0)) {
      if (dscores != nullptr)
        for (int e = lane; e < E; e += 32) store1(dscores, dt, row + e, 0.f);
      continue;
    }
    float z[PER], f[PER], slope[PER], m = -INFINITY, n = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      z[i] = e < E ? raw_to_float(load_raw1(scores, dt, row + e), dt) : -INFINITY;
      f[i] = e < E ? (float)counts[(size_t)s * E + e] : 0.f;
      m = fmaxf(m, z[i]);
      n += f[i];
    }
    m = warp_max(m);
    n = warp_sum(n);
    float sum = 0.f, dot = 0.f;
    const bool none = m == -INFINITY;   // no score above -inf (or only NaN ones): see below
    const float base = sigmoid ? fminf(m, 0.f) : m;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float zi = z[i];
      if (sigmoid) {   // sigmoid(z) e^-base without underflow, and 1 - sigmoid(z)
        const float e = expf(-fabsf(zi)), r = 1.f / (1.f + e);
        slope[i] = zi >= 0.f ? e * r : r;
        z[i] = zi == -INFINITY ? 0.f : expf((zi < 0.f ? zi : 0.f) - base) * r;
      } else {
        z[i] = zi == -INFINITY ? 0.f : expf(zi - base);
      }
      sum += z[i];
      dot += z[i] * f[i];
    }
    sum = warp_sum(sum);
    dot = warp_sum(dot);
    // p = z / sum; a token whose scores are all -inf has no probabilities and counts as zeros
    const float inv = none && sum == 0.f ? 0.f : 1.f / sum, scale = n > 0.f ? (float)E / n : 0.f;
    dot *= inv * scale;
    const float w = 1.f / (groups * (float)nkept[s]);
    if (lane == 0) acc += (double)(w * dot);
    if (dscores != nullptr) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        if (e < E)
          store1(dscores, dt, row + e, c * w * (z[i] * inv) * (f[i] * scale - dot) * (sigmoid ? slope[i] : 1.f));
      }
    }
  }
  if (lane == 0) sums[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int i = 0; i < kLossWarps; ++i) v += sums[i];
    part[blockIdx.x] = v;
    __threadfence();
    last = atomicAdd(&head->ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (last && warp == 0) {   // the blocks' sums, in a fixed order
    __threadfence();
    double v = 0.0;
    for (int i = lane; i < (int)gridDim.x; i += 32) v += __ldcg(part + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && loss != nullptr) *loss = (float)v;
  }
}

}  // namespace

BalanceLayout balance_layout(const moe_balance_config& c) {
  BalanceLayout L{};
  L.nkept = align256(sizeof(Head));
  L.part = align256(L.nkept + sizeof(int32_t) * (size_t)c.S);
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
  cudaError_t e = cudaMemsetAsync(ws, 0, L.part, s);
  if (e != cudaSuccess) return e;
  if (topk != nullptr || c.T == 0) {
    if (topk != nullptr && (e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)c.S * c.E, s)) != cudaSuccess)
      return e;
  }
  DeviceInfo di;
  if ((e = device_info(&di)) != cudaSuccess) return e;
  const int cb = (int)std::max<long long>(1, std::min<long long>(((long long)std::max(c.T, c.S) + 255) / 256, di.sms * 8));
  if ((e = launch_pdl(balance_count_kernel, dim3(cb), dim3(kCountThreads), 0, s, topk, off, mask, c.T, c.E, c.k, c.S,
                      counts, nkept, head, stats)) != cudaSuccess)
    return e;
  if (loss == nullptr && dscores == nullptr) return cudaSuccess;
  const int lb = (int)std::max<long long>(
      1, std::min<long long>(((long long)c.T + kLossWarps - 1) / kLossWarps, std::min(di.sms * 6, kMaxLossBlocks)));
  return launch_pdl(balance_loss_kernel, dim3(lb), dim3(kLossThreads), 0, s, scores, c.dtype, off, mask, coef,
                    (const int32_t*)counts, (const int32_t*)nkept, head, reinterpret_cast<double*>(base + L.part),
                    c.T, c.E, c.S, c.score == MOE_SCORE_SIGMOID ? 1 : 0, loss, dscores);
}

}  // namespace moe
