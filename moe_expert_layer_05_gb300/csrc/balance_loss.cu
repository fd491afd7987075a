// The router's balance loss: how often each expert was chosen against how much
// probability it was given,
//
//   loss = E / (k N^2) sum_e c[e] sum_t p[t, e],
//
// over the N tokens that count; c[e] the times expert e is among their k choices, p[t] the
// softmax of token t's logits, or their sigmoids divided by the sigmoids' sum.  1 where all is even.
// The choices are constants of the gradient, so the loss is linear in p with the slope
// w[e] = E c[e] / (k N^2), the same for every token:
//
//   d loss / d logits[t, e] = p[t, e] (w[e] - sum_j w[j] p[t, j])   (times 1 - sigmoid for sigmoid scores).
//
// G lanes a row (8, 16 or 32, the least that leaves a lane at most eight experts or fills a
// warp), lane l the experts l, l + G, ...  The forward keeps a lane's sums of p over its rows in
// registers; the blocks leave partial sums, and the last one to finish adds them in block
// order, so the bits do not depend on timing.
#include <cuda_runtime.h>

#include "entry_checks.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxBlocks = 304;            // forward: two on each SM
constexpr int kMaxTokens = 1 << 24;
constexpr uint32_t kAll = 0xffffffffu;

struct BalanceParams {
  const float* logits;       // [T, E]
  const int32_t* topk;       // [T, k]
  const int32_t* tokens;     // [T] or nullptr
  int T, E, k, score;
  float* part;               // [blocks][E] sums of p
  int32_t* part_count;       // [blocks][E + 1] choices, tokens
  float* loss;
  int32_t* counts;
  float* slope;              // [E]
  const float* dloss;
  float* dlogits;
  int* status;
};

template <int G>
__device__ __forceinline__ float row_max(float v) {
  #pragma unroll
  for (int m = G / 2; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, m));
  return v;
}
template <int G>
__device__ __forceinline__ float row_sum(float v) {
  #pragma unroll
  for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
  return v;
}

// x[i]: this lane's logits in, probabilities out (experts past E: -infinity in).
// rest[i] (sigmoid): 1 - sigmoid.  A row of -infinity alone has no probabilities: zeros.
template <int G, int NV>
__device__ __forceinline__ void probabilities(float (&x)[NV], float (&rest)[NV], bool sigmoid) {
  float m = x[0];
  #pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, x[i]);
  m = row_max<G>(m);
  float sum = 0.f;
  if (!sigmoid) {
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = expf(x[i] - m);
      sum += x[i];
    }
  } else {
    // sigmoids over exp(min(m, 0)): far below zero they have no fp32 value, their ratios do
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float t = expf(-fabsf(x[i])), r = 1.f / (1.f + t);
      const bool pos = x[i] >= 0.f;
      rest[i] = pos ? t * r : r;
      x[i] = r * (pos ? 1.f : m >= 0.f ? t : expf(x[i] - m));
      sum += x[i];
    }
  }
  sum = row_sum<G>(sum);
  const float inv = 1.f / sum;
  #pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = m == -INFINITY ? 0.f : x[i] * inv;
}

template <int G, int NV>
__device__ __forceinline__ void load_row(const BalanceParams& p, long long row, bool on, int l, float (&x)[NV]) {
  #pragma unroll
  for (int i = 0; i < NV; ++i)
    x[i] = on && l + G * i < p.E ? p.logits[row * p.E + l + G * i] : -INFINITY;
}

template <int G, int NV>
__global__ void __launch_bounds__(kThreads) balance_fwd_kernel(const BalanceParams p) {
  pdl_entry();
  __shared__ float s_sum[kWarps * (32 / G)][G * NV];
  __shared__ int s_count[kMaxE + 1];
  __shared__ double s_part[kThreads];
  __shared__ int s_last;
  const int lane = threadIdx.x & 31, l = lane % G, sub = threadIdx.x / G;
  constexpr int kRows = kThreads / G;                        // rows at a time
  for (int i = threadIdx.x; i <= p.E; i += kThreads) s_count[i] = 0;
  __syncthreads();
  float acc[NV];
  #pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.f;
  int counted = 0;
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  for (long long r0 = static_cast<long long>(blockIdx.x) * kRows; r0 < p.T; r0 += step) {
    const long long row = r0 + sub;
    const bool on = row < p.T && (p.tokens == nullptr || p.tokens[row] >= 0);
    float x[NV], rest[NV];
    load_row<G, NV>(p, row, on, l, x);
    if (on) {
      for (int j = l; j < p.k; j += G) {
        const int e = p.topk[row * p.k + j];
        if (e >= 0 && e < p.E)
          atomicAdd(&s_count[e], 1);
        else
          set_status(p.status, kErrBadIndex);
      }
      if (l == 0) ++counted;
    }
    probabilities<G, NV>(x, rest, p.score != 0);
    #pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] += x[i];
  }
  if (counted != 0) atomicAdd(&s_count[p.E], counted);
  #pragma unroll
  for (int i = 0; i < NV; ++i) s_sum[sub][l + G * i] = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    float a = 0.f;
    for (int s = 0; s < kRows; ++s) a += s_sum[s][e];
    p.part[static_cast<long long>(blockIdx.x) * p.E + e] = a;
  }
  for (int i = threadIdx.x; i <= p.E; i += kThreads)
    p.part_count[static_cast<long long>(blockIdx.x) * (p.E + 1) + i] = s_count[i];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(p.status + kBalanceDoneWord, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // the last block: an expert a thread
  int n = 0;
  for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += kThreads) n += __ldcg(p.part_count + b * (p.E + 1) + p.E);
  s_part[threadIdx.x] = n;
  __syncthreads();
  for (int h = kThreads / 2; h > 0; h >>= 1) {
    if (static_cast<int>(threadIdx.x) < h) s_part[threadIdx.x] += s_part[threadIdx.x + h];
    __syncthreads();
  }
  const double tokens = s_part[0];
  __syncthreads();
  double mine = 0.0;
  const int e = threadIdx.x;
  if (e < p.E) {
    double sum = 0.0;
    int c = 0;
    #pragma unroll 16
    for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
      sum += __ldcg(p.part + b * p.E + e);
      c += __ldcg(p.part_count + b * (p.E + 1) + e);
    }
    const double w = tokens > 0.0 ? p.E * static_cast<double>(c) / (p.k * tokens * tokens) : 0.0;
    p.counts[e] = c;
    p.slope[e] = static_cast<float>(w);
    mine = w * sum;
  }
  s_part[threadIdx.x] = mine;
  __syncthreads();
  for (int h = kThreads / 2; h > 0; h >>= 1) {
    if (static_cast<int>(threadIdx.x) < h) s_part[threadIdx.x] += s_part[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    p.loss[0] = static_cast<float>(s_part[0]);
    atomicExch(p.status + kBalanceDoneWord, 0);
  }
}

template <int G, int NV>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(const BalanceParams p) {
  pdl_entry();
  const int lane = threadIdx.x & 31, l = lane % G;
  constexpr int kRows = kThreads / G;
  float w[NV];
  #pragma unroll
  for (int i = 0; i < NV; ++i) w[i] = l + G * i < p.E ? p.slope[l + G * i] : 0.f;
  const float scale = p.dloss[0];
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  for (long long r0 = static_cast<long long>(blockIdx.x) * kRows; r0 < p.T; r0 += step) {
    const long long row = r0 + threadIdx.x / G;
    const bool on = row < p.T && (p.tokens == nullptr || p.tokens[row] >= 0);
    float x[NV], rest[NV];
    load_row<G, NV>(p, row, on, l, x);
    probabilities<G, NV>(x, rest, p.score != 0);
    float dot = 0.f;
    #pragma unroll
    for (int i = 0; i < NV; ++i) dot = fmaf(w[i], x[i], dot);
    dot = row_sum<G>(dot);
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      float d = x[i] * (w[i] - dot) * scale;
      if (p.score != 0) d *= rest[i];
      if (row < p.T && l + G * i < p.E) p.dlogits[row * p.E + l + G * i] = on ? d : 0.f;
    }
  }
}

int rows_at_a_time(int E) { return E <= 8 ? kThreads / 8 : E <= 16 ? kThreads / 16 : kThreads / 32; }
int fwd_blocks(int T, int E) {
  const int r = rows_at_a_time(E), b = static_cast<int>((static_cast<long long>(T) + r - 1) / r);
  return b < 1 ? 1 : b < kMaxBlocks ? b : kMaxBlocks;
}

template <class... Args>
cudaError_t run(void (*const (&kern)[6])(Args...), const BalanceParams& p, int blocks, cudaStream_t st) {
  const int E = p.E;
  const int i = E <= 8 ? 0 : E <= 16 ? 1 : E <= 32 ? 2 : E <= 64 ? 3 : E <= 128 ? 4 : 5;
  count_launches(1);
  return launch_k(kern[i], blocks, kThreads, 0, st, p);
}

bool sizes_ok(int32_t T, int32_t E) { return T >= 0 && T <= kMaxTokens && E > 0 && E <= kMaxE; }
bool score_ok(int32_t score) { return score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID; }

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::entry;

extern "C" {

size_t moe_balance_loss_workspace_bytes(int32_t T, int32_t E) {
  if (!sizes_ok(T, E)) return 0;
  return kStatusBytes + align_up(static_cast<size_t>(fwd_blocks(T, E)) * (2 * E + 1) * 4);
}

moe_status moe_balance_loss_forward(const float* logits, const int32_t* topk_idx, const int32_t* tokens, int32_t T,
                                    int32_t E, int32_t k, int32_t score, float* loss, int32_t* counts, float* slope,
                                    void* ws, size_t ws_bytes, void* stream) {
  if (!sizes_ok(T, E) || k <= 0 || k > kMaxK || k > E || !score_ok(score)) return MOE_ERR_INVALID_ARG;
  if (!ptr_ok(loss) || !ptr_ok(counts) || !ptr_ok(slope) || !ptr_ok(ws) || !opt_ok(tokens)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ptr_ok(logits) || !ptr_ok(topk_idx))) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_balance_loss_workspace_bytes(T, E)) return MOE_ERR_WORKSPACE;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  BalanceParams p = {};
  p.logits = logits;
  p.topk = topk_idx;
  p.tokens = tokens;
  p.T = T;
  p.E = E;
  p.k = k;
  p.score = score;
  const int blocks = fwd_blocks(T, E);
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kStatusBytes);
  p.part_count = reinterpret_cast<int32_t*>(p.part + static_cast<size_t>(blocks) * E);
  p.loss = loss;
  p.counts = counts;
  p.slope = slope;
  p.status = static_cast<int*>(ws);
  static void (*const kern[6])(BalanceParams) = {balance_fwd_kernel<8, 1>,  balance_fwd_kernel<16, 1>,
                                                 balance_fwd_kernel<32, 1>, balance_fwd_kernel<32, 2>,
                                                 balance_fwd_kernel<32, 4>, balance_fwd_kernel<32, 8>};
  return status_of(run(kern, p, blocks, static_cast<cudaStream_t>(stream)));
}

moe_status moe_balance_loss_backward(const float* logits, const float* slope, const int32_t* tokens, int32_t T,
                                     int32_t E, int32_t score, const float* dloss, float* dlogits, void* stream) {
  if (!sizes_ok(T, E) || !score_ok(score) || !ptr_ok(slope) || !ptr_ok(dloss) || !opt_ok(tokens))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ptr_ok(logits) || !ptr_ok(dlogits))) return MOE_ERR_INVALID_ARG;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  BalanceParams p = {};
  p.logits = logits;
  p.tokens = tokens;
  p.T = T;
  p.E = E;
  p.score = score;
  p.slope = const_cast<float*>(slope);
  p.dloss = dloss;
  p.dlogits = dlogits;
  const int r = rows_at_a_time(E), need = static_cast<int>((static_cast<long long>(T) + r - 1) / r);
  static void (*const kern[6])(BalanceParams) = {balance_bwd_kernel<8, 1>,  balance_bwd_kernel<16, 1>,
                                                 balance_bwd_kernel<32, 1>, balance_bwd_kernel<32, 2>,
                                                 balance_bwd_kernel<32, 4>, balance_bwd_kernel<32, 8>};
  return status_of(run(kern, p, need < 8 * kMaxBlocks ? need : 8 * kMaxBlocks, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
