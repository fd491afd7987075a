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

constexpr int kThreads = 512;
constexpr int kMaxBlocks = 152;            // forward: one on each SM
constexpr int kMaxTokens = 1 << 24;
constexpr uint32_t kAll = 0xffffffffu;

struct BalanceParams {
  const float* logits;       // [T, E]
  const int32_t* topk;       // [T, k]
  const int32_t* tokens;     // [T] or nullptr
  int T, E, k, score;
  uint4* part;               // [blocks][part_words(E)]
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

// e^x and 1 / x by the special function unit, off by a few U and, for e^x, by x's own rounding (|x| U).
__device__ __forceinline__ float exp_of(float x) { return ex2(x * 1.4426950408889634f); }
__device__ __forceinline__ float inverse(float x) { return __fdividef(1.f, x); }

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
      x[i] = exp_of(x[i] - m);
      sum += x[i];
    }
  } else {
    // sigmoids over exp(min(m, 0)): far below zero they have no fp32 value, their ratios do
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float t = exp_of(-fabsf(x[i])), r = inverse(1.f + t);
      const bool pos = x[i] >= 0.f;
      rest[i] = pos ? t * r : r;
      x[i] = r * (pos ? 1.f : m >= 0.f ? t : exp_of(x[i] - m));
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

// The sums of a block over its rows, and the choices, as it leaves them: E floats, then E + 1 ints (the
// last one its tokens), in words of four.
__host__ __device__ constexpr int sum_words(int E) { return (E + 3) / 4; }
__host__ __device__ constexpr int part_words(int E) { return sum_words(E) + (E + 4) / 4; }

template <int G, int NV>
__global__ void __launch_bounds__(kThreads) balance_fwd_kernel(const BalanceParams p) {
  pdl_entry();
  constexpr int kRows = kThreads / G;                        // rows at a time
  constexpr int kMaxWords = part_words(kMaxE);
  __shared__ float s_sum[kThreads / 32][G * NV > 4 ? G * NV : 4];
  __shared__ __align__(16) int s_out[4 * kMaxWords];         // this block's part
  __shared__ uint4 s_join[kThreads];
  __shared__ float s_red[kThreads / 32];
  __shared__ double s_unit;
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G, sub = threadIdx.x / G;
  const int ws = sum_words(p.E), words = part_words(p.E);
  for (int i = threadIdx.x; i < 4 * words; i += kThreads) s_out[i] = 0;
  __syncthreads();
  int* s_count = s_out + 4 * ws;
  float acc[NV];
  #pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.f;
  int counted = 0;
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  // (a row's loads are on their way while the row before it is worked on)
  float next[NV];
  int choice = 0;
  bool next_on = false;
  auto fetch = [&](long long row) {
    const bool in = row < p.T;
    next_on = in && (p.tokens == nullptr || p.tokens[row] >= 0);
    load_row<G, NV>(p, row, in, l, next);
    choice = in && l < p.k ? p.topk[row * p.k + l] : 0;
  };
  auto count = [&](int e) {
    if (e >= 0 && e < p.E)
      atomicAdd(&s_count[e], 1);
    else
      set_status(p.status, kErrBadIndex);
  };
  fetch(static_cast<long long>(blockIdx.x) * kRows + sub);
  for (long long r0 = static_cast<long long>(blockIdx.x) * kRows; r0 < p.T; r0 += step) {
    const long long row = r0 + sub;
    const bool on = next_on;
    const int first = choice;
    float x[NV], rest[NV];
    #pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = on ? next[i] : -INFINITY;
    fetch(row + step);
    if (on) {
      if (l < p.k) count(first);
      for (int j = l + G; j < p.k; j += G) count(p.topk[row * p.k + j]);     // (k above the lanes of a row)
      if (l == 0) ++counted;
    }
    probabilities<G, NV>(x, rest, p.score != 0);
    #pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] += x[i];
  }
  if (counted != 0) atomicAdd(&s_count[p.E], counted);
  // the rows of a warp, then the warps in order
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    #pragma unroll
    for (int m = G; m < 32; m <<= 1) acc[i] += __shfl_xor_sync(kAll, acc[i], m);
    if (lane < G) s_sum[warp][l + G * i] = acc[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    float a = 0.f;
    #pragma unroll
    for (int s = 0; s < kThreads / 32; ++s) a += s_sum[s][e];
    s_out[e] = __float_as_int(a);
  }
  __syncthreads();
  if (gridDim.x > 1) {
  uint4* part = p.part + static_cast<long long>(blockIdx.x) * words;
  for (int i = threadIdx.x; i < words; i += kThreads) part[i] = reinterpret_cast<const uint4*>(s_out)[i];
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(p.status + kBalanceDoneWord, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // The last block: thread = (strand, word); strand s adds the blocks s, s + strands, ..., the strands are added
  // in order.
  const int strands = kThreads / words, strand = threadIdx.x / words, w = threadIdx.x - strand * words;
  const bool sums = w < ws;
  float f[4] = {0.f, 0.f, 0.f, 0.f};
  int c[4] = {0, 0, 0, 0};
  auto add = [&](const uint4& v) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sums)
        f[i] += __uint_as_float(u[i]);
      else
        c[i] += static_cast<int>(u[i]);
    }
  };
  if (strand < strands) {
    #pragma unroll 16
    for (int b = strand; b < static_cast<int>(gridDim.x); b += strands) add(__ldcg(p.part + b * words + w));
  }
  auto pack = [&] {
    return sums ? make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]))
                : make_uint4(c[0], c[1], c[2], c[3]);
  };
  s_join[threadIdx.x] = pack();
  __syncthreads();
  if (strand == 0) {
    for (int s = 1; s < strands; ++s) add(s_join[s * words + w]);
    reinterpret_cast<uint4*>(s_out)[w] = pack();
  }
  __syncthreads();
  }
  // (one fp64 division for all: there are two lanes of it)
  if (threadIdx.x == 0) {
    const double n = s_count[p.E];
    s_unit = n > 0.0 ? p.E / (p.k * n * n) : 0.0;
  }
  __syncthreads();
  float mine = 0.f;
  const int e = threadIdx.x;
  if (e < p.E) {
    const float slope = static_cast<float>(s_count[e] * s_unit);
    p.counts[e] = s_count[e];
    p.slope[e] = slope;
    mine = slope * __int_as_float(s_out[e]);
  }
  #pragma unroll
  for (int m = 16; m > 0; m >>= 1) mine += __shfl_xor_sync(kAll, mine, m);
  if (lane == 0) s_red[warp] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    float loss = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) loss += s_red[i];
    p.loss[0] = loss;
    if (gridDim.x > 1) atomicExch(p.status + kBalanceDoneWord, 0);
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
  float next[NV];
  bool next_on = false;
  auto fetch = [&](long long row) {
    next_on = row < p.T && (p.tokens == nullptr || p.tokens[row] >= 0);
    load_row<G, NV>(p, row, row < p.T, l, next);
  };
  fetch(static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / G);
  for (long long r0 = static_cast<long long>(blockIdx.x) * kRows; r0 < p.T; r0 += step) {
    const long long row = r0 + threadIdx.x / G;
    const bool on = next_on;
    float x[NV], rest[NV];
    #pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = on ? next[i] : -INFINITY;
    fetch(row + step);
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

constexpr int kFwdRounds = 4;   // rows of a lane group before there is another block
int rows_at_a_time(int E) { return E <= 8 ? kThreads / 8 : E <= 16 ? kThreads / 16 : kThreads / 32; }
int fwd_blocks(int T, int E) {
  const long long r = kFwdRounds * rows_at_a_time(E), b = (T + r - 1) / r;
  return b < 1 ? 1 : b < kMaxBlocks ? static_cast<int>(b) : kMaxBlocks;
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
  return kStatusBytes + align_up(static_cast<size_t>(fwd_blocks(T, E)) * part_words(E) * sizeof(uint4));
}

moe_status moe_balance_loss_forward(const float* logits, const int32_t* topk_idx, const int32_t* tokens, int32_t T,
                                    int32_t E, int32_t k, int32_t score, float* loss, int32_t* counts, float* slope,
                                    void* ws, size_t ws_bytes, void* stream) {
  if (!sizes_ok(T, E) || k <= 0 || k > kMaxK || k > E || !score_ok(score)) return MOE_ERR_INVALID_ARG;
  if (!word_ok(loss) || !word_ok(counts) || !word_ok(slope) || !ptr_ok(ws) || !opt_ok(tokens)) return MOE_ERR_INVALID_ARG;
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
  p.part = reinterpret_cast<uint4*>(static_cast<char*>(ws) + kStatusBytes);
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
  if (!sizes_ok(T, E) || !score_ok(score) || !word_ok(slope) || !word_ok(dloss) || !opt_ok(tokens))
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
  return status_of(run(kern, p, need < 4 * kMaxBlocks ? need : 4 * kMaxBlocks, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
