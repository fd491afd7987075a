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
// G lanes a row, lane l the four experts from 4 l on (above 128 experts four more, 128 further
// on), so a row of a multiple of four is read in 16-byte words.  The forward keeps a lane's sums
// of p over its rows in registers; the blocks leave partial sums, and the last one to finish adds them,
// in an order that does not depend on timing.  Both directions read the logits once.
//
// Measured (device time, a call): 256 x 8 3.0 us forward and 1.5 backward, 4096 x 64 8.2 and 1.8, 16384 x 256 with
// sigmoids 12.5 and 7.6 (backward: 4.4 TB/s).  The forward is bound by what follows its rows: the wait for the
// slowest block, two fences, an atomic and the reads of the others' sums, each a round trip to the L2.
#include <cuda_runtime.h>

#include "entry_checks.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;              // backward
constexpr int kMaxBlocks = 152;            // forward: one on each SM
constexpr int kJoin = 11;                  // partial sums on their way at a time
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
// rest[i] (sigmoid): 1 - sigmoid.  A row of -infinity alone has no probabilities: zeros.  The maximum knows nothing of
// NaN, so it is the sum that tells such a row (0) from one with a NaN (NaN throughout).
template <int G, int NV>
__device__ __forceinline__ void probabilities(float (&x)[NV], float (&rest)[NV], bool sigmoid) {
  float m = x[0];
  #pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, x[i]);
  m = row_max<G>(m);
  if (m == -INFINITY) m = 0.f;
  float sum = 0.f;
  if (!sigmoid) {
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = exp_of(x[i] - m);
      sum += x[i];
    }
  } else {
    // sigmoids over exp(min(m, 0)): far below zero they have no fp32 value, their ratios do
    float e[NV];
    #pragma unroll
    for (int i = 0; i < NV; ++i) e[i] = exp_of(-fabsf(x[i]));
    const bool low = m < 0.f;
    if (__any_sync(kAll, low)) {
      #pragma unroll
      for (int i = 0; i < NV; ++i) rest[i] = low ? exp_of(x[i] - m) : e[i];
    } else {
      #pragma unroll
      for (int i = 0; i < NV; ++i) rest[i] = e[i];
    }
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float r = inverse(1.f + e[i]);
      const bool pos = x[i] >= 0.f;
      x[i] = pos ? r : r * rest[i];
      rest[i] = pos ? e[i] * r : r;
      sum += x[i];
    }
  }
  sum = row_sum<G>(sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  #pragma unroll
  for (int i = 0; i < NV; ++i) x[i] *= inv;
}

// Expert of a lane's value i.
template <int G>
__device__ __forceinline__ constexpr int expert_of(int l, int i) { return 4 * (l + G * (i / 4)) + i % 4; }

template <int G, int NV>
__device__ __forceinline__ void load_row(const BalanceParams& p, long long row, bool on, int l, float (&x)[NV]) {
  const float* src = p.logits + row * p.E;
  #pragma unroll
  for (int i = 0; i < NV; i += 4) {
    const int e = expert_of<G>(l, i);
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (on && e < p.E) {
      if (p.E % 4 == 0) {
        v = *reinterpret_cast<const float4*>(src + e);
      } else {
        v.x = src[e];
        if (e + 1 < p.E) v.y = src[e + 1];
        if (e + 2 < p.E) v.z = src[e + 2];
        if (e + 3 < p.E) v.w = src[e + 3];
      }
    }
    x[i] = v.x;
    x[i + 1] = v.y;
    x[i + 2] = v.z;
    x[i + 3] = v.w;
  }
}

// The sums of a block over its rows, and the choices, as it leaves them: E floats, then E + 1 ints (the
// last one its tokens), in words of four.
__host__ __device__ constexpr int sum_words(int E) { return (E + 3) / 4; }
__host__ __device__ constexpr int part_words(int E) { return sum_words(E) + (E + 4) / 4; }

// A block of the forward.  Rows of more than 128 experts want more of their loads on their way: 13.8 us with
// 512 threads, 12.5 with 1024 at 16384 x 256; with fewer experts the sums of more warps cost more than
// that gives (8.3 against 9.3 us at 4096 x 64).
__host__ __device__ constexpr int fwd_threads(int E) { return E > 128 ? 1024 : 512; }

template <int G, int NV>
__global__ void __launch_bounds__(fwd_threads(G * NV)) balance_fwd_kernel(const BalanceParams p) {
  pdl_entry();
  constexpr int TH = fwd_threads(G * NV);
  constexpr int kRows = TH / G;                        // rows at a time
  constexpr int kMaxWords = part_words(kMaxE);
  __shared__ union {
    float sum[TH / 32][G * NV];                        // of each warp
    uint4 join[TH];                                    // the last block's strands
  } s_mem;
  __shared__ __align__(16) int s_out[4 * kMaxWords];         // this block's part
  __shared__ float s_red[TH / 32];
  __shared__ double s_unit;
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G, sub = threadIdx.x / G;
  const int ws = sum_words(p.E), words = part_words(p.E);
  for (int i = threadIdx.x; i < 4 * words; i += TH) s_out[i] = 0;
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
    if (lane < G) s_mem.sum[warp][expert_of<G>(l, i)] = acc[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += TH) {
    float a = 0.f;
    #pragma unroll
    for (int s = 0; s < TH / 32; ++s) a += s_mem.sum[s][e];
    s_out[e] = __float_as_int(a);
  }
  __syncthreads();
  const bool sums = static_cast<int>(threadIdx.x) % words < ws;
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
  auto pack = [&] {
    return sums ? make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]))
                : make_uint4(c[0], c[1], c[2], c[3]);
  };
  const int w = threadIdx.x % words;
  uint4* out = reinterpret_cast<uint4*>(s_out);
  if (gridDim.x > 1) {
    if (static_cast<int>(threadIdx.x) < words) p.part[blockIdx.x * words + w] = out[w];
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(p.status + kBalanceDoneWord, 1) == static_cast<int>(gridDim.x) - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // The last one: thread = (strand, word); strand s adds the blocks s, s + strands, ..., the strands are added
    // in order.
    const int blocks = gridDim.x, strands = TH / words, strand = threadIdx.x / words;
    if (strand < strands) {
      // (a batch's loads go out together: one after the other each costs an L2 round trip)
      for (int b0 = strand; b0 < blocks; b0 += kJoin * strands) {
        uint4 v[kJoin];
        #pragma unroll
        for (int j = 0; j < kJoin; ++j) {
          const int b = b0 + j * strands;
          v[j] = b < blocks ? __ldcg(p.part + b * words + w) : make_uint4(0, 0, 0, 0);
        }
        #pragma unroll
        for (int j = 0; j < kJoin; ++j) add(v[j]);
      }
    }
    s_mem.join[threadIdx.x] = pack();
    __syncthreads();
    if (strand == 0) {
      for (int i = 1; i < strands; ++i) add(s_mem.join[i * words + w]);
      out[w] = pack();
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
    for (int i = 0; i < TH / 32; ++i) loss += s_red[i];
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
  for (int i = 0; i < NV; ++i) w[i] = expert_of<G>(l, i) < p.E ? p.slope[expert_of<G>(l, i)] : 0.f;
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
    if (row >= p.T) continue;
    float* dst = p.dlogits + row * p.E;
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] *= (w[i] - dot) * scale;
      if (p.score != 0) x[i] *= rest[i];
      if (!on) x[i] = 0.f;
    }
    #pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int e = expert_of<G>(l, i);
      if (e < p.E) {
        if (p.E % 4 == 0) {
          *reinterpret_cast<float4*>(dst + e) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
          #pragma unroll
          for (int c = 0; c < 4; ++c)
            if (e + c < p.E) dst[e + c] = x[i + c];
        }
      }
    }
  }
}

constexpr int kFwdRounds = 4;   // rows of a lane group before there is another block
int lanes_of(int E) { return E <= 8 ? 2 : E <= 16 ? 4 : E <= 32 ? 8 : E <= 64 ? 16 : 32; }
int fwd_blocks(int T, int E) {
  const long long r = kFwdRounds * (fwd_threads(E) / lanes_of(E)), b = (T + r - 1) / r;
  return b < 1 ? 1 : b < kMaxBlocks ? static_cast<int>(b) : kMaxBlocks;
}

template <class... Args>
cudaError_t run(void (*const (&kern)[6])(Args...), const BalanceParams& p, int blocks, int threads, cudaStream_t st) {
  const int E = p.E;
  const int i = E <= 8 ? 0 : E <= 16 ? 1 : E <= 32 ? 2 : E <= 64 ? 3 : E <= 128 ? 4 : 5;
  count_launches(1);
  return launch_k(kern[i], blocks, threads, 0, st, p);
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
  if (!word_ok(loss) || !word_ok(counts) || !word_ok(slope) || !ptr_ok(ws) || !opt_ok(tokens))
    return MOE_ERR_INVALID_ARG;
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
  static void (*const kern[6])(BalanceParams) = {balance_fwd_kernel<2, 4>,  balance_fwd_kernel<4, 4>,
                                                 balance_fwd_kernel<8, 4>,  balance_fwd_kernel<16, 4>,
                                                 balance_fwd_kernel<32, 4>, balance_fwd_kernel<32, 8>};
  return status_of(run(kern, p, blocks, fwd_threads(E), static_cast<cudaStream_t>(stream)));
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
  const int r = kThreads / lanes_of(E), need = static_cast<int>((static_cast<long long>(T) + r - 1) / r);
  static void (*const kern[6])(BalanceParams) = {balance_bwd_kernel<2, 4>,  balance_bwd_kernel<4, 4>,
                                                 balance_bwd_kernel<8, 4>,  balance_bwd_kernel<16, 4>,
                                                 balance_bwd_kernel<32, 4>, balance_bwd_kernel<32, 8>};
  const int blocks = need < 4 * kMaxBlocks ? need : 4 * kMaxBlocks;
  return status_of(run(kern, p, blocks, kThreads, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
