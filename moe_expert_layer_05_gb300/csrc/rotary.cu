// Rotary positions: each pair (a, b) of a head's first R values turned by the angle
// position * freq of its pair,
//
//   (a, b) -> scale (a cos - b sin, b cos + a sin),
//
// or by its negative (the gradient: the transposed rotation, times the same scale).  Pairs lie
// side by side (interleaved) or R/2 apart (half); values from R on are copied.
//
// Angles of far positions have no digits left in fp32, so a pair's frequency is taken in
// turns as a 64-bit binary fraction, and position * fraction modulo 2^64 is the angle's
// fraction of a turn: off by 2^-62 (for pairs of up to a radian a position) times the position,
// 2^-31 turns at the last one.
//
// A block works out the sines of its tokens once for all heads, while its first values
// are on their way; then a thread loads one piece of 16 values while it turns the one before, five
// blocks to an SM.  Bound by HBM: every value is read and written once.  16384 tokens of 40 heads of 128 beside
// 8 heads of values, 58 us (5.7 TB/s; four pieces at a time 62, six blocks 62, eight 75); one token 2.7 us.
#include <cuda_runtime.h>

#include <cmath>

#include "entry_checks.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;             // of one block, at most
constexpr int kAhead = 1;              // pieces a thread loads at a time, while it turns the ones before
constexpr int kMaxHeads = 1024, kMaxWidth = 512;      // (kTokens of the widest: 16 KB of sines)

struct RotaryParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  long long x_token, x_head, out_token, out_head;
  const int32_t* positions;
  const double* freq;
  int T, heads, R;
  int turned, tasks;                   // pieces of 16 values of a row: those that turn, all
  int words;                           // 16-byte words of a row
  int block_tokens;
  float scale;
  int interleaved, inverse;
};

// (a, b) of two neighbouring pairs i, i + 1 in words of their own (half layout)
__device__ __forceinline__ void turn_half(uint32_t& a, uint32_t& b, const float2& r0, const float2& r1) {
  const float a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
  a = pack_bf16x2(a0 * r0.x - b0 * r0.y, a1 * r1.x - b1 * r1.y);
  b = pack_bf16x2(b0 * r0.x + a0 * r0.y, b1 * r1.x + a1 * r1.y);
}
// one pair in one word (interleaved)
__device__ __forceinline__ void turn_pair(uint32_t& w, const float2& r) {
  const float a = bf16_lo(w), b = bf16_hi(w);
  w = pack_bf16x2(a * r.x - b * r.y, b * r.x + a * r.y);
}

// freq / (2 pi) modulo 1 as a 64-bit binary fraction: the mantissa times 2^64 / (2 pi), shifted.
// (In whole numbers: fp64 arithmetic has two lanes an SM.)
__device__ __forceinline__ unsigned long long turn_fraction(double freq) {
  constexpr unsigned long long kTurn = 0x28BE60DB9391054Aull;            // 2^64 / (2 pi)
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(freq));
  const int e = static_cast<int>(bits >> 52 & 0x7ff);
  if (e == 0) return 0;                                                  // below 2^-1022
  const unsigned long long m = (bits & 0xfffffffffffffull) | 1ull << 52;
  const unsigned long long lo = m * kTurn, hi = __umul64hi(m, kTurn);    // times 2^(e - 1075)
  const int s = 1075 - e;
  unsigned long long r;
  if (s <= 0)
    r = s > -64 ? lo << -s : 0;
  else if (s < 64)
    r = lo >> s | hi << (64 - s);
  else
    r = s < 128 ? hi >> (s - 64) : 0;
  return bits >> 63 ? 0 - r : r;
}

__global__ void __launch_bounds__(kThreads, 5) rotary_kernel(const RotaryParams p) {
  extern __shared__ __align__(16) float2 s_turn[];         // [token][pair]: cos, sin, times scale
  pdl_entry();
  const int t0 = static_cast<int>(blockIdx.x) * p.block_tokens;
  const int tokens = min(p.block_tokens, p.T - t0), pairs = p.R / 2;
  const int rows = tokens * p.heads, all = rows * p.tasks;
  // piece j of a row: words first, second
  auto first_word = [&](int j) { return j < p.turned ? (p.interleaved ? 2 * j : j) : 2 * j; };
  auto second_word = [&](int j) { return j < p.turned && !p.interleaved ? j + p.turned : 2 * j + 1; };
  auto src = [&](int row) {
    const int t = row / p.heads;
    return reinterpret_cast<const uint4*>(p.x + (t0 + t) * p.x_token + (row - t * p.heads) * p.x_head);
  };
  struct Piece {
    uint4 v, w;
  };
  Piece cur[kAhead], next[kAhead];
  auto load = [&](Piece (&q)[kAhead], int i0) {
    #pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * kThreads;
      if (i < all) {
        const int row = i / p.tasks, j = i - row * p.tasks;
        const uint4* w = src(row);
        q[u].v = w[first_word(j)];
        if (second_word(j) < p.words) q[u].w = w[second_word(j)];
      }
    }
  };
  load(cur, threadIdx.x);
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs;
    const unsigned long long frac = turn_fraction(p.freq[i - t * pairs]);
    const long long position = p.positions[t0 + t];
    const unsigned long long angle = static_cast<unsigned long long>(position) * frac;
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * (1.f / 2147483648.f), &s, &c);   // (half turns)
    s_turn[i] = make_float2(c * p.scale, (p.inverse ? -s : s) * p.scale);
  }
  __syncthreads();
  auto turn = [&](Piece (&q)[kAhead], int i0) {
    #pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= all) break;
      const int row = i / p.tasks, j = i - row * p.tasks, t = row / p.heads;
      uint4 v = q[u].v, w = q[u].w;
      if (j < p.turned) {
        const float4* r = reinterpret_cast<const float4*>(s_turn + t * pairs + 8 * j);
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 z = r[e];
          const float2 r0 = make_float2(z.x, z.y), r1 = make_float2(z.z, z.w);
          if (p.interleaved) {
            // pairs 8 j + 2 e, + 1: the piece's 32-bit words 2 e, 2 e + 1
            uint32_t& lo = e == 0 ? v.x : e == 1 ? v.z : e == 2 ? w.x : w.z;
            uint32_t& hi = e == 0 ? v.y : e == 1 ? v.w : e == 2 ? w.y : w.w;
            turn_pair(lo, r0);
            turn_pair(hi, r1);
          } else {
            uint32_t& x = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
            uint32_t& y = e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w;
            turn_half(x, y, r0, r1);
          }
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(p.out + (t0 + t) * p.out_token + (row - t * p.heads) * p.out_head);
      dst[first_word(j)] = v;
      if (second_word(j) < p.words) dst[second_word(j)] = w;
    }
  };
  constexpr int kRound = kAhead * kThreads;
  for (int i0 = threadIdx.x; i0 < all; i0 += 2 * kRound) {
    load(next, i0 + kRound);
    turn(cur, i0);
    load(cur, i0 + 2 * kRound);
    turn(next, i0 + kRound);
  }
}

// Tokens of a block: as many as fill whole rounds of kAhead pieces a thread best (40 heads of 128, 8 pieces each:
// four tokens make five rounds).
int tokens_of_block(int T, int heads, int tasks) {
  constexpr long long kRound = kThreads * kAhead;
  int best = 1;
  double most = 0.0;
  for (int t = 1; t <= kTokens && t <= T; ++t) {
    const long long n = static_cast<long long>(t) * heads * tasks;
    const double used = static_cast<double>(n) / ((n + kRound - 1) / kRound * kRound);
    if (used > most * 1.01) {
      most = used;
      best = t;
    }
  }
  return best;
}

bool stride_ok(long long s) { return s > 0 && s % 8 == 0 && s < (1LL << 38); }

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::entry;

extern "C" {

moe_status moe_rotary_frequencies(int32_t R, double base, int32_t scaling, double factor, int32_t original_length,
                                  double fast, double slow, double* freq, float* scale) {
  if (R <= 0 || R > kMaxWidth || R % 16 != 0 || !(base > 1.0) || !(base < 1e300) || freq == nullptr || scale == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (scaling != MOE_ROTARY_PLAIN && scaling != MOE_ROTARY_LINEAR && scaling != MOE_ROTARY_BY_PARTS)
    return MOE_ERR_INVALID_ARG;
  if (scaling != MOE_ROTARY_PLAIN && !(factor >= 1.0 && factor < 1e300)) return MOE_ERR_INVALID_ARG;
  if (scaling == MOE_ROTARY_BY_PARTS && !(original_length > 0 && slow > 0.0 && fast >= slow && fast < 1e300))
    return MOE_ERR_INVALID_ARG;
  double lo = 0.0, hi = 0.0;
  if (scaling == MOE_ROTARY_BY_PARTS) {
    // the pair (a real number) that turns n times within the original length
    const double per = R / (2.0 * log(base)), length = original_length / 6.283185307179586476925;
    lo = floor(per * log(length / fast));
    hi = ceil(per * log(length / slow));
    if (lo < 0.0) lo = 0.0;
    if (hi > R - 1) hi = R - 1;
  }
  for (int i = 0; i < R / 2; ++i) {
    const double f = pow(base, -2.0 * i / R);
    double slowed = scaling == MOE_ROTARY_LINEAR ? 1.0 : 0.0;       // the part of it divided by the factor
    if (scaling == MOE_ROTARY_BY_PARTS) {
      // (hi <= 0: the first pair, the fastest, turns no more than `slow` times)
      slowed = hi <= 0.0 ? 1.0 : (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
      slowed = slowed < 0.0 ? 0.0 : slowed > 1.0 ? 1.0 : slowed;
    }
    freq[i] = scaling == MOE_ROTARY_PLAIN ? f : f * (1.0 - slowed) + f / factor * slowed;
  }
  *scale = scaling == MOE_ROTARY_BY_PARTS ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
  return MOE_OK;
}

moe_status moe_rotary(const moe_heads* x, const int32_t* positions, const double* freq, int32_t T, int32_t heads,
                      int32_t width, int32_t R, int32_t interleaved, float scale, int32_t inverse, const moe_heads* out,
                      void* stream) {
  if (T < 0 || T > (1 << 24) || heads <= 0 || heads > kMaxHeads || width <= 0 || width > kMaxWidth || width % 8 != 0)
    return MOE_ERR_INVALID_ARG;
  if (R <= 0 || R > width || R % 16 != 0 || x == nullptr || out == nullptr || !ptr_ok(freq)) return MOE_ERR_INVALID_ARG;
  RotaryParams p = {};
  p.x = static_cast<const __nv_bfloat16*>(x->data);
  p.out = static_cast<__nv_bfloat16*>(out->data);
  p.x_head = heads > 1 ? x->head_stride : width;
  p.x_token = T > 1 ? x->token_stride : static_cast<long long>(heads) * p.x_head;
  p.out_head = heads > 1 ? out->head_stride : width;
  p.out_token = T > 1 ? out->token_stride : static_cast<long long>(heads) * p.out_head;
  if (T > 0) {
    if (!ptr_ok(x->data) || !ptr_ok(out->data) || !ptr_ok(positions)) return MOE_ERR_INVALID_ARG;
    if (!stride_ok(p.x_token) || !stride_ok(p.x_head) || !stride_ok(p.out_token) || !stride_ok(p.out_head))
      return MOE_ERR_INVALID_ARG;
    if (!((p.out_head >= width && p.out_token >= (heads - 1) * p.out_head + width) ||
          (p.out_token >= width && p.out_head >= (T - 1) * p.out_token + width)))
      return MOE_ERR_INVALID_ARG;
    if (x->data == out->data && (p.x_token != p.out_token || p.x_head != p.out_head)) return MOE_ERR_INVALID_ARG;
  }
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  p.positions = positions;
  p.freq = freq;
  p.T = T;
  p.heads = heads;
  p.R = R;
  p.turned = R / 16;
  p.words = width / 8;
  p.tasks = x->data == out->data ? p.turned : (p.words + 1) / 2;
  p.scale = scale;
  p.interleaved = interleaved != 0;
  p.inverse = inverse != 0;
  count_launches(1);
  p.block_tokens = tokens_of_block(T, heads, p.tasks);
  return status_of(launch_k(rotary_kernel, (T + p.block_tokens - 1) / p.block_tokens, kThreads,
                            static_cast<size_t>(p.block_tokens) * (R / 2) * sizeof(float2),
                            static_cast<cudaStream_t>(stream), p));
}

}  // extern "C"
