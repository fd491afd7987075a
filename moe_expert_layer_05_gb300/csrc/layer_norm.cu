// Layer norm over the hidden dimension with the residual sum in front of it,
// and its backward pass.
//
//   s = bf16(x + r),  mu = <s>,  rstd = 1 / sqrt(<(s - mu)^2> + eps),
//   y = (s - mu) rstd w + b;
//   with xh = (s - mu) rstd and g = w dy:
//   dx = rstd (g - <g> - xh <g xh>) (+ dsum),  dw = sum_t dy xh,  db = sum_t dy.
//
// All sums and statistics are fp32; a row is kept in registers between the
// passes over it, so each input is read once and each output written once:
// the kernels are bound by HBM.  The variance is taken about the mean (a
// second pass over the registers), so it does not cancel for rows whose mean
// is large against their spread.
#include <cuda_bf16.h>

#include <cstdint>

#include "entry_checks.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// Blocks of the backward pass, each of which leaves one row of partial sums
// of dw and db: two on each of the 152 SMs.
constexpr int kBwdBlocks = 304;

struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 unpack8(const uint4& u) {
  return F8{{bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y), bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w),
             bf16_hi(u.w)}};
}
__device__ __forceinline__ uint4 pack8(const F8& f) {
  return make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]), pack_bf16x2(f.v[4], f.v[5]),
                    pack_bf16x2(f.v[6], f.v[7]));
}

// Sum of two values over the block, the same bits in every thread: warps by
// shuffles, then every thread adds the warps' sums in order.  s: 2 * WARPS
// floats; the caller alternates between two such arrays, so one barrier
// separates a write from the reads of the call before last.
template <int WARPS>
__device__ __forceinline__ void block_sum2(float& a, float& b, float* s) {
  #pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    a += __shfl_xor_sync(kFull, a, d);
    b += __shfl_xor_sync(kFull, b, d);
  }
  if constexpr (WARPS > 1) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
      s[2 * warp] = a;
      s[2 * warp + 1] = b;
    }
    __syncthreads();
    a = 0.f;
    b = 0.f;
    #pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      a += s[2 * w];
      b += s[2 * w + 1];
    }
  }
}

// One block per row; thread t holds the 8-value words t, t + THREADS, ...
template <int THREADS, int NV>
__global__ void __launch_bounds__(THREADS) layer_norm_fwd_kernel(const uint4* __restrict__ x,
                                                                 const uint4* __restrict__ residual,
                                                                 const uint4* __restrict__ weight,
                                                                 const uint4* __restrict__ bias, int H, float eps,
                                                                 uint4* __restrict__ y, uint4* __restrict__ sum_out,
                                                                 float* __restrict__ mean, float* __restrict__ rstd) {
  pdl_entry();
  constexpr int WARPS = THREADS / 32;
  __shared__ float s_a[2 * WARPS], s_b[2 * WARPS];
  const int words = H / 8;
  const long long row = static_cast<long long>(blockIdx.x) * words;
  F8 v[NV];
  float sum = 0.f, unused = 0.f;
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * THREADS;
    v[i] = F8{};
    if (c < words) {
      v[i] = unpack8(x[row + c]);
      if (residual != nullptr) {
        const F8 r = unpack8(residual[row + c]);
        #pragma unroll
        for (int j = 0; j < 8; ++j) v[i].v[j] += r.v[j];
        // the stream goes on in bf16, and the statistics are those of the
        // rounded sum, which is what the backward pass has
        const uint4 p = pack8(v[i]);
        sum_out[row + c] = p;
        v[i] = unpack8(p);
      }
      #pragma unroll
      for (int j = 0; j < 8; ++j) sum += v[i].v[j];
    }
  }
  block_sum2<WARPS>(sum, unused, s_a);
  const float mu = sum / H;
  float sq = 0.f;
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (threadIdx.x + i * THREADS < words) {
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = v[i].v[j] - mu;
        sq += d * d;
      }
    }
  }
  block_sum2<WARPS>(sq, unused, s_b);
  const float rs = 1.0f / sqrtf(sq / H + eps);
  if (threadIdx.x == 0) {
    mean[blockIdx.x] = mu;
    rstd[blockIdx.x] = rs;
  }
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * THREADS;
    if (c < words) {
      const F8 w = unpack8(weight[c]);
      F8 b{};
      if (bias != nullptr) b = unpack8(bias[c]);
      F8 o;
      #pragma unroll
      for (int j = 0; j < 8; ++j) o.v[j] = (v[i].v[j] - mu) * rs * w.v[j] + b.v[j];
      y[row + c] = pack8(o);
    }
  }
}

// Blocks walk the rows (block b takes rows b, b + gridDim.x, ...); a thread
// keeps the sums of dw and db of its columns in registers and leaves them in
// part[block][0 / 1][H] at the end.
template <int THREADS, int NV>
__global__ void __launch_bounds__(THREADS) layer_norm_bwd_kernel(const uint4* __restrict__ dy,
                                                                 const uint4* __restrict__ s,
                                                                 const uint4* __restrict__ weight,
                                                                 const float* __restrict__ mean,
                                                                 const float* __restrict__ rstd,
                                                                 const uint4* __restrict__ dsum, int T, int H,
                                                                 uint4* __restrict__ dx, float* __restrict__ part) {
  pdl_entry();
  constexpr int WARPS = THREADS / 32;
  __shared__ float s_red[2][2 * WARPS];
  const int words = H / 8;
  F8 dw[NV] = {}, db[NV] = {};
  int flip = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x, flip ^= 1) {
    const long long row = static_cast<long long>(t) * words;
    const float mu = mean[t], rs = rstd[t];
    uint4 us[NV], ud[NV];
    float m1 = 0.f, m2 = 0.f;
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * THREADS;
      us[i] = ud[i] = make_uint4(0, 0, 0, 0);
      if (c < words) {
        us[i] = s[row + c];
        ud[i] = dy[row + c];
      }
    }
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * THREADS;
      if (c < words) {
        const F8 xs = unpack8(us[i]), d = unpack8(ud[i]), w = unpack8(weight[c]);
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (xs.v[j] - mu) * rs;
          const float g = d.v[j] * w.v[j];
          dw[i].v[j] += d.v[j] * xh;
          db[i].v[j] += d.v[j];
          m1 += g;
          m2 += g * xh;
        }
      }
    }
    block_sum2<WARPS>(m1, m2, s_red[flip]);
    m1 /= H;
    m2 /= H;
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * THREADS;
      if (c < words) {
        const F8 xs = unpack8(us[i]), d = unpack8(ud[i]), w = unpack8(weight[c]);
        F8 o;
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (xs.v[j] - mu) * rs;
          o.v[j] = (d.v[j] * w.v[j] - m1 - xh * m2) * rs;
        }
        if (dsum != nullptr) {
          const F8 e = unpack8(dsum[row + c]);
          #pragma unroll
          for (int j = 0; j < 8; ++j) o.v[j] += e.v[j];
        }
        dx[row + c] = pack8(o);
      }
    }
  }
  float4* out = reinterpret_cast<float4*>(part + static_cast<long long>(blockIdx.x) * 2 * H);
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * THREADS;
    if (c < words) {
      out[2 * c] = make_float4(dw[i].v[0], dw[i].v[1], dw[i].v[2], dw[i].v[3]);
      out[2 * c + 1] = make_float4(dw[i].v[4], dw[i].v[5], dw[i].v[6], dw[i].v[7]);
      out[H / 4 + 2 * c] = make_float4(db[i].v[0], db[i].v[1], db[i].v[2], db[i].v[3]);
      out[H / 4 + 2 * c + 1] = make_float4(db[i].v[4], db[i].v[5], db[i].v[6], db[i].v[7]);
    }
  }
}

// dw and db from the blocks' partial sums, added in block order in eight
// strands (strand s: blocks s, s + 8, ...) and the strands in order.
constexpr int kJoinCols = 32, kJoinStrands = 8;
__global__ void __launch_bounds__(kJoinCols * kJoinStrands) layer_norm_join_kernel(const float* __restrict__ part,
                                                                                  int blocks, int H,
                                                                                  float* __restrict__ dweight,
                                                                                  float* __restrict__ dbias) {
  pdl_entry();
  __shared__ float s_sum[kJoinStrands][kJoinCols];
  const int lane = threadIdx.x % kJoinCols, strand = threadIdx.x / kJoinCols;
  const int col = blockIdx.x * kJoinCols + lane;      // over [dw | db], 2 H columns
  float a = 0.f;
  if (col < 2 * H) {
    #pragma unroll 4
    for (int b = strand; b < blocks; b += kJoinStrands) a += part[static_cast<long long>(b) * 2 * H + col];
  }
  s_sum[strand][lane] = a;
  __syncthreads();
  if (strand == 0 && col < 2 * H) {
    float r = 0.f;
    #pragma unroll
    for (int i = 0; i < kJoinStrands; ++i) r += s_sum[i][lane];
    if (col < H)
      dweight[col] = r;
    else if (dbias != nullptr)
      dbias[col - H] = r;
  }
}

template <int THREADS, int NV>
cudaError_t fwd(const void* x, const void* residual, const void* weight, const void* bias, int T, int H, float eps,
                void* y, void* sum_out, float* mean, float* rstd, cudaStream_t st) {
  count_launches(1);
  return launch_k(layer_norm_fwd_kernel<THREADS, NV>, T, THREADS, 0, st, static_cast<const uint4*>(x),
                  static_cast<const uint4*>(residual), static_cast<const uint4*>(weight),
                  static_cast<const uint4*>(bias), H, eps, static_cast<uint4*>(y), static_cast<uint4*>(sum_out), mean,
                  rstd);
}

template <int THREADS, int NV>
cudaError_t bwd(int grid, const void* dy, const void* s, const void* weight, const float* mean, const float* rstd,
                const void* dsum, int T, int H, void* dx, float* part, cudaStream_t st) {
  count_launches(1);
  return launch_k(layer_norm_bwd_kernel<THREADS, NV>, grid, THREADS, 0, st, static_cast<const uint4*>(dy),
                  static_cast<const uint4*>(s), static_cast<const uint4*>(weight), mean, rstd,
                  static_cast<const uint4*>(dsum), T, H, static_cast<uint4*>(dx), part);
}

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::entry;

extern "C" {

size_t moe_layer_norm_workspace_bytes(int32_t T, int32_t H) {
  if (T < 0 || !hidden_ok(H)) return 0;
  const size_t blocks = T < kBwdBlocks ? T : kBwdBlocks;
  return kStatusBytes + align_up(blocks * 2 * H * sizeof(float));
}

moe_status moe_layer_norm_forward(const void* x, const void* residual, const void* weight, const void* bias, int32_t T,
                                  int32_t H, float eps, void* y, void* sum_out, float* mean, float* rstd,
                                  void* stream) {
  if (T < 0 || !hidden_ok(H) || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (!ptr_ok(weight) || !opt_ok(bias)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ptr_ok(x) || !opt_ok(residual) || !ptr_ok(y) || !ptr_ok(mean) || !ptr_ok(rstd)))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && residual != nullptr && !ptr_ok(sum_out)) return MOE_ERR_INVALID_ARG;
  if (residual == nullptr && sum_out != nullptr) return MOE_ERR_INVALID_ARG;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // four 8-value words per thread at most: the smallest block that holds a row
  cudaError_t e;
  if (H <= 1024)
    e = fwd<32, 4>(x, residual, weight, bias, T, H, eps, y, sum_out, mean, rstd, st);
  else if (H <= 4096)
    e = fwd<128, 4>(x, residual, weight, bias, T, H, eps, y, sum_out, mean, rstd, st);
  else if (H <= 8192)
    e = fwd<256, 4>(x, residual, weight, bias, T, H, eps, y, sum_out, mean, rstd, st);
  else
    e = fwd<512, 4>(x, residual, weight, bias, T, H, eps, y, sum_out, mean, rstd, st);
  return status_of(e);
}

moe_status moe_layer_norm_backward(const void* dy, const void* s, const void* weight, const float* mean,
                                   const float* rstd, const void* dsum, int32_t T, int32_t H, void* dx, float* dweight,
                                   float* dbias, void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || !hidden_ok(H)) return MOE_ERR_INVALID_ARG;
  if (!ptr_ok(weight) || !ptr_ok(dweight) || !opt_ok(dbias) || !ptr_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ptr_ok(dy) || !ptr_ok(s) || !ptr_ok(mean) || !ptr_ok(rstd) || !opt_ok(dsum) || !ptr_ok(dx)))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_layer_norm_workspace_bytes(T, H)) return MOE_ERR_WORKSPACE;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = T < kBwdBlocks ? T : kBwdBlocks;
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + kStatusBytes);
  cudaError_t e = cudaSuccess;
  if (T > 0) {
    if (H <= 512)
      e = bwd<32, 2>(grid, dy, s, weight, mean, rstd, dsum, T, H, dx, part, st);
    else if (H <= 2048)
      e = bwd<128, 2>(grid, dy, s, weight, mean, rstd, dsum, T, H, dx, part, st);
    else if (H <= 8192)
      e = bwd<512, 2>(grid, dy, s, weight, mean, rstd, dsum, T, H, dx, part, st);
    else
      e = bwd<1024, 2>(grid, dy, s, weight, mean, rstd, dsum, T, H, dx, part, st);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  count_launches(1);
  return status_of(launch_k(layer_norm_join_kernel, (2 * H + kJoinCols - 1) / kJoinCols, kJoinCols * kJoinStrands, 0,
                            st, part, grid, H, dweight, dbias));
}

}  // extern "C"
