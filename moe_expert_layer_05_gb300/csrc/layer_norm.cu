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
//
// Measured on one GB300, 16384 rows of 7168 (940 MB either way; a plain copy
// reaches 6.68 TB/s): forward with the residual 135 us (6.96 TB/s), backward
// with dsum 144 us (6.52 TB/s).
#include <cuda_bf16.h>

#include <atomic>
#include <cstdint>

#include "entry_checks.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// Blocks of the backward pass, each of which leaves one row of partial sums
// of dw and db: one on each of the 152 SMs.
constexpr int kBwdBlocks = 152;
constexpr int kBwdWarps = 16;

struct F8 {
  float v[8];
};
// The same eight values as four pairs.
struct P8 {
  F32x2 p[4];
};
__device__ __forceinline__ P8 pairs8(const uint4& u) {
  return P8{{bf16x2_f32x2(u.x), bf16x2_f32x2(u.y), bf16x2_f32x2(u.z), bf16x2_f32x2(u.w)}};
}
__device__ __forceinline__ F8 unpack8(const uint4& u) {
  return F8{{bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y), bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w),
             bf16_hi(u.w)}};
}
__device__ __forceinline__ uint4 pack8(const F8& f) {
  return make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]), pack_bf16x2(f.v[4], f.v[5]),
                    pack_bf16x2(f.v[6], f.v[7]));
}

// ---------------------------------------------------------------- forward
// A row is held by as many warps as it needs at 4 eight-value words per thread
// and no more: a block of its own, or (ONE_WARP) one warp of a block of
// kFwdRows rows.
constexpr int kNV = 4;
constexpr int kFwdRows = 4;

// Sum over the threads that hold a row, the same bits in every thread:
// shuffles, then every thread adds the warps' sums in order.
template <bool ONE_WARP>
__device__ __forceinline__ float row_sum(float a, float* red, int warps) {
  #pragma unroll
  for (int d = 16; d > 0; d >>= 1) a += __shfl_xor_sync(kFull, a, d);
  if constexpr (!ONE_WARP) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0.f;
    for (int w = 0; w < warps; ++w) a += red[w];
  }
  return a;
}

template <bool ONE_WARP>
__global__ void __launch_bounds__(512) layer_norm_fwd_kernel(const uint4* __restrict__ x,
                                                             const uint4* __restrict__ residual,
                                                             const uint4* __restrict__ weight,
                                                             const uint4* __restrict__ bias, int T, int H, int warps,
                                                             float eps, uint4* __restrict__ y,
                                                             uint4* __restrict__ sum_out, float* __restrict__ mean,
                                                             float* __restrict__ rstd) {
  pdl_entry();
  __shared__ float s_a[16], s_b[16];
  const int words = H / 8;
  const int gtid = ONE_WARP ? threadIdx.x & 31 : threadIdx.x, gthreads = ONE_WARP ? 32 : blockDim.x;
  const int t = ONE_WARP ? blockIdx.x * kFwdRows + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= T) return;
  const long long row = static_cast<long long>(t) * words;
  // every load of the row in flight before the first is used
  uint4 ux[kNV], ur[kNV];
  #pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = gtid + i * gthreads;
    ux[i] = ur[i] = make_uint4(0, 0, 0, 0);
    if (c < words) {
      ux[i] = x[row + c];
      if (residual != nullptr) ur[i] = residual[row + c];
    }
  }
  F8 v[kNV];
  float sum = 0.f;
  #pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = gtid + i * gthreads;
    v[i] = unpack8(ux[i]);
    if (residual != nullptr) {
      const F8 r = unpack8(ur[i]);
      #pragma unroll
      for (int j = 0; j < 8; ++j) v[i].v[j] += r.v[j];
      // the stream goes on in bf16, and the statistics are those of the
      // rounded sum, which is what the backward pass has
      const uint4 p = pack8(v[i]);
      if (c < words) sum_out[row + c] = p;
      v[i] = unpack8(p);
    }
    #pragma unroll
    for (int j = 0; j < 8; ++j) sum += v[i].v[j];
  }
  const float mu = row_sum<ONE_WARP>(sum, s_a, warps) / H;
  float sq = 0.f;
  #pragma unroll
  for (int i = 0; i < kNV; ++i) {
    if (gtid + i * gthreads < words) {
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = v[i].v[j] - mu;
        sq += d * d;
      }
    }
  }
  const float rs = 1.0f / sqrtf(row_sum<ONE_WARP>(sq, s_b, warps) / H + eps);
  if (gtid == 0) {
    mean[t] = mu;
    rstd[t] = rs;
  }
  #pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = gtid + i * gthreads;
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

// ---------------------------------------------------------------- backward
// A row is worked on by a group of `warps` warps, NV eight-value words per
// thread; a block, one per SM, has up to 16 warps, as many groups as the rows
// can use, and the groups of the whole grid take the rows in turn.  Each group
// streams its rows (s, dy and dsum: contiguous in memory) through a ring of row
// buffers in shared memory with bulk copies.  A thread takes its words of a
// row into registers at once, so the barrier of the row's sums also frees the
// buffer: the copy of a later row starts there while this one is finished, and
// all buffers but one are always in flight (4 x 43 KB at H = 7168).  The sums
// of dw and db of a thread's columns stay in registers; the groups of a block
// are added pairwise at the end and the block leaves one row
// part[block][0 / 1][H].
constexpr int kMaxStages = 4;
constexpr size_t kRingBytes = 200 * 1024;

// Barrier over the warps of one group of a block.
__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

__device__ __forceinline__ uint4 word_of(const uint4* __restrict__ row, int c, int words) {
  return c < words ? row[c] : make_uint4(0, 0, 0, 0);
}

struct BwdShape {
  int nv, warps, groups, threads, blocks, stages;
  size_t smem;
};
BwdShape bwd_shape(int T, int H, bool dsum) {
  BwdShape b;
  b.nv = H <= 8192 ? 2 : 4;          // (16 warps hold a row)
  b.warps = (H / 8 + 32 * b.nv - 1) / (32 * b.nv);
  const int most = kBwdWarps / b.warps, wanted = (T + kBwdBlocks - 1) / kBwdBlocks;
  b.groups = wanted < most ? (wanted > 0 ? wanted : 1) : most;
  b.threads = 32 * b.warps * b.groups;
  b.blocks = (T + b.groups - 1) / b.groups;
  if (b.blocks > kBwdBlocks) b.blocks = kBwdBlocks;
  const size_t rows = static_cast<size_t>(H) * 2 * (dsum ? 3 : 2) * b.groups;
  b.stages = static_cast<int>(kRingBytes / rows);
  if (b.stages > kMaxStages) b.stages = kMaxStages;
  b.smem = rows * b.stages;          // (holds the sums of half the groups, 8 H bytes each, at the end)
  return b;
}

template <int NV, bool DSUM>
__global__ void __launch_bounds__(512, 1) layer_norm_bwd_kernel(const uint4* __restrict__ dy, const uint4* __restrict__ s,
                                                                const uint4* __restrict__ weight,
                                                                const float* __restrict__ mean,
                                                                const float* __restrict__ rstd,
                                                                const uint4* __restrict__ dsum, int T, int H, int warps,
                                                                int stages, uint4* __restrict__ dx,
                                                                float* __restrict__ part, int* status,
                                                                unsigned long long wait_ns) {
  pdl_entry();
  extern __shared__ __align__(128) uint4 ring[];
  __shared__ uint64_t s_full[kBwdWarps][kMaxStages];
  __shared__ float2 s_red[2][kBwdWarps];
  __shared__ int s_abort;
  __shared__ int s_stop[kBwdWarps];      // a group's first row that started no later row's copy
  constexpr int ROWS = DSUM ? 3 : 2;
  const int words = H / 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / warps, gwarp = warp % warps, gtid = gwarp * 32 + lane, gthreads = warps * 32;
  const int groups = blockDim.x / gthreads;
  uint4* buf = ring + static_cast<size_t>(group) * stages * ROWS * words;
  const int t0 = blockIdx.x * groups + group, step = gridDim.x * groups;
  if (threadIdx.x == 0) {
    for (int g = 0; g < groups; ++g) {
      for (int i = 0; i < stages; ++i) mbar_init(&s_full[g][i], 1);
      s_stop[g] = T;
    }
    s_abort = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  const uint32_t bytes = static_cast<uint32_t>(H) * 2;
  auto load = [&](long long t, int stage) {      // one thread of the group
    if (t >= T) return;
    uint64_t* bar = &s_full[group][stage];
    uint4* to = buf + static_cast<size_t>(stage) * ROWS * words;
    const long long row = t * words;
    mbar_arrive_expect_tx(bar, ROWS * bytes);
    bulk_load(to, s + row, bytes, bar);
    bulk_load(to + words, dy + row, bytes, bar);
    if constexpr (DSUM) bulk_load(to + 2 * words, dsum + row, bytes, bar);
  };
  if (gtid == 0) {
    for (int i = 0; i < stages; ++i) load(t0 + static_cast<long long>(i) * step, i);
  }
  // (KEEP: weight, xh and g in registers; wider rows leave those to the sums
  // and take the row a second time from shared memory)
  constexpr bool KEEP = NV == 2;
  P8 w[KEEP ? NV : 1];
  if constexpr (KEEP) {
    #pragma unroll
    for (int i = 0; i < NV; ++i) w[i] = pairs8(word_of(weight, gtid + i * gthreads, words));
  }
  P8 dw[NV] = {}, db[NV] = {};
  const float inv_h = 1.0f / H;
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  float mu_next = t0 < T ? mean[t0] : 0.f, rs_next = t0 < T ? rstd[t0] : 0.f;
  for (long long t = t0; t < T; t += step) {
    const float mu = mu_next, rs = rs_next;
    if (t + step < T) {
      mu_next = mean[t + step];
      rs_next = rstd[t + step];
    }
    // (a wait that gave up raises s_abort; the group goes on to the end
    // together, on whatever the buffer holds, and starts no more copies)
    mbar_wait(&s_full[group][stage], phase, &s_abort, wait_ns);
    const uint4* row_s = buf + static_cast<size_t>(stage) * ROWS * words;
    // xh and g stay in registers for the second half of the row's work:
    // taking bf16 pairs apart is what the kernel's arithmetic mostly costs
    const F32x2 neg_mu = make_f32x2(-mu, -mu), rs2 = make_f32x2(rs, rs);
    F32x2 s1 = make_f32x2(0.f, 0.f), s2 = make_f32x2(0.f, 0.f);
    P8 norm[KEEP ? NV : 1], g[KEEP ? NV : 1];
    uint4 ue[KEEP ? NV : 1];
    #pragma unroll
    for (int i = 0; i < NV; ++i) {               // (words past the row: dy = 0 adds nothing)
      const int c = gtid + i * gthreads;
      const P8 xs = pairs8(word_of(row_s, c, words)), d = pairs8(word_of(row_s + words, c, words));
      if constexpr (DSUM && KEEP) ue[i] = word_of(row_s + 2 * words, c, words);
      const P8 wv = KEEP ? w[KEEP ? i : 0] : pairs8(word_of(weight, c, words));
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F32x2 xh = mul2(add2(xs.p[j], neg_mu), rs2), gj = mul2(d.p[j], wv.p[j]);
        dw[i].p[j] = fma2(d.p[j], xh, dw[i].p[j]);
        db[i].p[j] = add2(db[i].p[j], d.p[j]);
        s1 = add2(s1, gj);
        s2 = fma2(gj, xh, s2);
        if constexpr (KEEP) {
          norm[i].p[j] = xh;
          g[i].p[j] = gj;
        }
      }
    }
    const float2 f1 = split_f32x2(s1), f2 = split_f32x2(s2);
    float m1 = f1.x + f1.y, m2 = f2.x + f2.y;
    #pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
      m1 += __shfl_xor_sync(kFull, m1, k);
      m2 += __shfl_xor_sync(kFull, m2, k);
    }
    if (warps > 1) {                        // the group's warps, added in order
      float2* red = &s_red[flip][group * warps];
      if (lane == 0) red[gwarp] = make_float2(m1, m2);
      group_sync(group, gthreads);
      const float2 v = lane < warps ? red[lane] : make_float2(0.f, 0.f);
      m1 = v.x;
      m2 = v.y;
      #pragma unroll
      for (int k = 16; k > 0; k >>= 1) {
        m1 += __shfl_xor_sync(kFull, m1, k);
        m2 += __shfl_xor_sync(kFull, m2, k);
      }
      flip ^= 1;
    } else {
      __syncwarp();
    }
    auto refill = [&] {                    // every thread of the group has read the buffer
      if (gtid != 0) return;
      if (!*static_cast<volatile int*>(&s_abort))
        load(t + static_cast<long long>(stages) * step, stage);
      else
        s_stop[group] = min(s_stop[group], static_cast<int>(t));
    };
    if constexpr (KEEP) refill();
    // dx = rs g - rs <g> - xh rs <g xh>  (rs^2 would leave fp32 where rs does not)
    m1 *= -inv_h * rs;
    m2 *= -inv_h * rs;
    const F32x2 k1 = make_f32x2(m1, m1), k2 = make_f32x2(m2, m2);
    const long long row = t * words;
    #pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = gtid + i * gthreads;
      P8 o;
      if constexpr (KEEP) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) o.p[j] = fma2(norm[i].p[j], k2, fma2(g[i].p[j], rs2, k1));
      } else {
        const P8 xs = pairs8(word_of(row_s, c, words)), d = pairs8(word_of(row_s + words, c, words));
        const P8 wv = pairs8(word_of(weight, c, words));
        #pragma unroll
        for (int j = 0; j < 4; ++j)
          o.p[j] = fma2(mul2(add2(xs.p[j], neg_mu), rs2), k2, fma2(mul2(d.p[j], wv.p[j]), rs2, k1));
      }
      if constexpr (DSUM) {
        const P8 e = pairs8(KEEP ? ue[KEEP ? i : 0] : word_of(row_s + 2 * words, c, words));
        #pragma unroll
        for (int j = 0; j < 4; ++j) o.p[j] = add2(o.p[j], e.p[j]);
      }
      if (c < words)
        dx[row + c] = make_uint4(pack_bf16x2(o.p[0]), pack_bf16x2(o.p[1]), pack_bf16x2(o.p[2]), pack_bf16x2(o.p[3]));
    }
    if constexpr (!KEEP) {
      if (warps > 1) group_sync(group, gthreads);
      else __syncwarp();
      refill();
    }
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  __syncthreads();
  if (s_abort) {
    if (threadIdx.x == 0) set_status(status, kErrTimeout);
    if (gtid == 0 && t0 < T) {
      // copies still on their way, of the last `stages` rows that were started:
      // each is waited for, half a second at most
      const int rows = (T - t0 + step - 1) / step, stop = (s_stop[group] - t0 + step - 1) / step;
      const int started = min(rows, stop + stages);
      for (int k = max(started - stages, 0); k < started; ++k) {
        const unsigned long long since = global_timer_ns();
        while (!mbar_try_wait(&s_full[group][k % stages], k / stages & 1) &&
               global_timer_ns() - since < kWaitLimitNs / 4) {
        }
      }
    }
    __syncthreads();
    return;
  }
  // the groups' sums, added pairwise through shared memory
  P8* sums = reinterpret_cast<P8*>(ring);
  for (int n = groups; n > 1;) {
    const int half = (n + 1) / 2;
    if (group >= half && group < n) {
      P8* to = sums + static_cast<size_t>(group - half) * 2 * words;
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = gtid + i * gthreads;
        if (c < words) {
          to[c] = dw[i];
          to[words + c] = db[i];
        }
      }
    }
    __syncthreads();
    if (group < n - half) {
      const P8* from = sums + static_cast<size_t>(group) * 2 * words;
      #pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = gtid + i * gthreads;
        if (c < words) {
          const P8 a = from[c], b = from[words + c];
          #pragma unroll
          for (int j = 0; j < 4; ++j) {
            dw[i].p[j] = add2(dw[i].p[j], a.p[j]);
            db[i].p[j] = add2(db[i].p[j], b.p[j]);
          }
        }
      }
    }
    __syncthreads();
    n = half;
  }
  if (group != 0) return;
  P8* out = reinterpret_cast<P8*>(part + static_cast<long long>(blockIdx.x) * 2 * H);
  #pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = gtid + i * gthreads;
    if (c < words) {
      out[c] = dw[i];
      out[words + c] = db[i];
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

template <int NV, bool DSUM>
cudaError_t bwd(const BwdShape& b, const void* dy, const void* s, const void* weight, const float* mean,
                const float* rstd, const void* dsum, int T, int H, void* dx, float* part, int* status, cudaStream_t st) {
  auto kern = layer_norm_bwd_kernel<NV, DSUM>;
  static std::atomic<bool> attr_set[64];    // (per device)
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  const unsigned long long wait = gemm_wait_limit_ns();
  count_launches(1);
  return launch_k(kern, b.blocks, b.threads, b.smem, st, static_cast<const uint4*>(dy), static_cast<const uint4*>(s),
                  static_cast<const uint4*>(weight), mean, rstd, static_cast<const uint4*>(dsum), T, H, b.warps,
                  b.stages, static_cast<uint4*>(dx), part, status, wait != 0 ? wait : kWaitLimitNs);
}

bool rows_ok(int32_t T) { return T >= 0 && T <= (1 << 30); }

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::entry;

extern "C" {

size_t moe_layer_norm_workspace_bytes(int32_t T, int32_t H) {
  if (!rows_ok(T) || !hidden_ok(H)) return 0;
  const size_t blocks = T < kBwdBlocks ? T : kBwdBlocks;
  return kStatusBytes + align_up(blocks * 2 * H * sizeof(float));
}

moe_status moe_layer_norm_forward(const void* x, const void* residual, const void* weight, const void* bias, int32_t T,
                                  int32_t H, float eps, void* y, void* sum_out, float* mean, float* rstd,
                                  void* stream) {
  if (!rows_ok(T) || !hidden_ok(H) || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (!ptr_ok(weight) || !opt_ok(bias)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ptr_ok(x) || !opt_ok(residual) || !ptr_ok(y) || !ptr_ok(mean) || !ptr_ok(rstd)))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && residual != nullptr && !ptr_ok(sum_out)) return MOE_ERR_INVALID_ARG;
  if (residual == nullptr && sum_out != nullptr) return MOE_ERR_INVALID_ARG;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int warps = (H / 8 + 32 * kNV - 1) / (32 * kNV);
  auto kern = warps == 1 ? layer_norm_fwd_kernel<true> : layer_norm_fwd_kernel<false>;
  const int blocks = warps == 1 ? (T + kFwdRows - 1) / kFwdRows : T;
  count_launches(1);
  return status_of(launch_k(kern, blocks, 32 * (warps == 1 ? kFwdRows : warps), 0, st, static_cast<const uint4*>(x),
                            static_cast<const uint4*>(residual), static_cast<const uint4*>(weight),
                            static_cast<const uint4*>(bias), T, H, warps, eps, static_cast<uint4*>(y),
                            static_cast<uint4*>(sum_out), mean, rstd));
}

moe_status moe_layer_norm_backward(const void* dy, const void* s, const void* weight, const float* mean,
                                   const float* rstd, const void* dsum, int32_t T, int32_t H, void* dx, float* dweight,
                                   float* dbias, void* ws, size_t ws_bytes, void* stream) {
  if (!rows_ok(T) || !hidden_ok(H)) return MOE_ERR_INVALID_ARG;
  if (!ptr_ok(weight) || !ptr_ok(dweight) || !opt_ok(dbias) || !ptr_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ptr_ok(dy) || !ptr_ok(s) || !ptr_ok(mean) || !ptr_ok(rstd) || !opt_ok(dsum) || !ptr_ok(dx)))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_layer_norm_workspace_bytes(T, H)) return MOE_ERR_WORKSPACE;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const BwdShape b = bwd_shape(T, H, dsum != nullptr);
  int* status = static_cast<int*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + kStatusBytes);
  if (T > 0) {
    cudaError_t e;
    if (b.nv == 2)
      e = dsum != nullptr ? bwd<2, true>(b, dy, s, weight, mean, rstd, dsum, T, H, dx, part, status, st)
                          : bwd<2, false>(b, dy, s, weight, mean, rstd, dsum, T, H, dx, part, status, st);
    else
      e = dsum != nullptr ? bwd<4, true>(b, dy, s, weight, mean, rstd, dsum, T, H, dx, part, status, st)
                          : bwd<4, false>(b, dy, s, weight, mean, rstd, dsum, T, H, dx, part, status, st);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  count_launches(1);
  return status_of(launch_k(layer_norm_join_kernel, (2 * H + kJoinCols - 1) / kJoinCols, kJoinCols * kJoinStrands, 0,
                            st, part, b.blocks, H, dweight, dbias));
}

}  // extern "C"
