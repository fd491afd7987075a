// The 2-norm of all gradients of a model together, and their scaling to a limit.
//
//   norm = sqrt(sum over all tensors of the sum of squares),
//   out = g * min(1, limit / (norm + 1e-6)).
//
// The tensors' addresses and sizes travel with the launch (kList or kLongList of them; further
// ones in further launches), so nothing is copied to the device.  All tensors together are one
// list of chunks of 32 KB; blocks of fixed number take them in turn, so each partial sum is over
// the same chunks on every run, and the last block to finish adds the partial sums in order.
//
// A thread's 128 bytes of a chunk are squared and added up in fp32 and joined in fp64.  Squares leave
// fp32's range long before their root does: where such a sum is not in the middle of the
// range, the same values are squared in fp64.
//
// Bound by HBM: the norm reads everything once, the scaling reads and writes it once.  The
// scaling walks the chunks from the last to the first, of which the norm has left the last ones
// in L2.  2.3 GB: 336 us for the norm (6.8 TB/s) and 700 for the scaling (6.6); 15 tensors of
// 4.8 MB together: 5.6 and 4.2 us, the norm's mostly the join of its blocks.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "entry_checks.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWords = 8;                              // 16-byte words of a thread and chunk
constexpr int kChunkWords = kThreads * kWords;         // 32 KB
constexpr int kBlocks = 152 * 6;                       // of the norm, each its share of the chunks
constexpr long long kMaxClipBlocks = 1LL << 30;
constexpr int kList = 64, kLongList = 512;             // tensors of one launch
constexpr int kMaxTensors = 1 << 20;

template <int N>
struct TensorList {
  const uint4* src[N];
  uint4* dst[N];
  long long n[N];              // elements
  long long end[N];            // chunks up to and including this tensor's
  unsigned char fp32[N];
  int count;
};

// The tensor a chunk belongs to.
template <int N>
__device__ __forceinline__ int tensor_of(const TensorList<N>& list, long long chunk) {
  int lo = 0, hi = list.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (chunk < list.end[mid])
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ float squares(const uint4& v, bool fp32) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  float s = 0.f;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (fp32) {
      const float f = __uint_as_float(u[i]);
      s = fmaf(f, f, s);
    } else {
      const float a = bf16_lo(u[i]), b = bf16_hi(u[i]);
      s = fmaf(a, a, s);
      s = fmaf(b, b, s);
    }
  }
  return s;
}
__device__ __forceinline__ double squares64(const uint4& v, bool fp32) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  double s = 0.0;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double a = fp32 ? __uint_as_float(u[i]) : bf16_lo(u[i]), b = fp32 ? 0.f : bf16_hi(u[i]);
    s += a * a + b * b;
  }
  return s;
}

// Word w of a tensor of n elements: whole, or (the last one) what there is of it, then zeros.
__device__ __forceinline__ uint4 word_at(const uint4* src, long long w, long long n, bool fp32) {
  const int per = fp32 ? 4 : 8;
  const long long left = n - w * per;
  if (left >= per) return src[w];
  uint4 v = make_uint4(0, 0, 0, 0);
  if (left <= 0) return v;
  uint32_t u[4] = {0, 0, 0, 0};
  for (int i = 0; i < left; ++i) {
    if (fp32)
      u[i] = reinterpret_cast<const uint32_t*>(src + w)[i];
    else
      u[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(src + w)[i]) << (16 * (i & 1));
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// A thread's words of a chunk.  A whole chunk's loads stand side by side, without a branch between them.
__device__ __forceinline__ void load_chunk(const uint4* src, long long w0, long long n, bool fp32, uint4 (&v)[kWords]) {
  if ((w0 - threadIdx.x + kChunkWords) * (fp32 ? 4 : 8) <= n) {
    #pragma unroll
    for (int j = 0; j < kWords; ++j) v[j] = src[w0 + j * kThreads];
  } else {
    #pragma unroll
    for (int j = 0; j < kWords; ++j) v[j] = word_at(src, w0 + j * kThreads, n, fp32);
  }
}

__device__ __forceinline__ double block_sum(double v, double* s) {
  s[threadIdx.x] = v;
  __syncthreads();
  #pragma unroll
  for (int h = kThreads / 2; h > 0; h >>= 1) {
    if (static_cast<int>(threadIdx.x) < h) s[threadIdx.x] += s[threadIdx.x + h];
    __syncthreads();
  }
  const double r = s[0];
  __syncthreads();
  return r;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ TensorList<N> list,
                                                             double* __restrict__ part, int part0, int total,
                                                             float* __restrict__ norm, int* status) {
  pdl_entry();
  __shared__ double s_sum[kThreads];
  __shared__ int s_last;
  double sum = 0.0;
  const long long chunks = list.count > 0 ? list.end[list.count - 1] : 0;
  for (long long c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(list, c);
    const bool fp32 = list.fp32[i] != 0;
    const long long w0 = (c - (i > 0 ? list.end[i - 1] : 0)) * kChunkWords + threadIdx.x;
    uint4 v[kWords];
    load_chunk(list.src[i], w0, list.n[i], fp32, v);
    float s[2] = {0.f, 0.f};
    #pragma unroll
    for (int j = 0; j < kWords; ++j) s[j & 1] += squares(v[j], fp32);
    const float t = s[0] + s[1];
    if (t >= 0x1p-70f && t < 0x1p120f) {
      sum += t;
    } else {
      #pragma unroll
      for (int j = 0; j < kWords; ++j)
        if ((v[j].x | v[j].y | v[j].z | v[j].w) != 0u) sum += squares64(v[j], fp32);
    }
  }
  sum = block_sum(sum, s_sum);
  if (threadIdx.x == 0) {
    part[part0 + blockIdx.x] = sum;
    __threadfence();
    s_last = atomicAdd(status + kNormDoneWord, 1) == total - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double all = 0.0;
  for (int b = threadIdx.x; b < total; b += kThreads) all += __ldcg(part + b);
  all = block_sum(all, s_sum);
  if (threadIdx.x == 0) {
    norm[0] = static_cast<float>(sqrt(all));
    atomicExch(status + kNormDoneWord, 0);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    grad_clip_kernel(const __grid_constant__ TensorList<N> list, const float* __restrict__ norm, float limit,
                     int in_place) {
  pdl_entry();
  float c = limit / (norm[0] + 1e-6f);
  if (c >= 1.f || (limit == INFINITY && norm[0] == INFINITY)) {      // (infinity / infinity: no limit is none)
    if (in_place) return;
    c = 1.f;
  }
  const long long chunks = list.end[list.count - 1];
  for (long long c0 = blockIdx.x; c0 < chunks; c0 += gridDim.x) {
    const long long chunk = chunks - 1 - c0;
    const int i = tensor_of(list, chunk);
    const bool fp32 = list.fp32[i] != 0;
    const int per = fp32 ? 4 : 8;
    const long long w0 = (chunk - (i > 0 ? list.end[i - 1] : 0)) * kChunkWords + threadIdx.x, n = list.n[i];
    const bool whole = (w0 - threadIdx.x + kChunkWords) * per <= n;
    uint4 v[kWords];
    load_chunk(list.src[i], w0, n, fp32, v);
    #pragma unroll
    for (int j = 0; j < kWords; ++j) {
      uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      #pragma unroll
      for (int e = 0; e < 4; ++e)
        u[e] = fp32 ? __float_as_uint(__uint_as_float(u[e]) * c) : pack_bf16x2(bf16_lo(u[e]) * c, bf16_hi(u[e]) * c);
      const long long w = w0 + j * kThreads, left = n - w * per;
      if (whole || left >= per) {
        __stcs(list.dst[i] + w, make_uint4(u[0], u[1], u[2], u[3]));
      } else {
        for (int e = 0; e < left; ++e) {
          if (fp32)
            reinterpret_cast<uint32_t*>(list.dst[i] + w)[e] = u[e];
          else
            reinterpret_cast<uint16_t*>(list.dst[i] + w)[e] = static_cast<uint16_t>(u[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
}

bool list_ok(const moe_tensor* t, int32_t n) {
  if (n < 0 || n > kMaxTensors || (n > 0 && t == nullptr)) return false;
  for (int32_t i = 0; i < n; ++i) {
    if (t[i].n < 0 || t[i].n > (1LL << 40) || (t[i].type != MOE_TYPE_BF16 && t[i].type != MOE_TYPE_FP32)) return false;
    if (t[i].n > 0 && !entry::ptr_ok(t[i].data)) return false;
  }
  return true;
}
long long chunks_of(const moe_tensor& t) {
  const long long per = t.type == MOE_TYPE_FP32 ? 4 : 8;
  return ((t.n + per - 1) / per + kChunkWords - 1) / kChunkWords;
}

// Whether what a scaling writes overlaps nothing else of it: two threads would scale the same value.
struct Span {
  uintptr_t begin, end;
  bool written;
};
void add_spans(Span* s, size_t& count, const moe_tensor* t, int32_t n, bool written) {
  for (int32_t i = 0; i < n; ++i) {
    if (t[i].n == 0) continue;
    const uintptr_t at = reinterpret_cast<uintptr_t>(t[i].data);
    s[count++] = {at, at + static_cast<uintptr_t>(t[i].n) * (t[i].type == MOE_TYPE_FP32 ? 4 : 2), written};
  }
}
bool apart(Span* s, size_t count) {
  std::sort(s, s + count, [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any = 0, written = 0;          // where what came before ends
  for (size_t i = 0; i < count; ++i) {
    if (s[i].begin < (s[i].written ? any : written)) return false;
    any = std::max(any, s[i].end);
    if (s[i].written) written = std::max(written, s[i].end);
  }
  return true;
}
moe_status writes_apart(const moe_tensor* t, const moe_tensor* outs, int32_t n) {
  Span few[2 * kList], *s = few;
  if (n > kList) s = new (std::nothrow) Span[2 * static_cast<size_t>(n)];
  if (s == nullptr) return MOE_ERR_WORKSPACE;
  size_t count = 0;
  add_spans(s, count, t, n, outs == nullptr);
  if (outs != nullptr) add_spans(s, count, outs, n, true);
  const bool ok = apart(s, count);
  if (s != few) delete[] s;
  return ok ? MOE_OK : MOE_ERR_INVALID_ARG;
}
int launches_of(int32_t n) { return n <= kList ? 1 : (n + kLongList - 1) / kLongList; }

template <int N>
void fill(TensorList<N>& list, const moe_tensor* t, const moe_tensor* out, int count) {
  long long end = 0;
  list.count = count;
  for (int i = 0; i < count; ++i) {
    end += chunks_of(t[i]);
    list.src[i] = static_cast<const uint4*>(t[i].data);
    list.dst[i] = static_cast<uint4*>(out != nullptr ? out[i].data : t[i].data);
    list.n[i] = t[i].n;
    list.end[i] = end;
    list.fp32[i] = t[i].type == MOE_TYPE_FP32;
  }
}
long long all_chunks(const moe_tensor* t, int count) {
  long long chunks = 0;
  for (int i = 0; i < count; ++i) chunks += chunks_of(t[i]);
  return chunks > 1 ? chunks : 1;
}
int blocks_of(const moe_tensor* t, int count) {
  const long long chunks = all_chunks(t, count);
  return chunks < kBlocks ? static_cast<int>(chunks) : kBlocks;
}

template <int N>
cudaError_t norm_launch(const moe_tensor* t, int count, int blocks, double* part, int part0, int total, float* norm,
                        int* status, cudaStream_t st) {
  TensorList<N> list;
  fill(list, t, nullptr, count);
  count_launches(1);
  return launch_k(grad_norm_kernel<N>, blocks, kThreads, 0, st, list, part, part0, total, norm, status);
}
template <int N>
cudaError_t clip_launch(const moe_tensor* t, const moe_tensor* out, int count, const float* norm, float limit,
                        cudaStream_t st) {
  TensorList<N> list;
  fill(list, t, out, count);
  count_launches(1);
  // a block a chunk: 2.3 GB scaled in 700 us; 805 where 912 blocks take 80 each in turn
  const long long chunks = all_chunks(t, count);
  const int blocks = static_cast<int>(chunks < kMaxClipBlocks ? chunks : kMaxClipBlocks);
  return launch_k(grad_clip_kernel<N>, blocks, kThreads, 0, st, list, norm, limit, out == nullptr ? 1 : 0);
}

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::entry;

extern "C" {

size_t moe_grad_norm_workspace_bytes(int32_t n) {
  if (n < 0 || n > kMaxTensors) return 0;
  return kStatusBytes + align_up(static_cast<size_t>(launches_of(n)) * kBlocks * sizeof(double));
}

moe_status moe_grad_norm(const moe_tensor* grads, int32_t n, float* norm, void* ws, size_t ws_bytes, void* stream) {
  if (!list_ok(grads, n) || !word_ok(norm) || !ptr_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_grad_norm_workspace_bytes(n)) return MOE_ERR_WORKSPACE;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* part = reinterpret_cast<double*>(static_cast<char*>(ws) + kStatusBytes);
  const int per = n <= kList ? kList : kLongList;
  int total = 0;
  for (int32_t i = 0; i == 0 || i < n; i += per) total += blocks_of(grads + i, n - i < per ? n - i : per);
  int part0 = 0;
  for (int32_t i = 0; i == 0 || i < n; i += per) {
    const int count = n - i < per ? n - i : per, blocks = blocks_of(grads + i, count);
    const cudaError_t e =
        per == kList
            ? norm_launch<kList>(grads + i, count, blocks, part, part0, total, norm, static_cast<int*>(ws), st)
            : norm_launch<kLongList>(grads + i, count, blocks, part, part0, total, norm, static_cast<int*>(ws), st);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    part0 += blocks;
  }
  return MOE_OK;
}

moe_status moe_grad_clip(const moe_tensor* grads, const moe_tensor* outs, int32_t n, const float* norm, float limit,
                         void* stream) {
  if (!list_ok(grads, n) || !word_ok(norm) || !(limit >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (outs != nullptr) {
    if (!list_ok(outs, n)) return MOE_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i)
      if (outs[i].n != grads[i].n || outs[i].type != grads[i].type) return MOE_ERR_INVALID_ARG;
  }
  const moe_status apart = writes_apart(grads, outs, n);
  if (apart != MOE_OK) return apart;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int per = n <= kList ? kList : kLongList;
  // the tensors of the last launch first, too
  const int32_t last = n > 0 ? (n - 1) / per * per : -1;
  for (int32_t i = last; i >= 0; i -= per) {
    const int count = n - i < per ? n - i : per;
    const moe_tensor* out = outs != nullptr ? outs + i : nullptr;
    const cudaError_t e = per == kList ? clip_launch<kList>(grads + i, out, count, norm, limit, st)
                                       : clip_launch<kLongList>(grads + i, out, count, norm, limit, st);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
