// Token embedding with scaling, and the gradient of its table by sorted tokens.
//
//   out[i] = bf16(scale * table[tok[i]]),
//   dtable[v] = base[v] + scale * sum over the i with tok[i] = v of dy[i].
//
// The gradient never adds through atomics: the token positions are sorted by
// token (a stable radix sort), a run of equal tokens is summed in ascending
// position, and every row of dtable is written once, so the result does not
// depend on timing.  A frequent token's run is cut at multiples of kChunk
// sorted positions: whole chunks of one token are summed by blocks of their
// own, and the row adds their sums in order.  The sums are fp32.
//
// Both directions are bound by HBM: the lookup by the rows it reads and
// writes, the gradient mostly by the V x H fp32 words it writes.
#include <cuda_bf16.h>

#include <cstdint>

#include "entry_checks.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kDigitBits = 8;
constexpr int kBins = 1 << kDigitBits;
constexpr int kSortThreads = 256;
constexpr int kSortItems = 8;
constexpr int kSortTile = kSortThreads * kSortItems;   // pairs one block ranks
constexpr int kChunk = 64;                             // sorted positions summed by one block

// ---------------------------------------------------------------- lookup
// One block per token.  An id outside [0, V) gives a zero row; -1 is padding,
// any other one is reported.
__global__ void __launch_bounds__(128) embedding_fwd_kernel(const int32_t* __restrict__ tokens,
                                                            const uint4* __restrict__ table, int V, int words,
                                                            float scale, uint4* __restrict__ out, int* status) {
  pdl_entry();
  const int tok = tokens[blockIdx.x];
  const bool ok = tok >= 0 && tok < V;
  if (!ok && tok != -1 && threadIdx.x == 0) set_status(status, kErrBadIndex);
  const uint4* src = table + static_cast<long long>(ok ? tok : 0) * words;
  uint4* dst = out + static_cast<long long>(blockIdx.x) * words;
  for (int c = threadIdx.x; c < words; c += blockDim.x) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok) {
      v = src[c];
      v = make_uint4(pack_bf16x2(bf16_lo(v.x) * scale, bf16_hi(v.x) * scale),
                     pack_bf16x2(bf16_lo(v.y) * scale, bf16_hi(v.y) * scale),
                     pack_bf16x2(bf16_lo(v.z) * scale, bf16_hi(v.z) * scale),
                     pack_bf16x2(bf16_lo(v.w) * scale, bf16_hi(v.w) * scale));
    }
    dst[c] = v;
  }
}

// ---------------------------------------------------------------- sort
// Key of a position: its token, or V (after every token) where it has none.
__device__ __forceinline__ uint32_t key_of(const int32_t* __restrict__ tokens, int i, int V, int* status) {
  const int t = tokens[i];
  if (t >= 0 && t < V) return static_cast<uint32_t>(t);
  if (t != -1) set_status(status, kErrBadIndex);
  return static_cast<uint32_t>(V);
}

// Digit counts of each tile of kSortTile pairs: hist[tile][bin].  The first
// pass reads the tokens themselves (keys == nullptr) and marks every row of
// the table as without a run.
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(const int32_t* __restrict__ tokens,
                                                                 const uint32_t* __restrict__ keys, int n, int V,
                                                                 int shift, int32_t* __restrict__ hist,
                                                                 int32_t* __restrict__ first, int* status) {
  pdl_entry();
  __shared__ int s_cnt[kBins];
  s_cnt[threadIdx.x] = 0;
  __syncthreads();
  const long long i0 = static_cast<long long>(blockIdx.x) * kSortTile;
  #pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const long long i = i0 + j * kSortThreads + threadIdx.x;
    if (i < n) {
      const uint32_t k = keys != nullptr ? keys[i] : key_of(tokens, static_cast<int>(i), V, status);
      atomicAdd(&s_cnt[(k >> shift) & (kBins - 1)], 1);
    }
  }
  __syncthreads();
  hist[static_cast<long long>(blockIdx.x) * kBins + threadIdx.x] = s_cnt[threadIdx.x];
  if (keys == nullptr) {
    const long long stride = static_cast<long long>(gridDim.x) * kSortThreads;
    for (long long v = static_cast<long long>(blockIdx.x) * kSortThreads + threadIdx.x; v < V; v += stride)
      first[v] = -1;
  }
}

// Moves the pairs of one tile to their places for this digit, keeping the
// order of equal digits.  Warp w ranks the tile's pairs [256 w, 256 w + 256)
// in rounds of 32; the place of a pair is the number of pairs with a smaller
// digit anywhere, plus those with its digit in earlier tiles, in earlier
// warps, in earlier rounds, and in lower lanes.
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const int32_t* __restrict__ tokens,
                                                                    const uint32_t* __restrict__ keys,
                                                                    const int32_t* __restrict__ pos, int n, int V,
                                                                    int shift, const int32_t* __restrict__ hist,
                                                                    uint32_t* __restrict__ keys_out,
                                                                    int32_t* __restrict__ pos_out) {
  pdl_entry();
  constexpr int WARPS = kSortThreads / 32;
  __shared__ int s_cnt[WARPS][kBins];
  __shared__ int s_base[kBins];
  __shared__ int s_warp[WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  #pragma unroll
  for (int w = 0; w < WARPS; ++w) s_cnt[w][tid] = 0;
  // bin tid: pairs in all tiles, and in the tiles before this one
  int total = 0, before = 0;
  for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
    const int c = hist[static_cast<long long>(b) * kBins + tid];
    if (b < static_cast<int>(blockIdx.x)) before += c;
    total += c;
  }
  int inc = total;                       // exclusive scan of the totals over the bins
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(kFull, inc, d);
    if (lane >= d) inc += u;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int lower = 0;
  for (int w = 0; w < warp; ++w) lower += s_warp[w];
  s_base[tid] = lower + inc - total + before;
  __syncthreads();

  uint32_t key[kSortItems];
  int where[kSortItems], rank[kSortItems];
  const long long i0 = static_cast<long long>(blockIdx.x) * kSortTile + warp * 32 * kSortItems;
  #pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const long long i = i0 + j * 32 + lane;
    key[j] = 0xffffffffu;
    where[j] = 0;
    if (i < n) {
      key[j] = keys != nullptr ? keys[i] : key_of(tokens, static_cast<int>(i), V, nullptr);
      where[j] = keys != nullptr ? pos[i] : static_cast<int>(i);
    }
  }
  #pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const bool live = i0 + j * 32 + lane < n;
    const int d = live ? static_cast<int>((key[j] >> shift) & (kBins - 1)) : kBins;
    const unsigned peers = __match_any_sync(kFull, d);
    const int lead = __ffs(peers) - 1;
    int seen = 0;
    if (live && lane == lead) {
      seen = s_cnt[warp][d];
      s_cnt[warp][d] = seen + __popc(peers);
    }
    seen = __shfl_sync(kFull, seen, lead);
    rank[j] = seen + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
  }
  __syncthreads();
  int run = s_base[tid];                 // bin tid: first place of each warp's pairs
  #pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const int c = s_cnt[w][tid];
    s_cnt[w][tid] = run;
    run += c;
  }
  __syncthreads();
  #pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    if (i0 + j * 32 + lane < n) {
      const int d = static_cast<int>((key[j] >> shift) & (kBins - 1));
      const int to = s_cnt[warp][d] + rank[j];
      keys_out[to] = key[j];
      pos_out[to] = where[j];
    }
  }
}

// ---------------------------------------------------------------- runs
__device__ __forceinline__ void add_row8(float (&a)[8], const uint4& v) {
  a[0] += bf16_lo(v.x); a[1] += bf16_hi(v.x);
  a[2] += bf16_lo(v.y); a[3] += bf16_hi(v.y);
  a[4] += bf16_lo(v.z); a[5] += bf16_hi(v.z);
  a[6] += bf16_lo(v.w); a[7] += bf16_hi(v.w);
}

// Block (c, j): chunk c of the sorted positions, words [128 j, 128 j + 128) of
// the rows.  Marks where each token's run begins and, for a whole chunk of
// one token, leaves the sum of its rows in part[c].
__global__ void __launch_bounds__(128) embedding_runs_kernel(const uint32_t* __restrict__ keys,
                                                             const int32_t* __restrict__ pos, int n, int V, int words,
                                                             const uint4* __restrict__ dy, int32_t* __restrict__ first,
                                                             float4* __restrict__ part) {
  pdl_entry();
  __shared__ int s_pos[kChunk];
  const int i0 = blockIdx.x * kChunk, tid = threadIdx.x;
  const int end = min(n, i0 + kChunk);
  if (tid < end - i0) {
    const uint32_t k = keys[i0 + tid];
    s_pos[tid] = pos[i0 + tid];
    if (blockIdx.y == 0 && k < static_cast<uint32_t>(V) && (i0 + tid == 0 || keys[i0 + tid - 1] != k))
      first[k] = i0 + tid;
  }
  __syncthreads();
  if (end - i0 < kChunk || keys[i0] != keys[end - 1] || keys[i0] >= static_cast<uint32_t>(V)) return;
  const int c = blockIdx.y * 128 + tid;
  if (c >= words) return;
  float a[8] = {};
  #pragma unroll 8
  for (int r = 0; r < kChunk; ++r) add_row8(a, dy[static_cast<long long>(s_pos[r]) * words + c]);
  float4* o = part + (static_cast<long long>(blockIdx.x) * words + c) * 2;
  o[0] = make_float4(a[0], a[1], a[2], a[3]);
  o[1] = make_float4(a[4], a[5], a[6], a[7]);
}

// Row v of the gradient, by one block (grid x: rows, y: columns): the row's
// run is its positions up to a chunk border, whole chunks, and the rest.
__global__ void __launch_bounds__(128) embedding_rows_kernel(const uint32_t* __restrict__ keys,
                                                             const int32_t* __restrict__ pos, int n, int words,
                                                             const uint4* __restrict__ dy,
                                                             const int32_t* __restrict__ first,
                                                             const float4* __restrict__ part,
                                                             const uint4* __restrict__ base, float scale,
                                                             float4* __restrict__ dtable) {
  pdl_entry();
  const uint32_t v = blockIdx.x;
  const int c = blockIdx.y * 128 + threadIdx.x;
  if (c >= words) return;
  float a[8] = {};
  int i = first[v];
  if (i >= 0) {
    while (i < n && keys[i] == v) {
      if (i % kChunk == 0 && i + kChunk <= n && keys[i + kChunk - 1] == v) {
        const float4* p = part + (static_cast<long long>(i / kChunk) * words + c) * 2;
        const float4 p0 = p[0], p1 = p[1];
        a[0] += p0.x; a[1] += p0.y; a[2] += p0.z; a[3] += p0.w;
        a[4] += p1.x; a[5] += p1.y; a[6] += p1.z; a[7] += p1.w;
        i += kChunk;
      } else {
        add_row8(a, dy[static_cast<long long>(pos[i]) * words + c]);
        ++i;
      }
    }
    #pragma unroll
    for (int j = 0; j < 8; ++j) a[j] *= scale;
  }
  if (base != nullptr) add_row8(a, base[static_cast<long long>(v) * words + c]);
  float4* o = dtable + (static_cast<long long>(v) * words + c) * 2;
  o[0] = make_float4(a[0], a[1], a[2], a[3]);
  o[1] = make_float4(a[4], a[5], a[6], a[7]);
}

// ---------------------------------------------------------------- workspace
// Tiles of the sort; one where there is nothing to sort (its launch still
// marks the table's rows).
int sort_tiles(int n) { return n > 0 ? (n + kSortTile - 1) / kSortTile : 1; }

struct Ws {
  size_t keys[2], pos[2], hist, first, part, total;
};
Ws layout(int n, int V, int H) {
  Ws w;
  size_t off = entry::kStatusBytes;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = entry::align_up(off + bytes);
    return o;
  };
  const size_t N = n;
  for (int i = 0; i < 2; ++i) {
    w.keys[i] = take(N * 4);
    w.pos[i] = take(N * 4);
  }
  w.hist = take(static_cast<size_t>(sort_tiles(n)) * kBins * 4);
  w.first = take(static_cast<size_t>(V) * 4);
  w.part = take(N / kChunk * H * 4);
  w.total = off;
  return w;
}

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

constexpr int kMaxTokens = 1 << 24, kMaxVocab = 1 << 24;
bool sizes_ok(int32_t n, int32_t V, int32_t H) {
  return n >= 0 && n <= kMaxTokens && V > 0 && V <= kMaxVocab && entry::hidden_ok(H);
}

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::entry;

extern "C" {

size_t moe_embedding_workspace_bytes(int32_t n, int32_t V, int32_t H) {
  return sizes_ok(n, V, H) ? layout(n, V, H).total : 0;
}

moe_status moe_embedding_forward(const int32_t* tokens, int32_t n, const void* table, int32_t V, int32_t H, float scale,
                                 void* out, void* ws, void* stream) {
  if (!sizes_ok(n, V, H) || !ptr_ok(table) || !ptr_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (n > 0 && (!ptr_ok(tokens) || !ptr_ok(out))) return MOE_ERR_INVALID_ARG;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  count_launches(1);
  return status_of(launch_k(embedding_fwd_kernel, n, 128, 0, static_cast<cudaStream_t>(stream), tokens,
                            static_cast<const uint4*>(table), V, H / 8, scale, static_cast<uint4*>(out),
                            static_cast<int*>(ws)));
}

moe_status moe_embedding_backward(const int32_t* tokens, int32_t n, const void* dy, int32_t V, int32_t H, float scale,
                                  const void* base, float* dtable, void* ws, size_t ws_bytes, void* stream) {
  if (!sizes_ok(n, V, H) || !ptr_ok(dtable) || !opt_ok(base) || !ptr_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (n > 0 && (!ptr_ok(tokens) || !ptr_ok(dy))) return MOE_ERR_INVALID_ARG;
  const Ws w = layout(n, V, H);
  if (ws_bytes < w.total) return MOE_ERR_WORKSPACE;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* status = static_cast<int*>(ws);
  int32_t* first = at<int32_t>(ws, w.first);
  int32_t* hist = at<int32_t>(ws, w.hist);
  const int tiles = sort_tiles(n);
  int cur = 0, launches = 0;
  // digits of the keys 0 .. V
  for (int shift = 0; shift < 32 && (shift == 0 || (V >> shift) != 0); shift += kDigitBits) {
    const uint32_t* keys = shift == 0 ? nullptr : at<uint32_t>(ws, w.keys[cur]);
    const int32_t* pos = shift == 0 ? nullptr : at<int32_t>(ws, w.pos[cur]);
    const int to = shift == 0 ? 0 : cur ^ 1;
    if (launch_k(sort_hist_kernel, tiles, kSortThreads, 0, st, tokens, keys, n, V, shift, hist, first, status) !=
            cudaSuccess ||
        launch_k(sort_scatter_kernel, tiles, kSortThreads, 0, st, tokens, keys, pos, n, V, shift, hist,
                 at<uint32_t>(ws, w.keys[to]), at<int32_t>(ws, w.pos[to])) != cudaSuccess)
      return MOE_ERR_CUDA;
    launches += 2;
    cur = to;
  }
  const uint32_t* keys = at<uint32_t>(ws, w.keys[cur]);
  const int32_t* pos = at<int32_t>(ws, w.pos[cur]);
  const int words = H / 8;
  const unsigned cols = (words + 127) / 128;
  if (n > 0) {
    if (launch_k(embedding_runs_kernel, dim3((n + kChunk - 1) / kChunk, cols), 128, 0, st, keys, pos, n, V, words,
                 static_cast<const uint4*>(dy), first, at<float4>(ws, w.part)) != cudaSuccess)
      return MOE_ERR_CUDA;
    ++launches;
  }
  if (launch_k(embedding_rows_kernel, dim3(V, cols), 128, 0, st, keys, pos, n, words, static_cast<const uint4*>(dy),
               first, at<float4>(ws, w.part), static_cast<const uint4*>(base), scale,
               reinterpret_cast<float4*>(dtable)) != cudaSuccess)
    return MOE_ERR_CUDA;
  count_launches(launches + 1);
  return MOE_OK;
}

}  // extern "C"
