// Token embedding with scaling, and the gradient of its table by sorted tokens.
//
//   out[i] = bf16(scale * table[tok[i]]),
//   dtable[v] = base[v] + scale * sum over the i with tok[i] = v of dy[i].
//
// The gradient never adds through atomics: the token positions are sorted by
// token (a stable radix sort; up to kFewTokens are searched instead), a run of
// equal tokens is summed in ascending position, and every row of dtable is
// written once, so the result does not depend on timing.  A frequent token's run is cut at multiples of kChunk
// sorted positions: whole chunks of one token are summed by blocks of their
// own, and the row adds their sums in order.  The sums are fp32.
//
// Both directions are bound by HBM: the lookup by the rows it reads and
// writes, the gradient mostly by the V x H fp32 words it writes.  Measured on
// one GB300 (a plain copy reaches 6.68 TB/s): lookup of 16384 x 4096 31 us
// (6.24 TB/s); gradient of 16384 rows into 32000 x 7168 195 us (5.91 TB/s: sort
// 17, whole chunks 9, rows 165); 1003 rows into 50001 x 1024 on top of `base`
// 59 us (5.25 TB/s: sort 7, rows 49).
#include <cuda_bf16.h>

#include <atomic>
#include <cstdint>

#include "entry_checks.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kDigitBits = 9;                          // two passes up to V = 2^18
constexpr int kBins = 1 << kDigitBits;
constexpr int kSortThreads = 512;
constexpr int kSortItems = 8;
constexpr int kSortTile = kSortThreads * kSortItems;   // pairs one block ranks
constexpr int kChunk = 32;                             // sorted positions summed by one block

// ---------------------------------------------------------------- lookup
// An id outside [0, V) gives a zero row; -1 is padding, any other one is
// reported.  A thread has four 16-byte loads on their way: four words of one
// row (wide rows, one block each), or, with rows of up to 256 words, a word of
// four rows (`lanes` threads a row, a power of two): 16384 rows of 1032 in 10.7
// us, against 17.3 with a block each.
template <bool WIDE>
__global__ void __launch_bounds__(128) embedding_fwd_kernel(const int32_t* __restrict__ tokens, int n,
                                                            const uint4* __restrict__ table, int V, int words,
                                                            int lanes, float scale, uint4* __restrict__ out,
                                                            int* status) {
  pdl_entry();
  const int rows = 128 / lanes;                        // (narrow) rows of one of the four loads
  int tok[4];
  long long row[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    row[i] = WIDE ? blockIdx.x : static_cast<long long>(blockIdx.x) * 4 * rows + i * rows + threadIdx.x / lanes;
    tok[i] = (WIDE && i > 0) ? tok[0] : row[i] < n ? tokens[row[i]] : -1;
    if ((tok[i] < -1 || tok[i] >= V) && (WIDE ? threadIdx.x == 0 && i == 0 : threadIdx.x % lanes == 0))
      set_status(status, kErrBadIndex);
    if (tok[i] >= V) tok[i] = -1;
  }
  for (int c0 = WIDE ? threadIdx.x : threadIdx.x % lanes; c0 < words; c0 += WIDE ? 4 * 128 : lanes) {
    uint4 v[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = WIDE ? c0 + i * 128 : c0;
      v[i] = tok[i] >= 0 && c < words ? table[static_cast<long long>(tok[i]) * words + c] : make_uint4(0, 0, 0, 0);
    }
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = WIDE ? c0 + i * 128 : c0;
      const float by = tok[i] >= 0 ? scale : 0.f;      // (a zero row whatever the scale)
      if (c < words && row[i] < n)
        out[row[i] * words + c] = make_uint4(pack_bf16x2(bf16_lo(v[i].x) * by, bf16_hi(v[i].x) * by),
                                             pack_bf16x2(bf16_lo(v[i].y) * by, bf16_hi(v[i].y) * by),
                                             pack_bf16x2(bf16_lo(v[i].z) * by, bf16_hi(v[i].z) * by),
                                             pack_bf16x2(bf16_lo(v[i].w) * by, bf16_hi(v[i].w) * by));
    }
  }
}

__device__ __forceinline__ void add_row8(float (&a)[8], const uint4& v) {
  a[0] += bf16_lo(v.x); a[1] += bf16_hi(v.x);
  a[2] += bf16_lo(v.y); a[3] += bf16_hi(v.y);
  a[4] += bf16_lo(v.z); a[5] += bf16_hi(v.z);
  a[6] += bf16_lo(v.w); a[7] += bf16_hi(v.w);
}

// Eight fp32 values to a 16-byte aligned place: one 32-byte store where it is
// 32-byte aligned.
__device__ __forceinline__ void store8(float* p, const float (&a)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    st_global_v8(p, a);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(a[0], a[1], a[2], a[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(a[4], a[5], a[6], a[7]);
  }
}

// Words [begin, end) of two rows of the gradient without a token (those that
// `fill` says): base, or zero.  One warp, eight loads on their way.
__device__ __forceinline__ void fill_rows(const long long (&v)[2], const bool (&fill)[2], int words, int begin, int end,
                                          const uint4* __restrict__ base, float* __restrict__ dtable) {
  for (int c0 = begin + (threadIdx.x & 31); c0 < end; c0 += 128) {
    uint4 b[2][4];
    #pragma unroll
    for (int u = 0; u < 2; ++u) {
      #pragma unroll
      for (int k = 0; k < 4; ++k) {
        b[u][k] = make_uint4(0, 0, 0, 0);
        if (base != nullptr && fill[u] && c0 + 32 * k < end) b[u][k] = base[v[u] * words + c0 + 32 * k];
      }
    }
    #pragma unroll
    for (int u = 0; u < 2; ++u) {
      #pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a[8] = {};
        add_row8(a, b[u][k]);
        if (fill[u] && c0 + 32 * k < end) store8(dtable + (v[u] * words + c0 + 32 * k) * 8, a);
      }
    }
  }
}

// Narrow rows (up to 16 words): `lanes`, a power of two, for a row.  Calls f(row,
// word) for each of the block's rows [0, rows) and words, as many rows at a time
// as the block's threads hold.
template <class F>
__device__ __forceinline__ void narrow_rows(int rows, int words, F&& f) {
  int lanes = 16;
  while (lanes / 2 >= words) lanes /= 2;
  const int c = threadIdx.x % lanes;
  #pragma unroll 4
  for (int r = threadIdx.x / lanes; r < rows; r += 128 / lanes)
    if (c < words) f(r, c);
}
constexpr int kNarrow = 16;

// ---------------------------------------------------------------- few tokens
// Up to kFewTokens positions there is nothing to sort: one launch, in which
// block (b, j) writes words [128 j, 128 j + 128) of the table's rows b, b + grid,
// ... (strided, because token ids are mostly ordered by frequency), a warp a
// row.  The block looks through all tokens for the rows that have one; such a
// row's warp finds its positions, in ascending order, and sums them.  64 tokens
// into 11000 x 680 8.0 us (the sort's three launches: 12.3); at 256 both take 13.
constexpr int kFewTokens = 128;
__global__ void __launch_bounds__(128) embedding_few_kernel(const int32_t* __restrict__ tokens, int n, int V, int words,
                                                            const uint4* __restrict__ dy,
                                                            const uint4* __restrict__ base, float scale,
                                                            float* __restrict__ dtable, int* status) {
  pdl_entry();
  extern __shared__ uint32_t s_has[];                  // a bit for each of the block's rows
  __shared__ int s_tok[kFewTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int first = blockIdx.x, step = gridDim.x, rows = (V - first + step - 1) / step;
  const int c0 = blockIdx.y * 128 + lane;
  for (int i = tid; i < (rows + 31) / 32; i += 128) s_has[i] = 0;
  __syncthreads();
  for (int i = tid; i < kFewTokens; i += 128) {
    const int t = i < n ? tokens[i] : -1;
    s_tok[i] = t;
    if (first == 0 && blockIdx.y == 0 && (t < -1 || t >= V)) set_status(status, kErrBadIndex);
    const int off = t - first;
    if (t >= 0 && t < V && off >= 0 && off % step == 0) atomicOr(&s_has[off / step >> 5], 1u << (off / step & 31));
  }
  __syncthreads();
  auto has = [&](int r) { return ((s_has[r >> 5] >> (r & 31)) & 1u) != 0; };
  if (words <= kNarrow) {
    narrow_rows(rows, words, [&](int r, int c) {
      const long long at = (first + static_cast<long long>(r) * step) * words + c;
      if (has(r)) return;
      float a[8] = {};
      if (base != nullptr) add_row8(a, base[at]);
      store8(dtable + at * 8, a);
    });
  }
  for (int r = words <= kNarrow ? rows : warp; r < rows; r += 8) {
    const long long v[2] = {first + static_cast<long long>(r) * step, first + static_cast<long long>(r + 4) * step};
    const bool fill[2] = {!has(r), r + 4 < rows && !has(r + 4)};
    fill_rows(v, fill, words, blockIdx.y * 128, min(words, static_cast<int>(blockIdx.y) * 128 + 128), base, dtable);
  }
  for (int r = warp; r < rows; r += 4) {
    if (!has(r)) continue;
    const int v = first + r * step;
    const long long row = static_cast<long long>(v) * words;
    float a[4][8] = {};
    for (int i0 = 0; i0 < n; i0 += 32) {
      unsigned match = __ballot_sync(kFull, s_tok[i0 + lane] == v);
      while (match != 0) {                             // two positions at a time
        const int p0 = i0 + __ffs(match) - 1;
        match &= match - 1;
        const bool two = match != 0;
        const int p1 = two ? i0 + __ffs(match) - 1 : p0;
        match &= match - 1;
        uint4 e[2][4];
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (c0 + 32 * k < words) {
            e[0][k] = dy[static_cast<long long>(p0) * words + c0 + 32 * k];
            if (two) e[1][k] = dy[static_cast<long long>(p1) * words + c0 + 32 * k];
          }
        }
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (c0 + 32 * k < words) {
            add_row8(a[k], e[0][k]);
            if (two) add_row8(a[k], e[1][k]);
          }
        }
      }
    }
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + 32 * k;
      if (c < words) {
        #pragma unroll
        for (int j = 0; j < 8; ++j) a[k][j] *= scale;
        if (base != nullptr) add_row8(a[k], base[row + c]);
        store8(dtable + (row + c) * 8, a[k]);
      }
    }
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

// Up to kClusterSort positions: the whole sort in one launch, by BLOCKS blocks:
// one up to kBlockSort positions (1003 in 7 us), a cluster of eight beyond
// (16384 in 17 us).  Each block holds its share of the pairs, in registers
// while it ranks them and in shared memory between the passes.  A pass ranks
// the pairs as sort_scatter_kernel does, with the digit counts of every warp in
// shared memory; the blocks read each other's counts and write the pairs to
// their places in each other's shared memory, and the sorted pairs are copied
// out in one piece.  (Written to their places in global memory they cost a
// sector each.)
constexpr int kCluster = 8;
constexpr int kClusterThreads = 512;                  // (one for each bin)
constexpr int kClusterWarps = kClusterThreads / 32;
constexpr int kClusterItems = 16;                     // pairs per thread at most
constexpr int kClusterSort = kCluster * kClusterThreads * kClusterItems;
constexpr int kBlockSort = 2 * kClusterThreads;       // (beyond, a cluster's eight times fewer rounds are faster)
__host__ __device__ constexpr int sort_rounds(int n, int blocks) {
  return (n + blocks * kClusterThreads - 1) / (blocks * kClusterThreads);
}
size_t sort_smem(int n, int blocks) {
  return static_cast<size_t>(kClusterWarps) * kBins * 2 + static_cast<size_t>(sort_rounds(n, blocks)) * kClusterThreads * 8;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Barrier over the blocks that sort together.
template <int BLOCKS>
__device__ __forceinline__ void sort_sync() {
  if constexpr (BLOCKS > 1) cluster_sync();
  else __syncthreads();
}
template <int BLOCKS>
__device__ __forceinline__ void cluster_sort(const int32_t* __restrict__ tokens, int n, int V, int passes,
                                             uint32_t* __restrict__ keys_out, int32_t* __restrict__ pos_out,
                                             int* status, uint8_t* s_raw) {
  __shared__ uint32_t s_total[kBins];                 // this block's pairs of each digit
  __shared__ uint32_t s_base[kBins];                  // where they go
  __shared__ int s_warp[kClusterWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t me = BLOCKS > 1 ? cluster_ctarank() : 0;
  const int rounds = sort_rounds(n, BLOCKS), slice = rounds * kClusterThreads;
  uint16_t* s_cnt = reinterpret_cast<uint16_t*>(s_raw);              // [warp][bin]
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_cnt + kClusterWarps * kBins);
  uint32_t* s_pos = s_key + slice;
  uint16_t* my_cnt = s_cnt + warp * kBins;
  const int mine = min(max(n - static_cast<int>(me) * slice, 0), slice);   // pairs of this block
  const int w0 = warp * 32 * rounds + lane;                                // this lane's: w0, w0 + 32, ...
  uint32_t key[kClusterItems], where[kClusterItems];
  uint16_t rank[kClusterItems];
  #pragma unroll
  for (int j = 0; j < kClusterItems; ++j) {
    const int i = w0 + j * 32, g = static_cast<int>(me) * slice + i;
    key[j] = (j < rounds && i < mine) ? key_of(tokens, g, V, status) : 0xffffffffu;
    where[j] = static_cast<uint32_t>(g);
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * kDigitBits;
    for (int i = lane; i < kBins / 2; i += 32) reinterpret_cast<uint32_t*>(my_cnt)[i] = 0;
    __syncwarp();
    #pragma unroll
    for (int j = 0; j < kClusterItems; ++j) {
      if (j < rounds) {
        const bool live = w0 + j * 32 < mine;
        const int d = live ? static_cast<int>((key[j] >> shift) & (kBins - 1)) : kBins;
        const unsigned peers = __match_any_sync(kFull, d);
        const int lead = __ffs(peers) - 1;
        int seen = 0;
        if (live && lane == lead) {
          seen = my_cnt[d];
          my_cnt[d] = static_cast<uint16_t>(seen + __popc(peers));
        }
        seen = __shfl_sync(kFull, seen, lead);
        rank[j] = static_cast<uint16_t>(seen + __popc(peers & ((1u << lane) - 1u)));
        __syncwarp();
      }
    }
    __syncthreads();
    if (tid < kBins) {                    // bin tid: where each warp's pairs begin among this block's
      uint32_t run = 0;
      #pragma unroll 8
      for (int w = 0; w < kClusterWarps; ++w) {
        const uint32_t c = s_cnt[w * kBins + tid];
        s_cnt[w * kBins + tid] = static_cast<uint16_t>(run);
        run += c;
      }
      s_total[tid] = run;
    }
    sort_sync<BLOCKS>();
    int total = 0, before = 0;            // bin tid: pairs of all blocks, and of those before this one
    if (tid < kBins) {
      if constexpr (BLOCKS > 1) {
        #pragma unroll
        for (uint32_t r = 0; r < BLOCKS; ++r) {
          const int c = static_cast<int>(ld_cluster_u32(mapa_shared(smem_u32(&s_total[tid]), r)));
          total += c;
          if (r < me) before += c;
        }
      } else {
        total = static_cast<int>(s_total[tid]);
      }
    }
    int inc = total;
    #pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(kFull, inc, d);
      if (lane >= d) inc += u;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    if (tid < kBins) {
      int lower = 0;
      for (int w = 0; w < warp; ++w) lower += s_warp[w];
      s_base[tid] = static_cast<uint32_t>(lower + inc - total + before);
    }
    __syncthreads();
    #pragma unroll
    for (int j = 0; j < kClusterItems; ++j) {
      if (j < rounds && w0 + j * 32 < mine) {
        const int d = static_cast<int>((key[j] >> shift) & (kBins - 1));
        const uint32_t to = s_base[d] + my_cnt[d] + rank[j];
        if constexpr (BLOCKS > 1) {
          const uint32_t block = (to / kClusterThreads) / static_cast<uint32_t>(rounds);
          const uint32_t at = to - block * static_cast<uint32_t>(slice);
          st_cluster_u32(mapa_shared(smem_u32(s_key + at), block), key[j]);
          st_cluster_u32(mapa_shared(smem_u32(s_pos + at), block), where[j]);
        } else {
          s_key[to] = key[j];
          s_pos[to] = where[j];
        }
      }
    }
    sort_sync<BLOCKS>();                  // every block's pairs are in their places
    if (pass + 1 < passes) {
      #pragma unroll
      for (int j = 0; j < kClusterItems; ++j) {
        const int i = w0 + j * 32;
        if (j < rounds && i < mine) {
          key[j] = s_key[i];
          where[j] = s_pos[i];
        }
      }
      if constexpr (BLOCKS == 1) __syncthreads();
    }
  }
  const long long g0 = static_cast<long long>(me) * slice;
  for (int i = tid; i < mine; i += kClusterThreads) {
    keys_out[g0 + i] = s_key[i];
    pos_out[g0 + i] = static_cast<int32_t>(s_pos[i]);
  }
}

// More positions: two launches a pass.  Digit counts of each tile of kSortTile
// pairs: hist[tile][bin].  The first pass reads the tokens themselves (keys ==
// nullptr).
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(const int32_t* __restrict__ tokens,
                                                                 const uint32_t* __restrict__ keys, int n, int V,
                                                                 int shift, int32_t* __restrict__ hist, int* status) {
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

// ---------------------------------------------------------------- rows
// First launch (up to kClusterSort positions): the first block or cluster sorts;
// the others clear the flags of the rows that have a token.
constexpr int kClearRows = 1 << 14;     // flags one other block clears
template <int BLOCKS>
__device__ __forceinline__ void sort_launch(const int32_t* __restrict__ tokens, int n, int V, int passes,
                                            uint32_t* __restrict__ keys_out, int32_t* __restrict__ pos_out,
                                            uint8_t* __restrict__ has, int* status) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  if (blockIdx.x < BLOCKS) {
    cluster_sort<BLOCKS>(tokens, n, V, passes, keys_out, pos_out, status, s_raw);
    return;
  }
  const int block = blockIdx.x - BLOCKS, blocks = gridDim.x - BLOCKS;
  for (int v = block * kClusterThreads + threadIdx.x; v < V; v += blocks * kClusterThreads) has[v] = 0;
}
__global__ void __launch_bounds__(kClusterThreads)
    block_sort_kernel(const int32_t* __restrict__ tokens, int n, int V, int passes, uint32_t* __restrict__ keys_out,
                      int32_t* __restrict__ pos_out, uint8_t* __restrict__ has, int* status) {
  pdl_entry();
  sort_launch<1>(tokens, n, V, passes, keys_out, pos_out, has, status);
}
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kClusterThreads)
    cluster_sort_kernel(const int32_t* __restrict__ tokens, int n, int V, int passes, uint32_t* __restrict__ keys_out,
                        int32_t* __restrict__ pos_out, uint8_t* __restrict__ has, int* status) {
  pdl_entry();
  sort_launch<kCluster>(tokens, n, V, passes, keys_out, pos_out, has, status);
}

// For more positions: the flags of the rows that have a token, cleared here and
// set by embedding_chunks_kernel.
__global__ void __launch_bounds__(256) clear_has_kernel(uint8_t* __restrict__ has, int V) {
  pdl_entry();
  const int v = blockIdx.x * 256 + threadIdx.x;
  if (v < V) has[v] = 0;
}

// Block q: chunk c = q / cols of the sorted positions, words [128 j, 128 j +
// 128), j = q % cols, of the rows.  Flags the rows that have a token and, for a
// whole chunk of one token, leaves the sum of its rows in part[c].
__global__ void __launch_bounds__(128) embedding_chunks_kernel(const uint32_t* __restrict__ keys,
                                                               const int32_t* __restrict__ pos, int n, int V, int words,
                                                               int cols, const uint4* __restrict__ dy,
                                                               uint8_t* __restrict__ has, float* __restrict__ part) {
  pdl_entry();
  const int chunk = blockIdx.x / cols, col = blockIdx.x % cols;
  const int i0 = chunk * kChunk, tid = threadIdx.x;
  const int end = min(n, i0 + kChunk);
  if (col == 0 && i0 + tid < end) {
    const uint32_t k = keys[i0 + tid];
    if (k < static_cast<uint32_t>(V)) has[k] = 1;
  }
  const uint32_t k0 = keys[i0], k1 = keys[end - 1];
  if (end - i0 < kChunk || k0 != k1 || k0 >= static_cast<uint32_t>(V)) return;
  const int c = col * 128 + tid;
  if (c >= words) return;
  float a[8] = {};
  #pragma unroll
  for (int r0 = 0; r0 < kChunk; r0 += 8) {
    uint4 d[8];
    #pragma unroll
    for (int r = 0; r < 8; ++r) d[r] = dy[static_cast<long long>(pos[i0 + r0 + r]) * words + c];
    #pragma unroll
    for (int r = 0; r < 8; ++r) add_row8(a, d[r]);
  }
  store8(part + (static_cast<long long>(chunk) * words + c) * 8, a);
}

// Two kinds of blocks, taking turns as long as there are both.  One, (b, j):
// the rows whose runs begin at sorted positions [4 b, 4 b + 4), words [128 j,
// 128 j + 128).  The batch's rows of dy (and of base) are loaded together; a run
// that goes on past it is followed through the positions up to the next chunk,
// the sums of the whole chunks, and the positions in the chunk where it ends --
// so a block reads at most 63 rows of dy, however often a token occurs.  The
// other fills those of rows_each rows that have no token.  64 registers and so
// 32 warps on an SM: with batches of 8 and 114 registers the filling blocks
// were too few (1003 tokens, 50001 x 1024: 70 us, against 61).
constexpr int kBatch = 4;
constexpr int kFollow = 6;              // a followed run's rows of dy on their way at a time
__global__ void __launch_bounds__(128, 8) embedding_rows_kernel(const uint32_t* __restrict__ keys,
                                                                const int32_t* __restrict__ pos, int n, int V,
                                                                int words, int cols, int run_blocks,
                                                                const uint4* __restrict__ dy,
                                                                const uint8_t* __restrict__ has,
                                                                const float4* __restrict__ part, int rows_each,
                                                                const uint4* __restrict__ base, float scale,
                                                                float* __restrict__ dtable) {
  pdl_entry();
  const int tid = threadIdx.x;
  int block = blockIdx.x;
  {
    const int turns = min(run_blocks, static_cast<int>(gridDim.x) - run_blocks);
    bool fills = run_blocks == turns;                  // the kind that is left after the turns
    if (block < 2 * turns) {
      fills = block & 1;
      block >>= 1;
    } else {
      block -= turns;
    }
    if (fills) {
      const long long v0 = static_cast<long long>(block) * rows_each;
      if (words <= kNarrow) {
        narrow_rows(static_cast<int>(min(static_cast<long long>(rows_each), V - v0)), words, [&](int r, int c) {
          if (has[v0 + r] != 0) return;
          float a[8] = {};
          if (base != nullptr) add_row8(a, base[(v0 + r) * words + c]);
          store8(dtable + ((v0 + r) * words + c) * 8, a);
        });
        return;
      }
      // two rows a warp, or (wide rows) a quarter of two rows
      const int warp = tid >> 5, apart = words < 512 ? 4 : 1;
      const int quarter = (words + 3) / 4, begin = apart == 4 ? 0 : warp * quarter;
      for (int r = apart == 4 ? warp : 0; r < rows_each; r += 2 * apart) {
        const long long v[2] = {v0 + r, v0 + r + apart};
        const bool fill[2] = {v[0] < V && has[v[0]] == 0, r + apart < rows_each && v[1] < V && has[v[1]] == 0};
        fill_rows(v, fill, words, begin, apart == 4 ? words : min(words, begin + quarter), base, dtable);
      }
      return;
    }
  }
  const int c_ = block % cols * 128 + tid;
  block /= cols;
  const int i0 = block * kBatch, len = min(n - i0, kBatch);
  const bool mine = c_ < words;           // (the other lanes of the last warp go along: they share the lookups)
  const int c = mine ? c_ : 0, lane = tid & 31;
  const uint32_t none = static_cast<uint32_t>(V);   // keys from here on are no token
  uint32_t key[kBatch];
  int at[kBatch];
  const uint32_t before = i0 > 0 ? keys[i0 - 1] : 0xffffffffu;
  #pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    key[u] = u < len ? keys[i0 + u] : none;
    at[u] = u < len ? pos[i0 + u] : 0;
  }
  float a[8] = {};
  auto row_out = [&](uint32_t v, const uint4& b) {
    #pragma unroll
    for (int j = 0; j < 8; ++j) a[j] *= scale;
    add_row8(a, b);
    if (mine) store8(dtable + (static_cast<long long>(v) * words + c) * 8, a);
    #pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = 0.f;
  };
  auto whole = [&](int i, uint32_t k) { return i % kChunk == 0 && i + kChunk <= n && keys[i + kChunk - 1] == k; };
  uint4 d[kBatch], b[kBatch];
  #pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    d[u] = b[u] = make_uint4(0, 0, 0, 0);
    const bool begins = key[u] < none && key[u] != before;   // (its run begins in this batch)
    if (begins) d[u] = dy[static_cast<long long>(at[u]) * words + c];
    if (begins && base != nullptr && (u == 0 || key[u] != key[u - 1]))
      b[u] = base[static_cast<long long>(key[u]) * words + c];
  }
  uint32_t cur = none;                    // the run being summed (none: not yet one that begins here)
  uint4 cur_base = make_uint4(0, 0, 0, 0);
  int i = i0 + len;                       // where it goes on
  if (key[0] < none && key[0] != before && whole(i0, key[0])) {
    cur = key[0];                         // (a whole chunk: by its sum, below)
    cur_base = b[0];
    i = i0;
  } else {
    #pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (key[u] != before && key[u] != cur) {
        if (cur < none) row_out(cur, cur_base);
        cur = key[u];
        cur_base = b[u];
      }
      if (cur < none && key[u] == cur) add_row8(a, d[u]);
    }
  }
  if (cur >= none) return;
  // Positions up to `stop`, at most a chunk further (one lookup: a lane each);
  // false where the run ends before.
  auto follow = [&](int stop) {
    const uint32_t k = i + lane < stop ? keys[i + lane] : none;
    const int p = i + lane < stop ? pos[i + lane] : 0;
    const int count = __popc(__ballot_sync(kFull, k == cur));     // (sorted: the first ones)
    for (int r = 0; r < count; r += kFollow) {
      uint4 e[kFollow];
      #pragma unroll
      for (int u = 0; u < kFollow; ++u) {
        const int row = __shfl_sync(kFull, p, (r + u) & 31);
        if (r + u < count) e[u] = dy[static_cast<long long>(row) * words + c];
      }
      #pragma unroll
      for (int u = 0; u < kFollow; ++u)
        if (r + u < count) add_row8(a, e[u]);
    }
    i += count;
    return i == stop;
  };
  if (follow(min(n, (i + kChunk - 1) / kChunk * kChunk))) {
    // whole chunks, 32 looked up at a time, then the chunk it ends in
    for (int more = 32; more == 32;) {
      const int chunk = i / kChunk;
      const long long last = static_cast<long long>(chunk + lane + 1) * kChunk - 1;
      more = __popc(__ballot_sync(kFull, last < n && keys[last] == cur));
      for (int r = 0; r < more; r += 4) {
        float4 q[4][2];
        #pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (r + u < more) {
            const float4* src = part + (static_cast<long long>(chunk + r + u) * words + c) * 2;
            q[u][0] = src[0];
            q[u][1] = src[1];
          }
        }
        #pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (r + u < more) {
            a[0] += q[u][0].x; a[1] += q[u][0].y; a[2] += q[u][0].z; a[3] += q[u][0].w;
            a[4] += q[u][1].x; a[5] += q[u][1].y; a[6] += q[u][1].z; a[7] += q[u][1].w;
          }
        }
      }
      i += more * kChunk;
    }
    follow(min(n, i + kChunk));
  }
  row_out(cur, cur_base);
}

// ---------------------------------------------------------------- workspace
struct Ws {
  size_t keys[2], pos[2], hist, has, part, total;
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
  w.hist = take((N + kSortTile - 1) / kSortTile * kBins * 4);
  w.has = take(V);
  w.part = take(N / kChunk * H * 4);
  w.total = off;
  return w;
}

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// Once per device: the sorts' shared memory.
cudaError_t sort_attr() {
  static std::atomic<bool> set[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(cluster_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sort_smem(kClusterSort, kCluster)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(block_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sort_smem(kBlockSort, 1)));
  if (e == cudaSuccess) set[dev].store(true, std::memory_order_release);
  return e;
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
  const int words = H / 8;
  const bool wide = words > 256;
  int lanes = 128;
  while (!wide && lanes / 2 >= words) lanes /= 2;
  const int per_block = wide ? 1 : 4 * (128 / lanes);
  return status_of(launch_k(wide ? embedding_fwd_kernel<true> : embedding_fwd_kernel<false>,
                            (n + per_block - 1) / per_block, 128, 0, static_cast<cudaStream_t>(stream), tokens, n,
                            static_cast<const uint4*>(table), V, words, lanes, scale, static_cast<uint4*>(out),
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
  const int words = H / 8;
  const uint4* b16 = static_cast<const uint4*>(base);
  const int cols = (words + 127) / 128;
  if (n <= kFewTokens) {
    // 64 KB a block, less where that would leave SMs without a block
    const int wide = words < 128 ? words : 128;
    const int even = static_cast<int>((static_cast<long long>(V) * cols + 1215) / 1216);
    const int rows = even < 4 ? 4 : even < 65536 / (wide * 32) ? even : 65536 / (wide * 32);
    const int blocks = (V + rows - 1) / rows;
    count_launches(1);
    return status_of(launch_k(embedding_few_kernel, dim3(blocks, cols), 128, (V / blocks + 32) / 32 * 4 + 4, st, tokens, n,
                              V, words, static_cast<const uint4*>(dy), b16, scale, dtable, status));
  }
  uint8_t* has = at<uint8_t>(ws, w.has);
  int passes = 1;                                    // digits of the keys 0 .. V
  while (passes * kDigitBits < 32 && (V >> (passes * kDigitBits)) != 0) ++passes;
  int cur = 0, launches = 0;
  if (n <= kClusterSort) {
    if (sort_attr() != cudaSuccess) return MOE_ERR_CUDA;
    const int clear = (V + kClearRows - 1) / kClearRows, blocks = n <= kBlockSort ? 1 : kCluster;
    if (launch_k(blocks == 1 ? block_sort_kernel : cluster_sort_kernel,
                 blocks + (clear + blocks - 1) / blocks * blocks, kClusterThreads, sort_smem(n, blocks), st, tokens, n,
                 V, passes, at<uint32_t>(ws, w.keys[0]), at<int32_t>(ws, w.pos[0]), has, status) != cudaSuccess)
      return MOE_ERR_CUDA;
    launches = 1;
  } else {
    int32_t* hist = at<int32_t>(ws, w.hist);
    const int tiles = (n + kSortTile - 1) / kSortTile;
    if (launch_k(clear_has_kernel, (V + 255) / 256, 256, 0, st, has, V) != cudaSuccess) return MOE_ERR_CUDA;
    for (int pass = 0; pass < passes; ++pass) {
      const uint32_t* keys = pass == 0 ? nullptr : at<uint32_t>(ws, w.keys[cur]);
      const int32_t* pos = pass == 0 ? nullptr : at<int32_t>(ws, w.pos[cur]);
      const int to = pass == 0 ? 0 : cur ^ 1, shift = pass * kDigitBits;
      if (launch_k(sort_hist_kernel, tiles, kSortThreads, 0, st, tokens, keys, n, V, shift, hist, status) !=
              cudaSuccess ||
          launch_k(sort_scatter_kernel, tiles, kSortThreads, 0, st, tokens, keys, pos, n, V, shift, hist,
                   at<uint32_t>(ws, w.keys[to]), at<int32_t>(ws, w.pos[to])) != cudaSuccess)
        return MOE_ERR_CUDA;
      cur = to;
    }
    launches = 1 + 2 * passes;
  }
  const uint32_t* keys = at<uint32_t>(ws, w.keys[cur]);
  const int32_t* pos = at<int32_t>(ws, w.pos[cur]);
  const uint4* dy16 = static_cast<const uint4*>(dy);
  const long long sums = static_cast<long long>((n + kChunk - 1) / kChunk) * cols;
  const long long runs = static_cast<long long>((n + kBatch - 1) / kBatch) * cols;
  // rows one block fills: 64 KB, less where that would leave SMs without a block
  int fill_rows = words * 32 >= 65536 ? 1 : 65536 / (words * 32);
  if (fill_rows > (V + 1215) / 1216) fill_rows = (V + 1215) / 1216 < 4 ? 4 : (V + 1215) / 1216;
  const long long fills = (static_cast<long long>(V) + fill_rows - 1) / fill_rows;
  if (sums > 0) {
    if (launch_k(embedding_chunks_kernel, static_cast<unsigned>(sums), 128, 0, st, keys, pos, n, V, words, cols, dy16,
                 has, at<float>(ws, w.part)) != cudaSuccess)
      return MOE_ERR_CUDA;
    ++launches;
  }
  if (runs + fills > 0) {
    if (launch_k(embedding_rows_kernel, static_cast<unsigned>(runs + fills), 128, 0, st, keys, pos, n, V, words, cols,
                 static_cast<int>(runs), dy16, has, at<float4>(ws, w.part), fill_rows, b16, scale,
                 dtable) != cudaSuccess)
      return MOE_ERR_CUDA;
    ++launches;
  }
  count_launches(launches);
  return MOE_OK;
}

}  // extern "C"
