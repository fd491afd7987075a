// Causal attention over packed sequences with grouped heads, and its gradient.
//
//   o[i] = sum_j p[i, j] v[j],  p[i, j] = exp(scale <q[i], k[j]> - lse[i]),  start(i) <= j <= i,
//   lse[i] = log sum_j exp(scale <q[i], k[j]>);
//   delta[i] = <do[i], o[i]>,  ds[i, j] = p[i, j] (<do[i], v[j]> - delta[i]),
//   dv[j] = sum_i p[i, j] do[i],  dk[j] = scale sum_i ds[i, j] q[i],  dq[i] = scale sum_j ds[i, j] k[j],
//
// start(i): the first row of row i's sequence.  The rows are cut into tiles of 128
// whatever the sequences: a tile's keys are the rows from its first row's start to its
// own last one, and what a row does not see is masked.  So the tile list needs the
// number of rows alone, which the host knows, and each CTA reads from cu_seqlens where
// its own rows' sequences begin and end (row_map, find_map).  A key tile ends where the row
// tile does, so each row finds its own key in the first tile it meets and its
// maximum is finite from then on.
//
// Every product is a tcgen05.mma on 128-row tiles that TMA brings (zeros outside
// the tensor and past the head's width); a warp or two issue them, and eight (forward) or
// sixteen warps work on the scores in TMEM.
//
// Measured at 8192 rows of one sequence, 32/8 heads of 128 (a library's bf16 product of 8192 x 8192 x 8192: 1927
// TFLOP/s): forward 326 us (1687), gradients 1080 (1273, of five products; the two kernels compute seven, of which
// the scores and dp twice).  Eight packed sequences of 1 to 3907 rows: 144 and 458 us.  Heads of 64, 32768 rows, 8/1
// heads: forward 890 us (1235).  One row: 6.6 us.
//
// Rounded between the products, as operands of the tensor cores have to be: the probabilities (relative to a
// reference within 2^8 of their maximum; the sum that divides them is of the fp32 values), p for dv, ds for dq and
// dk.  Each is off by 2^-8 of itself at most, independently, which leaves out 2.0e-3 and the gradients 2.4e-3
// off as a whole, of which the results' own rounding is 1.5e-3 and 1.7e-3.  In two parts, as the statistics below,
// they would double the products.
//
// Values that are not finite: a product with a probability of zero is still a NaN
// on the tensor cores.  Where a tile has masked places the operand along the
// contraction is therefore looked through first, and what is not finite there is
// put to zero (clean_tile); the forward gives it back at the end to the rows that do see it.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <type_traits>

#include "entry_checks.h"
#include "gemm_common.h"

namespace moe {
namespace {

constexpr int kRows = 128;                 // rows of a tile
constexpr int kMaxSmem = 232448;
// Warps that work on the scores, then four more, of which one loads and one issues the products.
constexpr int kFwdArith = 256, kFwdThreads = kFwdArith + 128;
constexpr int kBwdArith = 512, kBwdThreads = kBwdArith + 128;
constexpr int kParts = kBwdArith / kRows;  // gradients: threads that share a row, 32 columns each
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kMaxTokens = 1 << 24, kMaxHeads = 1024, kMaxHeadDim = 128, kMaxSequences = 1 << 24;
constexpr float kMinScale = 0x1p-64f;      // (lse / scale and score * scale stay in fp32's range)

struct Heads {                             // [T, heads, D] bf16, strides in elements
  __nv_bfloat16* p;
  long long token, head;
};

struct AttnParams {
  const int32_t* cu;       // [B + 1]
  int B, T, Hq, Hkv, D;
  float scale, scale2;     // scale, scale * log2 e
  int mode;                // forward: what an item's tiles of 128 rows are (kTwoHeads, kTwoTiles, kOneTile)
  int tiles;               // tiles along the rows
  int split;               // dk, dv: CTAs that share a group's heads
  Heads q, o, d0, d1;      // forward: q, out, v; gradients: dq or dk, dv
  float* lse;              // [Hq, T]
  uint4* stats;            // [2][Hq, pitch]: -lse / scale, -delta, each as eight bf16 (split_row)
  long long pitch;
  int* status;
  unsigned long long wait_ns;
};

// Registers move from the warps that load and issue to those that work on the scores; the block is
// launched with as many as a thread of it can have.
constexpr int kFwdRegs = 216, kFwdOtherRegs = 72, kBwdRegs = 104, kBwdOtherRegs = 64;
static_assert(kFwdArith * kFwdRegs + 128 * kFwdOtherRegs <= kFwdThreads * 168, "registers of a block");
static_assert(kBwdArith * kBwdRegs + 128 * kBwdOtherRegs <= kBwdThreads * 96, "registers of a block");
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// A value that is the same in all lanes, known as such to the compiler.
template <class T>
__device__ __forceinline__ T uniform(T v) { return __shfl_sync(0xffffffffu, v, 0); }

// Whether what a kernel keeps in shared memory ends inside what it was given.
__device__ __forceinline__ bool smem_fits(const uint8_t* base, const void* end) {
  uint32_t given;
  asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(given));
  return static_cast<const uint8_t*>(end) <= base + given;
}

// ---------------------------------------------------------------- sequences
// Where the sequences of rows r0 .. r0 + R - 1 begin and end.
struct RowMap {
  int first, last;         // rows of any sequence: [first, last)
  int start, end;          // of the sequence of row r0 (last boundary <= r0); next boundary past the rows
  uint32_t bits[8];        // boundaries at r0 + 1 .. r0 + R - 1
};

// All threads of the CTA; one pass over cu_seqlens with independent loads, however
// many sequences.  Boundaries that do not ascend or lie outside [0, T] leave the
// ranges inside [0, T] all the same.
template <int R>
__device__ __forceinline__ void row_map(const AttnParams& p, int r0, RowMap* m) {
  int c = static_cast<int>(threadIdx.x) <= p.B ? p.cu[threadIdx.x] : 0;     // (on its way across the barrier)
  if (threadIdx.x < 8) m->bits[threadIdx.x] = 0u;
  if (threadIdx.x == 0) {
    m->start = 0;
    m->end = p.T;
    m->first = max(c, 0);
  }
  __syncthreads();
  int lo = 0, hi = p.T;
  for (int i = threadIdx.x; i <= p.B; i += blockDim.x) {
    if (i != static_cast<int>(threadIdx.x)) c = p.cu[i];
    if (i == p.B) m->last = min(c, p.T);
    if (c <= r0)
      lo = max(lo, c);
    else if (c >= r0 + R)
      hi = min(hi, c);
    else
      atomicOr(&m->bits[(c - r0) >> 5], 1u << ((c - r0) & 31));
    if (blockIdx.x == 0 && (c < 0 || c > p.T || (i > 0 && p.cu[i - 1] > c))) set_status(p.status, kErrBadIndex);
  }
  lo = __reduce_max_sync(kFull, lo);
  hi = __reduce_min_sync(kFull, hi);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&m->start, lo);
    atomicMin(&m->end, hi);
  }
  __syncthreads();
}
__device__ __forceinline__ int start_of(const RowMap* m, int r0, int row) {
  const int off = row - r0;
  uint32_t b = m->bits[off >> 5] & (0xffffffffu >> (31 - (off & 31)));
  for (int w = off >> 5;;) {
    if (b != 0) return r0 + 32 * w + 31 - __clz(b);
    if (--w < 0) return m->start;
    b = m->bits[w];
  }
}
__device__ __forceinline__ int end_of(const RowMap* m, int r0, int row, int words) {
  const int off = row - r0;
  uint32_t b = m->bits[off >> 5] & (0xfffffffeu << (off & 31));
  for (int w = off >> 5;;) {
    if (b != 0) return r0 + 32 * w + __ffs(b) - 1;
    if (++w >= words) return m->end;
    b = m->bits[w];
  }
}

// The same by one warp, for kernels whose CTAs work through many tiles: the boundaries ascend, so a search by 32 at
// a time finds the last one at or before r0.  mine: boundary number `lane`, or INT_MAX past the last.
template <int R>
__device__ __forceinline__ void find_map(const AttnParams& p, int r0, int mine, int first, int last, RowMap* m) {
  const int lane = threadIdx.x & 31;
  if (lane < 8) m->bits[lane] = 0u;
  __syncwarp();
  int at = 0, n = p.B + 1;                 // it is the first of these n, or further on among them (or there is none)
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int k = __popc(__ballot_sync(kFull, lane * step < n && p.cu[at + lane * step] <= r0));
    if (k == 0) break;
    at += (k - 1) * step;
    n = min(step, n - (k - 1) * step);
  }
  int lo = 0, hi = p.T;
  for (int i = at + lane;; i += 32) {
    const bool in = i <= p.B;
    const int c = i == lane ? mine : in ? p.cu[i] : INT_MAX;
    if (c <= r0)
      lo = max(lo, c);
    else if (c >= r0 + R)
      hi = min(hi, c);
    else
      atomicOr(&m->bits[(c - r0) >> 5], 1u << ((c - r0) & 31));
    if (__any_sync(kFull, !in || c >= r0 + R)) break;
  }
  lo = __reduce_max_sync(kFull, lo);
  hi = __reduce_min_sync(kFull, hi);
  if (lane == 0) {
    m->first = first;
    m->last = last;
    m->start = lo;
    m->end = hi;
  }
  __syncwarp();
}
// Boundaries that do not ascend or lie outside [0, T] are reported; a warp of each CTA, its share.
__device__ __forceinline__ void check_boundaries(const AttnParams& p) {
  const int lane = threadIdx.x & 31, step = static_cast<int>(gridDim.x) * 32;
  for (int i = static_cast<int>(blockIdx.x) * 32 + lane; i <= p.B; i += step) {
    const int c = p.cu[i];
    if (c < 0 || c > p.T || (i > 0 && p.cu[i - 1] > c)) set_status(p.status, kErrBadIndex);
  }
}
// The next of `items` for one of `grid` CTAs, each of which began with the one of its own number and takes them until
// there is none: of as many takes as items the last puts the counter back to zero.
__device__ __forceinline__ int take_item(int* status, int items, int grid) {
  const int before = atomicAdd(status + kAttentionItemWord, 1);
  if (before == items - 1) atomicExch(status + kAttentionItemWord, 0);
  return before + grid;
}

// A count over all of a CTA's items, of which only places and phases are asked for: stages and barriers come round
// after 16, 6, 4 or 2, so 48 may be taken off (kept above the first round, and from overflowing in very long calls).
__device__ __forceinline__ int wrapped(int count) { return count < 96 ? count : 48 + count % 48; }

// Bits lo .. hi of 32: the columns that a row sees.  (As bits: a comparison with each end takes three
// instructions a place, of a kind that the SM starts every other cycle.)
__device__ __forceinline__ uint32_t seen(int lo, int hi) {
  const uint32_t from = lo <= 0 ? ~0u : lo > 31 ? 0u : ~0u << lo, to = hi >= 31 ? ~0u : hi < 0 ? 0u : ~(~1u << hi);
  return from & to;
}

// 32 values of a row: zero where it does not see.
__device__ __forceinline__ void blank(uint32_t (&v)[32], uint32_t on) {
  #pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!(on >> x & 1u)) v[x] = 0u;
}

// ---------------------------------------------------------------- tiles
template <int DP>
struct Tile {
  static constexpr int kBytes = kRows * DP * 2;
  static constexpr int kChunk = kRows * 128;           // 64 columns of all rows, 128-byte swizzled
  static constexpr int kStages = DP == 128 ? 4 : 8;    // forward: key and value tiles in flight
  static constexpr int kBuffers = DP == 128 ? 2 : 3;   // forward: of scores in TMEM
  static constexpr uint32_t kScores = idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t kSums = idesc_bf16_f32(128, DP, false, true);
};

template <int DP>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int row) {
  #pragma unroll
  for (int c = 0; c < DP / 64; ++c) tma_load_3d(dst + c * Tile<DP>::kChunk, map, bar, 64 * c, head, row);
}

// The warp that issues the products runs converged, one lane issuing (mma_bf16_ss_warp).
// Descriptors of a tile's first rows and columns: as the operand of the scores (columns along the
// contraction) and of the sums (rows along it).
__device__ __forceinline__ uint64_t scores_desc(const uint8_t* tile) {
  return smem_desc_sw128(smem_u32(tile), 16, 1024);
}
__device__ __forceinline__ uint64_t sums_desc(const uint8_t* tile) {
  return smem_desc_sw128(smem_u32(tile), kRows * 128, 1024);
}

// Descriptor of 128 rows of 16 columns, not swizzled: the first eight columns as 16 bytes a row at
// `rows`, the other eight at `rest`, further on.
__device__ __forceinline__ uint64_t rows_desc(const uint8_t* rows, const uint8_t* rest) {
  return static_cast<uint64_t>((smem_u32(rows) & 0x3FFFFu) >> 4) |
         static_cast<uint64_t>((smem_u32(rest) - smem_u32(rows)) >> 4) << 16 |   // between the two halves
         static_cast<uint64_t>(128u >> 4) << 32 |                               // between groups of eight rows
         static_cast<uint64_t>(1) << 46;                                        // descriptor version for tcgen05
}

// D[128 x 128] = A[128 rows, DP] B[128 rows, DP]^T
template <int DP>
__device__ __forceinline__ void mma_scores(uint32_t leader, uint32_t d, uint64_t a, uint64_t b) {
  #pragma unroll
  for (int c = 0; c < DP / 64; ++c)
    #pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint64_t off = (c * Tile<DP>::kChunk + kk * 32) >> 4;
      mma_bf16_ss_warp(leader, d, a + off, b + off, Tile<DP>::kScores, (c | kk) != 0 ? 1u : 0u);
    }
}

// D[128 x DP] (+)= W[128 x 128] B[128 rows, DP], W in TMEM as one thread's packed values after the other's: SPAN steps
// of 16 rows along the contraction side by side, the next ones 16 SPAN columns further (where the
// thread's scores were); steps [from, to) of eight.
template <int DP, int SPAN>
__device__ __forceinline__ void mma_sums(uint32_t leader, uint32_t d, uint32_t w, uint64_t b, bool add, int from = 0,
                                         int to = 8) {
  #pragma unroll
  for (int kk = from; kk < to; ++kk)
    mma_bf16_ts_warp(leader, d, w + kk / SPAN * (16 * SPAN) + kk % SPAN * 8, b + kk * (2048 >> 4), Tile<DP>::kSums,
                     (add || kk != 0) ? 1u : 0u);
}

// Words t, t + n, ... of a tile: what is not finite becomes zero, after found().
template <int DP, class F>
__device__ __forceinline__ void clean_tile(uint8_t* tile, int t, int n, F found) {
  uint4* w = reinterpret_cast<uint4*>(tile);
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  __nv_bfloat162 acc[2] = {zero, zero};
  auto add = [&](int k, uint32_t v) { acc[k] = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&v), zero, acc[k]); };
  #pragma unroll 8
  for (int i = t; i < Tile<DP>::kBytes / 16; i += n) {
    const uint4 v = w[i];
    add(0, v.x);
    add(1, v.y);
    add(0, v.z);
    add(1, v.w);
  }
  const __nv_bfloat162 all = __hadd2(acc[0], acc[1]);
  if ((*reinterpret_cast<const uint32_t*>(&all) & 0x7fff7fffu) == 0) return;      // (a sum of zeros)
  found();
  auto part = [](uint32_t v) {
    if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
    if ((v & 0x7f800000u) == 0x7f800000u) v &= 0x0000ffffu;
    return v;
  };
  for (int i = t; i < Tile<DP>::kBytes / 16; i += n) {
    const uint4 v = w[i];
    w[i] = make_uint4(part(v.x), part(v.y), part(v.z), part(v.w));
  }
  fence_proxy_async_smem();
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float as_f(uint32_t v) { return __uint_as_float(v); }

// A converged warp's wait.  It returns when the phase is complete, or when a wait of the block has given up: the
// warp then goes through the rest of its loops, whose waits all return, on whatever the buffers hold, and
// what it leaves behind does not count (MOE_ERR_TIMEOUT).  A vote whether to go on would double its 60 cycles.
__device__ __forceinline__ void warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned long long ns) {
  mbar_wait(bar, parity, abort, ns);
  __syncwarp();
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  tc_fence_before_sync();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Loads that may still be on their way when a warp has given up: the last parity of each barrier.
struct Issued {
  uint32_t mask = 0, parity = 0;
  __device__ __forceinline__ void note(int slot, uint32_t ph) {
    mask |= 1u << slot;
    parity = (parity & ~(1u << slot)) | (ph << slot);
  }
  __device__ __forceinline__ void drain(uint64_t* bars) const {
    for (int s = 0; s < 32; ++s)
      if (mask >> s & 1u) mbar_wait_drain(bars + s, parity >> s & 1u);
  }
};

// 32 columns of a warp's 32 rows, a row a thread, rounded: through 2 KB of shared memory, so that a row's 64 bytes
// leave together.  `out`: the first row; rows: which of them are stored; columns from D on are not.
__device__ __forceinline__ void store_cols(uint8_t* staging, __nv_bfloat16* out, long long stride, uint32_t rows,
                                           int col, int D, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  uint4* s = reinterpret_cast<uint4*>(staging);
  #pragma unroll
  for (int w = 0; w < 4; ++w)
    s[lane * 4 + (w ^ (lane >> 1 & 3))] =
        make_uint4(pack_bf16x2(v[8 * w], v[8 * w + 1]), pack_bf16x2(v[8 * w + 2], v[8 * w + 3]),
                   pack_bf16x2(v[8 * w + 4], v[8 * w + 5]), pack_bf16x2(v[8 * w + 6], v[8 * w + 7]));
  __syncwarp();
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2), w = lane & 3;
    if ((rows >> r & 1u) && col + 8 * w < D)
      *reinterpret_cast<uint4*>(out + r * stride + col + 8 * w) = s[r * 4 + (w ^ (r >> 1 & 3))];
  }
  __syncwarp();
}

// A warp's 32 rows of 64 columns in shared memory, rounded, the 16-byte words of a row turned round by its number:
// a row a thread going in, whole rows after one another coming out.
__device__ __forceinline__ uint4* staged_word(uint8_t* staging, int r, int w) {
  return reinterpret_cast<uint4*>(staging) + r * 8 + (w ^ (r & 7));
}
__device__ __forceinline__ void put_cols(uint8_t* staging, int r, int col, const float (&v)[32]) {
  #pragma unroll
  for (int w = 0; w < 4; ++w)
    *staged_word(staging, r, col / 8 + w) =
        make_uint4(pack_bf16x2(v[8 * w], v[8 * w + 1]), pack_bf16x2(v[8 * w + 2], v[8 * w + 3]),
                   pack_bf16x2(v[8 * w + 4], v[8 * w + 5]), pack_bf16x2(v[8 * w + 6], v[8 * w + 7]));
}
// Eight columns of a row of values: what is not finite among them is added to the row's sums; true: these are all NaN.
__device__ __forceinline__ bool give_back(uint4* sums, const uint4& v) {
  const uint32_t y[4] = {v.x, v.y, v.z, v.w};
  uint32_t* to = reinterpret_cast<uint32_t*>(sums);
  uint32_t found = 0u, nan = ~0u;
  #pragma unroll
  for (int i = 0; i < 4; ++i) found |= __vcmpeq2(y[i] & 0x7f807f80u, 0x7f807f80u);
  if (found == 0u) return false;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t on = __vcmpeq2(y[i] & 0x7f807f80u, 0x7f807f80u);
    const uint32_t add = (y[i] & on) | (0x80008000u & ~on);                 // (-0 changes nothing)
    const __nv_bfloat162 r =
        __hadd2(*reinterpret_cast<const __nv_bfloat162*>(to + i), *reinterpret_cast<const __nv_bfloat162*>(&add));
    to[i] = *reinterpret_cast<const uint32_t*>(&r);
    nan &= __vcmpgtu2(to[i] & 0x7fff7fffu, 0x7f807f80u);
  }
  return nan == ~0u;
}
// The first D columns of the rows that `rows` names.
__device__ __forceinline__ void store_rows(uint8_t* staging, __nv_bfloat16* out, long long stride, uint32_t rows,
                                           int D) {
  const int lane = threadIdx.x & 31, w = lane & 7;
  #pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 4) {
    const int r = r0 + (lane >> 3);
    if ((rows >> r & 1u) && 8 * w < D)
      *reinterpret_cast<uint4*>(out + r * stride + 8 * w) = *staged_word(staging, r, w);
  }
}

// Lanes a and a ^ M (a without the bit): a's second word against the other's first.
template <int M>
__device__ __forceinline__ void exchange(uint4& first, uint4& second) {
  const bool high = (threadIdx.x & M) != 0;
  const uint4 give = high ? first : second;
  const uint4 got = make_uint4(__shfl_xor_sync(kFull, give.x, M), __shfl_xor_sync(kFull, give.y, M),
                               __shfl_xor_sync(kFull, give.z, M), __shfl_xor_sync(kFull, give.w, M));
  if (high)
    first = got;
  else
    second = got;
}

// ---------------------------------------------------------------- forward
// A CTA has two tiles of 128 query rows, each with four warps, and one stream of key
// and value tiles for both: two heads of a group on the same rows, or (groups of an
// odd size) 256 rows of one head (or one tile, where there are few).  The CTAs stay and take such
// items one after the other: one's outputs are written while the next one's first
// products run.  (A CTA for each lost 14 thousand cycles an item before its first key
// tile and after its last, of 2800 a key tile; this one 9.)  The tensor cores alternate between them: while one
// tile's scores are exponentiated, the other's products run.  TMEM: buffers of scores of
// 128 columns (their first 64 become the probabilities), sums DP columns a tile.
//
// Heads of up to 64 leave room for three buffers, taken in turn by both tiles: a tile's next scores are
// there when it has exponentiated the last ones.  Scores and sums are then issued by a warp
// each (one for both waits for one while the other could go on: 322 us against 264 at 8192 rows,
// 32 heads of 64; with a buffer a tile 300).  Wide heads have a buffer a tile and one issuing warp (two: 0.53 ms
// against 0.41).
//
// What bounds it: a step, one key tile against both tiles of rows, is 2540 cycles at heads of 128, of which the
// tensor cores work 2048.  The rest is the chain of one tile (scores, maximum, exponentials, sums,
// next scores), of which TMEM has room for two.
//
// A barrier that is waited for by parity has to be seen before its next phase ends.  With three buffers a tile's next
// probabilities can be there before the last ones' arrival has been looked at, so their barriers are two, in turns.
// The tiles of an item: two heads of a group on the same rows, 256 rows of one head, or 128 of one.
constexpr int kTwoHeads = 0, kTwoTiles = 1, kOneTile = 2;
struct FwdItem {
  RowMap map;
  int item;                                // -1: no more
  int q0, top, kv;
  int from[2], to[2], base[2], head[2], ib, n;
  int loaded;                              // tiles in the ring: 2 n, or the first ones of an item without rows
  int mixed;                               // 256 rows of one head: key tiles from here on are masked for one half
  int bad_lo, bad_hi;                      // key rows of tiles in which clean_tile found something
};
struct FwdBook {
  uint64_t full[8], q_full;                // (one after the other: Issued counts on it)
  uint64_t empty[8], q_empty, s_full[2][2], p_full[2][2][2], o_full[2], o_empty[2], drain;
  uint64_t free[3];                        // three buffers: the sums that read this one are done
  uint64_t item_full[2], item_empty[2], ending;
  uint32_t tmem;
  int abort_flag;
  FwdItem item[2];
};

constexpr int kFwdLoadWarp = kFwdArith / 32, kFwdMmaWarp = kFwdLoadWarp + 1, kFwdItemWarp = kFwdLoadWarp + 3;
constexpr int kFwdStaging = kFwdArith / 32 * 4096;       // 32 rows of 64 columns a warp

// Item i of the grid: the last tiles first, they have the longest rows of keys.
__device__ __forceinline__ void fwd_place(const AttnParams& p, int i, int& q0, int& first_head) {
  const int per = p.mode == kTwoHeads ? p.Hq / 2 : p.Hq;
  q0 = (p.tiles - 1 - i / per) * (p.mode == kTwoTiles ? 2 * kRows : kRows);
  first_head = i % per * (p.mode == kTwoHeads ? 2 : 1);
}

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attention_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
  using C = Tile<DP>;
  constexpr int ST = C::kStages, L = C::kBuffers;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* q_smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = q_smem + 2 * C::kBytes;
  uint8_t* out_smem = ring + ST * C::kBytes;
  FwdBook& bk = *reinterpret_cast<FwdBook*>(out_smem + kFwdStaging);
  if (!smem_fits(smem_raw, &bk + 1)) {
    pdl_wait();
    if (threadIdx.x == 0) set_status(p.status, kErrLaunch);
    return;
  }
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (warp == kFwdLoadWarp && lane == 0) {          // (it uses them before the first barrier of all threads)
    for (int s = 0; s < 8; ++s) {
      mbar_init(&bk.full[s], 1);
      mbar_init(&bk.empty[s], 1);
    }
    mbar_init(&bk.q_full, 1);
    mbar_init(&bk.q_empty, 1);
    for (int u = 0; u < 2; ++u) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(&bk.s_full[u][x], 1);
        mbar_init(&bk.p_full[u][x][0], 4);
        mbar_init(&bk.p_full[u][x][1], 4);
      }
      mbar_init(&bk.o_full[u], 1);
      mbar_init(&bk.o_empty[u], 4);
      mbar_init(&bk.item_full[u], 1);
      mbar_init(&bk.item_empty[u], 1 + (L == 2 ? 1 : 2) + kFwdArith / 32);      // loads, products, arithmetic
    }
    for (int s = 0; s < 3; ++s) mbar_init(&bk.free[s], 2);      // the scores have been issued, the sums are done
    mbar_init(&bk.ending, 1);
    mbar_init(&bk.drain, L == 2 ? 1 : 2);
    bk.abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == kFwdMmaWarp) {
    tmem_alloc(&bk.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  pdl_wait();

  // The first queries, and where both tiles have the same rows the first keys, do not wait for the sequences'
  // boundaries.
  const bool early = p.mode != kTwoTiles;
  const int filled_by = p.mode == kOneTile ? 1 : 2;           // tiles of queries
  if (warp == kFwdLoadWarp && lane == 0 && early) {
    int q0, h;
    fwd_place(p, blockIdx.x, q0, h);
    mbar_arrive_expect_tx(&bk.q_full, filled_by * C::kBytes);
    for (int u = 0; u < filled_by; ++u) load_tile<DP>(q_smem + u * C::kBytes, &tmQ, &bk.q_full, h + u, q0);
    for (int s = 0; s < 2; ++s) {
      mbar_arrive_expect_tx(&bk.full[s], C::kBytes);
      load_tile<DP>(ring + s * C::kBytes, s ? &tmV : &tmK, &bk.full[s], h / (p.Hq / p.Hkv), q0);
    }
  }
  // Item `item` as number `it` of this CTA, by the item warp; its queries are sent for to the L2.
  int mine = INT_MAX, first_row = 0, last_row = 0;
  auto place = [&](int item, int it) {
    FwdItem& m = bk.item[it & 1];
    int q0, h;
    fwd_place(p, item, q0, h);
    for (int r = it > 0 ? lane : 2 * kRows; r < filled_by * kRows; r += 32) {
      const int row = q0 + (p.mode == kTwoTiles ? r : r & (kRows - 1));
      const int head = h + (p.mode == kTwoTiles ? 0 : r / kRows);
      if (row < p.T) {
        const __nv_bfloat16* q = p.q.p + row * p.q.token + head * p.q.head;
        prefetch_l2(q);
        prefetch_l2(q + p.D - 1);
      }
    }
    find_map<2 * kRows>(p, q0, mine, first_row, last_row, &m.map);
    if (lane == 0) {
      // key tile i: rows [top - 128 (i + 1), top - 128 i); query tile u meets tiles [from[u], to[u])
      const int top = q0 + (p.mode == kTwoTiles ? 2 * kRows : kRows);
      for (int u = 0; u < 2; ++u) {
        const int base = q0 + (p.mode == kTwoTiles ? kRows * u : 0);
        const int a = max(base, first_row), b = min(base + kRows, last_row);
        m.base[u] = base;
        m.head[u] = h + (p.mode == kTwoHeads ? u : 0);
        m.from[u] = p.mode == kTwoTiles ? 1 - u : 0;
        const bool on = a < b && u < filled_by;
        m.to[u] = m.from[u] + (on ? (base + kRows - start_of(&m.map, q0, a) + kRows - 1) / kRows : 0);
      }
      const bool on0 = m.to[0] > m.from[0], on1 = m.to[1] > m.from[1];
      m.ib = on1 ? m.from[1] : m.from[0];
      m.n = (on0 || on1) ? max(m.to[0], m.to[1]) - m.ib : 0;
      m.loaded = m.n > 0 ? 2 * m.n : (early && it == 0 ? 2 : 0);
      // (a boundary between a tile's rows masks their keys in front of it; the second tile's last one is the furthest)
      m.mixed = INT_MAX;
      if (p.mode == kTwoTiles && on1)
        m.mixed = (top - start_of(&m.map, q0, min(m.base[1] + kRows, last_row) - 1)) / kRows;
      m.q0 = q0;
      m.top = top;
      m.kv = h / (p.Hq / p.Hkv);
      m.bad_lo = INT_MAX;
      m.bad_hi = -1;
      m.item = item;
    }
    __syncwarp();
  };
  if (warp == kFwdItemWarp) {
    if (lane <= p.B) mine = p.cu[lane];     // (the first boundaries stay with it)
    const int begin = p.B < 32 ? __shfl_sync(kFull, mine, 0) : p.cu[0];
    const int end = p.B < 32 ? __shfl_sync(kFull, mine, p.B) : p.cu[p.B];
    first_row = max(begin, 0);
    last_row = min(end, p.T);
    place(blockIdx.x, 0);
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = uniform(bk.tmem);
  volatile int* abort = &bk.abort_flag;
  const unsigned long long lim = p.wait_ns;
  // The next item for a role; false: no more (or a wait has given up).
  auto next_item = [&](int it) {
    mbar_wait(&bk.item_full[it & 1], (it >> 1) & 1, abort, lim);
    return *const_cast<volatile int*>(&bk.item[it & 1].item) >= 0 && *abort == 0;
  };

  if (warp >= kFwdLoadWarp) {
   fewer_registers<kFwdOtherRegs>();
   if (warp == kFwdItemWarp) {
    // ------------------------------------------------ the items
    const int items = p.tiles * (p.mode == kTwoHeads ? p.Hq / 2 : p.Hq), grid = gridDim.x;
    int next = blockIdx.x;
    for (int it = 0;; ++it) {
      if (it >= 2) warp_wait(&bk.item_empty[it & 1], ((it >> 1) & 1) ^ 1u, abort, lim);
      if (next >= items || uniform(*abort) != 0) {
        if (lane == 0) {
          bk.item[it & 1].item = -1;
          mbar_arrive(&bk.item_full[it & 1]);
        }
        break;
      }
      if (it > 0) place(next, it);          // (the first one has been placed)
      if (lane == 0) mbar_arrive(&bk.item_full[it & 1]);
      // The next one when this one's last loads have been issued.  (No earlier: a CTA that holds its next item from the
      // start of a long one keeps it from those that end before; 186 us against 156 at sequences of 1 to 3907 rows.)
      warp_wait(&bk.ending, it & 1, abort, lim);
      next = uniform(lane == 0 ? take_item(p.status, items, grid) : 0);
    }
    while (next < items) next = uniform(lane == 0 ? take_item(p.status, items, grid) : 0);      // (given up)
    check_boundaries(p);
   } else if (warp == kFwdLoadWarp) {
    if (lane == 0) {
      Issued got;
      int turn = 0, filled = 0;
      bool go = true;
      if (early) {
        got.note(8, 0);
        got.note(0, 0);
        got.note(1, 0);
      }
      for (int it = 0; go && next_item(it); ++it) {
        const FwdItem& m = bk.item[it & 1];
        const int loaded = m.loaded, ib = m.ib, top = m.top, kv = m.kv;
        if (loaded > 0) {
          const bool here = early && it == 0;
          if (!here) {
            if (filled > 0 && !mbar_wait(&bk.q_empty, (filled - 1) & 1, abort, lim)) break;
            mbar_arrive_expect_tx(&bk.q_full, filled_by * C::kBytes);
            for (int u = 0; u < filled_by; ++u)
              load_tile<DP>(q_smem + u * C::kBytes, &tmQ, &bk.q_full, m.head[u], m.base[u]);
            got.note(8, filled & 1);
          }
          ++filled;
          for (int s = here ? 2 : 0; s < loaded; ++s) {           // key, value, key, ...
            const int slot = (turn + s) % ST;
            const uint32_t ph = ((turn + s) / ST) & 1;
            if (turn + s >= ST && !mbar_wait(&bk.empty[slot], ph ^ 1u, abort, lim)) {
              go = false;
              break;
            }
            mbar_arrive_expect_tx(&bk.full[slot], C::kBytes);
            load_tile<DP>(ring + slot * C::kBytes, (s & 1) ? &tmV : &tmK, &bk.full[slot], kv,
                          top - kRows * (ib + (s >> 1) + 1));
            got.note(slot, ph);
          }
          turn = wrapped(turn + loaded);
          filled = wrapped(filled);
        }
        mbar_arrive(&bk.item_empty[it & 1]);
        mbar_arrive(&bk.ending);
      }
      got.drain(bk.full);                    // (they have landed by the end, unless another warp gave up)
    }
   } else if (warp == kFwdMmaWarp || (L > 2 && warp == kFwdMmaWarp + 1)) {
    const uint32_t leader = elect_one() ? 1u : 0u;
    const uint64_t q_desc = scores_desc(q_smem), k_desc = scores_desc(ring), v_desc = sums_desc(ring);
    // this warp's counts over all items: tiles in the ring, fillings of the queries, key tiles met by each tile of
    // rows, items with rows of each, and the buffer of scores and its round
    int turn = 0, filled = 0, met0 = 0, met1 = 0, outs0 = 0, outs1 = 0;
    uint32_t b = 0;
    int round = 0;
    for (int it = 0; uniform(next_item(it) ? 1 : 0) != 0; ++it) {
      const FwdItem& m = bk.item[it & 1];
      const int f0 = uniform(m.from[0]), f1 = uniform(m.from[1]), e0 = uniform(m.to[0]), e1 = uniform(m.to[1]);
      const int first = uniform(m.ib), n = uniform(m.n), loaded = uniform(m.loaded), last = first + n - 1;
      const int mixed = uniform(m.mixed);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bk.item_empty[it & 1]);
      auto full = [&](int s) { warp_wait(&bk.full[s % ST], (s / ST) & 1, abort, lim); };
      auto release = [&](int s) { mma_commit_warp(leader, &bk.empty[s % ST]); };
      auto scores = [&](int u, int i, uint32_t buffer) {
        if (i > last) return;
        const int s = turn + 2 * (i - first), f = u ? f1 : f0, x = (u ? met1 : met0) + i - f;
        if (u == 0) {
          full(s);
          tc_fence_after_sync();
        }
        if (i >= f && i < (u ? e1 : e0)) {
          mma_scores<DP>(leader, tmem + buffer, q_desc + u * (C::kBytes >> 4), k_desc + (s % ST) * (C::kBytes >> 4));
          mma_commit_warp(leader, &bk.s_full[u][x & 1]);
        }
        if (u == 1) {
          release(s);
          if (i == last) mma_commit_warp(leader, &bk.q_empty);
        }
      };
      // the sums of tile u over value tile i
      auto sums = [&](int u, int i, uint32_t buffer) {
        const int s = turn + 2 * (i - first) + 1, f = u ? f1 : f0, e = u ? e1 : e0, x = (u ? met1 : met0) + i - f;
        if (u == 0) full(s);
        if (i >= f && i < e) {
          const int outs = u ? outs1 : outs0;
          if (i == f && outs > 0) warp_wait(&bk.o_empty[u], (outs - 1) & 1, abort, lim);
          // Where the second tile of rows looks through the value tile (masked there, perhaps not here) the first
          // one's product waits for it: what is not finite shall be there for both or for neither.  (The other way
          // round the first tile's probabilities, which come after its own look, have been waited for.)
          const int x1 = met1 + i - f1;
          const bool both = p.mode == kTwoTiles && u == 0 && i >= f1 && i < e1 && (i == f0 || i >= mixed);
          #pragma unroll 1
          for (int w = both ? 1 : 0; w >= 0; --w) {
            const int y = w ? x1 : x;
            warp_wait(&bk.p_full[w ? 1 : u][y & 1][0], (y >> 1) & 1, abort, lim);
          }
          // (the first half of the keys while the second is still exponentiated)
          #pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (half) warp_wait(&bk.p_full[u][x & 1][half], (x >> 1) & 1, abort, lim);
            tc_fence_after_sync();
            mma_sums<DP, 8>(leader, tmem + 128 * L + DP * u, tmem + buffer, v_desc + (s % ST) * (C::kBytes >> 4),
                            i > f || half, 4 * half, 4 * half + 4);
          }
          if (i + 1 == e) mma_commit_warp(leader, &bk.o_full[u]);
        }
        if (u == 1) release(s);
      };
      if (n == 0) {
        if (loaded > 0 && warp == kFwdMmaWarp) {         // (loaded before it was known that nothing asks for it)
          warp_wait(&bk.q_full, filled & 1, abort, lim);
          mma_commit_warp(leader, &bk.q_empty);
          for (int s = turn; s < turn + loaded; ++s) {
            full(s);
            release(s);
          }
        }
      } else if (L == 2) {
        warp_wait(&bk.q_full, filled & 1, abort, lim);
        scores(0, first, 0);
        scores(1, first, 128);
        for (int i = first; i <= last; ++i) {
          sums(0, i, 0);
          scores(0, i + 1, 0);
          sums(1, i, 128);
          scores(1, i + 1, 128);
        }
      } else if (warp == kFwdMmaWarp) {
        warp_wait(&bk.q_full, filled & 1, abort, lim);
        for (int i = first; i <= last; ++i) {
          #pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (round > 0) warp_wait(&bk.free[b], (round - 1) & 1, abort, lim);
            tc_fence_after_sync();
            scores(u, i, 128 * b);
            // (Without it the warp of the sums, which has nothing to wait for where a tile does not meet the keys,
            // could end a second phase before this one has looked at the first.)
            if (lane == 0) mbar_arrive(&bk.free[b]);
            __syncwarp();
            if (++b == L) {
              b = 0;
              ++round;
            }
          }
        }
      } else {
        for (int i = first; i <= last; ++i) {
          #pragma unroll
          for (int u = 0; u < 2; ++u) {
            sums(u, i, 128 * b);
            mma_commit_warp(leader, &bk.free[b]);
            b = b + 1 == L ? 0 : b + 1;
          }
        }
      }
      turn = wrapped(turn + loaded);
      filled = wrapped(filled + (loaded > 0));
      met0 = wrapped(met0 + e0 - f0);
      met1 = wrapped(met1 + e1 - f1);
      outs0 = wrapped(outs0 + (e0 > f0));
      outs1 = wrapped(outs1 + (e1 > f1));
      round = wrapped(round);
    }
    mma_commit_warp(leader, &bk.drain);      // (TMEM is given back after them, whoever gave up)
    mbar_wait_drain(&bk.drain, 0);
   }
  } else {
   more_registers<kFwdRegs>();
   // ------------------------------------------------ a thread a row
   const int u = warp >> 2;
   const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
   const uint32_t to_ = tmem + 128 * L + DP * u + lanes;
   int turn = 0, met = 0, outs = 0, scored = 0;   // as in the warp that issues; outs: items with rows of this tile
   for (int it = 0; uniform(next_item(it) ? 1 : 0) != 0; ++it) {
    FwdItem& m = bk.item[it & 1];
    const int f = m.from[u], e = m.to[u], ib = m.ib, n = m.n, q0 = m.q0, top = m.top;
    if (e > f) {
     const int r0 = m.base[u], h = m.head[u], kv = m.kv;
     const int row = r0 + (warp & 3) * 32 + lane;
     const bool valid = row >= m.map.first && row < m.map.last;
     const int key_lo = valid ? start_of(&m.map, q0, row) : INT_MIN / 2, key_hi = valid ? row : INT_MAX / 2;
     // keys from here on are seen by every row of the tile (up to the diagonal)
     const int all_from = start_of(&m.map, q0, min(r0 + kRows, m.map.last) - 1);
     // probabilities are relative to a reference that follows the maximum once it is 2^8 above
     const float slack = 8.f / p.scale2;
     float ref = -INFINITY, sum = 0.f;
     uint32_t s[4][32];
     int buffer = (scored + 2 * (f - ib) + u) % L;
     for (int i = f; i < e; ++i) {
      const int x = met + i - f;
      warp_wait(&bk.s_full[u][x & 1], (x >> 1) & 1, abort, lim);
      tc_fence_after_sync();
      const uint32_t ts = tmem + 128 * buffer + lanes;
      if (L > 2) buffer = buffer > 0 ? buffer - 1 : L - 1;      // (two on)
      const int k0 = top - kRows * (i + 1);
      const bool masked = i == f || k0 < all_from;
      #pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_x32(ts + 32 * c, s[c]);
      #pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_wait(s[c]);
      if (masked) {
        #pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t on = seen(key_lo - k0 - 32 * c, key_hi - k0 - 32 * c);
          if (__all_sync(kFull, on == kFull)) continue;
          #pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!(on >> j & 1u)) s[c][j] = 0xff800000u;
        }
        const int at = turn + 2 * (i - ib) + 1;
        warp_wait(&bk.full[at % ST], (at / ST) & 1, abort, lim);
        clean_tile<DP>(ring + (at % ST) * C::kBytes, threadIdx.x & 127, 128, [&] {
          atomicMin(&m.bad_lo, k0);
          atomicMax(&m.bad_hi, k0 + kRows - 1);
          __threadfence_block();                 // (the other tile of rows finds the zeros: it shall know)
        });
      }
      uint32_t w[32];
      // probabilities of half the keys, packed, and their sum
      auto exps = [&](int half) {
        const float off = ref == -INFINITY ? 0.f : -ref * p.scale2;
        const F32x2 off2 = make_f32x2(off, off), mul2_ = make_f32x2(p.scale2, p.scale2);
        F32x2 part[2];
        #pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t(&x)[32] = s[2 * half + c];
          part[c] = make_f32x2(0.f, 0.f);
          #pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 y = split_f32x2(fma2(make_f32x2(as_f(x[2 * j]), as_f(x[2 * j + 1])), mul2_, off2));
            const F32x2 q = make_f32x2(ex2(y.x), ex2(y.y));
            part[c] = add2(part[c], q);
            w[16 * c + j] = pack_bf16x2(q);
          }
        }
        return add2(part[0], part[1]);
      };
      float mx[8];
      #pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t* y = s[c >> 1] + 16 * (c & 1);
        mx[c] = max3(as_f(y[0]), as_f(y[1]), as_f(y[2]));
        #pragma unroll
        for (int j = 3; j < 15; j += 2) mx[c] = max3(mx[c], as_f(y[j]), as_f(y[j + 1]));
      }
      #pragma unroll
      for (int c = 0; c < 8; c += 2) mx[c] = max3(mx[c], as_f(s[c >> 1][15]), as_f(s[c >> 1][31]));
      const float top_ = max3(max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[4]), max3(mx[5], mx[6], mx[7]), ref);
      const bool grow = top_ > ref + slack;
      if (__any_sync(kFull, grow)) {
        const float a = grow ? ex2((ref - top_) * p.scale2) : 1.f;
        if (grow) ref = top_;
        sum *= a;
        if (i > f) {
          // (with two buffers this tile's scores come after the sums so far)
          if (L > 2) {
            const int k = scored + 2 * (i - ib) + u - 2;          // (its sums have to be done)
            warp_wait(&bk.free[k % L], (k / L) & 1, abort, lim);
            tc_fence_after_sync();
          }
          #pragma unroll 1
          for (int c = 0; c < DP / 16; ++c) {
            uint32_t o[16];
            tmem_ld_x16(to_ + 16 * c, o);
            tmem_ld_wait(o);
            #pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(as_f(o[j]) * a);
            tmem_st_x16(to_ + 16 * c, o);
          }
        }
      }
      F32x2 total = exps(0);
      tmem_st_x32(ts, w);
      tmem_st_wait();
      warp_arrive(&bk.p_full[u][x & 1][0], lane);
      total = add2(total, exps(1));
      tmem_st_x32(ts + 32, w);
      tmem_st_wait();
      warp_arrive(&bk.p_full[u][x & 1][1], lane);
      const float2 t = split_f32x2(total);
      sum += t.x + t.y;
     }
     warp_wait(&bk.o_full[u], outs & 1, abort, lim);
     tc_fence_after_sync();
     #pragma unroll
     for (int c = 0; c < DP / 32; ++c) tmem_ld_x32(to_ + 32 * c, s[c]);
     #pragma unroll
     for (int c = 0; c < DP / 32; ++c) tmem_ld_wait(s[c]);
     warp_arrive(&bk.o_empty[u], lane);
     const float inv = 1.f / sum;
     if (valid) p.lse[static_cast<long long>(h) * p.T + row] = (ref == -INFINITY ? 0.f : ref * p.scale) + logf(sum);
     const int bad_lo = *const_cast<volatile int*>(&m.bad_lo), bad_hi = *const_cast<volatile int*>(&m.bad_hi);
     const uint32_t rows = __ballot_sync(kFull, valid);
     uint8_t* staging = out_smem + warp * 4096;
     #pragma unroll
     for (int col = 0; col < DP; col += 64) {
      #pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v[32];
        #pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = as_f(s[col / 32 + c][j]) * inv;
        put_cols(staging, lane, 32 * c, v);
      }
      if (valid) {
        // what clean_tile took out, for the rows that see it; eight columns that are all NaN have seen enough
        uint32_t words = (1u << min((p.D - col) / 8, 8)) - 1u;
        for (int j = max(key_lo, bad_lo); words != 0 && j <= min(key_hi, bad_hi); ++j) {
          const uint4* src = reinterpret_cast<const uint4*>(p.d0.p + j * p.d0.token + kv * p.d0.head + col);
          for (int w = 0; w < 8; ++w)
            if ((words >> w & 1u) && give_back(staged_word(staging, lane, w), src[w])) words &= ~(1u << w);
        }
      }
      __syncwarp();
      store_rows(staging, p.o.p + (row - lane) * p.o.token + h * p.o.head + col, p.o.token, rows, p.D - col);
      __syncwarp();
     }
     outs = wrapped(outs + 1);
    }
    turn = wrapped(turn + m.loaded);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bk.item_empty[it & 1]);
    met = wrapped(met + e - f);
    scored = wrapped(scored + 2 * n);
   }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  pdl_launch_next();
  if (threadIdx.x == 0 && bk.abort_flag) set_status(p.status, kErrTimeout);
  if (warp == kFwdMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- gradients
// Four threads share a row of scores, 32 columns each.  (Two, with half as many warps, left the loop
// waiting for its own latencies a third of the time: a step of dk and dv 2900 cycles, whatever the width.)
constexpr int kBwdLoadWarp = kBwdArith / 32, kBwdMmaWarp = kBwdLoadWarp + 1;

// A value as three bf16 whose sum has its 24 bits, and five zeros.
__device__ __forceinline__ uint4 split_row(float v) {
  const __nv_bfloat16 a = __float2bfloat16(v);
  const float r = v - __bfloat162float(a);
  const __nv_bfloat16 b = __float2bfloat16(r), c = __float2bfloat16(r - __bfloat162float(b));
  const uint32_t lo = __bfloat16_as_ushort(a), hi = __bfloat16_as_ushort(b);
  return make_uint4(lo | hi << 16, __bfloat16_as_ushort(c), 0u, 0u);
}

// dq: 128 query rows of one head against their key tiles, CTAs that stay as in the forward.  TMEM: dq DP columns
// from 0, scores at 128, two buffers of dp at 256 and 384 (each becomes ds).  Both products of the next key
// tile run while this one's ds is worked out, the scores once they have been read.  A step is 1630
// cycles at heads of 128, of which the tensor cores work 1536; an item takes 10 thousand besides (a CTA for each
// took 3 thousand more).
//
// out, for delta, comes through a place of the keys (TMA; read from memory by the threads it
// kept the first step waiting as long).  Sixteen warps work on one step, 32 columns a thread (two
// groups of four, a row a thread, every other step: 1180 us against 1150 for the gradients at 8192 rows).
//
// delta comes from the rounded out, an error of out's rounding in each of its products.  Where a
// row sees few keys that is of the size of ds; rows that begin within their first key tile
// take delta = sum_j p dp there instead.  Either goes to stats, for dk.
constexpr int kKStages = 3;                // key tiles in flight: one is held from its scores to its dq
struct DqItem {
  RowMap map;
  int item, n;                             // item -1: no more; n: key tiles
  int q0, head, kv;
};
struct DqBook {
  uint64_t q_full, k_full[kKStages], v_full[2];              // (one after the other: Issued counts on it)
  uint64_t q_empty, o_read, k_empty[kKStages], v_empty[2], s_full, s_empty, dp_full[2], dp_empty[2], ds_full[2];
  uint64_t out_full, out_empty, drain, item_full[2], item_empty[2], ending;
  uint64_t sums_read, sums_full;           // delta's parts have been read, other parts are in their place
  uint32_t tmem;
  int abort_flag;
  DqItem item[2];
  float sums[kParts][kRows];               // parts of rows' sums
};
constexpr int kBwdItemWarp = kBwdLoadWarp + 3;

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attention_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDo,
                        const __grid_constant__ CUtensorMap tmO, const AttnParams p) {
  using C = Tile<DP>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* q_smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* do_smem = q_smem + C::kBytes;
  uint8_t* k_smem = do_smem + C::kBytes;
  uint8_t* v_smem = k_smem + kKStages * C::kBytes;
  DqBook& bk = *reinterpret_cast<DqBook*>(v_smem + 2 * C::kBytes);
  if (!smem_fits(smem_raw, &bk + 1)) {
    pdl_wait();
    if (threadIdx.x == 0) set_status(p.status, kErrLaunch);
    return;
  }
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (warp == kBwdLoadWarp && lane == 0) {
    mbar_init(&bk.q_full, 1);
    mbar_init(&bk.q_empty, 1 + kBwdArith / 32);              // dp's products, and delta's reads
    mbar_init(&bk.o_read, kBwdArith / 32);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&bk.k_full[s], 1);
      mbar_init(&bk.k_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bk.v_full[s], 1);
      mbar_init(&bk.v_empty[s], 1);
      mbar_init(&bk.dp_full[s], 1);
      mbar_init(&bk.dp_empty[s], 1);
      mbar_init(&bk.ds_full[s], kBwdArith / 32);
      mbar_init(&bk.item_full[s], 1);
      mbar_init(&bk.item_empty[s], 3 + kBwdArith / 32);      // loads, the two that issue, arithmetic
    }
    mbar_init(&bk.s_full, 1);
    mbar_init(&bk.s_empty, kBwdArith / 32);
    mbar_init(&bk.out_full, 1);
    mbar_init(&bk.out_empty, kBwdArith / 32);
    mbar_init(&bk.sums_read, kBwdArith / 32);
    mbar_init(&bk.sums_full, kBwdArith / 32);
    mbar_init(&bk.ending, 1);
    mbar_init(&bk.drain, 2);
    bk.abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
    prefetch_tensormap(&tmDo);
    prefetch_tensormap(&tmO);
  }
  if (warp == kBwdMmaWarp) {
    tmem_alloc(&bk.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  pdl_wait();
  // Item `item` as number `it` of this CTA, by the item warp: the last tiles first, they have the longest rows of keys.
  int mine = INT_MAX, first_row = 0, last_row = 0;
  auto place = [&](int item, int it) {
    DqItem& m = bk.item[it & 1];
    const int q0 = (p.tiles - 1 - item / p.Hq) * kRows, h = item % p.Hq;
    find_map<kRows>(p, q0, mine, first_row, last_row, &m.map);
    if (lane == 0) {
      const int a = max(q0, first_row), b = min(q0 + kRows, last_row);
      m.n = a < b ? (q0 + kRows - start_of(&m.map, q0, a) + kRows - 1) / kRows : 0;
      m.q0 = q0;
      m.head = h;
      m.kv = h / (p.Hq / p.Hkv);
      m.item = item;
    }
    __syncwarp();
  };
  if (warp == kBwdItemWarp) {
    if (lane <= p.B) mine = p.cu[lane];     // (the first boundaries stay with it)
    const int begin = p.B < 32 ? __shfl_sync(kFull, mine, 0) : p.cu[0];
    const int end = p.B < 32 ? __shfl_sync(kFull, mine, p.B) : p.cu[p.B];
    first_row = max(begin, 0);
    last_row = min(end, p.T);
    place(blockIdx.x, 0);
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = uniform(bk.tmem);
  volatile int* abort = &bk.abort_flag;
  const unsigned long long lim = p.wait_ns;
  // The next item for a role; false: no more (or a wait has given up).
  auto next_item = [&](int it) {
    mbar_wait(&bk.item_full[it & 1], (it >> 1) & 1, abort, lim);
    return *const_cast<volatile int*>(&bk.item[it & 1].item) >= 0 && *abort == 0;
  };

  if (warp >= kBwdLoadWarp) {
   fewer_registers<kBwdOtherRegs>();
   if (warp == kBwdItemWarp) {
    // ------------------------------------------------ the items (as in the forward)
    const int items = p.tiles * p.Hq, grid = gridDim.x;
    int next = blockIdx.x;
    for (int it = 0;; ++it) {
      if (it >= 2) warp_wait(&bk.item_empty[it & 1], ((it >> 1) & 1) ^ 1u, abort, lim);
      if (next >= items || uniform(*abort) != 0) {
        if (lane == 0) {
          bk.item[it & 1].item = -1;
          mbar_arrive(&bk.item_full[it & 1]);
        }
        break;
      }
      if (it > 0) place(next, it);          // (the first one has been placed)
      if (lane == 0) mbar_arrive(&bk.item_full[it & 1]);
      warp_wait(&bk.ending, it & 1, abort, lim);
      next = uniform(lane == 0 ? take_item(p.status, items, grid) : 0);
    }
    while (next < items) next = uniform(lane == 0 ? take_item(p.status, items, grid) : 0);      // (given up)
    check_boundaries(p);
   } else if (warp == kBwdLoadWarp) {
    if (lane == 0) {
      Issued got;
      int turn = 0, vturn = 0, live = 0;     // tiles through the stages of k and v, items with rows
      bool go = true;
      for (int it = 0; go && next_item(it); ++it) {
        const DqItem& m = bk.item[it & 1];
        const int n = m.n, q0 = m.q0, h = m.head, kv = m.kv;
        // a place among the keys: for out first, then for them
        auto place_k = [&](const CUtensorMap* map, int head, int row) {
          const int s = turn % kKStages;
          const uint32_t ph = (turn / kKStages) & 1;
          if (turn >= kKStages && !mbar_wait(&bk.k_empty[s], ph ^ 1u, abort, lim)) return false;
          mbar_arrive_expect_tx(&bk.k_full[s], C::kBytes);
          load_tile<DP>(k_smem + s * C::kBytes, map, &bk.k_full[s], head, row);
          got.note(1 + s, ph);
          ++turn;
          return true;
        };
        if (n > 0) {
          if (live > 0 && !mbar_wait(&bk.q_empty, (live - 1) & 1, abort, lim)) break;
          mbar_arrive_expect_tx(&bk.q_full, 2 * C::kBytes);
          load_tile<DP>(q_smem, &tmQ, &bk.q_full, h, q0);
          load_tile<DP>(do_smem, &tmDo, &bk.q_full, h, q0);
          got.note(0, live & 1);
          ++live;
          if (!place_k(&tmO, h, q0)) break;
          for (int j = 0; j < n && go; ++j) {
            const int row = q0 - kRows * j, s = vturn & 1;
            const uint32_t ph = (vturn >> 1) & 1;
            if (!place_k(&tmK, kv, row) || (vturn >= 2 && !mbar_wait(&bk.v_empty[s], ph ^ 1u, abort, lim))) {
              go = false;
              break;
            }
            mbar_arrive_expect_tx(&bk.v_full[s], C::kBytes);
            load_tile<DP>(v_smem + s * C::kBytes, &tmV, &bk.v_full[s], kv, row);
            got.note(1 + kKStages + s, ph);
            ++vturn;
          }
          turn = wrapped(turn);
          vturn = wrapped(vturn);
          live = wrapped(live);
        }
        mbar_arrive(&bk.item_empty[it & 1]);
        mbar_arrive(&bk.ending);
      }
      got.drain(&bk.q_full);
    }
   } else {
    // One warp issues the scores and dp, the other dq: what one waits for costs the other nothing.
    const uint32_t leader = elect_one() ? 1u : 0u;
    constexpr uint64_t kNext = C::kBytes >> 4;
    const uint64_t q_desc = scores_desc(q_smem), do_desc = scores_desc(do_smem), k_desc = scores_desc(k_smem),
                   v_desc = scores_desc(v_smem), kt_desc = sums_desc(k_smem);
    // the place among the keys (of kKStages) and its round, key tiles met, items with rows
    uint32_t ks = 0, kr = 0;
    int at = 0, live = 0;
    auto next_place = [&] {
      if (++ks == kKStages) {
        ks = 0;
        kr ^= 1;
      }
    };
    for (int it = 0; uniform(next_item(it) ? 1 : 0) != 0; ++it) {
      const int n = uniform(bk.item[it & 1].n);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bk.item_empty[it & 1]);
      if (n == 0) continue;
      if (warp == kBwdMmaWarp) {
        warp_wait(&bk.q_full, live & 1, abort, lim);
        next_place();                        // (out's)
        for (int j = 0; j < n; ++j) {
          // (the scores once the last ones have been read; dp's buffer once the ds before the last is dq's)
          const uint32_t b = at & 1;
          warp_wait(&bk.k_full[ks], kr, abort, lim);
          if (at > 0) warp_wait(&bk.s_empty, (at - 1) & 1, abort, lim);
          tc_fence_after_sync();
          mma_scores<DP>(leader, tmem + 128, q_desc, k_desc + ks * kNext);
          mma_commit_warp(leader, &bk.s_full);
          warp_wait(&bk.v_full[b], (at >> 1) & 1, abort, lim);
          if (at >= 2) warp_wait(&bk.dp_empty[b], ((at >> 1) & 1) ^ 1u, abort, lim);
          tc_fence_after_sync();
          mma_scores<DP>(leader, tmem + 256 + 128 * b, do_desc, v_desc + b * kNext);
          mma_commit_warp(leader, &bk.dp_full[b]);
          mma_commit_warp(leader, &bk.v_empty[b]);
          next_place();
          ++at;
        }
        mma_commit_warp(leader, &bk.q_empty);
      } else {
        warp_wait(&bk.o_read, live & 1, abort, lim);
        if (lane == 0) mbar_arrive(&bk.k_empty[ks]);
        next_place();
        if (live > 0) warp_wait(&bk.out_empty, (live - 1) & 1, abort, lim);
        for (int j = 0; j < n; ++j) {
          const uint32_t b = at & 1;
          warp_wait(&bk.ds_full[b], (at >> 1) & 1, abort, lim);
          tc_fence_after_sync();
          mma_sums<DP, 2>(leader, tmem, tmem + 256 + 128 * b, kt_desc + ks * kNext, j > 0);
          mma_commit_warp(leader, &bk.dp_empty[b]);
          mma_commit_warp(leader, &bk.k_empty[ks]);
          next_place();
          ++at;
        }
        mma_commit_warp(leader, &bk.out_full);
      }
      at = wrapped(at);
      live = wrapped(live + 1);
    }
    mma_commit_warp(leader, &bk.drain);
    mbar_wait_drain(&bk.drain, 0);
   }
  } else {
   more_registers<kBwdRegs>();
   const int part = warp >> 2;
   const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
   const int lr = (warp & 3) * 32 + lane;
   const F32x2 mul2_ = make_f32x2(p.scale2, p.scale2);
   int steps = 0, live = 0;                  // key tiles met, items with rows; their sum: places among the keys
   for (int it = 0; uniform(next_item(it) ? 1 : 0) != 0; ++it) {
    const DqItem& m = bk.item[it & 1];
    const int n = m.n, q0 = m.q0, row = q0 + lr;
    if (n > 0) {
    const bool valid = row >= m.map.first && row < m.map.last;
    const int key_lo = valid ? start_of(&m.map, q0, row) : p.T, key_hi = valid ? row : -1;
    const int all_from = start_of(&m.map, q0, min(q0 + kRows, m.map.last) - 1);
    const float lse = valid ? -p.lse[static_cast<long long>(m.head) * p.T + row] * kLog2e : 0.f;
    // <do, o>: a quarter of the columns a thread
    warp_wait(&bk.q_full, live & 1, abort, lim);
    const int turn = steps + live;
    warp_wait(&bk.k_full[turn % kKStages], (turn / kKStages) & 1, abort, lim);
    {
      const uint8_t* o_smem = k_smem + turn % kKStages * C::kBytes;
      float d = 0.f;
      #pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        const int w = DP / 32 * part + i, at = w / 8 * C::kChunk + lr * 128 + ((w ^ lr) & 7) * 16;
        const uint4 x = *reinterpret_cast<const uint4*>(o_smem + at), y = *reinterpret_cast<const uint4*>(do_smem + at);
        d += bf16_lo(x.x) * bf16_lo(y.x) + bf16_hi(x.x) * bf16_hi(y.x) + bf16_lo(x.y) * bf16_lo(y.y) +
             bf16_hi(x.y) * bf16_hi(y.y) + bf16_lo(x.z) * bf16_lo(y.z) + bf16_hi(x.z) * bf16_hi(y.z) +
             bf16_lo(x.w) * bf16_lo(y.w) + bf16_hi(x.w) * bf16_hi(y.w);
      }
      bk.sums[part][lr] = d;
    }
    warp_arrive(&bk.o_read, lane);
    if (lane == 0) mbar_arrive(&bk.q_empty);
    // (By counted barriers, whose waits end: at a named one the others would stand if one warp had given up.)
    warp_wait(&bk.o_read, live & 1, abort, lim);
    float delta = -((bk.sums[0][lr] + bk.sums[1][lr]) + (bk.sums[2][lr] + bk.sums[3][lr]));
    warp_arrive(&bk.sums_read, lane);
    const F32x2 lse2 = make_f32x2(lse, lse);
    auto step = [&](int j, auto masked_c) {
      constexpr bool masked = decltype(masked_c)::value;
      const int at = steps + j, b = at & 1;
      warp_wait(&bk.s_full, at & 1, abort, lim);
      tc_fence_after_sync();
      const int k0 = q0 - kRows * j;
      const uint32_t on = masked ? seen(key_lo - k0 - 32 * part, key_hi - k0 - 32 * part) : kFull;
      const bool whole = !masked || __all_sync(kFull, on == kFull);           // (of the warp's places)
      uint32_t s[32], d[32], w[16];
      tmem_ld_x32(tmem + lanes + 128 + 32 * part, s);
      tmem_ld_wait(s);
      warp_arrive(&bk.s_empty, lane);
      #pragma unroll
      for (int x = 0; x < 32; x += 2) {
        float2 y = split_f32x2(fma2(make_f32x2(as_f(s[x]), as_f(s[x + 1])), mul2_, lse2));
        y.x = ex2(y.x);
        y.y = ex2(y.y);
        if (masked) {
          if (!(on >> x & 1u)) y.x = 0.f;
          if (!(on >> x & 2u)) y.y = 0.f;
        }
        s[x] = __float_as_uint(y.x);
        s[x + 1] = __float_as_uint(y.y);
      }
      if (masked) {
        const int k = steps + live + 1 + j;
        warp_wait(&bk.k_full[k % kKStages], (k / kKStages) & 1, abort, lim);
        clean_tile<DP>(k_smem + (k % kKStages) * C::kBytes, threadIdx.x, kBwdArith, [] {});
      }
      warp_wait(&bk.dp_full[b], (at >> 1) & 1, abort, lim);
      const uint32_t tdp = tmem + lanes + 256 + 128 * b + 32 * part;
      tc_fence_after_sync();
      tmem_ld_x32(tdp, d);
      tmem_ld_wait(d);
      if (!whole) blank(d, on);               // (so that ds is zero there whatever the tensors hold)
      if (masked && j == 0 && all_from >= q0) {
        // (some rows begin within this key tile)
        F32x2 sum = make_f32x2(0.f, 0.f);
        #pragma unroll
        for (int x = 0; x < 32; x += 2)
          sum = fma2(make_f32x2(as_f(s[x]), as_f(s[x + 1])), make_f32x2(as_f(d[x]), as_f(d[x + 1])), sum);
        const float2 t = split_f32x2(sum);
        warp_wait(&bk.sums_read, live & 1, abort, lim);
        bk.sums[part][lr] = t.x + t.y;
        warp_arrive(&bk.sums_full, lane);
        warp_wait(&bk.sums_full, live & 1, abort, lim);
        if (key_lo >= k0) delta = -((bk.sums[0][lr] + bk.sums[1][lr]) + (bk.sums[2][lr] + bk.sums[3][lr]));
      } else if (masked && j == 0) {
        warp_arrive(&bk.sums_full, lane);    // (a phase an item)
      }
      const F32x2 delta2 = make_f32x2(delta, delta);
      #pragma unroll
      for (int x = 0; x < 32; x += 2) {
        const float2 y = split_f32x2(mul2(make_f32x2(as_f(s[x]), as_f(s[x + 1])),
                                    add2(make_f32x2(as_f(d[x]), as_f(d[x + 1])), delta2)));
        w[x / 2] = pack_bf16x2(y.x, y.y);
      }
      tmem_st_x16(tdp, w);
      tmem_st_wait();
      warp_arrive(&bk.ds_full[b], lane);
      if (masked && j == 0 && valid && part == 0) {
        // (where do is not finite, nor is delta: p of this row shall not be either)
        uint4* stats = p.stats + m.head * p.pitch + row;
        stats[0] = split_row(isfinite(delta) ? lse / p.scale2 : delta - delta);
        stats[p.Hq * p.pitch] = split_row(delta);
      }
    };
    for (int j = 0; j < n; ++j) {
      if (j == 0 || q0 - kRows * j < all_from)
        step(j, std::true_type{});
      else
        step(j, std::false_type{});
    }
    warp_wait(&bk.out_full, live & 1, abort, lim);
    tc_fence_after_sync();
    const int col = 32 * part;
    uint32_t o[32];
    tmem_ld_x32(tmem + lanes + col, o);
    tmem_ld_wait(o);
    warp_arrive(&bk.out_empty, lane);
    // A row's 64 bytes by four lanes, which turn their words round among themselves: shared memory has the next
    // item's tiles on their way to it.
    uint4 w[4];
    #pragma unroll
    for (int x = 0; x < 4; ++x)
      w[x] = make_uint4(pack_bf16x2(as_f(o[8 * x]) * p.scale, as_f(o[8 * x + 1]) * p.scale),
                        pack_bf16x2(as_f(o[8 * x + 2]) * p.scale, as_f(o[8 * x + 3]) * p.scale),
                        pack_bf16x2(as_f(o[8 * x + 4]) * p.scale, as_f(o[8 * x + 5]) * p.scale),
                        pack_bf16x2(as_f(o[8 * x + 6]) * p.scale, as_f(o[8 * x + 7]) * p.scale));
    exchange<1>(w[0], w[1]);
    exchange<1>(w[2], w[3]);
    exchange<2>(w[0], w[2]);
    exchange<2>(w[1], w[3]);
    const uint32_t rows = __ballot_sync(kFull, valid);
    const int at_col = col + 8 * (lane & 3);
    __nv_bfloat16* out = p.d0.p + (row - lane) * p.d0.token + m.head * p.d0.head + at_col;
    #pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = (lane & ~3) + x;         // word lane % 4 of this row
      if ((rows >> r & 1u) && at_col < p.D) *reinterpret_cast<uint4*>(out + r * p.d0.token) = w[x];
    }
    steps = wrapped(steps + n);
    live = wrapped(live + 1);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bk.item_empty[it & 1]);
   }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  pdl_launch_next();
  if (threadIdx.x == 0 && bk.abort_flag) set_status(p.status, kErrTimeout);
  if (warp == kBwdMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// dk and dv: 128 key rows of one key-value head against the query tiles of every head of
// its group, so that the group's sum is a sum in TMEM.  Scores transposed (a thread a
// key), so that the probabilities lie in TMEM as the A operand of the sums.  TMEM: dk, dv
// DP columns from 0 and 128, scores at 256 (which become p), dp at 384 (ds).  In the
// order dv(j), scores(j + 1), dk(j), dp(j + 1) each buffer is free again when its turn
// comes.  A step is 2440 cycles at heads of 128, of which the tensor cores work 2176.
//
// A thread's columns are queries, each with an lse and a delta of its own.  Read from shared memory
// they cost it 128 KB a step, as much as the tiles (a step 2900 cycles, whatever the width); so
// the products subtract them: one more step of the contraction, three bf16 parts of -lse / scale (or
// -delta) against ones.
//
// The heads of a group may be shared out among the CTAs of a cluster (p.split of them): each leaves
// its sums in its shared memory, and each adds up its share of the rows over all of them, in
// the order of the CTAs, through distributed shared memory.
constexpr int kRowBytes = kRows * 16;      // a block of statistics
struct DkvBook {
  uint64_t kv_full, q_full[2], do_full[2];
  uint64_t q_empty[2], do_empty[2], s_full, p_full, dp_full, ds_full, done;
  uint32_t tmem;
  int abort_flag;
  RowMap map;
};

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attention_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDo,
                         const AttnParams p) {
  using C = Tile<DP>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* k_smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* v_smem = k_smem + C::kBytes;
  uint8_t* q_smem = v_smem + C::kBytes;
  uint8_t* do_smem = q_smem + 2 * C::kBytes;
  uint8_t* lse_smem = do_smem + 2 * C::kBytes;           // two blocks of 128 rows of 16 bytes, with q
  uint8_t* delta_smem = lse_smem + 2 * kRowBytes;        // the same, with do
  uint8_t* ones_smem = delta_smem + 2 * kRowBytes;       // 128 rows of three ones and five zeros
  uint8_t* zero_smem = ones_smem + kRowBytes;            // the other half of each operand's 16 columns
  float4* sums = reinterpret_cast<float4*>(q_smem);      // [dk, dv][128][DP], in place of q and do
  DkvBook& bk = *reinterpret_cast<DkvBook*>(zero_smem + kRowBytes);
  if (!smem_fits(smem_raw, &bk + 1)) {
    pdl_wait();
    if (threadIdx.x == 0) set_status(p.status, kErrLaunch);
    return;
  }
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (warp == kBwdLoadWarp && lane == 0) {          // (it uses them before the first barrier of all threads)
    mbar_init(&bk.kv_full, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bk.q_full[s], 1);
      mbar_init(&bk.q_empty[s], 1);
      mbar_init(&bk.do_full[s], 1);
      mbar_init(&bk.do_empty[s], 1);
    }
    mbar_init(&bk.s_full, 1);
    mbar_init(&bk.p_full, kBwdArith / 32);
    mbar_init(&bk.dp_full, 1);
    mbar_init(&bk.ds_full, kBwdArith / 32);
    mbar_init(&bk.done, 1);
    bk.abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
    prefetch_tensormap(&tmDo);
  }
  if (threadIdx.x < kRows) {
    reinterpret_cast<uint4*>(ones_smem)[threadIdx.x] = make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u);
    reinterpret_cast<uint4*>(zero_smem)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == kBwdMmaWarp) {
    tmem_alloc(&bk.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  pdl_wait();
  const int split = p.split, rank = static_cast<int>(blockIdx.x) % split, item = static_cast<int>(blockIdx.x) / split;
  const int kv = item % p.Hkv, k0 = item / p.Hkv * kRows;
  // The keys and the first queries do not wait for the sequences' boundaries.
  const int group = p.Hq / p.Hkv, h0 = kv * group + rank * (group / split);
  if (warp == kBwdLoadWarp && lane == 0) {
    mbar_arrive_expect_tx(&bk.kv_full, 2 * C::kBytes);
    load_tile<DP>(k_smem, &tmK, &bk.kv_full, kv, k0);
    load_tile<DP>(v_smem, &tmV, &bk.kv_full, kv, k0);
    mbar_arrive_expect_tx(&bk.q_full[0], C::kBytes + kRowBytes);
    load_tile<DP>(q_smem, &tmQ, &bk.q_full[0], h0, k0);
    bulk_load(lse_smem, p.stats + h0 * p.pitch + k0, kRowBytes, &bk.q_full[0]);
    mbar_arrive_expect_tx(&bk.do_full[0], C::kBytes + kRowBytes);
    load_tile<DP>(do_smem, &tmDo, &bk.do_full[0], h0, k0);
    bulk_load(delta_smem, p.stats + (p.Hq + h0) * p.pitch + k0, kRowBytes, &bk.do_full[0]);
  }
  row_map<kRows>(p, k0, &bk.map);
  tc_fence_after_sync();
  const uint32_t tmem = uniform(bk.tmem);
  volatile int* abort = &bk.abort_flag;
  const unsigned long long lim = p.wait_ns;
  // query tiles k0, k0 + 128, ... up to the end of the last key's sequence, for each of this CTA's heads
  const int a = max(k0, bk.map.first), b = min(k0 + kRows, bk.map.last);
  const int end = a < b ? end_of(&bk.map, k0, b - 1, kRows / 32) : k0;
  const int nq = a < b ? (end - k0 + kRows - 1) / kRows : 0, n = nq * (group / split);

  if (warp >= kBwdLoadWarp) {
   fewer_registers<kBwdOtherRegs>();
   if (warp == kBwdLoadWarp) {
    if (lane == 0) {
      Issued got;
      got.note(0, 0);
      got.note(1, 0);
      got.note(3, 0);
      int h = h0, row = k0;
      for (int j = 1; j < n; ++j) {
        row += kRows;
        if (row >= k0 + nq * kRows) {
          row = k0;
          ++h;
        }
        const int s = j & 1;
        const uint32_t ph = (j >> 1) & 1;
        if (j >= 2 && !mbar_wait(&bk.q_empty[s], ph ^ 1u, abort, lim)) break;
        mbar_arrive_expect_tx(&bk.q_full[s], C::kBytes + kRowBytes);
        load_tile<DP>(q_smem + s * C::kBytes, &tmQ, &bk.q_full[s], h, row);
        bulk_load(lse_smem + s * kRowBytes, p.stats + h * p.pitch + row, kRowBytes, &bk.q_full[s]);
        got.note(1 + s, ph);
        if (j >= 2 && !mbar_wait(&bk.do_empty[s], ph ^ 1u, abort, lim)) break;
        mbar_arrive_expect_tx(&bk.do_full[s], C::kBytes + kRowBytes);
        load_tile<DP>(do_smem + s * C::kBytes, &tmDo, &bk.do_full[s], h, row);
        bulk_load(delta_smem + s * kRowBytes, p.stats + (p.Hq + h) * p.pitch + row, kRowBytes, &bk.do_full[s]);
        got.note(3 + s, ph);
      }
      got.drain(&bk.kv_full);
    }
   } else if (n > 0 && warp == kBwdMmaWarp) {
    // (One warp for all: one for the scores and dv and one for dp and dk took 0.82 ms where this takes 0.66.)
    const uint32_t leader = elect_one() ? 1u : 0u;
    const uint64_t k_desc = scores_desc(k_smem), v_desc = scores_desc(v_smem), q_desc = scores_desc(q_smem),
                   do_desc = scores_desc(do_smem), qt_desc = sums_desc(q_smem), dot_desc = sums_desc(do_smem),
                   ones_desc = rows_desc(ones_smem, zero_smem);
    constexpr uint64_t kNext = C::kBytes >> 4;
    const int tiles = uniform(n);
    auto scores = [&](int j) {
      mma_scores<DP>(leader, tmem + 256, k_desc, q_desc + (j & 1) * kNext);
      mma_bf16_ss_warp(leader, tmem + 256, ones_desc, rows_desc(lse_smem + (j & 1) * kRowBytes, zero_smem), C::kScores,
                       1u);
      mma_commit_warp(leader, &bk.s_full);
    };
    auto dprob = [&](int j) {
      mma_scores<DP>(leader, tmem + 384, v_desc, do_desc + (j & 1) * kNext);
      mma_bf16_ss_warp(leader, tmem + 384, ones_desc, rows_desc(delta_smem + (j & 1) * kRowBytes, zero_smem),
                       C::kScores, 1u);
      mma_commit_warp(leader, &bk.dp_full);
    };
    warp_wait(&bk.kv_full, 0, abort, lim);
    warp_wait(&bk.q_full[0], 0, abort, lim);
    tc_fence_after_sync();
    scores(0);
    warp_wait(&bk.do_full[0], 0, abort, lim);
    tc_fence_after_sync();
    dprob(0);
    for (int j = 0; j < tiles; ++j) {
      warp_wait(&bk.p_full, j & 1, abort, lim);
      tc_fence_after_sync();
      mma_sums<DP, 2>(leader, tmem + 128, tmem + 256, dot_desc + (j & 1) * kNext, j > 0);
      if (j + 2 < tiles) mma_commit_warp(leader, &bk.do_empty[j & 1]);
      if (j + 1 < tiles) {
        warp_wait(&bk.q_full[(j + 1) & 1], ((j + 1) >> 1) & 1, abort, lim);
        scores(j + 1);
      }
      warp_wait(&bk.ds_full, j & 1, abort, lim);
      tc_fence_after_sync();
      mma_sums<DP, 2>(leader, tmem, tmem + 384, qt_desc + (j & 1) * kNext, j > 0);
      if (j + 2 < tiles) mma_commit_warp(leader, &bk.q_empty[j & 1]);
      if (j + 1 < tiles) {
        warp_wait(&bk.do_full[(j + 1) & 1], ((j + 1) >> 1) & 1, abort, lim);
        dprob(j + 1);
      }
    }
    mma_commit_warp(leader, &bk.done);
    mbar_wait_drain(&bk.done, 0);
   }
  } else {
   more_registers<kBwdRegs>();
   if (n > 0) {
    const int part = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int key = k0 + (warp & 3) * 32 + lane;
    const bool valid = key >= bk.map.first && key < bk.map.last;
    const int all_to = end_of(&bk.map, k0, a, kRows / 32);      // queries up to here see every key (from the diagonal)
    const F32x2 mul2_ = make_f32x2(p.scale2, p.scale2);
    auto step = [&](int j, int q0, auto masked_c) {
      constexpr bool masked = decltype(masked_c)::value;
      warp_wait(&bk.s_full, j & 1, abort, lim);
      tc_fence_after_sync();
      uint32_t on = kFull;                    // queries of the key's sequence, from its own on
      if (masked) {
        const int to = valid ? end_of(&bk.map, k0, key, kRows / 32) : INT_MAX;
        on = seen(key - q0 - 32 * part, to - 1 - q0 - 32 * part);
      }
      uint32_t s[32], d[32], w[16];
      tmem_ld_x32(tmem + lanes + 256 + 32 * part, s);
      tmem_ld_wait(s);
      const bool whole = !masked || __all_sync(kFull, on == kFull);           // (of the warp's places)
      if (masked) {
        warp_wait(&bk.do_full[j & 1], (j >> 1) & 1, abort, lim);
        clean_tile<DP>(do_smem + (j & 1) * C::kBytes, threadIdx.x, kBwdArith, [] {});
      }
      #pragma unroll
      for (int x = 0; x < 32; x += 2) {
        float2 y = split_f32x2(mul2(make_f32x2(as_f(s[x]), as_f(s[x + 1])), mul2_));
        y.x = ex2(y.x);
        y.y = ex2(y.y);
        if (masked) {
          if (!(on >> x & 1u)) y.x = 0.f;
          if (!(on >> x & 2u)) y.y = 0.f;
        }
        s[x] = __float_as_uint(y.x);
        s[x + 1] = __float_as_uint(y.y);
        w[x / 2] = pack_bf16x2(y.x, y.y);
      }
      tmem_st_x16(tmem + lanes + 256 + 32 * part, w);
      tmem_st_wait();
      warp_arrive(&bk.p_full, lane);
      if (masked) {
        warp_wait(&bk.q_full[j & 1], (j >> 1) & 1, abort, lim);
        clean_tile<DP>(q_smem + (j & 1) * C::kBytes, threadIdx.x, kBwdArith, [] {});
      }
      warp_wait(&bk.dp_full, j & 1, abort, lim);
      tc_fence_after_sync();
      tmem_ld_x32(tmem + lanes + 384 + 32 * part, d);
      tmem_ld_wait(d);
      if (!whole) blank(d, on);               // (so that ds is zero there whatever the tensors hold)
      #pragma unroll
      for (int x = 0; x < 32; x += 2) {
        const F32x2 prob = make_f32x2(as_f(s[x]), as_f(s[x + 1]));
        const float2 y = split_f32x2(mul2(prob, make_f32x2(as_f(d[x]), as_f(d[x + 1]))));
        w[x / 2] = pack_bf16x2(y.x, y.y);
      }
      tmem_st_x16(tmem + lanes + 384 + 32 * part, w);
      tmem_st_wait();
      warp_arrive(&bk.ds_full, lane);
    };
    int q0 = k0;
    for (int j = 0; j < n; ++j) {
      if (q0 == k0 || q0 + kRows > all_to)
        step(j, q0, std::true_type{});
      else
        step(j, q0, std::false_type{});
      q0 += kRows;
      if (q0 >= k0 + nq * kRows) q0 = k0;
    }
    warp_wait(&bk.done, 0, abort, lim);
    tc_fence_after_sync();
    {
      // eight warps store dk, the others dv
      const int half = part >> 1;
      const Heads& to = half == 0 ? p.d0 : p.d1;
      const float mul = half == 0 ? p.scale : 1.f;
      __nv_bfloat16* out = to.p + (key - lane) * to.token + kv * to.head;
      const uint32_t keys = __ballot_sync(kFull, valid);
      float4* row = sums + (half * kRows + key - k0) * (DP / 4);
      #pragma unroll
      for (int c = part & 1; c < DP / 32; c += 2) {
        uint32_t o[32];
        float v[32];
        tmem_ld_x32(tmem + lanes + 128 * half + 32 * c, o);
        tmem_ld_wait(o);
        #pragma unroll
        for (int x = 0; x < 32; ++x) v[x] = as_f(o[x]) * mul;
        if (split == 1) {
          store_cols(q_smem + warp * 2048, out, to.token, keys, 32 * c, p.D, v);
        } else {
          #pragma unroll
          for (int x = 0; x < 8; ++x)
            row[(8 * c + x) ^ (key & (DP / 4 - 1))] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
        }
      }
    }
   }
  }
  if (split > 1 && n > 0) {                 // (n is the same in all CTAs of a cluster)
    __syncwarp();
    cluster_sync();
    const int each = (kRows + split - 1) / split, r0 = rank * each, rows = min(each, kRows - r0);
    for (int i = threadIdx.x; i < 2 * rows * (DP / 8); i += kBwdThreads) {
      const int w = i % (DP / 8), r = r0 + i / (DP / 8) % rows, half = i / (DP / 8) / rows, key = k0 + r;
      const float4* mine = sums + (half * kRows + r) * (DP / 4);
      const int turned = key & (DP / 4 - 1);
      const uint32_t lo = smem_u32(mine + ((2 * w) ^ turned)), hi = smem_u32(mine + ((2 * w + 1) ^ turned));
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      for (int c = 0; c < split; ++c) {
        x = add4(x, ld_cluster_v4(mapa_shared(lo, c)));
        y = add4(y, ld_cluster_v4(mapa_shared(hi, c)));
      }
      const Heads& to = half == 0 ? p.d0 : p.d1;
      if (key >= bk.map.first && key < bk.map.last && 8 * w < p.D)
        *reinterpret_cast<uint4*>(to.p + key * to.token + kv * to.head + 8 * w) =
            make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w), pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    }
    cluster_sync();                         // (the others read this CTA's shared memory until here)
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  pdl_launch_next();
  if (threadIdx.x == 0 && bk.abort_flag) set_status(p.status, kErrTimeout);
  if (warp == kBwdMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- host
// What a kernel uses, and up to 1 KB in front of it for the first 1024-byte boundary (of which there
// may be less: each kernel looks).
constexpr int smem_of(int used) { return used + 1024 < kMaxSmem ? used + 1024 : kMaxSmem; }
template <int DP>
constexpr int fwd_smem() {
  return (2 + Tile<DP>::kStages) * Tile<DP>::kBytes + kFwdStaging + static_cast<int>(sizeof(FwdBook));
}
template <int DP>
constexpr int dq_smem() { return (4 + kKStages) * Tile<DP>::kBytes + static_cast<int>(sizeof(DqBook)); }
template <int DP>
constexpr int dkv_smem() {
  return 6 * Tile<DP>::kBytes + 6 * kRowBytes + static_cast<int>(sizeof(DkvBook));
}
static_assert(fwd_smem<128>() <= kMaxSmem && dq_smem<128>() <= kMaxSmem && dkv_smem<128>() <= kMaxSmem,
              "shared memory");

// Launch of blocks with much shared memory, in clusters of `cluster`.  (Each takes an SM's registers for itself, so no
// two blocks of an SM wait for each other's TMEM, which the blocks of two clusters might do in a ring.)
template <class... KArgs, class... Args>
cudaError_t launch_big(void (*kern)(KArgs...), std::atomic<bool>* attr_set, int grid, int threads, int smem,
                       cudaStream_t st, int cluster, Args&&... args) {
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // (see launch_k)
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// CTAs that share the heads of a group in dk and dv's kernel.  As few as leave no CTA more than 5/4 of an SM's share of
// one long sequence's tiles: a CTA of the first keys has tiles * group / split of them, an SM (tiles + 1) tiles
// q_heads / 2 / 152.  Large batches take one: clusters of four leave SMs of a GPC idle (8192 rows, 32/8 heads of
// 128, both kernels: 1.08 ms alone, 1.20 in pairs, 1.36 by four); small ones gain (2048 rows, 32/4 heads: 0.23, 0.14,
// 0.11 and, by eight, 0.18 ms; 1000 rows, 6/2 heads of 80: 51 us, 36 by three).
int group_split(const AttnParams& p) {
  const int group = p.Hq / p.Hkv;
  int best = 1;
  for (int c = 2; c <= 8 && static_cast<long long>(best) * (p.tiles + 1) * p.Hkv < 243; ++c)
    if (group % c == 0) best = c;
  return best;
}

// The tiles of an item of the forward: two, which share the keys' loads and keep the tensor cores busy in turn; but one
// where an SM would have none otherwise.  (One, two, by tiles * heads: 32, a row of 32/8 heads of 128: 6.6, 7.0 us;
// 48, 1003 rows, 6/2 of 80: 15.1, 18.0; 128, 4000 rows, 4 of 128: 43, 49; 152, 2400 rows, 8/1 of 64: 19.7, 24.2; 512,
// 2048 rows, 32/8 of 128: 50, 31; 2048, 8192 rows: 557, 326.  Past the limit one stays ahead for a while, as most of
// its SMs still have one tile: 208: 67, 76; 304: 101, 108 and 67, 80 (heads of 64); 312: 42, 44; 384: 92, 71.)
int forward_mode(const AttnParams& p) {
  if (static_cast<long long>(p.tiles) * p.Hq <= num_sms()) return kOneTile;
  return p.Hq / p.Hkv % 2 == 0 ? kTwoHeads : kTwoTiles;
}

// How a tensor's strides count where a dimension has one element: as if it were dense.
Heads heads_of(const moe_heads* t, int T, int heads, int D) {
  Heads h;
  h.p = static_cast<__nv_bfloat16*>(t->data);
  h.head = heads > 1 ? t->head_stride : D;
  h.token = T > 1 ? t->token_stride : (heads > 1 ? static_cast<long long>(heads) * h.head : D);
  return h;
}
bool stride_ok(long long s) { return s > 0 && s % 8 == 0 && s < (1LL << 38); }
bool heads_ok(const moe_heads* t, int T, int heads, int D, bool output) {
  if (t == nullptr || !entry::ptr_ok(t->data)) return false;
  const Heads h = heads_of(t, T, heads, D);
  if (!stride_ok(h.token) || !stride_ok(h.head)) return false;
  if (!output) return true;
  // each element its own place
  return (h.head >= D && h.token >= (heads - 1) * h.head + D) || (h.token >= D && h.head >= (T - 1) * h.token + D);
}
bool config_ok(const moe_attention_config* c) {
  if (c == nullptr || c->T < 0 || c->T > kMaxTokens || c->sequences < 0 || c->sequences > kMaxSequences) return false;
  if (c->q_heads <= 0 || c->q_heads > kMaxHeads || c->kv_heads <= 0 || c->q_heads % c->kv_heads != 0) return false;
  if (c->head_dim <= 0 || c->head_dim > kMaxHeadDim || c->head_dim % 8 != 0) return false;
  return c->scale >= kMinScale && c->scale <= 1.f / kMinScale;
}
long long stats_pitch(int T) { return (static_cast<long long>(T) + kRows - 1) / kRows * kRows; }

AttnParams params_of(const moe_attention_config* c, const int32_t* cu, void* ws) {
  AttnParams p = {};
  p.cu = cu;
  p.B = c->sequences;
  p.T = c->T;
  p.Hq = c->q_heads;
  p.Hkv = c->kv_heads;
  p.D = c->head_dim;
  p.scale = c->scale;
  p.scale2 = c->scale * kLog2e;
  p.tiles = (c->T + kRows - 1) / kRows;
  p.status = static_cast<int*>(ws);
  p.stats = reinterpret_cast<uint4*>(static_cast<char*>(ws) + entry::kStatusBytes);
  p.pitch = stats_pitch(c->T);
  const unsigned long long wait = gemm_wait_limit_ns();
  p.wait_ns = wait != 0 ? wait : kWaitLimitNs;
  return p;
}

bool make_map(CUtensorMap* m, const moe_heads* t, int T, int heads, int D) {
  const Heads h = heads_of(t, T, heads, D);
  return make_tmap_heads(m, h.p, D, heads, T, h.head, h.token);
}

template <int DP>
cudaError_t forward(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                    cudaStream_t st) {
  static std::atomic<bool> attr_set[kMaxDevices];
  const int items = p.tiles * (p.mode == kTwoHeads ? p.Hq / 2 : p.Hq), sms = num_sms();
  return launch_big(attention_fwd_kernel<DP>, attr_set, items < sms ? items : sms, kFwdThreads, smem_of(fwd_smem<DP>()),
                    st, 1, tq, tk, tv, p);
}
template <int DP>
cudaError_t backward(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& td,
                     const CUtensorMap& to, AttnParams p, const Heads& dq, const Heads& dk, const Heads& dv,
                     cudaStream_t st) {
  static std::atomic<bool> dq_set[kMaxDevices], dkv_set[kMaxDevices];
  p.d0 = dq;
  const int items = p.tiles * p.Hq, sms = num_sms();
  const cudaError_t e =
      launch_big(attention_dq_kernel<DP>, dq_set, items < sms ? items : sms, kBwdThreads, smem_of(dq_smem<DP>()), st, 1,
                 tq, tk, tv, td, to, p);
  if (e != cudaSuccess) return e;
  p.d0 = dk;
  p.d1 = dv;
  p.split = group_split(p);
  return launch_big(attention_dkv_kernel<DP>, dkv_set, p.tiles * p.Hkv * p.split, kBwdThreads,
                    smem_of(dkv_smem<DP>()), st, p.split, tq, tk, tv, td, p);
}

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::entry;

extern "C" {

size_t moe_attention_workspace_bytes(const moe_attention_config* cfg) {
  if (!config_ok(cfg)) return 0;
  return kStatusBytes + align_up(static_cast<size_t>(cfg->q_heads) * stats_pitch(cfg->T) * 2 * sizeof(uint4));
}

moe_status moe_attention_forward(const moe_attention_config* cfg, const moe_heads* q, const moe_heads* k,
                                 const moe_heads* v, const int32_t* cu_seqlens, const moe_heads* out, float* lse,
                                 void* ws, size_t ws_bytes, void* stream) {
  if (!config_ok(cfg) || !ptr_ok(ws)) return MOE_ERR_INVALID_ARG;
  const int T = cfg->T, Hq = cfg->q_heads, Hkv = cfg->kv_heads, D = cfg->head_dim;
  const bool none = T == 0 || cfg->sequences == 0;
  if (!none && (!ptr_ok(cu_seqlens) || !ptr_ok(lse) || !heads_ok(q, T, Hq, D, false) ||
                !heads_ok(k, T, Hkv, D, false) ||
                !heads_ok(v, T, Hkv, D, false) || !heads_ok(out, T, Hq, D, true)))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kStatusBytes) return MOE_ERR_WORKSPACE;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  if (none) return MOE_OK;
  AttnParams p = params_of(cfg, cu_seqlens, ws);
  p.mode = forward_mode(p);
  if (p.mode == kTwoTiles) p.tiles = (p.tiles + 1) / 2;
  p.o = heads_of(out, T, Hq, D);
  p.d0 = heads_of(v, T, Hkv, D);
  p.q = heads_of(q, T, Hq, D);
  p.lse = lse;
  CUtensorMap tq, tk, tv;
  if (!make_map(&tq, q, T, Hq, D) || !make_map(&tk, k, T, Hkv, D) || !make_map(&tv, v, T, Hkv, D))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return status_of(D <= 64 ? forward<64>(tq, tk, tv, p, st) : forward<128>(tq, tk, tv, p, st));
}

moe_status moe_attention_backward(const moe_attention_config* cfg, const moe_heads* q, const moe_heads* k,
                                  const moe_heads* v, const int32_t* cu_seqlens, const moe_heads* out, const float* lse,
                                  const moe_heads* dout, const moe_heads* dq, const moe_heads* dk, const moe_heads* dv,
                                  void* ws, size_t ws_bytes, void* stream) {
  if (!config_ok(cfg) || !ptr_ok(ws)) return MOE_ERR_INVALID_ARG;
  const int T = cfg->T, Hq = cfg->q_heads, Hkv = cfg->kv_heads, D = cfg->head_dim;
  const bool none = T == 0 || cfg->sequences == 0;
  if (!none && (!ptr_ok(cu_seqlens) || !ptr_ok(lse) || !heads_ok(q, T, Hq, D, false) ||
                !heads_ok(k, T, Hkv, D, false) ||
                !heads_ok(v, T, Hkv, D, false) || !heads_ok(out, T, Hq, D, false) || !heads_ok(dout, T, Hq, D, false) ||
                !heads_ok(dq, T, Hq, D, true) || !heads_ok(dk, T, Hkv, D, true) || !heads_ok(dv, T, Hkv, D, true)))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_attention_workspace_bytes(cfg)) return MOE_ERR_WORKSPACE;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  if (none) return MOE_OK;
  AttnParams p = params_of(cfg, cu_seqlens, ws);
  p.lse = const_cast<float*>(lse);
  CUtensorMap tq, tk, tv, td, to;
  if (!make_map(&tq, q, T, Hq, D) || !make_map(&tk, k, T, Hkv, D) || !make_map(&tv, v, T, Hkv, D) ||
      !make_map(&td, dout, T, Hq, D) || !make_map(&to, out, T, Hq, D))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Heads hq = heads_of(dq, T, Hq, D), hk = heads_of(dk, T, Hkv, D), hv = heads_of(dv, T, Hkv, D);
  return status_of(D <= 64 ? backward<64>(tq, tk, tv, td, to, p, hq, hk, hv, st)
                           : backward<128>(tq, tk, tv, td, to, p, hq, hk, hv, st));
}

}  // extern "C"
