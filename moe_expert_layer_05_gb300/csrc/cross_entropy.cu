// Softmax cross entropy of a vocabulary head, and its gradient, without ever
// holding the logits:
//
//   z[t, v] = <x[t], w[v]>,  lse[t] = log sum_v exp z[t, v],
//   loss[t] = lse[t] - z[t, label[t]];
//   d[t, v] = dloss[t] (exp(z[t, v] - lse[t]) - [v = label[t]]),
//   dx = d w,  dw = d^T x.
//
// Forward: one tcgen05 GEMM whose epilogue reduces each half of a 256-column
// tile of logits to a maximum and a sum of exponentials per row
// (ce_stats_tile), and a kernel that joins the pairs in order.  The logits stay
// in TMEM.  Up to kFewRows tokens they are dot products instead (ce_few_kernel).
//
// Backward, per piece of the vocabulary: the piece's logits again, turned into
// d in the GEMM's epilogue (ce_grad_tile) and kept for this piece only, in
// bf16 -- the operand type of the tensor cores' next two products: a rounding
// of 2^-9 per element, of the size of the gradients' own rounding to bf16 at
// the end -- then dx += d w_piece into fp32 slabs and dw_piece = d^T x.  That
// holds where the roundings of many rows average out (the gradients' rel-L2 error
// is 2.2e-3, their own rounding 1.7e-3), and was up to 4e-3 elsewhere.  So what
// the rows' weights have in common stays out of d and multiplies the gradients in
// fp32 (ce_unit), and up to kTwoParts tokens d is kept in two bf16 parts, as
// twice the rows: 1.7e-3 with equal weights or few tokens, at 0.3 % and (64
// tokens, H = 4096, 32000 entries) 5 % of the time.  dx's
// contraction runs over the vocabulary and has few tiles, so it is cut into
// parts with a slab each, which are added in order and rounded once.  Pieces
// follow one another on the stream, so the fp32 additions into a slab have one
// order and the result does not depend on timing.
//
// Where a row is sure of its label, d is what is left of exp(z - lse) - 1, of the
// size of fp32's rounding of z.  The backward therefore makes each logit by the same
// additions as the forward: whole, in segments (kWhole), or as a dot product
// (kFewRows); and both keep the rounding of a product with log2 e out of
// differences.  Such rows' gradients are then as near to the exact ones as the plain
// fp32 form's (300 rows, 1 - p of 5e-5, H from 1024 to 16384: 1.00 to 1.06 times its
// error).
//
// Bound by the tensor cores where there are some hundred tokens or more, and
// there by the power limit over many passes.  Measured on one GB300 (cuBLAS
// bf16: 1914 TFLOP/s in a burst, 1721 sustained): forward of 8192 tokens, H =
// 4096, 32000 entries 1.26 ms (1.70 PFLOP/s); a training step of 4096 tokens, H
// = 4096, 131072 entries 10.4 to 10.9 ms (1.61 to 1.69 PFLOP/s: 4.4 TFLOP forward, 13.2
// backward); at H = 7168, 4096 tokens and 32000 entries 4.7 ms (1.59), of which the
// forward 1.12 (1.68).  With few tokens bound by reading the weight: one token, H = 4096,
// 32000 entries 45 us (5.9 TB/s), 131072 entries 153 us (7.0 TB/s).  Between
// them by the launches and the rounds of tiles: 1003 tokens, H = 1000, 5003
// entries 71 us, five launches, 80 tiles on 76 CTA pairs.
#include <cuda.h>
#include <cuda_runtime.h>

#include "entry_checks.h"
#include "gemm_common.h"

namespace moe {
namespace {

constexpr int kTile = 256;           // vocabulary entries of one logits tile
constexpr int kMaxTokens = 1 << 24, kMaxVocab = 1 << 24;
constexpr int kMaxSlabs = 16;
constexpr int kFewRows = 2;          // tokens up to which the logits are matrix-vector products
constexpr int kFewBlocks = 304;      // their blocks: two on each SM

// Elements of d kept at a time where the caller names no piece: 256 MB of bf16, but
// pieces of kMinPiece entries at least (above 32768 tokens d is 8 KB a token).
constexpr long long kPieceElements = 1LL << 27;
constexpr int kMinPiece = 4096;

// Logits of up to kWhole products are added up whole by the tensor cores (losses
// 8e-7 off at that length), longer ones in segments.  Both directions do it alike:
// where a row is sure of its label, the gradient is what is left of exp(z - lse) -
// 1, and a z added up differently from lse's would make it that difference
// (1.6e-4 at a logit of 20 and H = 7168, where 1 - p is 5e-5).
constexpr int kWhole = 4096, kSegment = 2048;

int round_up(int v, int m) { return (v + m - 1) / m * m; }

// Vocabulary entries of one piece: whole tiles, the pieces as even as they come.
int piece_of(int T, int V, int piece) {
  long long most = piece;
  if (piece <= 0) {
    most = kPieceElements / (T > 0 ? T : 1);
    if (most < kMinPiece) most = kMinPiece;
  }
  const int tiles = (V + kTile - 1) / kTile;
  const long long per = most < kTile ? 1 : piece > 0 ? (most + kTile - 1) / kTile : most / kTile;
  const int pieces = static_cast<int>((tiles + per - 1) / per);
  return (tiles + pieces - 1) / pieces * kTile;
}

// Tokens up to which d has two parts: their rows fit in one 128-row tile that has
// to be read and multiplied whole anyway.  (The tiles' stores are 32 rows high; for
// up to kFewRows tokens d comes by entries.)
constexpr int kTwoParts = 64;
int low_row(int T) {                                                    // first row of the lower parts; 0: none
  return T <= kFewRows ? T : T <= kTwoParts ? round_up(T, 32) : 0;
}
int d_rows(int T) { return T <= kTwoParts ? 2 * low_row(T) : T; }       // rows of d, of x in dw, of dx's slabs

// Up to 128 tokens the logits and dx run on 128-row tiles of one CTA,
// otherwise on 256-row tiles of CTA pairs.
bool small_rows(int T) { return T <= 128; }

// k-blocks of one part of a contraction over kb k-blocks whose output has
// `tiles` tiles for `units` CTAs or pairs.  Few tiles leave SMs idle in whole
// rounds, so the contraction is cut into as many parts as make rounds x (part +
// a tile's start and end, some 8 k-blocks) least.  dx at T = 4096, H = 4096
// (256 tiles on 76 pairs): two parts take 7 rounds of half the length instead
// of 4.  A further part has to save 1 %: it is a slab more of workspace.
int kb_per_split(int tiles, int units, int kb) {
  int best = kb;
  long long least = -1;
  for (int splits = 1; splits <= kMaxSlabs && splits <= kb; ++splits) {
    const int per = (kb + splits - 1) / splits;
    const int parts = (kb + per - 1) / per;
    const long long rounds = (static_cast<long long>(tiles) * parts + units - 1) / units;
    const long long cost = rounds * (per + 8) + parts;        // (a slab more to write and to add)
    if (least < 0 || cost * 100 < least * 99) {
      least = cost;
      best = per;
    }
  }
  return best;
}

int dx_per_split(int T, int H, int kb) {
  const int n_tiles = (H + kTile - 1) / kTile;
  return small_rows(T) ? kb_per_split(n_tiles, 152, kb) : kb_per_split((T + 255) / 256 * n_tiles, 76, kb);
}
// The weight gradient's contraction, over the tokens, is cut only where its
// tiles do not make one round.
constexpr int kDwBlock = 128;        // tokens of one of its k-blocks
int dw_per_split(int T, int H, int rows) {
  const int tiles = (rows + 255) / 256 * ((H + kTile - 1) / kTile), kb = (T + kDwBlock - 1) / kDwBlock;
  return tiles < 76 ? kb_per_split(tiles, 76, kb) : kb;
}

size_t dw_slab_bytes(int T, int H, int rows) {
  const int kb = (T + kDwBlock - 1) / kDwBlock, per = dw_per_split(T, H, rows);
  return per < kb ? static_cast<size_t>((kb + per - 1) / per) * round_up(rows, 256) * H * 4 : 0;
}

struct Ws {
  size_t stats, label_logit;         // forward
  size_t d, xz, slabs, dw_slabs;     // backward
  int piece, slab_count;
  size_t total;
};
Ws layout(int T, int H, int V, int piece) {
  Ws w;
  size_t off = entry::kStatusBytes, end = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = entry::align_up(off + bytes);
    return o;
  };
  const size_t rows = T;
  size_t parts = 2 * ((V + kTile - 1) / kTile);
  if (T <= kFewRows && parts < kFewBlocks) parts = kFewBlocks;
  w.stats = take(parts * rows * sizeof(float2));
  w.label_logit = take(rows * 4);
  end = off;
  off = entry::kStatusBytes;
  const size_t dr = d_rows(T);
  w.piece = piece_of(d_rows(T), V, piece);
  const int kb = w.piece / 64, per = dx_per_split(d_rows(T), H, kb);
  w.slab_count = (kb + per - 1) / per;
  w.d = take(dr * w.piece * 2);
  w.xz = take(dr * H * 2);
  w.slabs = take(static_cast<size_t>(w.slab_count) * dr * H * 4);
  // (the last piece may be smaller, and its contraction cut into more parts)
  const int first = V < w.piece ? V : w.piece, last = V - (V - 1) / w.piece * w.piece;
  const size_t sf = dw_slab_bytes(d_rows(T), H, first), sl = dw_slab_bytes(d_rows(T), H, last);
  w.dw_slabs = take(sf > sl ? sf : sl);
  w.total = end > off ? end : off;
  return w;
}

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// ---------------------------------------------------------------- logits GEMM
template <Epi EP, bool PAIR>
cudaError_t gemm_logits(const void* x, int T, int H, const void* w_rows, int rows, void* d, int ld, CeParams ce,
                        const SideJob& side, int* status, cudaStream_t st) {
  using C = GemmCfg<256, false, false, Sched::kDenseM, EP, 0, false, PAIR, false, true>;
  CUtensorMap ta, tb, tc;
  if (!make_tmap_bf16(&ta, x, H, T, 64, 128) || !make_tmap_bf16(&tb, w_rows, H, rows, 64, C::B_BOX_ROWS))
    return cudaErrorInvalidValue;
  tc = ta;
  if (d != nullptr && !make_tmap_out_bf16(&tc, d, ld, d_rows(T))) return cudaErrorInvalidValue;
  GemmParams p = gemm_params_zero();
  p.E = 1;
  p.m_rows = T;
  p.k_len = round_up(H, C::BK);          // (zeros past H)
  p.n_tiles = (rows + kTile - 1) / kTile;
  p.rows_cap = T;
  p.status = status;
  // groups of up to 16 row blocks, their rows of x within 32 MB of the L2:
  // 8192 x 4096 against 32000 entries 1.31 ms (all 32 row blocks at once: 1.38)
  const int group = (32 << 20) / (512 * H);
  p.m_group = group > 16 ? 16 : group < 4 ? 4 : group;
  p.seg_kb = kSegment / C::BK;
  p.ce = ce;
  p.side = side;
  const int tiles = (T + C::TILE_M - 1) / C::TILE_M * p.n_tiles;
  if constexpr (PAIR)
    return launch_gemm_pair<C>(ta, tb, tc, tc, p, tiles, st);
  else
    return launch_gemm<C>(ta, tb, tc, tc, p, tiles < num_sms() ? tiles : num_sms(), st);
}

// dx slabs (+)= d[T, cols] w_rows[cols, H] (T: rows of d)
template <bool PAIR>
cudaError_t gemm_dx(const void* d, int ld, int T, const void* w_rows, int rows, int H, int per, float* slabs,
                    int slab_count, bool add, int* status, cudaStream_t st) {
  using C = GemmCfg<256, false, true, Sched::kSplitK, Epi::kStoreF32, 0, false, PAIR, false, true>;
  CUtensorMap ta, tb, tc;
  if (!make_tmap_bf16(&ta, d, ld, T, 64, 128) || !make_tmap_bf16(&tb, w_rows, H, rows, 64, 64) ||
      !make_tmap_slabs_f32(&tc, slabs, H, T, slab_count))
    return cudaErrorInvalidValue;
  GemmParams p = gemm_params_zero();
  p.E = 1;
  p.m_rows = T;
  p.k_len = round_up(rows, kTile);       // whole tiles of d, zero past the vocabulary
  p.n_tiles = (H + kTile - 1) / kTile;
  p.rows_cap = T;
  p.valid_cols = H;
  p.kb_per_split = per;
  p.c_add = add ? 1 : 0;
  p.status = status;
  const int splits = (p.k_len / C::BK + per - 1) / per;
  const int tiles = (T + C::TILE_M - 1) / C::TILE_M * p.n_tiles * splits;
  if constexpr (PAIR)
    return launch_gemm_pair<C>(ta, tb, tc, tc, p, tiles, st);
  else
    return launch_gemm<C>(ta, tb, tc, tc, p, tiles < num_sms() ? tiles : num_sms(), st);
}

// dw_rows[rows, H] = d[T, rows]^T x[T, H]: in bf16, or (parts > 1) as fp32 slabs
// [parts][rows rounded up to 256][H] of parts of the contraction (T: rows of d).
cudaError_t gemm_dw(const void* d, int ld, int T, const void* x, int H, void* dw_rows, int rows, int per, float* slabs,
                    const CeParams& ce, const SideJob& side, int* status, cudaStream_t st) {
  using C = GemmCfg<256, true, true, Sched::kRoutedK, Epi::kStoreBf16, 0, false, true, false, true>;
  using CS = GemmCfg<256, true, true, Sched::kRoutedK, Epi::kStoreF32, 0, false, true, false, true>;
  static_assert(C::BK == kDwBlock && CS::BK == kDwBlock, "k-blocks of the weight gradient");
  const int kb = (T + kDwBlock - 1) / kDwBlock, parts = (kb + per - 1) / per;
  CUtensorMap ta, tb, tc;
  GemmParams p = gemm_params_zero();
  p.E = parts;
  p.m_rows = parts > 1 ? round_up(rows, 256) : rows;
  p.k_len = T;
  p.kb_per_split = per;
  p.m_tiles_w = (rows + 255) / 256;
  p.n_tiles = (H + kTile - 1) / kTile;
  p.valid_cols = H;
  p.ce = ce;
  p.side = side;
  p.status = status;
  if (!make_tmap_bf16(&ta, d, ld, T, 64, kDwBlock) || !make_tmap_bf16(&tb, x, H, T, 64, kDwBlock))
    return cudaErrorInvalidValue;
  const int tiles = parts * p.m_tiles_w * p.n_tiles;
  if (parts > 1) {
    if (!make_tmap_out_f32(&tc, slabs, H, static_cast<uint64_t>(parts) * p.m_rows)) return cudaErrorInvalidValue;
    return launch_gemm_pair<CS>(ta, tb, tc, tc, p, tiles, st);
  }
  if (!make_tmap_out_bf16(&tc, dw_rows, H, rows)) return cudaErrorInvalidValue;
  return launch_gemm_pair<C>(ta, tb, tc, tc, p, tiles, st);
}

// ---------------------------------------------------------------- few tokens
// Up to kFewRows tokens the logits are matrix-vector products: the head's
// weight is read once, in whole rows, and nothing else counts.  (The tensor
// cores' tiles read 128 bytes of each of 256 rows at a time, which costs HBM a
// quarter of its rate: one token, 131072 x 4096, in 190 us, against 153 here,
// 7.0 TB/s; from four tokens on the arithmetic here takes longer than that.)
// A warp takes STEP entries at a time, lanes the words of their rows (two for one
// token, one for two: 45 and 47 us at 32000 x 4096, 54 with two and two); x
// stays in shared memory.  Lane t keeps token t's running maximum and sum; the
// warps of a block are joined in order and leave one pair stats[block][t], and
// the last block to finish joins the blocks' pairs, in an order of its own
// that does not depend on who is last.
constexpr int kFewWarps = 16;

// Two (maximum, sum) pairs as one.  The exponents are differences of maxima, so
// that the side that has the maximum keeps its sum to the bit: a product rounded
// before the subtraction would leave it a factor that grows with every join
// (losses of sure rows 1.9e-4 off over 131072 entries, a logit of 90).
__device__ __forceinline__ float2 ce_join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x), top = m == -INFINITY ? 0.f : m;
  return make_float2(m, a.y * ex2((a.x - top) * kLog2e) + b.y * ex2((b.x - top) * kLog2e));
}

// lse and loss of one row from its joined pair.
__device__ __forceinline__ void ce_row_out(float2 a, int row, const int32_t* __restrict__ labels, int V,
                                           const float* label_logit, float* __restrict__ loss,
                                           float* __restrict__ lse, int* status) {
  const float l = a.x + logf(a.y);
  const int label = labels[row];
  const bool scored = label >= 0 && label < V;
  if (!scored && label != -1) set_status(status, kErrBadIndex);
  lse[row] = l;
  loss[row] = scored ? l - __ldcg(label_logit + row) : 0.f;    // (another block may have written it)
}

// Logits of STEP entries (their rows of w) and TT tokens, by one warp: mine[r] is
// token t's of entry r in lane t.  Both directions call this: where a row is sure of
// its label, z and lse have to come of the same additions.
template <int TT, int STEP>
__device__ __forceinline__ void few_logits(const uint4* const (&rows)[STEP], int words, const uint4* s_x, int lane,
                                           float (&mine)[STEP]) {
  F32x2 acc[STEP][TT];
  #pragma unroll
  for (int r = 0; r < STEP; ++r)
    #pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = make_f32x2(0.f, 0.f);
  for (int c0 = lane; c0 < words; c0 += 4 * 32) {
    uint4 u[4][STEP];
    #pragma unroll
    for (int i = 0; i < 4; ++i)
      #pragma unroll
      for (int r = 0; r < STEP; ++r)
        u[i][r] = c0 + 32 * i < words ? rows[r][c0 + 32 * i] : make_uint4(0, 0, 0, 0);
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + 32 * i;
      if (c < words) {
        F32x2 wv[STEP][4];
        #pragma unroll
        for (int r = 0; r < STEP; ++r) {
          wv[r][0] = bf16x2_f32x2(u[i][r].x);
          wv[r][1] = bf16x2_f32x2(u[i][r].y);
          wv[r][2] = bf16x2_f32x2(u[i][r].z);
          wv[r][3] = bf16x2_f32x2(u[i][r].w);
        }
        #pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint4 xu = s_x[t * words + c];
          const F32x2 xv[4] = {bf16x2_f32x2(xu.x), bf16x2_f32x2(xu.y), bf16x2_f32x2(xu.z), bf16x2_f32x2(xu.w)};
          #pragma unroll
          for (int r = 0; r < STEP; ++r)
            #pragma unroll
            for (int j = 0; j < 4; ++j) acc[r][t] = fma2(wv[r][j], xv[j], acc[r][t]);
        }
      }
    }
  }
  #pragma unroll
  for (int r = 0; r < STEP; ++r) {
    mine[r] = 0.f;
    #pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float2 f = split_f32x2(acc[r][t]);
      float z = f.x + f.y;
      #pragma unroll
      for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
      if (lane == t) mine[r] = z;
    }
  }
}

template <int TT, int STEP>
__global__ void __launch_bounds__(32 * kFewWarps) ce_few_kernel(const uint4* __restrict__ x,
                                                                const uint4* __restrict__ w,
                                                                const int32_t* __restrict__ labels, int T, int words,
                                                                int V, float2* stats, float* label_logit,
                                                                float* __restrict__ loss, float* __restrict__ lse,
                                                                int* status) {
  pdl_entry();
  extern __shared__ __align__(16) uint4 s_x[];          // [TT][words], zero past T
  __shared__ float2 s_part[kFewWarps][TT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < TT * words; i += blockDim.x)
    s_x[i] = i < T * words ? x[i] : make_uint4(0, 0, 0, 0);
  __syncthreads();
  const int label = lane < T ? labels[lane] : -1;
  float2 run = make_float2(-INFINITY, 0.f);
  const int stride = gridDim.x * kFewWarps * STEP;
  for (int v0 = (blockIdx.x * kFewWarps + warp) * STEP; v0 < V; v0 += stride) {
    const uint4* rows[STEP];
    #pragma unroll
    for (int r = 0; r < STEP; ++r) rows[r] = w + static_cast<long long>(min(v0 + r, V - 1)) * words;
    float mine[STEP];
    few_logits<TT, STEP>(rows, words, s_x, lane, mine);
    #pragma unroll
    for (int r = 0; r < STEP; ++r) {
      if (v0 + r < V && lane < T) {
        run = ce_join(run, make_float2(mine[r], 1.f));
        if (label == v0 + r) label_logit[lane] = mine[r];
      }
    }
  }
  if (lane < TT) s_part[warp][lane] = run;
  __syncthreads();
  if (warp == 0 && lane < T) {
    float2 a = s_part[0][lane];
    #pragma unroll
    for (int i = 1; i < kFewWarps; ++i) a = ce_join(a, s_part[i][lane]);
    stats[blockIdx.x * T + lane] = a;
  }
  __shared__ int s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(status + kFewDoneWord, 1) == static_cast<int>(gridDim.x) - 1 ? 1 : 0;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  if (threadIdx.x == 0) atomicExch(status + kFewDoneWord, 0);      // zero for the next launch
  if (warp < T) {                           // warp t: token t
    float2 a = make_float2(-INFINITY, 0.f);
    for (int i = lane; i < static_cast<int>(gridDim.x); i += 32) a = ce_join(a, __ldcg(stats + i * T + warp));
    #pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      a = ce_join(a, make_float2(__shfl_xor_sync(0xffffffffu, a.x, d), __shfl_xor_sync(0xffffffffu, a.y, d)));
    if (lane == 0) ce_row_out(a, warp, labels, V, label_logit, loss, lse, status);
  }
}

// d of one piece (w: its rows) for as few tokens, as ce_grad_tile's: in two bf16
// parts, rows t and T + t, zero from the piece's last entry to the end of its last
// tile.  Block 0 also leaves the copy of x that the weight gradient reads, twice,
// without the rows that are not scored (xz: null but for the first piece).
template <int TT, int STEP>
__global__ void __launch_bounds__(32 * kFewWarps) ce_few_grad_kernel(const uint4* __restrict__ x,
                                                                     const uint4* __restrict__ w, int T, int words,
                                                                     int entries, const CeParams ce, int ld,
                                                                     __nv_bfloat16* __restrict__ d,
                                                                     uint4* __restrict__ xz, int* status) {
  pdl_entry();
  extern __shared__ __align__(16) uint4 s_x[];          // [TT][words], zero past T
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < TT * words; i += blockDim.x)
    s_x[i] = i < T * words ? x[i] : make_uint4(0, 0, 0, 0);
  __syncthreads();
  const float unit = ce_unit_of(ce, lane);
  const int label = lane < T ? ce.labels[lane] : -1;
  const bool scored = label >= 0 && label < ce.vocab;
  const float lse = scored ? ce.lse[lane] : 0.f, dl = scored ? ce.dloss[lane] / unit : 0.f;
  if (blockIdx.x == 0 && xz != nullptr) {
    if (warp == 0 && !scored && label != -1) set_status(status, kErrBadIndex);
    const unsigned rows_scored = __ballot_sync(0xffffffffu, scored);
    for (int i = threadIdx.x; i < T * words; i += blockDim.x)
      xz[i] = xz[T * words + i] = (rows_scored >> (i / words)) & 1u ? s_x[i] : make_uint4(0, 0, 0, 0);
  }
  const int end = (entries + kTile - 1) / kTile * kTile;
  const int stride = gridDim.x * kFewWarps * STEP;
  for (int v0 = (blockIdx.x * kFewWarps + warp) * STEP; v0 < end; v0 += stride) {
    const uint4* rows[STEP];
    #pragma unroll
    for (int r = 0; r < STEP; ++r) rows[r] = w + static_cast<long long>(min(v0 + r, entries - 1)) * words;
    float mine[STEP];
    few_logits<TT, STEP>(rows, words, s_x, lane, mine);
    if (lane < T) {
      #pragma unroll
      for (int r = 0; r < STEP; ++r) {                  // (kTile is a multiple of STEP: v0 + r < end)
        float g = ex2((mine[r] - lse) * kLog2e);
        if (label == ce.v0 + v0 + r) g -= 1.f;
        g = scored && v0 + r < entries ? g * dl : 0.f;
        const __nv_bfloat16 upper = __float2bfloat16_rn(g);
        __nv_bfloat16* to = d + static_cast<long long>(lane) * ld + v0 + r;
        to[0] = upper;
        to[static_cast<long long>(T) * ld] = __float2bfloat16_rn(g - __bfloat162float(upper));
      }
    }
  }
}

// Launches either kernel for `entries` entries: dynamic shared memory for x, as
// many blocks as there is work for.
template <int TT, int STEP, class Kern, class... Args>
cudaError_t launch_few(Kern kern, std::atomic<bool> (&attr_set)[kMaxDevices], int H, int entries, cudaStream_t st,
                       Args... args) {
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TT * entry::kMaxH * 2);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  const int need = (entries + kFewWarps * STEP - 1) / (kFewWarps * STEP);
  count_launches(1);
  return launch_k(kern, need < kFewBlocks ? need : kFewBlocks, 32 * kFewWarps, static_cast<size_t>(TT) * H * 2, st,
                  args...);
}

template <int TT, int STEP>
cudaError_t loss_few(const void* x, const void* w, int T, int H, int V, const CeParams& ce, float* loss, float* lse,
                     int* status, cudaStream_t st) {
  static std::atomic<bool> attr_set[kMaxDevices];
  return launch_few<TT, STEP>(ce_few_kernel<TT, STEP>, attr_set, H, V, st, static_cast<const uint4*>(x),
                              static_cast<const uint4*>(w), ce.labels, T, H / 8, V, ce.stats, ce.label_logit, loss,
                              lse, status);
}

template <int TT, int STEP>
cudaError_t grad_few(const void* x, const void* w_rows, int T, int H, int rows, const CeParams& ce, int ld, void* d,
                     void* xz, int* status, cudaStream_t st) {
  static std::atomic<bool> attr_set[kMaxDevices];
  return launch_few<TT, STEP>(ce_few_grad_kernel<TT, STEP>, attr_set, H, round_up(rows, kTile), st,
                              static_cast<const uint4*>(x), static_cast<const uint4*>(w_rows), T, H / 8, rows, ce, ld,
                              static_cast<__nv_bfloat16*>(d), static_cast<uint4*>(xz), status);
}

// ---------------------------------------------------------------- row kernels
constexpr int kJoinRows = 32, kJoinStrands = 16;

// lse and loss of each row from its half tiles' (maximum, sum): strand s takes
// pairs s, s + 16, ... in order, then the strands are joined in order.
__global__ void __launch_bounds__(kJoinRows * kJoinStrands) ce_join_kernel(const float2* __restrict__ stats, int parts,
                                                                          const float* __restrict__ label_logit,
                                                                          const int32_t* __restrict__ labels, int T,
                                                                          int V, float* __restrict__ loss,
                                                                          float* __restrict__ lse, int* status) {
  pdl_entry();
  __shared__ float2 s_part[kJoinStrands][kJoinRows];
  const int lane = threadIdx.x % kJoinRows, strand = threadIdx.x / kJoinRows;
  const int row = blockIdx.x * kJoinRows + lane;
  float2 a = make_float2(-INFINITY, 0.f);
  if (row < T) {
    #pragma unroll 4
    for (int i = strand; i < parts; i += kJoinStrands) a = ce_join(a, stats[static_cast<long long>(i) * T + row]);
  }
  s_part[strand][lane] = a;
  __syncthreads();
  if (strand != 0 || row >= T) return;
  #pragma unroll
  for (int i = 1; i < kJoinStrands; ++i) a = ce_join(a, s_part[i][lane]);
  ce_row_out(a, row, labels, V, label_logit, loss, lse, status);
}

// The weight gradient's slabs added in order, rounded to bf16.  n4 = values of
// the output / 4, stride4 = those of a slab.
__global__ void __launch_bounds__(256) ce_dw_kernel(const float4* __restrict__ slabs, int count, long long n4,
                                                    long long stride4, uint2* __restrict__ dw) {
  pdl_entry();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 a = slabs[i];
  #pragma unroll 4
  for (int s = 1; s < count; ++s) {
    const float4 b = slabs[s * stride4 + i];
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
  }
  dw[i] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
}

bool sizes_ok(int32_t T, int32_t H, int32_t V, int32_t piece) {
  return T >= 0 && T <= kMaxTokens && V > 0 && V <= kMaxVocab && entry::hidden_ok(H) && piece >= 0 &&
         // tiles are counted in 32 bits
         (static_cast<long long>(T) / 128 + 1) * (V / kTile + 1) < (1LL << 30);
}

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::entry;

#define MOE_TRY(expr)                                 \
  do {                                                \
    if ((expr) != cudaSuccess) return MOE_ERR_CUDA;   \
  } while (0)

extern "C" {

size_t moe_cross_entropy_workspace_bytes(int32_t T, int32_t H, int32_t V, int32_t piece) {
  return sizes_ok(T, H, V, piece) ? layout(T, H, V, piece).total : 0;
}

moe_status moe_cross_entropy_forward(const void* x, const void* w, const int32_t* labels, int32_t T, int32_t H,
                                     int32_t V, float* loss, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (!sizes_ok(T, H, V, 0) || !ptr_ok(w) || !ptr_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ptr_ok(x) || !ptr_ok(labels) || !ptr_ok(loss) || !ptr_ok(lse))) return MOE_ERR_INVALID_ARG;
  const Ws l = layout(T, H, V, 0);
  if (ws_bytes < l.label_logit + static_cast<size_t>(T) * 4) return MOE_ERR_WORKSPACE;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* status = static_cast<int*>(ws);
  CeParams ce{};
  ce.labels = labels;
  ce.vocab = V;
  ce.stats = at<float2>(ws, l.stats);
  ce.label_logit = at<float>(ws, l.label_logit);
  if (T == 1) return status_of(loss_few<1, 2>(x, w, T, H, V, ce, loss, lse, status, st));
  if (T <= kFewRows) return status_of(loss_few<kFewRows, 1>(x, w, T, H, V, ce, loss, lse, status, st));
  const bool small = small_rows(T);
  if (H > kWhole)
    MOE_TRY(small ? (gemm_logits<Epi::kCeStatsSeg, false>(x, T, H, w, V, nullptr, 0, ce, SideJob{}, status, st))
                  : (gemm_logits<Epi::kCeStatsSeg, true>(x, T, H, w, V, nullptr, 0, ce, SideJob{}, status, st)));
  else
    MOE_TRY(small ? (gemm_logits<Epi::kCeStats, false>(x, T, H, w, V, nullptr, 0, ce, SideJob{}, status, st))
                  : (gemm_logits<Epi::kCeStats, true>(x, T, H, w, V, nullptr, 0, ce, SideJob{}, status, st)));
  count_launches(1);
  MOE_TRY(launch_k(ce_join_kernel, (T + kJoinRows - 1) / kJoinRows, kJoinRows * kJoinStrands, 0, st, ce.stats,
                   2 * ((V + kTile - 1) / kTile), ce.label_logit, labels, T, V, loss, lse, status));
  return MOE_OK;
}

moe_status moe_cross_entropy_backward(const void* x, const void* w, const int32_t* labels, const float* lse,
                                      const float* dloss, int32_t T, int32_t H, int32_t V, int32_t piece, void* dx,
                                      void* dw, void* ws, size_t ws_bytes, void* stream) {
  if (!sizes_ok(T, H, V, piece) || !ptr_ok(w) || !ptr_ok(dw) || !ptr_ok(ws)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ptr_ok(x) || !ptr_ok(labels) || !ptr_ok(lse) || !ptr_ok(dloss) || !ptr_ok(dx)))
    return MOE_ERR_INVALID_ARG;
  const Ws l = layout(T, H, V, piece);
  if (ws_bytes < l.total) return MOE_ERR_WORKSPACE;
  if (!device_is_gb300()) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) return status_of(cudaMemsetAsync(dw, 0, static_cast<size_t>(V) * H * 2, st));
  int* status = static_cast<int*>(ws);
  void* d = at<char>(ws, l.d);
  void* xz = at<char>(ws, l.xz);
  float* slabs = at<float>(ws, l.slabs);
  const bool small = small_rows(T);
  CeParams ce{};
  ce.labels = labels;
  ce.vocab = V;
  ce.lse = lse;
  ce.dloss = dloss;
  ce.rows = T;
  ce.low = low_row(T);
  const int D = d_rows(T);
  const int per = dx_per_split(D, H, l.piece / 64);
  SideJob copy{};                            // beside the first piece's logits: x without its unscored rows
  copy.src = static_cast<const uint4*>(x);
  copy.dst = xz;
  copy.n = D;
  copy.words = H / 8;
  for (int v0 = 0; v0 < V; v0 += l.piece) {
    const int rows = V - v0 < l.piece ? V - v0 : l.piece;
    const size_t at_w = static_cast<size_t>(v0) * H * 2;
    const char* w_rows = static_cast<const char*>(w) + at_w;
    char* dw_rows = static_cast<char*>(dw) + at_w;
    ce.v0 = v0;
    if (T <= kFewRows) {
      void* x_to = v0 == 0 ? xz : nullptr;
      MOE_TRY(T == 1 ? (grad_few<1, 2>(x, w_rows, T, H, rows, ce, l.piece, d, x_to, status, st))
                     : (grad_few<kFewRows, 1>(x, w_rows, T, H, rows, ce, l.piece, d, x_to, status, st)));
    } else if (H > kWhole) {
      MOE_TRY(small ? (gemm_logits<Epi::kCeGradSeg, false>(x, T, H, w_rows, rows, d, l.piece, ce, copy, status, st))
                    : (gemm_logits<Epi::kCeGradSeg, true>(x, T, H, w_rows, rows, d, l.piece, ce, copy, status, st)));
    } else {
      MOE_TRY(small ? (gemm_logits<Epi::kCeGrad, false>(x, T, H, w_rows, rows, d, l.piece, ce, copy, status, st))
                    : (gemm_logits<Epi::kCeGrad, true>(x, T, H, w_rows, rows, d, l.piece, ce, copy, status, st)));
    }
    if (small) {
      MOE_TRY(gemm_dx<false>(d, l.piece, D, w_rows, rows, H, per, slabs, l.slab_count, v0 > 0, status, st));
    } else {
      MOE_TRY(gemm_dx<true>(d, l.piece, D, w_rows, rows, H, per, slabs, l.slab_count, v0 > 0, status, st));
    }
    copy.n = 0;
    SideJob join{};                          // beside the last piece's weight gradient: dx from its slabs
    if (v0 + l.piece >= V) {
      join.src = reinterpret_cast<const uint4*>(slabs);
      join.dst = dx;
      join.n = static_cast<long long>(T) * H / 4;
      join.stride = static_cast<long long>(ce.low > 0 ? ce.low : T) * H / 4;
      join.words = ce.low > 0 ? 2 * l.slab_count : l.slab_count;   // (the lower part of each after its upper one)
    }
    const int dw_per = dw_per_split(D, H, rows), dw_kb = (D + kDwBlock - 1) / kDwBlock;
    float* dw_slabs = at<float>(ws, l.dw_slabs);
    MOE_TRY(gemm_dw(d, l.piece, D, xz, H, dw_rows, rows, dw_per, dw_slabs, ce, join, status, st));
    if (dw_per < dw_kb) {
      const long long n4 = static_cast<long long>(rows) * H / 4;
      count_launches(1);
      MOE_TRY(launch_k(ce_dw_kernel, static_cast<unsigned>((n4 + 255) / 256), 256, 0, st,
                       reinterpret_cast<const float4*>(dw_slabs), (dw_kb + dw_per - 1) / dw_per, n4,
                       static_cast<long long>(round_up(rows, 256)) * H / 4, reinterpret_cast<uint2*>(dw_rows)));
    }
  }
  return MOE_OK;
}

}  // extern "C"
