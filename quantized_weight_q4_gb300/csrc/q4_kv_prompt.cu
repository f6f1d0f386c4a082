// Attention of prompts over the paged 8-bit cache on the tensor cores (sm_103a):
// the form for many new tokens a sequence.
//
// 4 D flops for each query and visible key: bound by the tensor cores, and by
// the exponentials beside them.  Two launches:
//
// * q4_kv_expand_kernel turns the pages of each sequence into consecutive
//   rows of codes as fp16 (exact), once for all the queries that will read
//   them: 2 bytes written for each code, against 4 D flops for each query.
//   Beside them it writes a record of each 128-token tile: the scales of its
//   eight blocks of 16 tokens, and which tokens exist.
// * q4_kv_prompt_kernel: a CTA takes 256 query rows of one kv head (the query
//   heads that share it, token-major) as two MMA tiles of 128, and walks over
//   the visible tiles of 128 tokens.  One warp copies K and V tiles with TMA
//   into a ring, one warp issues the MMAs, and four warps a tile (a thread a
//   row) take the scores from tensor memory, form the weights and put them
//   back as the fp16 A operand of the second product.  While one tile's rows
//   are in the softmax the tensor cores work on the other's.  The running
//   maximum moves only when it has grown by 2^8, so the sums in tensor memory
//   are seldom rescaled.
// * Scales are applied in fp32.  A block's key scale is part of the row's
//   constant that multiplies its scores; its value scale is an addend of the
//   exponent, so that the weight that is rounded to fp16 is p_j * scale
//   (relative to a power of two above the scales that the row has seen), and
//   the sum of p_j takes it out again.  Codes times scales as fp16 rows
//   instead would round keys and values to 11 bits: a key channel that stands
//   out then moves scores by 2^-12 of its share of them (that form: 410 us for
//   the prompt below, and 471 for the pieces).
// * Weights times scales are rounded to fp16, the type of the second product:
//   2^-11 of each, below the 2^-8 of the bf16 result.  Two terms, as the split
//   form has, would add half of all products again.
//
// Measured (8 kv heads of 128, 32 query heads): a prompt of 8192 tokens 424 us
// both launches, 1296 TFLOP/s of visible products (69% of the measured bf16
// peak of cuBLAS; tiles on the diagonal do up to twice the visible work); six
// pieces of up to 1537 tokens on up to 9000 cached ones 490 us, 1195 TFLOP/s.
// What is left is the chain of a
// tile (scores out of tensor memory, 128 exponentials a thread, weights back)
// where two tiles an SM do not cover one another, and for the pieces the last
// round of CTAs and the expansion.  The MMA warp runs its loop as a whole, with
// one lane issuing: elected before the loop, its single lane took 532 us.
#include <cfloat>
#include <type_traits>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"
#include "q4_kv_tc.cuh"

namespace q4 {
namespace {

using namespace gemm;

constexpr int kTile = 128;                // tokens of a K / V tile, rows of an MMA tile
constexpr int kTileRows = 2 * kTile;      // query rows of a CTA
constexpr int kThreads = 384;             // 2 x 4 softmax warps; a TMA warp, an MMA warp and two idle ones
constexpr int kTmaWarp = 8, kMmaWarp = 9;
// registers a thread: 384 x 168 at launch; the softmax warps hold a row's 128 scores
constexpr int kSoftmaxRegs = 216, kOtherRegs = 56;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "the shares must fit the launch's registers");
constexpr int kStages = 5;                // K and V tiles in flight
constexpr float kLazy = 8.0f;
constexpr float kUnit = 7.0f;             // weights are 2^7 at the reference: up to 2^15 with kLazy, below fp16's 65504
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr int kBlocks = kTile / kKvBlock;   // blocks of a tile
constexpr int kNoScale = -1024;             // exponent of a tile whose values are all zero
// A block's value scale counts as at least 2^kLeast of its tile's largest, one of 0 as 2^kZero (its codes are written as
// 0), and a tile's as at least 2^kZero of the row's reference: in fp16 its weights are 0 from 2^-32 on, while in their
// sum they count in full down to 2^-39.
constexpr float kLeast = -60.0f, kZero = -40.0f;

// What the softmax needs of 128 tokens of a head: a word for each lane of a warp.
struct TileInfo {
  float ks[kBlocks];         // key scales
  float lv[kBlocks];         // log2(value scale) - e
  float iv[kBlocks];         // 2^-lv
  unsigned seen[4];          // bit i: token i exists
  int e;                     // value scales are in (0, 2^e), the largest in the upper half; kNoScale: all are 0
  int full;                  // 1: all tokens exist
  int pad[2];
};
static_assert(sizeof(TileInfo) == 128 && kBlocks == 8, "a word for each lane");
constexpr int kLaneLv = 8, kLaneSeen = 24, kLaneE = 28, kLaneFull = 29;   // lanes of the words

struct ExpandParams {
  KvView c;
  KvBatch b;
  int group, split_rows;
  int rows_cap;              // rows of kv
  __half* kv;                // [2][heads][rows_cap][dim] codes
  TileInfo* info;            // [heads][rows_cap / 128]
  int* kv_cum;               // [B + 1] first tile of each sequence's tokens
  int* order;                // [B] sequences, the longest last
  int* q_cum;                // [B + 1] first tile of the query rows of each of those
  uint4* zeros;              // out, when rows of no sequence are this kernel's to clear, or null
  long long row_bytes;
  float* lse;                // with zeros: their sums of exponentials, or null
  int Hq;
  long long window, sinks;
  int tree;
  unsigned* err;
};

struct PromptParams {
  CUtensorMap kv;            // fp16 [2 * heads][rows_cap][dim], boxes of 64 x 128, 128-byte swizzle
  KvAttnCall a;
  int group, split_rows;
  int rows_cap;
  const TileInfo* info;
  const int* kv_cum;
  const int* order;
  const int* q_cum;
};

// 2^e, -126 <= e <= 127 (beyond: the nearest of those).
__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + max(-126, min(127, e))) << 23);
}
// The e in [-126, 126] with x < 2^e, x >= 2^(e - 1) within that range; x > 0.
__device__ __forceinline__ int exponent_above(float x) {
  return max(-126, min(126, static_cast<int>(__float_as_uint(x) >> 23) - 126));
}
// The larger; a NaN stays.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Sequences in this form have more query rows than the split form takes.
__device__ __forceinline__ bool is_prompt(int nq, int group, int split_rows) {
  return static_cast<long long>(nq) * group > split_rows;
}

// Tiles counted at most: lengths on the device may be anything, and a sum past this (of more tiles than any workspace
// holds) stays at it.
constexpr int kMostTiles = 1 << 29;
__device__ __forceinline__ int add_tiles(int a, int b) { return min(a + b, kMostTiles); }

// Exclusive prefix sums of n_of(b), each in [0, kMostTiles], into cum[0 .. B]; every thread of the block calls it.
template <int THREADS, typename F>
__device__ __forceinline__ void prefix(int B, int* cum, F n_of) {
  __shared__ int s_warp[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (B + THREADS - 1) / THREADS;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < B) {
      sum = add_tiles(sum, n_of(b));
      cum[b + 1] = sum;
    }
  }
  int up = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up = add_tiles(up, x);
  }
  if (lane == 31) s_warp[warp] = up;
  int before = __shfl_up_sync(0xffffffffu, up, 1);
  if (lane == 0) before = 0;
  __syncthreads();
  for (int i = 0; i < warp; ++i) before = add_tiles(before, s_warp[i]);
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < B) cum[b + 1] = add_tiles(cum[b + 1], before);
  }
  if (tid == 0) cum[0] = 0;
  __syncthreads();
}

// The b with cum[b] <= i < cum[b + 1].
__device__ __forceinline__ int find_seq(const int* cum, int B, int i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Tiles of n tokens or rows.
__device__ __forceinline__ int tiles_of(long long n, int each) {
  return static_cast<int>(min((max(n, 0LL) + each - 1) / each, static_cast<long long>(kMostTiles)));
}

__device__ __forceinline__ int kv_tiles(const KvBatch& b, int i, int group, int split_rows) {
  const int nq = b.cu[i + 1] - b.cu[i];
  return is_prompt(nq, group, split_rows) ? tiles_of(b.kv_len[i], kTile) : 0;
}

__device__ __forceinline__ int q_tiles(const KvBatch& b, int i, int group, int split_rows) {
  const int nq = b.cu[i + 1] - b.cu[i];
  return is_prompt(nq, group, split_rows) ? tiles_of(static_cast<long long>(nq) * group, kTileRows) : 0;
}

// First token that a window leaves to the queries from number j of a sequence on, and the tiles of the sinks before its
// tile.  A drafted token that sees no new one has the position before the first, whatever its number.
__device__ __forceinline__ int window_start(long long window, int tree, int len, int nq, int j) {
  const long long f = static_cast<long long>(len) - nq - window + (tree ? 0 : j + 1);
  return window > 0 && f > 0 ? static_cast<int>(f) : 0;
}
__device__ __forceinline__ int sink_tiles(long long sinks, int first) {
  return static_cast<int>(min(static_cast<long long>(first), (sinks + kTile - 1) / kTile));
}

// ---------------------------------------------------------------------------
// Pages to fp16 rows
// ---------------------------------------------------------------------------
constexpr int kExpandThreads = 256;

// Sequences by their number of tiles (of cum), in 256 classes, the longest last.  Which of a class comes first is
// left open: it moves work between SMs and changes no result.
__device__ __forceinline__ void order_by_length(int B, const int* cum, int* order) {
  constexpr int kClasses = kExpandThreads;
  __shared__ int s_count[kClasses], s_from[kClasses + 1], s_longest;
  const int tid = threadIdx.x;
  s_count[tid] = 0;
  if (tid == 0) s_longest = 1;
  __syncthreads();
  int longest = 0;
  for (int b = tid; b < B; b += kExpandThreads) longest = max(longest, cum[b + 1] - cum[b]);
  if (longest > 1) atomicMax(&s_longest, longest);
  __syncthreads();
  auto class_of = [&](int b) { return static_cast<int>(static_cast<long long>(cum[b + 1] - cum[b]) * (kClasses - 1) / s_longest); };
  for (int b = tid; b < B; b += kExpandThreads) atomicAdd(&s_count[class_of(b)], 1);
  __syncthreads();
  prefix<kExpandThreads>(kClasses, s_from, [&](int c) { return s_count[c]; });
  for (int b = tid; b < B; b += kExpandThreads) order[atomicAdd(&s_from[class_of(b)], 1)] = b;
  __syncthreads();
}

__global__ void __launch_bounds__(kExpandThreads) q4_kv_expand_kernel(const __grid_constant__ ExpandParams p) {
  extern __shared__ int s_cum[];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, h = blockIdx.y, B = p.b.B;
  prefix<kExpandThreads>(B, s_cum, [&](int b) { return kv_tiles(p.b, b, p.group, p.split_rows); });
  if (p.zeros) {
    const long long from = max(0, min(p.b.T, p.b.cu[B])) * p.row_bytes / 16, all = p.b.T * p.row_bytes / 16;
    const long long at = (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * kExpandThreads + tid;
    for (long long i = from + at; i < all; i += static_cast<long long>(gridDim.x) * gridDim.y * kExpandThreads)
      p.zeros[i] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (long long i = static_cast<long long>(max(0, min(p.b.T, p.b.cu[B]))) * p.Hq + at; i < static_cast<long long>(p.b.T) * p.Hq;
           i += static_cast<long long>(gridDim.x) * gridDim.y * kExpandThreads)
        p.lse[i] = -INFINITY;
  }
  const int tile = blockIdx.x, total = s_cum[B];
  if (tile == 0 && h == 0) {   // for the attention kernel
    for (int i = tid; i <= B; i += kExpandThreads) p.kv_cum[i] = s_cum[i];
    order_by_length(B, s_cum, p.order);
    prefix<kExpandThreads>(B, s_cum, [&](int i) { return q_tiles(p.b, p.order[i], p.group, p.split_rows); });
    for (int i = tid; i <= B; i += kExpandThreads) p.q_cum[i] = s_cum[i];
    __syncthreads();
    prefix<kExpandThreads>(B, s_cum, [&](int b) { return kv_tiles(p.b, b, p.group, p.split_rows); });
  }
  if (tile >= total) return;
  const int b = find_seq(s_cum, B, tile), t0 = (tile - s_cum[b]) * kTile, len = p.b.kv_len[b];
  // tiles, and blocks of others, that no query sees are not read: their pages may have left the table
  const int start = window_start(p.window, p.tree, len, p.b.cu[b + 1] - p.b.cu[b], 0);
  if (t0 + kTile <= start && t0 >= p.sinks) return;
  auto row_of = [&](int pos) {
    return pos >= len || ((pos | (kKvBlock - 1)) < start && (pos & ~(kKvBlock - 1)) >= p.sinks)
               ? -1LL : kv_row(p.c, p.b.table, p.b.table_stride, b, pos, h);
  };
  // the record: a lane for each block of 16 tokens
  if (tid < 32) {
    const int pos = t0 + lane * kKvBlock;
    long long row = -1;
    unsigned have = 0;
    if (lane < kBlocks && pos < len) {
      row = row_of(pos);
      if (row >= 0) have = 0xffffu >> (kKvBlock - min(kKvBlock, len - pos));
      else if (h == 0 && (pos + kKvBlock > start || pos < p.sinks)) atomicOr(p.err, kDevErrIndex);
    }
    const float ks = row >= 0 ? p.c.ks[row >> 4] : 0.f, vs = row >= 0 ? p.c.vs[row >> 4] : 0.f;
    const int e = __reduce_max_sync(0xffffffffu, vs > 0.f ? exponent_above(vs) : kNoScale);
    const unsigned next = __shfl_down_sync(0xffffffffu, have, 1);
    const int full = __all_sync(0xffffffffu, lane >= kBlocks || have == 0xffffu);
    TileInfo* info = p.info + static_cast<long long>(h) * (p.rows_cap / kTile) + tile;
    if (lane < kBlocks) {
      const float lv = vs != 0.f ? fmaxf(log2f(vs * power_of_two(-e)), kLeast) : kZero;
      info->ks[lane] = ks;
      info->lv[lane] = lv;
      info->iv[lane] = exp2f(-lv);
      if ((lane & 1) == 0) info->seen[lane >> 1] = have | next << 16;
      if (lane == 0) info->e = e, info->full = full;
    }
  }
  // 16 codes a thread
  const int D = p.c.dim, chunks = D / 16;
  for (int i = tid; i < kTile * chunks; i += kExpandThreads) {
    const int t = i / chunks, c = i % chunks, pos = t0 + t;
    const long long row = row_of(pos);
    const bool value = row >= 0 && p.c.vs[row >> 4] != 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (x ? value : row >= 0) w = *reinterpret_cast<const uint4*>((x ? p.c.v : p.c.k) + row * D + c * 16);
      uint4 f[2];
      widen4(w.x, f[0].x, f[0].y), widen4(w.y, f[0].z, f[0].w);
      widen4(w.z, f[1].x, f[1].y), widen4(w.w, f[1].z, f[1].w);
      uint4* to = reinterpret_cast<uint4*>(
          p.kv + ((static_cast<long long>(x) * p.c.heads + h) * p.rows_cap + static_cast<long long>(tile) * kTile + t) * D + c * 16);
      to[0] = f[0];
      to[1] = f[1];
    }
  }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
__device__ __forceinline__ float low2(f32x2 a) {
  float x, y;
  unpack2(a, x, y);
  return x;
}

constexpr int kScaleWords = 6 * kBlocks;   // of a softmax warp

template <int D>
struct Cfg {
  static constexpr int kHalf = kTile * 128;             // 128 rows of 64 fp16: one swizzled box
  static constexpr int kTileBytes = kHalf * (D / 64);   // a Q, K or V tile
  static constexpr int kSmem = 1024 + 2 * kTileBytes + kStages * kTileBytes + 256 + 8 * kScaleWords * 4;
  static constexpr uint32_t kTmemCols = 512;
  // instruction descriptors: fp16 operands, fp32 sums, 128 rows; q . k: both K-major, 128 columns;
  // p . v: V MN-major, D columns
  static constexpr uint32_t kIdescQk = (1u << 4) | (static_cast<uint32_t>(kTile >> 3) << 17) | (8u << 24);
  static constexpr uint32_t kIdescPv = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (8u << 24);
};

// Columns 0 .. n of 32: all from 31 on, none below 0.
__device__ __forceinline__ uint32_t columns_to(int n) { return n < 0 ? 0u : n >= 31 ? ~0u : (2u << n) - 1u; }

// Word i of a drafted token's bits (row `row` of the packed tokens): 0 outside.
__device__ __forceinline__ uint32_t tree_word(const KvAttnCall& a, long long row, int i) {
  return i >= 0 && i < a.tree_words ? static_cast<uint32_t>(__ldg(a.tree + row * a.tree_words + i)) : 0u;
}

// MORE: with sinks, drafted tokens' bits or sums of exponentials (each may be absent); a form of its own, so that
// calls without them keep their code.
template <int D, bool MORE>
__global__ void __launch_bounds__(kThreads, 1) q4_kv_prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sq = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = sq + 2 * C::kTileBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kStages * C::kTileBytes);
  uint64_t* empty = full + kStages;
  uint64_t* q_ready = empty + kStages;
  uint64_t* s_full = q_ready + 1;       // [2] scores of a tile are in tensor memory
  uint64_t* p_ready = s_full + 2;       // [2] its weights are, and its sums rescaled
  uint64_t* o_done = p_ready + 2;       // [2] its sums include the latest weights
  uint64_t* drain = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  float* s_scales = reinterpret_cast<float*>(ring + kStages * C::kTileBytes + 256);   // of the softmax warps
  __shared__ int s_fail;
  __shared__ int s_where[4];

  const KvAttnCall& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.b.B;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    mbar_init(q_ready, kTileRows);
    for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_ready[i], kTile), mbar_init(&o_done[i], 1);
    mbar_init(drain, 1);
    s_fail = 0;
  }
  fence_barrier_init();
  pdl_wait();   // before tensor memory is taken: the kernel before may need this SM's

  // ---- which rows: the longest sequences go first, and of one its last tiles, which see the most (six pieces of 414 to
  // 1537 tokens on up to 9000: 470 us, 513 us in the order given) ----
  if (warp == 0) {
    const long long t = static_cast<long long>(__ldg(p.q_cum + B)) * a.c.heads - 1 - blockIdx.x;
    const int qt = t < 0 ? 0 : static_cast<int>(t / a.c.heads);
    const int at = t < 0 ? 0 : warp_count_le(B, qt, [&](int j) { return __ldg(p.q_cum + j); });
    const int b = t < 0 ? -1 : __ldg(p.order + at);
    if (lane == 0) {
      s_where[0] = b;
      if (b >= 0) {
        s_where[1] = qt - __ldg(p.q_cum + at);
        s_where[2] = static_cast<int>(t % a.c.heads);
        s_where[3] = __ldg(p.kv_cum + b);   // first tile of the sequence's K and V
      }
    }
  }
  __syncthreads();
  const int b = s_where[0];
  if (b < 0) return;
  const int qt = s_where[1], h = s_where[2], tile0 = s_where[3];
  const int c0 = a.b.cu[b], nq = a.b.cu[b + 1] - c0, len = a.b.kv_len[b];
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();   // the next kernel may take tensor memory early: this one has its own
  const uint32_t tmem = *tmem_slot;
  // tensor memory: scores (and weights) of the two tiles, then their sums
  const uint32_t t_s[2] = {tmem, tmem + kTile}, t_o[2] = {tmem + 2 * kTile, tmem + 2 * kTile + D};

  // tiles of tokens that any row sees
  const int row0 = qt * kTileRows;
  const int j0 = row0 / p.group, j1 = min(nq - 1, (row0 + kTileRows - 1) / p.group);
  const int last = a.causal && !(MORE && a.tree) ? min(len - 1, len - nq + j1) : len - 1;
  const int first = window_start(a.window, MORE && a.tree, len, nq, j0) / kTile;
  const int stay = MORE ? sink_tiles(a.sinks, first) : 0;   // the sinks' tiles come first
  auto tile_of = [&](int i) { return MORE && i < stay ? i : i + first - stay; };
  const bool fits = (static_cast<long long>(tile0) + tiles_of(len, kTile)) * kTile <= p.rows_cap;
  if (!fits && tid == 0) atomicOr(a.err, kDevErrIndex);   // longer sequences than the call said
  const int n = fits && last >= 0 ? max(0, last / kTile + 1 - first + stay) : 0;

  if (warp >= kTmaWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kTmaWarp) {
    if (lane == 0) {
      int it = 0;
      for (; it < 2 * n && !s_fail; ++it) {
        const int st = it % kStages;
        if (it >= kStages && !gwait(&empty[st], ((it / kStages) - 1) & 1, &s_fail, a.err)) break;
        mbar_arrive_expect_tx(&full[st], C::kTileBytes);
        const int row = (tile0 + tile_of(it >> 1)) * kTile, z = (it & 1) * a.c.heads + h;
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tma_load_3d(ring + st * C::kTileBytes + x * C::kHalf, &p.kv, x * 64, row, z, &full[st]);
      }
      for (int g = it - 1; g >= 0 && g >= it - kStages; --g) (void)mbar_wait(&full[g % kStages], (g / kStages) & 1);
    }
  } else if (warp == kMmaWarp) {
    if (n > 0) {
      const uint32_t leader = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, poll_wait(bar, parity, &s_fail, a.err));
      };
      // descriptors count 16 bytes
      const uint64_t q_desc = smem_desc(smem_u32(sq), 16, 1024, kSwizzle128);
      const uint64_t k_desc = smem_desc(smem_u32(ring), 16, 1024, kSwizzle128);
      const uint64_t v_desc = smem_desc(smem_u32(ring), C::kHalf, 1024, kSwizzle128);
      auto qk = [&](int g, int st) {   // scores of tile g with the K tile in stage st
        const uint64_t qd = q_desc + g * (C::kTileBytes >> 4), kd = k_desc + st * (C::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int off = ((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4;
          lead_mma(leader, t_s[g], qd + off, kd + off, C::kIdescQk, kk > 0 ? 1u : 0u);
        }
        lead_commit(leader, &s_full[g]);
      };
      auto pv = [&](int g, int st, uint32_t more) {
        const uint64_t vd = v_desc + st * (C::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          lead_mma_ts(leader, t_o[g], t_s[g] + kk * 8, vd + kk * (2048 >> 4), C::kIdescPv, kk > 0 ? 1u : more);
        lead_commit(leader, &o_done[g]);
      };
      // copies alternate between K and V; stage and parity of the next one
      int st = 0;
      uint32_t phase = 0;
      auto next_copy = [&]() {
        if (++st == kStages) st = 0, phase ^= 1;
      };
      bool ok = wait(q_ready, 0) && wait(&full[0], 0);
      if (ok) {
        qk(0, 0);
        qk(1, 0);
        lead_commit(leader, &empty[0]);
        next_copy();
      }
      for (int i = 0; ok && i < n; ++i) {
        const bool next = i + 1 < n;
        const int v = st;
        ok = wait(&full[v], phase);
        next_copy();
        const int k = st;
        ok = ok && wait(&p_ready[0], i & 1);
        if (!ok) break;
        tc_fence_after();
        pv(0, v, i > 0);
        if (next) {
          ok = wait(&full[k], phase);
          if (!ok) break;
          qk(0, k);
        }
        ok = wait(&p_ready[1], i & 1);
        if (!ok) break;
        tc_fence_after();
        pv(1, v, i > 0);
        lead_commit(leader, &empty[v]);
        if (next) {
          qk(1, k);
          lead_commit(leader, &empty[k]);
          next_copy();
        }
      }
      // no MMA may still run when the tensor memory is freed
      lead_commit(leader, drain);
      (void)mbar_wait(drain, 0);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ================= softmax: a thread a row =================
    const int g = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;   // row of tile g
    const int row = row0 + g * kTile + r, j = row / p.group;
    const bool have = j < nq && c0 >= 0 && c0 + j < a.b.T;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    float rowc;
    {
      // the row as fp16, scaled by a power of two; the sign of `scale` goes with it
      uint4 w[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) w[i] = make_uint4(0, 0, 0, 0);
      if (have) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (static_cast<long long>(c0) + j) * a.q_stride +
                                                        (h * p.group + row % p.group) * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = __ldg(q + i);
      }
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) m = max(m, max(x[k] << 16 & 0x7fffffffu, x[k] & 0x7fff0000u));
      }
      const int e = m ? max(-126, min(126, 13 + 127 - static_cast<int>(m >> 23))) : 0;
      const float f = copysignf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23), a.scale);
      rowc = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * fabsf(a.scale) * kLog2e;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        __half2 y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[k] = __floats2half2_rn(__uint_as_float(x[k] << 16) * f, __uint_as_float(x[k] & 0xffff0000u) * f);
        *reinterpret_cast<uint4*>(sq + g * C::kTileBytes + (i >> 3) * C::kHalf + r * 128 + (((i & 7) ^ (r & 7)) << 4)) =
            *reinterpret_cast<uint4*>(y);
      }
      fence_async_smem();
      mbar_arrive(q_ready);
    }
    // positions the row sees: (from, to]; one that does not exist sees all, so that no tile is on its edge
    int qpos = len - nq + j;
    const int to = !have ? 0x7fffffff : MORE && a.tree ? len - nq - 1 : a.causal ? qpos : len - 1;
    if (MORE && a.tree && have) {   // as many new tokens as its path has; they are seen by their bits alone
      int path = 0;
      for (int i = 0; i < nq; i += 32)
        path += __popc(tree_word(a, static_cast<long long>(c0) + j, i >> 5) & columns_to(nq - 1 - i));
      qpos = len - nq + path - 1;
    }
    const long long f = have && a.window > 0 ? static_cast<long long>(qpos) - a.window : -1LL;
    const int from = f < -1 ? -1 : static_cast<int>(f);
    float m = -INFINITY, l = 0.f;
    int e = kNoScale;             // the sums are relative to 2^e, above the value scales that the row has seen
    bool ok = true;
    // a word of the tile's record for each lane, read a tile ahead, and by way of shared memory every scale for all
    const int* info = reinterpret_cast<const int*>(p.info + static_cast<long long>(h) * (p.rows_cap / kTile) + tile0) + lane;
    int next_rec = n > 0 ? __ldg(info + 32 * tile_of(0)) : 0;
    const uint32_t my_scales = smem_u32(s_scales + warp * kScaleWords);   // key scales, lv and iv, each twice
    const uint32_t put = my_scales + 8 * lane;
    const f32x2 rowc2 = dup2(rowc);
    for (int i = 0; i < n; ++i) {
      const int t0 = tile_of(i) * kTile, rec = next_rec;
      if (i + 1 < n) next_rec = __ldg(info + 32 * tile_of(i + 1));
      __syncwarp();               // the last tile's scales have been read
      if (lane < 24) asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(put), "r"(rec) : "memory");
      __syncwarp();
      uint32_t scales;            // the loads from it stay behind the stores
      asm volatile("mov.u32 %0, %1;" : "=r"(scales) : "r"(my_scales) : "memory");
      const int tile_e = __shfl_sync(0xffffffffu, rec, kLaneE);
      const int full = __shfl_sync(0xffffffffu, rec, kLaneFull);
      // tiles on the edge of what a row sees, or with tokens that do not exist (the same for the whole warp)
      const bool mine = t0 + kTile - 1 > to || (t0 <= from && !(MORE && t0 + kTile <= a.sinks)) || full == 0;
      const bool edge = __any_sync(0xffffffffu, mine);
      ok = gwait(&s_full[g], i & 1, &s_fail, a.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[kTile];
#pragma unroll
      for (int x = 0; x < 4; ++x) tmem_ld32_async(t_s[g] + lanes + 32 * x, s + 32 * x);
      f32x2 mul[kBlocks];         // a block's scores to powers of two
#pragma unroll
      for (int k = 0; k < kBlocks; k += 2) {
        lds_pairs(scales + 8 * k, mul[k], mul[k + 1]);
        mul[k] = mul2(mul[k], rowc2), mul[k + 1] = mul2(mul[k + 1], rowc2);
      }
      tmem_wait_ld();
      if (edge) {
        uint32_t bits[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) bits[x] = __shfl_sync(0xffffffffu, rec, kLaneSeen + x);
        const int lo = from - t0, hi = to - t0;
        if (MORE) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int at = t0 + 32 * x;
            uint32_t see = columns_to(to - at) & ~columns_to(from - at);
            if (at < a.sinks) see |= columns_to(to - at) & columns_to(static_cast<int>(min(a.sinks - at, 32LL)) - 1);
            if (a.tree && have) {
              const int k = at - (len - nq);   // place among the new tokens
              const long long row = static_cast<long long>(c0) + j;
              see |= __funnelshift_r(tree_word(a, row, k >> 5), tree_word(a, row, (k >> 5) + 1), k & 31);
            }
            bits[x] &= see;
          }
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (!((bits[c >> 5] >> (c & 31)) & 1u)) s[c] = 0xff800000u;
        } else {
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (c <= lo || c > hi || !((bits[c >> 5] >> (c & 31)) & 1u)) s[c] = 0xff800000u;
        }
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) mul[k] = dup2(max_nan(low2(mul[k]), 1e-30f));   // masked scores stay -inf
      }
      float now = -INFINITY, top[kBlocks];
#pragma unroll
      for (int k = 0; k < kBlocks; ++k) {
        top[k] = __uint_as_float(s[kKvBlock * k]);
#pragma unroll
        for (int c = 1; c < kKvBlock; ++c) top[k] = fmaxf(top[k], __uint_as_float(s[kKvBlock * k + c]));
        now = fmaxf(now, top[k] * low2(mul[k]));
      }
      int te = tile_e;
      if (edge) {                 // only scales of blocks that the row sees something of
        te = kNoScale;
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
          const int up = tile_e + __float2int_ru(__int_as_float(__shfl_sync(0xffffffffu, rec, kLaneLv + k)));
          te = top[k] > -INFINITY ? max(te, up) : te;
        }
      }
      if (__any_sync(0xffffffffu, now > m + kLazy || te > e)) {   // also from -inf
        const float next = fmaxf(m, now);
        const float k = next > -INFINITY ? ex2(m - next) : 1.f;
        m = next;
        l *= k;
        const float ko = k * power_of_two(e - max(e, te));
        e = max(e, te);
        if (i > 0) {
          ok = gwait(&o_done[g], (i - 1) & 1, &s_fail, a.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t o[32];
            tmem_ld32_async(t_o[g] + lanes + 32 * x, o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * ko);
            tmem_st32(t_o[g] + lanes + 32 * x, o);
          }
        }
      }
      // the tile's scales against the row's reference
      const int down = tile_e == kNoScale ? 0 : max(tile_e - e, static_cast<int>(kZero));
      const float off = (m > -INFINITY ? kUnit - m : 0.f) + static_cast<float>(down);
      uint32_t w[kTile / 2];
      f32x2 sum2[2] = {0ull, 0ull};
      const f32x2 off2 = dup2(off);
#pragma unroll
      for (int k = 0; k < kBlocks; ++k) {
        f32x2 lv[2], iv[2];
        lds_pairs(scales + 64 + 8 * (k & ~1), lv[0], lv[1]);
        lds_pairs(scales + 128 + 8 * (k & ~1), iv[0], iv[1]);
        const f32x2 add = add2(off2, lv[k & 1]);
#pragma unroll
        for (int c = k * kKvBlock / 2; c < (k + 1) * kKvBlock / 2; ++c) {
          float x, y;
          unpack2(fma2(pack2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), mul[k], add), x, y);
          x = ex2(x), y = ex2(y);
          sum2[c & 1] = fma2(pack2(x, y), iv[k & 1], sum2[c & 1]);
          const __half2 two = __floats2half2_rn(x, y);
          w[c] = *reinterpret_cast<const uint32_t*>(&two);
        }
      }
      tmem_st32(t_s[g] + lanes, w);
      tmem_st32(t_s[g] + lanes + 32, w + 32);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_ready[g]);
      float x, y;
      unpack2(add2(sum2[0], sum2[1]), x, y);
      l = fmaf(x + y, power_of_two(-down), l);
      asm volatile("" : "+f"(l));   // what was loaded is used before the next tile's stores
    }
    // the rows' results
    if (n > 0 && ok) {
      ok = gwait(&o_done[g], (n - 1) & 1, &s_fail, a.err);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    if (ok) {
      // a row that sees nothing: zeros; a NaN stays
      const float k = l > 0.f ? power_of_two(e) / l : l == 0.f ? 0.f : l;
      const long long at = ((static_cast<long long>(c0) + j) * a.Hq + h * p.group + row % p.group) * D;
      if (MORE && a.lse && have) a.lse[at / D] = l > 0.f ? (m + log2f(l) - kUnit) * kLn2 : l == 0.f ? -INFINITY : l;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32_async(t_o[g] + lanes + 32 * x, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0;
        }
        if (have) {
          uint4* to4 = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at + 32 * x);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            __nv_bfloat162 y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              y[i] = __floats2bfloat162_rn(__uint_as_float(o[8 * c + 2 * i]) * k, __uint_as_float(o[8 * c + 2 * i + 1]) * k);
            to4[c] = *reinterpret_cast<uint4*>(y);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <typename P>
cudaError_t launch_pdl(void (*kernel)(P), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  size_t info, kv_cum, order, q_cum, kv, total;
};
Layout layout(const KvView& c, int B, long long rows_cap) {
  Layout l;
  l.info = 0;
  l.kv_cum = up256(static_cast<size_t>(rows_cap / kTile) * c.heads * sizeof(TileInfo));
  l.order = l.kv_cum + up256((static_cast<size_t>(B) + 1) * sizeof(int));
  l.q_cum = l.order + up256(static_cast<size_t>(B) * sizeof(int));
  l.kv = l.q_cum + up256((static_cast<size_t>(B) + 1) * sizeof(int));
  l.total = l.kv + static_cast<size_t>(rows_cap) * c.heads * c.dim * 2 * sizeof(__half);
  return l;
}

}  // namespace

long long kv_prompt_rows(int B, long long max_kv, long long total_kv) {
  const long long each = (max_kv + kTile - 1) / kTile * kTile * B;
  const long long all = total_kv > 0 ? (total_kv + static_cast<long long>(kTile - 1) * B) / kTile * kTile : each;
  return all < each ? all : each;
}

size_t kv_prompt_bytes(const KvView& c, int B, long long rows) { return layout(c, B, rows).total; }

cudaError_t launch_kv_prompt(const KvAttnCall& a, int split_rows, long long rows, void* ws, cudaStream_t st) {
  const Layout l = layout(a.c, a.b.B, rows);
  uint8_t* w = static_cast<uint8_t*>(ws);
  ExpandParams x = {};
  x.c = a.c;
  x.b = a.b;
  x.group = a.Hq / a.c.heads;
  x.split_rows = split_rows;
  x.rows_cap = static_cast<int>(rows);
  x.kv = reinterpret_cast<__half*>(w + l.kv);
  x.info = reinterpret_cast<TileInfo*>(w + l.info);
  x.kv_cum = reinterpret_cast<int*>(w + l.kv_cum);
  x.order = reinterpret_cast<int*>(w + l.order);
  x.q_cum = reinterpret_cast<int*>(w + l.q_cum);
  // without a split form beside it, rows of no sequence are this form's
  x.zeros = split_rows == 0 ? static_cast<uint4*>(a.out) : nullptr;
  x.row_bytes = static_cast<long long>(a.Hq) * a.c.dim * 2;
  x.lse = a.lse;
  x.Hq = a.Hq;
  x.window = a.window;
  x.sinks = a.sinks;
  x.tree = a.tree != nullptr;
  x.err = a.err;
  PromptParams p = {};
  p.a = a;
  p.group = x.group;
  p.split_rows = split_rows;
  p.rows_cap = x.rows_cap;
  p.info = x.info;
  p.kv_cum = x.kv_cum;
  p.order = x.order;
  p.q_cum = x.q_cum;
  const auto encode = encoder();
  if (!encode) return cudaErrorUnknown;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.c.dim), static_cast<cuuint64_t>(rows), 2ull * a.c.heads};
  const cuuint64_t strides[2] = {dims[0] * 2, dims[0] * 2 * dims[1]};
  const cuuint32_t box[3] = {64, kTile, 1}, ones[3] = {1, 1, 1};
  if (encode(&p.kv, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, x.kv, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorUnknown;
  cudaError_t e = launch_pdl(q4_kv_expand_kernel, dim3(static_cast<unsigned>(rows / kTile), a.c.heads), kExpandThreads,
                             (static_cast<size_t>(a.b.B) + 1) * 4, st, x);
  if (e != cudaSuccess) return e;
  const long long tiles = (static_cast<long long>(a.b.T) * p.group + kTileRows - 1) / kTileRows + a.b.B;
  if (tiles * a.c.heads > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(tiles * a.c.heads));
  const auto run = [&](auto dim, auto more) {
    constexpr int D = decltype(dim)::value;
    constexpr bool kMore = decltype(more)::value;
    static std::atomic<unsigned long long> allowed;
    const cudaError_t x = allow_smem(q4_kv_prompt_kernel<D, kMore>, Cfg<D>::kSmem, allowed);
    return x != cudaSuccess ? x : launch_pdl(q4_kv_prompt_kernel<D, kMore>, grid, kThreads, Cfg<D>::kSmem, st, p);
  };
  const auto by_dim = [&](auto more) {
    return a.c.dim == 128 ? run(std::integral_constant<int, 128>{}, more) : run(std::integral_constant<int, 64>{}, more);
  };
  return kv_attn_more(a) ? by_dim(std::true_type{}) : by_dim(std::false_type{});
}

}  // namespace q4
