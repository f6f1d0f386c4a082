// Attention over the paged 8-bit cache on the tensor cores, split over the
// cached tokens (sm_103a): the form for some tens to hundreds of query rows a
// sequence, as drafts of several tokens have, with bf16 queries and results.
//
//   out[t, h] = sum_j p_j v_j,  p = softmax_j(scale * q[t, h] . k_j)
//
// 128 rows against each code: too many to widen the codes for every 16 of them
// (the split form), too few to write the codes out as fp16 first (the prompt
// form), and too few CTAs if each walks over all of a sequence.  So:
//
// * The unit of work is a tile of 128 tokens of a kv head for up to 128 query
//   rows (token-major).  The units of all sequences form one line, with some
//   empty ones before each (sequence, rows, head) for what starting one costs,
//   that is cut evenly over the CTAs; shares of what was cut are joined by the
//   last CTA to have one.
// * In a CTA one warp looks blocks up and copies their codes into a ring (in
//   registers of the warps that widen them they would not be far enough ahead);
//   eight warps put them as exact fp16 into shared memory in the order of the
//   MMA's operands; one warp issues the MMAs; eight warps (two threads a row,
//   each half of a tile's tokens) turn scores into weights.  Two tiles of scores take turns in tensor memory, so
//   that the next one's products run beside a tile's softmax.
// * Scales are applied in fp32: a block's key scale is part of the factor of
//   its scores, its value scale multiplies the weight before that is rounded
//   to fp16, relative to a power of two above the scales that the row has seen.
//
// Measured (bf16, 32 query heads on 8 kv heads of 128): 16 drafts of 7 to 61
// tokens on 492 to 6062 cached ones 82 us (both other forms, one after another:
// 237 us); 19 drafts of 32 tokens on 4000 67 us.  A tile takes 1.6 us, of which
// the softmax's chain is 1.2 (scores from tensor memory, 64 exponentials a
// thread, the pair's vote, weights back) and 0.8 what the codes' way takes of
// shared memory's bandwidth (copied in, read, written as fp16, read by two
// products); starting a (sequence, rows, head) takes 5 to 10 us of dependent
// lookups, joining a cut one 3 to 5.
#include <algorithm>
#include <cfloat>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"
#include "q4_kv_tc.cuh"

namespace q4 {
namespace {

using namespace gemm;

constexpr int kTile = 128;                // tokens and query rows of a tile
constexpr int kThreads = 640;             // 8 softmax warps, 8 that widen codes, one each for MMAs and copies, two idle ones
constexpr int kSoftmax = 2 * kTile, kWidenWarp = 8, kWidenWarps = 8, kMmaWarp = 16, kCopyWarp = 17, kWiden = kWidenWarps * 32;
// registers a thread: 640 x 96 at launch
constexpr int kSoftmaxRegs = 152, kWidenRegs = 56, kOtherRegs = 56;
static_assert(128 * (2 * kSoftmaxRegs + 2 * kWidenRegs + kOtherRegs) <= kThreads * 96, "the shares must fit the launch's registers");
constexpr int kStages = 2;                // of keys, and of values, as fp16
constexpr int kRaw = 4;                   // of codes: keys and values of a tile in turn
constexpr int kRecs = 8;                  // records of tiles: copies are six tiles at most before the softmax
constexpr int kBlocks = kTile / kKvBlock;
constexpr int kSegCost = 6;               // what starting a (sequence, rows, head) costs, in tiles (3 / 4 / 6 / 8: 92 / 85 / 85 / 86 us when it was chosen)
constexpr int kLeastTiles = 6;            // of a CTA, about: a share to join costs as much as several
constexpr float kLazy = 8.0f;             // the reference moves once a score exceeds it by 2^kLazy
constexpr float kUnit = 7.0f;             // weights are 2^7 at the reference: up to 2^15, below fp16's 65504
constexpr int kNoScale = -1024;           // exponent of blocks whose values are all zero
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct DraftParams {
  KvAttnCall a;
  int group, max_rows;       // sequences with more query rows are left to the prompt form
  unsigned* tickets;         // [ranges], zero
  float4* part;              // [ranges][2][D / 4 + 1][kTile] shares: sums; their maximum, weights' sum and exponent
};

// What the softmax needs of a tile of tokens.
struct Rec {
  float ks[kBlocks], vs[kBlocks];
  uint16_t seen[kBlocks];    // tokens of each block that exist
};

// One (sequence, rows, head) of the line, and the tiles a CTA takes of it.
struct Segment {
  int b, h, rows0;
  int c0, nq, len;
  int first, stay;           // tiles of the sinks, [0, stay), come before those from `first` on
  int start;                 // first token that a window leaves
  int lo, hi;                // this CTA's tiles of these (maybe none)
  long long from, to;        // units of the whole: [from, to)
  __device__ __forceinline__ int tile(int i) const { return i < stay ? i : i - stay + first; }
};

template <int D>
struct Cfg {
  static constexpr int kHalf = kTile * 128;             // 128 rows of 64 fp16: a swizzled box
  static constexpr int kTileBytes = kHalf * (D / 64);
  static constexpr int kRawBytes = kTile * D;
  static constexpr size_t smem(int B) {
    return 1024 + 2 * kStages * kTileBytes + kRaw * kRawBytes + 256 + static_cast<size_t>(B + 1) * 8;
  }
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kIdescQk = (1u << 4) | (static_cast<uint32_t>(kTile >> 3) << 17) | (8u << 24);
  static constexpr uint32_t kIdescPv = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (8u << 24);
};

__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + max(-126, min(127, e))) << 23);
}
__device__ __forceinline__ uint32_t columns_to(int n) { return n < 0 ? 0u : n >= 31 ? ~0u : (2u << n) - 1u; }
__device__ __forceinline__ uint32_t tree_word(const KvAttnCall& a, long long row, int i) {
  return i >= 0 && i < a.tree_words ? static_cast<uint32_t>(__ldg(a.tree + row * a.tree_words + i)) : 0u;
}
// Barriers of the softmax warps: of all, and of the two that share 32 rows (`pair`), with or without a vote.
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory"); }
__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(2 + pair) : "memory"); }
__device__ __forceinline__ bool pair_any(int pair, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y) : "r"(static_cast<uint32_t>(x)), "r"(2 + pair) : "memory");
  return y != 0;
}

// The tiles that the queries of a sequence see something of, at least one.
__device__ __forceinline__ void seq_tiles(const KvAttnCall& a, int nq, int len, int& start, int& first, int& stay, int& n) {
  const long long f = a.window > 0 ? static_cast<long long>(len) - nq - a.window + (a.tree ? 0 : 1) : 0;
  start = f > 0 ? static_cast<int>(f) : 0;
  const int hi = max(1, static_cast<int>((kv_tokens(a.c, a.b.table_stride, len) + kTile - 1LL) / kTile));
  first = min(start / kTile, hi - 1);
  stay = static_cast<int>(min(static_cast<long long>(first), (a.sinks + kTile - 1) / kTile));
  n = stay + hi - first;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) q4_kv_draft_kernel(const __grid_constant__ DraftParams p) {
  using C = Cfg<D>;
  constexpr int kParts = D / 16, kEach = kTile * kParts / kWiden;   // 16-byte parts of a row; of a tile, that a thread widens
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sk = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sv = sk + kStages * C::kTileBytes;
  uint8_t* raw = sv + kStages * C::kTileBytes;
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(raw + kRaw * C::kRawBytes);
  uint64_t* raw_empty = raw_full + kRaw;
  uint64_t* k_full = raw_empty + kRaw;
  uint64_t* k_empty = k_full + kStages;
  uint64_t* v_full = k_empty + kStages;
  uint64_t* v_empty = v_full + kStages;
  uint64_t* s_full = v_empty + kStages;  // [2] scores of a tile are in tensor memory
  uint64_t* p_ready = s_full + 2;        // [2] its weights are, and the sums rescaled
  uint64_t* o_done = p_ready + 2;        // [2] the sums include its weights: two, as a row may wait for a tile while the
  uint64_t* q_ready = o_done + 2;        //     one before it is not done
  uint64_t* drain = q_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  long long* s_cum = reinterpret_cast<long long*>(raw + kRaw * C::kRawBytes + 256);   // [B + 1] first unit of each sequence
  __shared__ __align__(16) Rec s_rec[kRecs];
  __shared__ long long s_warp[kThreads / 32];
  __shared__ float s_far[2][kTile];      // what the two threads of a row tell each other
  __shared__ int s_scale[2][kTile];
  __shared__ int s_fail, s_last, s_go;

  const KvAttnCall& a = p.a;
  // numbers that warps branch on come from one lane, so that they are known to be the same in all: exchanges and votes
  // behind a branch that may part lanes take much longer (the batch above 84 us)
  auto same = [](auto x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int tid = threadIdx.x, lane = tid & 31, warp = same(tid >> 5), B = a.b.B;
  if (tid == 0) {
    for (int i = 0; i < kRaw; ++i) mbar_init(&raw_full[i], 1 + kBlocks), mbar_init(&raw_empty[i], kWiden);
    for (int i = 0; i < kStages; ++i)
      mbar_init(&k_full[i], kWiden), mbar_init(&k_empty[i], 1), mbar_init(&v_full[i], kWiden), mbar_init(&v_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_ready[i], kSoftmax), mbar_init(&o_done[i], 1);
    mbar_init(q_ready, kSoftmax), mbar_init(drain, 1);
    s_fail = 0;
  }
  fence_barrier_init();
  pdl_wait();   // before tensor memory is taken: the kernel before may need this SM's
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);

  // ---- the line of units ----
  {
    const int per = (B + kThreads - 1) / kThreads;
    long long sum = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < B) {
        const int nq = a.b.cu[b + 1] - a.b.cu[b], len = a.b.kv_len[b];
        const long long rows = static_cast<long long>(min(nq, a.b.T)) * p.group;
        if (nq > 0 && kv_tokens(a.c, a.b.table_stride, len) < len) atomicOr(a.err, kDevErrIndex);
        int start, first, stay, n;
        seq_tiles(a, nq, len, start, first, stay, n);
        if (nq > 0 && rows <= p.max_rows) sum += (rows + kTile - 1) / kTile * a.c.heads * (n + kSegCost);
        s_cum[b + 1] = sum;
      }
    }
    long long up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    if (lane == 31) s_warp[warp] = up;
    __syncthreads();
    long long before = up - sum;
    for (int i = 0; i < warp; ++i) before += s_warp[i];
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < B) s_cum[b + 1] += before;
    }
    if (tid == 0) s_cum[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  // scores (and weights) of two tiles, sums, and the queries: from there they take nothing of shared memory's bandwidth,
  // which the codes' way through it all but fills
  const uint32_t t_s[2] = {tmem, tmem + kTile}, t_o = tmem + 2 * kTile, t_q = tmem + 3 * kTile;
  const long long units = s_cum[B];
  const long long ranges = max(1LL, min(static_cast<long long>(gridDim.x), units / (kSegCost + kLeastTiles)));
  auto even_cut = [&](long long i) { return units / ranges * i + min(i, units % ranges); };
  // the even range that holds unit u
  auto owner_of = [&](long long u) {
    const long long q = units / ranges, r = units % ranges;
    return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q;
  };
  // a cut before the first tile of a (sequence, rows, head) is one before its start
  auto range_of = [&](long long i) {
    const long long u = even_cut(i);
    if (u >= units) return units;
    int lo = 0, hi = B - 1;                     // the last b with s_cum[b] <= u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_cum[mid] <= u) lo = mid; else hi = mid - 1;
    }
    int start, first, stay, n;
    seq_tiles(a, a.b.cu[lo + 1] - a.b.cu[lo], a.b.kv_len[lo], start, first, stay, n);
    const long long into = (u - s_cum[lo]) % (n + kSegCost);
    return into <= kSegCost ? u - into : u;
  };
  const long long range = blockIdx.x;
  const long long u0 = same(range < ranges ? range_of(range) : units), u1 = same(range < ranges ? range_of(range + 1) : units);

  auto locate = [&](long long u, Segment& s) {
    int lo = 0, hi = B - 1;                     // the last b with s_cum[b] <= u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_cum[mid] <= u) lo = mid; else hi = mid - 1;
    }
    s.b = lo;
    s.c0 = a.b.cu[lo];
    s.nq = a.b.cu[lo + 1] - s.c0;
    s.len = a.b.kv_len[lo];
    int n;
    seq_tiles(a, s.nq, s.len, s.start, s.first, s.stay, n);
    const int each = n + kSegCost;
    const long long pair = (u - s_cum[lo]) / each;
    s.h = static_cast<int>(pair % a.c.heads);
    s.rows0 = static_cast<int>(pair / a.c.heads) * kTile;
    s.from = s_cum[lo] + pair * each;
    s.to = s.from + each;
    s.lo = max(0, static_cast<int>(u - s.from) - kSegCost);
    s.hi = max(0, static_cast<int>(min(s.to, u1) - s.from) - kSegCost);
  };

  if (warp >= kWidenWarp && warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWidenRegs));
    // ================= codes to fp16 tiles =================
    const int w = tid - kWidenWarp * 32, part = w % kParts, half = part >> 2;
    int it = 0, stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    // this thread's parts of a tile: part w % kParts of every (kWiden / kParts)th token from w / kParts on
    auto widen = [&](uint8_t* to, uint64_t* done, uint64_t* empty, uint32_t parity, bool wait) {
      ok = __all_sync(0xffffffffu, quick_wait(&raw_full[stage], phase, &s_fail, a.err));
      if (!ok) return;
      const uint8_t* from = raw + stage * C::kRawBytes + part * 16;
      uint4 x[kEach];
#pragma unroll
      for (int n = 0; n < kEach; ++n) {
        const int token = n * (kWiden / kParts) + w / kParts;
        x[n] = *reinterpret_cast<const uint4*>(from + token * D);
        if (s_rec[it % kRecs].seen[token >> 4] == 0) x[n] = make_uint4(0, 0, 0, 0);   // nothing was copied
      }
      if (wait) ok = __all_sync(0xffffffffu, quick_wait(empty, parity, &s_fail, a.err));
      if (!ok) return;
#pragma unroll
      for (int n = 0; n < kEach; ++n) {
        const int token = n * (kWiden / kParts) + w / kParts;
        uint4 f[2];
        widen4(x[n].x, f[0].x, f[0].y), widen4(x[n].y, f[0].z, f[0].w);
        widen4(x[n].z, f[1].x, f[1].y), widen4(x[n].w, f[1].z, f[1].w);
        uint8_t* row = to + half * C::kHalf + token * 128;
        const int c = (2 * part & 7) ^ (token & 7);
        // the halves' lanes begin with different ones: no bank twice
        *reinterpret_cast<uint4*>(row + ((c ^ half) << 4)) = half ? f[1] : f[0];
        *reinterpret_cast<uint4*>(row + ((c ^ 1 ^ half) << 4)) = half ? f[0] : f[1];
      }
      fence_async_smem();
      mbar_arrive(done);
      mbar_arrive(&raw_empty[stage]);
      if (++stage == kRaw) stage = 0, phase ^= 1;
    };
    Segment s;
    for (long long u = u0; ok && u < u1; u = s.to) {
      locate(u, s);
      for (int i = s.lo; ok && i < s.hi; ++i, ++it) {
        const int st = it % kStages;
        widen(sk + st * C::kTileBytes, &k_full[st], &k_empty[st], ((it / kStages) - 1) & 1, it >= kStages);
        if (ok) widen(sv + st * C::kTileBytes, &v_full[st], &v_empty[st], ((it / kStages) - 1) & 1, it >= kStages);
      }
    }
  } else if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kMmaWarp) {
      const uint32_t leader = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t parity) { return poll_wait(bar, parity, &s_fail, a.err); };
      const uint64_t k_desc = smem_desc(smem_u32(sk), 16, 1024, kSwizzle128);
      const uint64_t v_desc = smem_desc(smem_u32(sv), C::kHalf, 1024, kSwizzle128);
      auto qk = [&](int it) {
        const int st = it % kStages;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int off = ((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4;
          lead_mma_ts(leader, t_s[it & 1], t_q + kk * 8, k_desc + (st * C::kTileBytes >> 4) + off, C::kIdescQk, kk > 0 ? 1u : 0u);
        }
        lead_commit(leader, &s_full[it & 1]);
        lead_commit(leader, &k_empty[st]);
      };
      int it = 0, segs = 0;                     // tiles and (sequence, rows, head)s so far
      bool ok = true;
      Segment s;
      for (long long u = u0; ok && u < u1; u = s.to) {
        locate(u, s);
        const int n = s.hi - s.lo;
        if (n <= 0) continue;
        ok = wait(q_ready, segs++ & 1) && wait(&k_full[it % kStages], (it / kStages) & 1);
        if (!ok) break;
        tc_fence_after();
        qk(it);
        for (int i = 0; i < n; ++i, ++it) {
          if (i + 1 < n) {
            ok = wait(&k_full[(it + 1) % kStages], ((it + 1) / kStages) & 1);
            if (!ok) break;
            qk(it + 1);
          }
          ok = wait(&p_ready[it & 1], (it >> 1) & 1) && wait(&v_full[it % kStages], (it / kStages) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            lead_mma_ts(leader, t_o, t_s[it & 1] + kk * 8, v_desc + ((it % kStages) * C::kTileBytes >> 4) + kk * (2048 >> 4),
                        C::kIdescPv, kk > 0 || i > 0 ? 1u : 0u);
          lead_commit(leader, &o_done[it & 1]);
          lead_commit(leader, &v_empty[it % kStages]);
        }
      }
      // no MMA may still run when the tensor memory is freed
      lead_commit(leader, drain);
      (void)mbar_wait(drain, 0);
    } else if (warp == kCopyWarp) {
      // ================= pages to the ring =================
      Segment s = {};
      long long u = u0;
      int i = 0;
      bool more = u0 < u1;
      auto settle = [&]() {                     // to the next tile there is
        while (i >= s.hi) {
          if (u >= u1) {
            more = false;
            return;
          }
          locate(u, s);
          u = s.to;
          i = s.lo;
        }
      };
      // The next four tiles, a lane for each of their blocks: its page, asked for four tiles before it is used, its place
      // in the page, its tokens.
      int tiles = 0, page = -1, sub = 0;
      unsigned seen = 0;
      auto look_up = [&]() {
        tiles = 0, seen = 0, page = -1;
        for (; tiles < 32 / kBlocks && more; ++tiles) {
          const int pos = s.tile(i) * kTile + lane % kBlocks * kKvBlock, pi = pos >> a.c.page_log2;
          if (lane / kBlocks == tiles && pos < s.len && (pos + kKvBlock > s.start || pos < a.sinks)) {
            seen = 0xffffu >> (kKvBlock - min(kKvBlock, s.len - pos));
            sub = (s.h << (a.c.page_log2 - 4)) + ((pos & (a.c.page - 1)) >> 4);
            page = pi < a.b.table_stride ? __ldg(a.b.table + s.b * a.b.table_stride + pi) : -1;
          }
          ++i;
          settle();
        }
      };
      if (more) settle();
      look_up();
      const int run = min(a.c.page, kTile) / kKvBlock;   // blocks side by side
      int it = 0, copied = 0, stage = 0;        // tiles and halves of tiles so far
      uint32_t phase = 1;
      bool ok = true;
      while (tiles > 0 && ok) {
        int at = -1;                            // this lane's block of the cache
        if (seen != 0) {
          if (static_cast<unsigned>(page) < static_cast<unsigned>(a.c.pages))
            at = ((page * a.c.heads) << (a.c.page_log2 - 4)) + sub;
          else
            atomicOr(a.err, kDevErrIndex);
        }
        const unsigned tokens = at >= 0 ? seen : 0u;
        const int n = tiles;
        for (int g = 0; g < n && ok; ++g, ++it) {
          const int blk = __shfl_sync(0xffffffffu, at, g * kBlocks + lane % kBlocks);
          const unsigned have = __shfl_sync(0xffffffffu, tokens, g * kBlocks + lane % kBlocks);
          const bool mine = lane < kBlocks;
          // blocks of one page lie side by side: the first one's lane copies all of them if there is any
          const unsigned any = __ballot_sync(0xffffffffu, mine && blk >= 0) >> (lane & ~(run - 1)) & ((1u << run) - 1u);
          const int from = __ffs(any) - 1, first = __shfl_sync(0xffffffffu, blk, ((lane & ~(run - 1)) + max(from, 0)) & 31) - from;
          const bool copies = mine && (lane & (run - 1)) == 0 && any != 0;
          const unsigned bytes = __popc(__ballot_sync(0xffffffffu, copies)) * run * (kKvBlock * D);
          for (int v = 0; v < 2; ++v) {
            uint64_t* bar = &raw_full[stage];
            if (copied >= kRaw) ok = __all_sync(0xffffffffu, quick_wait(&raw_empty[stage], phase, &s_fail, a.err));
            if (!ok) break;
            Rec& r = s_rec[it % kRecs];
            if (v == 0 && mine) {
              r.seen[lane] = static_cast<uint16_t>(have);
              if (blk < 0) r.ks[lane] = r.vs[lane] = 0.f;
            }
            // lane 0's arrival comes behind the lanes' stores, and so publishes them: the other arrivals of this phase
            // follow the lanes' asynchronous copies alone
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (copies)
              asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                               smem_u32(raw + stage * C::kRawBytes + lane * (kKvBlock * D))),
                           "l"((v ? a.c.v : a.c.k) + static_cast<long long>(first) * (kKvBlock * D)), "r"(run * (kKvBlock * D)),
                           "r"(smem_u32(bar))
                           : "memory");
            if (v == 0 && mine && blk >= 0) {   // the scales come with the keys
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&r.ks[lane])), "l"(a.c.ks + blk) : "memory");
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&r.vs[lane])), "l"(a.c.vs + blk) : "memory");
            }
            // an arrival of each of eight lanes, after its asynchronous copies
            if (mine) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
            ++copied;
            if (++stage == kRaw) stage = 0, phase ^= 1;
          }
          if (g == 0) look_up();                // behind the first copies: nothing waits for it yet
        }
      }
      // after a failure nobody else waits for the copies in flight
      if (s_fail)
        for (int n = max(0, copied - kRaw); n < copied; ++n) (void)mbar_wait(&raw_full[n % kRaw], (n / kRaw) & 1);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ================= softmax: two threads a row, half of a tile's tokens and of the sums each =================
    constexpr int kCols = kTile / 2, kMine = kBlocks / 2;
    const int half = warp >> 2, pair = warp & 3, r = pair * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(pair * 32) << 16;
    const uint32_t t_mine = t_o + lanes + half * (D / 2);
    int it = 0;
    Segment s;
    // after a failed wait, of whichever warp, these go on without results: they meet in barriers
    for (long long u = u0; u < u1; u = s.to) {
      locate(u, s);
      s.to = same(s.to);
      const int n = same(s.hi - s.lo), row = s.rows0 + r, j = row / p.group, head = s.h * p.group + row % p.group;
      const long long t = static_cast<long long>(s.c0) + j;
      const bool have = j < s.nq && s.c0 >= 0 && t < a.b.T;
      const int base = s.len - s.nq;
      float rowc = 0.f;
      int qpos = base + j;
      if (n > 0) {
        // the row as fp16, scaled by a power of two; the sign of `scale` goes with it
        uint4 w[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = make_uint4(0, 0, 0, 0);
        if (have) {
          const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + t * a.q_stride + head * D);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) w[i] = __ldg(q + i);
          if (a.tree) {   // as many new tokens as its path has; they are seen by their bits alone
            int path = 0;
            for (int i = 0; i < s.nq; i += 32) path += __popc(tree_word(a, t, i >> 5) & columns_to(s.nq - 1 - i));
            qpos = base + path - 1;
          }
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
        // 64 elements of it: of D = 128 half each, of D = 64 all by the first
        if (D == 128 || half == 0) {
          uint32_t packed[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 mine = D == 128 && half ? w[(D / 8 - 8) + i] : w[i];
            const uint32_t x[4] = {mine.x, mine.y, mine.z, mine.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __half2 y = __floats2half2_rn(__uint_as_float(x[k] << 16) * f, __uint_as_float(x[k] & 0xffff0000u) * f);
              packed[4 * i + k] = *reinterpret_cast<const uint32_t*>(&y);
            }
          }
          tmem_st32(t_q + lanes + 32 * half, packed);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(q_ready);
      }
      // positions the row sees: (from, to]; one that does not exist sees all, so that no tile is on its edge
      const int to = !have ? 0x7fffffff : a.tree ? base - 1 : a.causal ? qpos : s.len - 1;
      const long long lowest = have && a.window > 0 ? static_cast<long long>(qpos) - a.window : -1LL;
      const int from = lowest < -1 ? -1 : static_cast<int>(lowest);
      float m = -INFINITY, l = 0.f; // the same maximum for both threads; the sum of this one's tokens
      int e = kNoScale;             // the sums are relative to 2^e, above the value scales that the row has seen
      for (int i = 0; i < n; ++i, ++it) {
        const int t0 = s.tile(s.lo + i) * kTile + half * kCols;
        (void)quick_wait(&s_full[it & 1], (it >> 1) & 1, &s_fail, a.err);
        __syncwarp();
        tc_fence_after();
        const Rec& rec = s_rec[it % kRecs];
        const uint2 exist = *reinterpret_cast<const uint2*>(rec.seen + half * kMine);
        uint32_t bits[2] = {exist.x, exist.y};
        const bool mine = t0 + kCols - 1 > to || (t0 <= from && t0 + kCols > a.sinks) || (bits[0] & bits[1]) != ~0u;
        const bool edge = __any_sync(0xffffffffu, mine);
        uint32_t v[kCols];
#pragma unroll
        for (int x = 0; x < 2; ++x) tmem_ld32_async(t_s[it & 1] + lanes + half * kCols + 32 * x, v + 32 * x);
        const float4 ks4 = *reinterpret_cast<const float4*>(rec.ks + half * kMine), vs4 = *reinterpret_cast<const float4*>(rec.vs + half * kMine);
        const float vs[kMine] = {vs4.x, vs4.y, vs4.z, vs4.w};
        float mul[kMine] = {ks4.x * rowc, ks4.y * rowc, ks4.z * rowc, ks4.w * rowc};   // a block's scores to powers of two
        tmem_wait_ld();
        if (edge) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int at = t0 + 32 * x;
            uint32_t see = columns_to(to - at) & ~columns_to(from - at);
            if (at < a.sinks) see |= columns_to(to - at) & columns_to(static_cast<int>(min(a.sinks - at, 32LL)) - 1);
            if (a.tree && have) {
              const int k = at - base;   // place among the new tokens
              see |= __funnelshift_r(tree_word(a, t, k >> 5), tree_word(a, t, (k >> 5) + 1), k & 31);
            }
            bits[x] &= see;
          }
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (!((bits[c >> 5] >> (c & 31)) & 1u)) v[c] = 0xff800000u;
#pragma unroll
          for (int k = 0; k < kMine; ++k) mul[k] = fmaxf(mul[k], 1e-30f);   // masked scores stay -inf
        }
        float now = -INFINITY;
        int te = kNoScale;          // of the blocks that the row sees something of
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          float top = __uint_as_float(v[kKvBlock * k]);
#pragma unroll
          for (int c = 1; c < kKvBlock; ++c) top = fmaxf(top, __uint_as_float(v[kKvBlock * k + c]));
          now = fmaxf(now, top * mul[k]);
          if (top > -INFINITY && vs[k] > 0.f) te = max(te, max(-126, min(126, static_cast<int>(__float_as_uint(vs[k]) >> 23) - 126)));
        }
        // the vote: also, both have read their scores, whose place the weights take
        if (pair_any(pair, now > m + kLazy || te > e)) {   // also from -inf
          s_far[half][r] = now, s_scale[half][r] = te;
          pair_sync(pair);
          now = fmaxf(now, s_far[half ^ 1][r]), te = max(te, s_scale[half ^ 1][r]);
          const float next = fmaxf(m, now);
          const float k = next > -INFINITY ? ex2(m - next) : 1.f;
          m = next;
          l *= k;
          const float ko = k * power_of_two(e - max(e, te));
          e = max(e, te);
          if (i > 0) {
            (void)quick_wait(&o_done[(it - 1) & 1], ((it - 1) >> 1) & 1, &s_fail, a.err);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              uint32_t o[32];
              tmem_ld32_async(t_mine + 32 * x, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * ko);
              tmem_st32(t_mine + 32 * x, o);
            }
          }
        }
        const f32x2 off2 = dup2(m > -INFINITY ? kUnit - m : 0.f);
        const float unit = power_of_two(-e);   // 2^e is above the scales: a weight stays below 2^15
        f32x2 sum2[2] = {0ull, 0ull};
        uint32_t w[kCols / 2];
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          const f32x2 f = dup2(mul[k]), vk = dup2(fminf(vs[k] * unit, 1.f));   // larger: a block that the row does not see
#pragma unroll
          for (int c = k * kKvBlock / 2; c < (k + 1) * kKvBlock / 2; ++c) {
            float x, y;
            unpack2(fma2(pack2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), f, off2), x, y);
            const f32x2 two = pack2(ex2(x), ex2(y));
            sum2[c & 1] = add2(sum2[c & 1], two);
            unpack2(mul2(two, vk), x, y);
            const __half2 z = __floats2half2_rn(x, y);
            w[c] = *reinterpret_cast<const uint32_t*>(&z);
          }
        }
        tmem_st32(t_s[it & 1] + lanes + half * (kCols / 2), w);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_ready[it & 1]);
        float x, y;
        unpack2(add2(sum2[0], sum2[1]), x, y);
        l += x + y;
      }
      if (n > 0) (void)quick_wait(&o_done[(it - 1) & 1], ((it - 1) >> 1) & 1, &s_fail, a.err);
      s_far[half][r] = l;
      rows_sync();
      if (tid == 0) s_go = !s_fail;
      l = s_far[0][r] + s_far[1][r];
      rows_sync();
      const bool whole = s.from >= u0 && s.to <= u1;
      // the ranges that share what is cut, with the cuts before its tiles at its start
      auto first_owner = [&]() { return owner_of(s.from + kSegCost); };
      auto last_owner = [&]() { return owner_of(s.to - 1); };
      // by one thread: whether this CTA is the last of them, which leaves the counter at zero
      auto take_ticket = [&](long long o0, long long o1) {
        const bool last = atom_add_acq_rel_gpu(p.tickets + o0, 1u) == static_cast<unsigned>(o1 - o0);
        if (last) p.tickets[o0] = 0;
        return last;
      };
      if (!s_go) {                // the same for all of them
        if (!whole && tid == 0) take_ticket(first_owner(), last_owner());   // without a share: the next call finds all counters at zero
        continue;
      }
      tc_fence_after();
      constexpr int kShare = kTile * (D / 4 + 1);
      if (whole) {
        const float k = l > 0.f ? power_of_two(e) / l : l == 0.f ? 0.f : l;   // a row that sees nothing: zeros; a NaN stays
        if (a.lse && have && half == 0) a.lse[t * a.Hq + head] = l > 0.f ? (m + log2f(l) - kUnit) * kLn2 : l == 0.f ? -INFINITY : l;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          uint32_t o[32];
          tmem_ld32_async(t_mine + 32 * x, o);
          tmem_wait_ld();
          if (have) {
            uint4* to4 = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (t * a.Hq + head) * D + half * (D / 2) + 32 * x);
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
        tc_fence_before();
        continue;
      }
      // partial sums: slot 0 for what began in an earlier CTA, 1 for what begins here
      float4* slot = p.part + (range * 2 + (s.from >= u0 ? 1 : 0)) * kShare + r;
      const int q0 = half * (D / 8);   // this thread's first four sums
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32_async(t_mine + 32 * x, o);
          tmem_wait_ld();
        }
        if (have) {
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            reinterpret_cast<uint4*>(slot)[(q0 + 8 * x + c / 4) * kTile] = n > 0 ? make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]) : make_uint4(0, 0, 0, 0);
        }
      }
      tc_fence_before();
      if (have && half == 0) slot[D / 4 * kTile] = make_float4(m, l, __int_as_float(e), 0.f);
      rows_sync();
      const long long o0 = first_owner(), o1 = last_owner();
      if (tid == 0) s_last = take_ticket(o0, o1);
      rows_sync();
      if (s_last && have) {
        const int shares = static_cast<int>(o1 - o0) + 1;
        auto share = [&](int i) { return p.part + ((o0 + i) * 2 + (i == 0 ? 1 : 0)) * kShare + r; };
        float mm = -INFINITY;
        int ee = kNoScale;
#pragma unroll 4
        for (int i = 0; i < shares; ++i) {
          const float4 x = __ldcg(share(i) + D / 4 * kTile);
          mm = fmaxf(mm, x.x), ee = max(ee, __float_as_int(x.z));
        }
        float ll = 0.f;
#pragma unroll 4
        for (int i = 0; i < shares; ++i) {
          const float4 x = __ldcg(share(i) + D / 4 * kTile);
          ll += x.x > -INFINITY ? x.y * ex2(x.x - mm) : x.y;   // without a key: 0
        }
        const float k = ll > 0.f ? power_of_two(ee) / ll : ll == 0.f ? 0.f : ll;
        if (a.lse && half == 0) a.lse[t * a.Hq + head] = ll > 0.f ? (mm + log2f(ll) - kUnit) * kLn2 : ll == 0.f ? -INFINITY : ll;
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
          float4 y[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) y[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
          for (int i = 0; i < shares; ++i) {
            const float4* from_share = share(i);
            const float4 x = __ldcg(from_share + D / 4 * kTile);
            const float f = x.x > -INFINITY ? ex2(x.x - mm) * power_of_two(__float_as_int(x.z) - ee) : 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 z = __ldcg(from_share + (q0 + c / 4 + q) * kTile);
              y[q].x = fmaf(f, z.x, y[q].x), y[q].y = fmaf(f, z.y, y[q].y);
              y[q].z = fmaf(f, z.z, y[q].z), y[q].w = fmaf(f, z.w, y[q].w);
            }
          }
          uint4* to4 = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (t * a.Hq + head) * D + half * (D / 2) + c);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            __nv_bfloat162 z[4] = {__floats2bfloat162_rn(y[2 * q].x * k, y[2 * q].y * k), __floats2bfloat162_rn(y[2 * q].z * k, y[2 * q].w * k),
                                   __floats2bfloat162_rn(y[2 * q + 1].x * k, y[2 * q + 1].y * k),
                                   __floats2bfloat162_rn(y[2 * q + 1].z * k, y[2 * q + 1].w * k)};
            to4[q] = *reinterpret_cast<uint4*>(z);
          }
        }
      }
    }
  }
  // rows of no sequence: zeros
  const long long end = max(0, min(a.b.T, a.b.cu[B])), row_elems = static_cast<long long>(a.Hq) * D;
  const long long mine = static_cast<long long>(blockIdx.x) * kThreads + tid, step = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = end * row_elems / 8 + mine; i < a.b.T * row_elems / 8; i += step)
    static_cast<uint4*>(a.out)[i] = make_uint4(0, 0, 0, 0);
  if (a.lse)
    for (long long i = end * a.Hq + mine; i < static_cast<long long>(a.b.T) * a.Hq; i += step) a.lse[i] = -INFINITY;
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D>
cudaError_t launch(const DraftParams& p, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(q4_kv_draft_kernel<D>, Cfg<D>::smem(kKvMaxSeqs), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::smem(p.a.b.B);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_kv_draft_kernel<D>, p);
}

}  // namespace

size_t kv_draft_bytes(int dim, int sms) {
  return kv_attn_header_bytes() + static_cast<size_t>(sms) * 2 * kTile * (dim + 4) * 4;
}

cudaError_t launch_kv_draft(const KvAttnCall& a, int max_rows, void* ws, int sms, cudaStream_t st) {
  if (static_cast<size_t>(sms) * sizeof(unsigned) > kv_attn_header_bytes()) return cudaErrorInvalidConfiguration;
  DraftParams p = {};
  p.a = a;
  p.group = a.Hq / a.c.heads;
  p.max_rows = max_rows;
  p.tickets = static_cast<unsigned*>(ws);
  p.part = reinterpret_cast<float4*>(static_cast<uint8_t*>(ws) + kv_attn_header_bytes());
  return a.c.dim == 128 ? launch<128>(p, sms, st) : launch<64>(p, sms, st);
}

}  // namespace q4
