// The attention weight of cached tokens, summed over the queries that see them
// (sm_103a):
//
//   weight[h, j] (+)= sum_{t, g of h} exp(scale * q[t, g] . k_j - lse[t, g])
//
// lse comes from the attention over the same queries, so a weight needs the
// token's key and all queries, and no other token.  The work is therefore laid
// out by tokens: a warp owns blocks of 16 tokens of a head, forms their scores
// with eight query rows at a time, and adds the exponentials of a token over
// the rows.  Every sum has one owner and one order, with no atomics.
//
// * The keys are the MMA's 16 rows and eight query rows its columns: a thread
//   then holds two tokens' scores with two queries, and two exchanges end a
//   sum.  A lane's elements of a key are the 16 (D = 128: twice 16) bytes that
//   it loads; the products take the elements of queries in the same order.
// * Codes are integers up to 127, exact in fp16, as are bf16 queries scaled by
//   a power of two a row; fp32 queries are two fp16 terms (22 bits).
// * Keys are read once, through a ring of asynchronous copies of each warp; the
//   queries of a (sequence, head) lie in shared memory in the order of the
//   MMA's operand.
// * The blocks of all sequences and heads form one line, with some empty ones
//   before each (sequence, head) for what starting it costs, cut evenly over
//   the CTAs whatever the lengths.
//
// With few queries HBM bounds it at best: D + 4 bytes a token and head, against
// 2 D flops and an exponential for each query.  Measured (bf16, 32 query heads on
// 8 kv heads of 128): one or two queries of 64 sequences of 50 to 8192 tokens
// 56 us, 5.4 TB/s; instructions are issued in 67% of the cycles, over a quarter of them
// widening codes.  One query over 390 tokens of 32 heads takes 8 us in a graph, over 3000 of 8 heads too.
// Many fp32 queries have no other form: keys are read, and their codes widened, again for every 64 rows, and two
// products a pair: a prompt of 8192 takes 6.3 ms.
#include <algorithm>
#include <cfloat>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"

namespace q4 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// CTAs of an SM (with rings of 4 blocks for two of them).  One query each over 64 sequences of 50 to 8191 tokens two / three
// / four: 74 / 63 / 58 us; over 4 of 4000 9 / 10 / 12; 16 queries each over 16 of 1000 to 4000 35 / 34 / 37
constexpr int kCtas = 3;
constexpr int kStages = 2;                // blocks of a warp's ring
constexpr int kTileRows = 8;              // query rows of an MMA's columns
constexpr int kChunkTiles = 8;            // of them in shared memory at a time
constexpr int kChunkRows = kTileRows * kChunkTiles;
constexpr int kSegCost = 5 * kWarps;      // what starting a (sequence, head) costs, in blocks of one tile of rows (2 / 3 / 5 / 8 a warp: 64 / 62 / 56 / 57 us)
constexpr int kLeastUnits = 3 * kWarps;   // of a CTA, with starts: kSegCost + kWarps gave short calls too few CTAs (one query on 3000 tokens, 8 heads, 10.3 us against 7.9; on 4 x 4000 12.9 against 10.2; 64 x 50 to 8191 the same)
constexpr long long kMostCost = 4096;     // of a block, so that no line, whatever the lengths, is too long for 64 bits
constexpr int kSplitRows = 64;            // query rows of a head up to which a sequence of bf16 queries takes this form
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What the fp16 rounding `w` of (lo, hi) leaves, as fp16.
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_f16(lo - f.x, hi - f.y);
}

// The blocks of a sequence that a call reads or writes: those of the sinks, [0, sinks), and [lo, hi).
struct Blocks {
  int sinks, lo, hi;
  __device__ __forceinline__ int count() const { return sinks + hi - lo; }
  __device__ __forceinline__ int real(int i) const { return i < sinks ? i : i - sinks + lo; }
};

struct Seq {
  int c0, nq, len, held;   // packed row of its first query, queries, cached tokens, tokens that have a weight already
  Blocks blocks;
  long long rows, cost;    // query rows of a head; what a block of tokens costs, in tiles of rows
};

// max_rows: sequences with more query rows are left to the tensor cores.
__device__ __forceinline__ Seq sequence(const KvWeighCall& a, int group, int max_rows, int b) {
  Seq s;
  s.c0 = a.b.cu[b];
  s.nq = max(0, a.b.cu[b + 1] - s.c0);
  s.len = max(0, a.b.kv_len[b]);
  s.held = a.held ? max(0, min(a.held[b], s.len)) : max(0, s.len - s.nq);
  s.rows = static_cast<long long>(s.nq) * group;
  s.cost = max(1LL, min((s.rows + kTileRows - 1) / kTileRows, kMostCost));
  const int hi = (kv_tokens(a.c, a.b.table_stride, s.len) + kKvBlock - 1) / kKvBlock;
  int lo = s.nq > 0 ? 0 : hi;
  if (a.window > 0 && s.nq > 0) {
    const long long first = static_cast<long long>(s.len) - s.nq - a.window + 1;
    lo = first > 0 ? min(static_cast<int>(first / kKvBlock), hi) : 0;
  }
  if (s.held < s.len) lo = min(lo, s.held / kKvBlock);   // those from held on are written
  const int sinks = a.window > 0 && s.nq > 0
                        ? static_cast<int>(min(static_cast<long long>(lo), (a.sinks + kKvBlock - 1) / kKvBlock)) : 0;
  s.blocks = {sinks, lo, hi};
  if (s.rows > max_rows) s.blocks = {0, 0, 0};
  return s;
}

template <int D, bool SPLIT>
constexpr size_t smem_bytes(int B) {
  return static_cast<size_t>(kChunkRows) * D * 2 * (SPLIT ? 2 : 1) + kChunkRows * (8 + 8) +
         static_cast<size_t>(kWarps) * kStages * kKvBlock * D + static_cast<size_t>(B + 1) * 8;
}

// SPLIT: queries in two fp16 terms.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, kCtas) q4_kv_weigh_kernel(const __grid_constant__ KvWeighCall a, int group,
                                                                        int max_rows) {
  constexpr int KT = D / 16, kParts = D / 64;   // k steps; 16-byte parts of a key that a lane has
  constexpr int kWords = SPLIT ? 4 : 2;         // of a lane's operand of a step and tile of rows
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint32_t* s_q = reinterpret_cast<uint32_t*>(smem_raw);                   // [tile][step][lane][kWords]
  float2* s_row = reinterpret_cast<float2*>(s_q + kChunkRows * D / 2 * (SPLIT ? 2 : 1));   // score of a unit product, -lse: base 2
  int2* s_see = reinterpret_cast<int2*>(s_row + kChunkRows);               // positions a row sees: (x, y]
  uint8_t* s_ring = reinterpret_cast<uint8_t*>(s_see + kChunkRows);        // [warp][stage] a block's codes
  long long* s_cum = reinterpret_cast<long long*>(s_ring + kWarps * kStages * kKvBlock * D);   // [B + 1] first unit of each sequence
  __shared__ long long s_warp[kWarps];
  // the warp's number from one lane, so that what depends on it is known to be the same in all: exchanges of lanes behind
  // a branch that may part them take much longer (the batch above 71 us)
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), B = a.b.B;
  const int g = lane >> 2, c = lane & 3;
  // a lane copies every 32nd 16 bytes of a block; of D = 128 every other token's halves change places: no bank twice
  constexpr uint32_t kBlockBytes = kKvBlock * D, kOdd = D == 128 ? 64 : 0;
  const uint32_t ring = smem_u32(s_ring + warp * kStages * kBlockBytes);
  const uint32_t put = (lane * 16) ^ (D == 128 && (lane >> 3 & 1) ? kOdd : 0);
  const uint32_t take = (g * D + c * 16) ^ (g & 1 ? kOdd : 0);   // of token g; g + 8 is as odd
  pdl_launch_dependents();
  pdl_wait();

  // ---- the line of units ----
  {
    const int per = (B + kThreads - 1) / kThreads;
    long long sum = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < B) {
        const Seq s = sequence(a, group, max_rows, b);
        if (kv_tokens(a.c, a.b.table_stride, s.len) < s.len) atomicOr(a.err, kDevErrIndex);
        const int n = s.blocks.count();
        sum += n > 0 ? static_cast<long long>(n + kSegCost) * s.cost * a.c.heads : 0;
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
    __syncthreads();
  }
  const long long units = s_cum[B];
  const long long ranges = max(1LL, min(static_cast<long long>(gridDim.x), units / kLeastUnits));
  if (blockIdx.x >= ranges) return;
  auto range_of = [&](long long i) { return units / ranges * i + min(i, units % ranges); };
  const long long u0 = range_of(blockIdx.x), u1 = range_of(blockIdx.x + 1);

  for (long long u = u0; u < u1;) {
    // ---- the next (sequence, head), and this CTA's blocks of it ----
    int b = 0;
    for (int lo = 0, hi = B - 1; lo <= hi;) {   // the last b with s_cum[b] <= u
      const int mid = (lo + hi) >> 1;
      if (s_cum[mid] <= u) b = mid, lo = mid + 1; else hi = mid - 1;
    }
    const Seq s = sequence(a, group, max_rows, b);
    const int nb = s.blocks.count();
    const long long pair_cost = static_cast<long long>(nb + kSegCost) * s.cost;
    const int h = static_cast<int>((u - s_cum[b]) / pair_cost);
    const long long first = s_cum[b] + h * pair_cost;
    // a block belongs to the CTA whose range holds its first unit
    auto block_at = [&](long long unit) {
      return static_cast<int>(max(0LL, min(static_cast<long long>(nb), (unit - first + s.cost - 1) / s.cost - kSegCost)));
    };
    const int from = block_at(u0 > first ? u0 : first), end = block_at(min(u1, first + pair_cost));
    u = first + pair_cost;
    if (from >= end) continue;
    const int32_t* table = a.b.table + b * a.b.table_stride;

    for (long long row0 = 0; row0 == 0 || row0 < s.rows; row0 += kChunkRows) {
      const int rows = static_cast<int>(min(static_cast<long long>(kChunkRows), s.rows - row0));
      const int tiles = (rows + kTileRows - 1) / kTileRows;
      // ---- queries, a warp a row: D / 4 lanes with four elements each ----
      __syncthreads();
      for (int r = warp; r < tiles * kTileRows; r += kWarps) {
        const long long row = row0 + r;
        const int j = static_cast<int>(row / group), head = h * group + static_cast<int>(row % group);
        const bool have = r < rows && s.c0 >= 0 && s.c0 + j < a.b.T;
        const long long t = static_cast<long long>(s.c0) + j;
        const float lse = have ? __ldg(a.lse + t * a.Hq + head) : INFINITY;
        const bool adds = fabsf(lse) <= FLT_MAX;   // a row that sees nothing, or is no number, adds nothing
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (adds && lane < D / 4) {
          const long long at = t * a.q_stride + head * D + 4 * lane;
          if (a.q_bf16) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at));
            x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xffff0000u);
            x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xffff0000u);
          } else {
            const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at));
            x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
          }
        }
        const float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
        const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        // 2^(13 - exponent of the largest), within fp32's normal numbers
        const int up = top > 0.f ? max(-126, min(126, 13 + 127 - static_cast<int>(__float_as_uint(top) >> 23))) : 0;
        const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        if (lane < D / 4) {
          // element 4 lane: 16-byte part lane / 4 of the key, the step's word lane % 4 of it
          const int part = lane >> 2, step = (part >> 2) * 4 + (lane & 3);
          uint32_t* to = s_q + (((r / kTileRows) * KT + step) * 32 + (r % kTileRows) * 4 + (part & 3)) * kWords;
          const uint32_t w0 = pack_f16(x[0] * f, x[1] * f), w1 = pack_f16(x[2] * f, x[3] * f);
          if (SPLIT)
            *reinterpret_cast<uint4*>(to) = make_uint4(w0, w1, pack_rest(x[0] * f, x[1] * f, w0), pack_rest(x[2] * f, x[3] * f, w1));
          else
            *reinterpret_cast<uint2*>(to) = make_uint2(w0, w1);
        }
        if (lane == 0) {
          s_row[r] = adds ? make_float2(__uint_as_float(static_cast<uint32_t>(127 - up) << 23) * a.scale * kLog2e, -lse * kLog2e)
                          : make_float2(0.f, -INFINITY);
          const int pos = s.len - s.nq + j;
          const long long lo = a.window > 0 ? static_cast<long long>(pos) - a.window : -1LL;
          s_see[r] = make_int2(lo < -1 ? -1 : static_cast<int>(lo), !adds ? -1 : a.causal ? pos : s.len - 1);
        }
      }
      __syncthreads();
      // blocks that every row of the chunk sees whole, and those that any sees something of
      const int p0 = s.len - s.nq + static_cast<int>(row0 / group), p1 = s.len - s.nq + static_cast<int>((row0 + max(rows, 1) - 1) / group);
      const int whole_hi = max(0, a.causal ? p0 + 1 : s.len) / kKvBlock;
      const int whole_lo = a.window > 0 && p1 >= a.window ? static_cast<int>((p1 - a.window + kKvBlock) / kKvBlock) : 0;
      const long long seen_lo = a.window > 0 ? p0 - a.window + 1 : 0;   // first position in p0's window
      const int seen_hi = a.causal ? p1 : s.len - 1;
      auto is_seen = [&](int blk) {
        return rows > 0 && blk * kKvBlock <= seen_hi && (blk * kKvBlock + kKvBlock > seen_lo || blk * kKvBlock < a.sinks);
      };
      // ---- the warp's blocks, 32 of them at a time: a lane looks one up ----
      for (int i0 = from + warp; i0 < end; i0 += 32 * kWarps) {
        const int count = min(32, (end - i0 + kWarps - 1) / kWarps);
        int my_at = -1, my_blk = 0;               // block of the cache (-1: nothing to do), block of the sequence
        unsigned my_kind = 0;                     // bit 0: some row sees of it, bit 1: not every row sees all of it
        float my_scale = 0.f;
        if (lane < count) {
          my_blk = s.blocks.real(i0 + lane * kWarps);
          const int pi = (my_blk * kKvBlock) >> a.c.page_log2;
          const int page = pi < a.b.table_stride ? __ldg(table + pi) : -1;
          const bool seen = is_seen(my_blk);
          if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.c.pages)) {
            atomicOr(a.err, kDevErrIndex);
          } else if (seen || row0 == 0) {
            my_at = ((page * a.c.heads + h) << (a.c.page_log2 - 4)) + (my_blk & ((a.c.page >> 4) - 1));
            const bool edge = my_blk >= whole_hi || (my_blk < whole_lo && (my_blk + 1LL) * kKvBlock > a.sinks);
            my_kind = (seen ? 1u : 0u) | (edge ? 2u : 0u);
            if (seen) my_scale = __ldg(a.c.ks + my_at);
          }
        }
        // keys of the block that lane n looked up; always closes a group, so that groups count blocks
        auto copy = [&](int n, uint32_t to) {
          const int at = __shfl_sync(0xffffffffu, my_at, n & 31);
          const unsigned kind = __shfl_sync(0xffffffffu, my_kind, n & 31);
          if (n < count && at >= 0 && (kind & 1u)) {
            const int8_t* from_k = a.c.k + static_cast<long long>(at) * kBlockBytes + lane * 16;
#pragma unroll
            for (uint32_t x = 0; x < kBlockBytes / 512; ++x)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + put + x * 512), "l"(from_k + x * 512) : "memory");
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto work = [&](int n, uint32_t block) {
          const int at = __shfl_sync(0xffffffffu, my_at, n);
          const unsigned kind = __shfl_sync(0xffffffffu, my_kind, n);
          if (at < 0) return;
          const int blk = __shfl_sync(0xffffffffu, my_blk, n);
          // this lane's token (c = 0: g, c = 1: g + 8) and what it has already
          const int pos = blk * kKvBlock + g + 8 * c;
          float* w = a.weight + static_cast<long long>(at) * kKvBlock + g + 8 * c;
          const bool mine = c < 2 && pos < s.len;
          const float had = mine && (row0 > 0 || pos < s.held) ? *w : 0.f;
          float sum[2] = {0.f, 0.f};
          if (kind & 1u) {
            const float ks = __shfl_sync(0xffffffffu, my_scale, n);
            uint4 k[2][kParts];
#pragma unroll
            for (int x = 0; x < kParts; ++x) {
              const uint32_t from_k = block + (take ^ (64 * x));
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(k[0][x].x), "=r"(k[0][x].y), "=r"(k[0][x].z), "=r"(k[0][x].w) : "r"(from_k));
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(k[1][x].x), "=r"(k[1][x].y), "=r"(k[1][x].z), "=r"(k[1][x].w) : "r"(from_k + 8 * D));
            }
            for (int t8 = 0; t8 < tiles; ++t8) {
              float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
              const uint32_t* q = s_q + (t8 * KT * 32 + lane) * kWords;
#pragma unroll
              for (int t = 0; t < KT; ++t) {
                const uint4 x = k[0][t >> 2], y = k[1][t >> 2];
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
                uint32_t f[4];
                widen4(xw[t & 3], f[0], f[2]);
                widen4(yw[t & 3], f[1], f[3]);
                if (SPLIT) {
                  const uint4 z = *reinterpret_cast<const uint4*>(q + t * 32 * kWords);
                  mma(acc[0], f, z.x, z.y);
                  mma(acc[1], f, z.z, z.w);
                } else {
                  const uint2 z = *reinterpret_cast<const uint2*>(q + t * 32 * kWords);
                  mma(acc[t & 1], f, z.x, z.y);
                }
              }
              // the thread's queries 2 c and 2 c + 1 of the tile
              const float4 r = *reinterpret_cast<const float4*>(s_row + t8 * kTileRows + 2 * c);
              const float f0 = ks * r.x, f1 = ks * r.z;
              float e[4];
              e[0] = fmaf(acc[0][0] + acc[1][0], f0, r.y), e[1] = fmaf(acc[0][1] + acc[1][1], f1, r.w);
              e[2] = fmaf(acc[0][2] + acc[1][2], f0, r.y), e[3] = fmaf(acc[0][3] + acc[1][3], f1, r.w);
              if (kind & 2u) {
                const int4 see = *reinterpret_cast<const int4*>(s_see + t8 * kTileRows + 2 * c);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                  const int p = blk * kKvBlock + g + (v >> 1) * 8, lo = v & 1 ? see.z : see.x, hi = v & 1 ? see.w : see.y;
                  if (p > hi || (p <= lo && p >= a.sinks)) e[v] = -INFINITY;
                }
              }
              sum[0] += ex2(e[0]) + ex2(e[1]);
              sum[1] += ex2(e[2]) + ex2(e[3]);
            }
            // the lanes of c = 0, 2 end the first token's sum, those of c = 1, 3 the second's
            const float keep = c & 1 ? sum[1] : sum[0], give = c & 1 ? sum[0] : sum[1];
            sum[0] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], 2);
          }
          if (mine && (kind & 1u || pos >= s.held)) *w = had + sum[0];
        };
        uint32_t stage = ring;
        auto next = [&](uint32_t at) { return at + kBlockBytes == ring + kStages * kBlockBytes ? ring : at + kBlockBytes; };
#pragma unroll
        for (int n = 0; n < kStages; ++n) copy(n, ring + n * kBlockBytes);
        for (int n = 0; n < count; ++n) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
          __syncwarp();
          work(n, stage);
          __syncwarp();
          copy(n + kStages, stage);
          stage = next(stage);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
      }
    }
  }
}

template <int D, bool SPLIT>
cudaError_t launch(const KvWeighCall& a, int group, int max_rows, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(q4_kv_weigh_kernel<D, SPLIT>, smem_bytes<D, SPLIT>(kKvMaxSeqs), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms * kCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D, SPLIT>(a.b.B);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_kv_weigh_kernel<D, SPLIT>, a, group, max_rows);
}

}  // namespace

cudaError_t launch_kv_weigh(const KvWeighCall& a, long long max_q, int sms, cudaStream_t st) {
  const int group = a.Hq / a.c.heads;
  const long long most = std::min<long long>(max_q, a.b.T) * group;
  const bool prompt = a.q_bf16 && most > kSplitRows && group <= kv_weigh_prompt_group();
  if (prompt && a.b.B == 1) return launch_kv_weigh_prompt(a, 0, sms, st);
  const int max_rows = prompt ? kSplitRows : 0x7fffffff;
  cudaError_t e;
  if (a.c.dim == 128)
    e = a.q_bf16 ? launch<128, false>(a, group, max_rows, sms, st) : launch<128, true>(a, group, max_rows, sms, st);
  else
    e = a.q_bf16 ? launch<64, false>(a, group, max_rows, sms, st) : launch<64, true>(a, group, max_rows, sms, st);
  return e == cudaSuccess && prompt ? launch_kv_weigh_prompt(a, kSplitRows, sms, st) : e;
}

}  // namespace q4
