// Attention over the paged 8-bit cache, split over the cached tokens
// (sm_103a): the form for few new tokens a sequence.
//
//   out[t, h] = sum_j p_j v_j,  p = softmax_j(scale * q[t, h] . k_j)
// over the cached tokens j that the query sees.  With few queries this reads
// each code once and does 4 D flops for it and each query that shares it: HBM
// bounds it, so the work is laid out by the codes.
//
// * The unit of work is a block: 16 tokens of one kv head, for one tile of
//   query rows (the queries that share the head: token-major, up to 16 rows).
//   The units of all sequences, heads and tiles form one line (with some empty
//   ones before each (sequence, tile, head), for what starting one costs), which
//   is cut into equal ranges, whatever the sequences' lengths.  A range is
//   worked on by a team of warps, a whole CTA or a quarter of one.  A team whose
//   range begins or ends inside a (sequence, tile, head) writes its share of the
//   sum (with the maximum and the weights' sum) to the workspace; the last of
//   the teams that share it adds the shares in order.
// * Each warp of a team streams blocks of its own (every fourth or sixteenth)
//   through its own ring of asynchronous copies, so that no warp waits for
//   another until the shares of the warps are added.
// * Codes are integers up to 127, exact in fp16, as are bf16 queries scaled
//   by a power of two per row; fp32 queries and the softmax weights are split
//   into two fp16 terms (22 bits) that fill the two halves of the MMA's 16
//   rows (SPLIT: 8 rows of queries), so fp32 calls keep fp32 accuracy at the
//   same cost.  Products accumulate in fp32.
// * A block's scale is one number per MMA tile: the key scale multiplies the
//   scores, the value scale the weights, relative to the largest so far.
//
// Measured (8 kv heads of 128, 32 query heads, bf16): 64 sequences of 4096
// tokens 96 us, 5.6 TB/s of codes and scales; 64 sequences of 50 to 8191
// tokens 96 us, 5.5 TB/s; one of 131,071 54 us, 4.9 TB/s; one of 390 with 32
// kv heads 10 us.  HBM is 70% busy on the long ones; the rest is the widening
// of codes to fp16: about 430 instructions for each block and warp, of which
// 32 are MMAs and 180 turn codes into fp16 pairs, issued in 51% of the cycles
// by the 16 warps that 128 registers a thread leave room for.  Short ones wait
// for a chain of page lookup, copy, product and join.
// Two blocks a step, under one softmax, need more registers than there are
// (an earlier step: 136 us for 127).
#include <algorithm>
#include <cfloat>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"

namespace q4 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;                 // rows of an MMA tile
constexpr int kTeams = 4;                 // teams of a CTA at most
constexpr int kStages = 2;                // ring stages of a warp, one block each
// Weight of the softmax reference with the value scale the sums are relative to.  The reference moves once a
// score exceeds it by 2^kLazy, or a value scale kMoreScale times (moving costs a multiplication of every sum);
// the weight is as large as that leaves of fp16's range (2^9 * 2^4 * 4 < 65504).  fp16 holds a weight to 11
// bits down to 2^-23 of the reference and to within 2^-34 of it below that.  With SPLIT the second term is
// the rest times kRestScale, so that the two hold 22 bits, and within 2^-45: small weights can matter
// together, where the largest weight's value is near zero.
constexpr float kUnitWeight = 512.0f;
constexpr float kLazy = 4.0f;
constexpr float kMoreScale = 4.0f;
constexpr float kRestScale = 2048.0f;
constexpr float kLog2e = 1.4426950408889634f;

struct AttnParams {
  KvAttnCall a;
  int group;                              // query heads of one kv head
  int max_rows;                           // sequences with more query rows are left to the prompt form
  unsigned* tickets;                      // [ranges], zero
  float* part;                            // [ranges][2][kRows][dim + 2] shares
};

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

// The first product of a sum.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// `scale` times the rest of (lo, hi) that its fp16 rounding `w` leaves, as fp16.
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t w, float scale) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_f16((lo - f.x) * scale, (hi - f.y) * scale);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// Two 16 x 16 byte matrices, transposed: lane l gives the address of row l % 16 of matrix l / 16; register
// 2 m + x gets rows 4 (l % 4) .. + 3 of column 8 x + l / 4 of matrix m.
__device__ __forceinline__ uint4 ldmatrix_t8(uint32_t a) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// One (sequence, row tile, kv head) of the line of units, and the blocks a CTA takes of it.
struct Segment {
  int b, h, tile;
  int c0, nq, len;         // packed row of the first new token, new tokens, cached tokens
  int lo, hi;              // this CTA's blocks (maybe none)
  long long first, last;   // units of the whole (sequence, tile, head): [first, last)
};

template <int D>
struct Stage {
  static constexpr int kCodes = kKvBlock * D;           // bytes of keys (values)
  static constexpr int kBytes = 2 * kCodes;
};

template <int D>
constexpr size_t smem_bytes(int B) {
  return kStages * Stage<D>::kBytes + static_cast<size_t>(kWarps) * kStages * Stage<D>::kBytes +   // rings
         static_cast<size_t>(kWarps / 2) * kRows * (D + 8) * 4 +                    // the warps' sums, two after one another
         static_cast<size_t>(kWarps) * kRows * 2 * 4 +                        // their maxima and weights
         static_cast<size_t>(kWarps) * kStages * 8 +                          // scales
         static_cast<size_t>(B + 1) * 8 + 64;
}

// Range of blocks [lo, hi) the queries of a sequence may see, at least one block where there are queries.
__device__ __forceinline__ void seq_blocks(const KvAttnCall& a, int nq, int len, int& lo, int& hi) {
  hi = max(1, (len + kKvBlock - 1) / kKvBlock);
  lo = 0;
  if (a.window > 0) {
    const long long first = a.causal ? static_cast<long long>(len) - nq - a.window + 1 : 0;
    lo = first > 0 ? min(static_cast<int>(first / kKvBlock), hi - 1) : 0;
  }
}

// Four elements (d ..) of query row `row` (token-major) of a (sequence, head), v over the weights' sum l.
template <int D>
__device__ __forceinline__ void store4(const AttnParams& p, const Segment& s, int row, int d, float4 v, float l) {
  const KvAttnCall& a = p.a;
  const int j = row / p.group;
  if (s.c0 < 0 || s.c0 + j >= a.b.T) return;
  const long long at = ((static_cast<long long>(s.c0) + j) * a.Hq + s.h * p.group + row % p.group) * D + d;
  auto over = [&](float y) { return l > 0.f ? y / l : l == 0.f ? 0.f : l; };   // no key: zeros; a NaN stays
  v = make_float4(over(v.x), over(v.y), over(v.z), over(v.w));
  if (a.out_bf16) {
    __nv_bfloat162 y[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) = *reinterpret_cast<uint2*>(y);
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
  }
}

// Barrier of a team's threads.
template <int CREW>
__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(CREW) : "memory");
}

// The sum of all shares of a (sequence, tile, head), the first in range o0, by the team that arrived last.  t_o, s_m,
// s_l: shared memory of the team and of all warps.  Every share's factor is found once, and a thread's elements of
// several shares are on their way together (an element at a time with its factors: the ragged batch 103 us for 96,
// one sequence of 16,000 tokens 31 us for 22).
template <int D, int ROWS, int TEAM>
__device__ __forceinline__ void join(const AttnParams& p, const Segment& s, int row0, int rows, long long o0, int shares,
                                  int team, int mine, float* t_o, float* s_m, float* s_l) {
  constexpr int crew = TEAM * 32, kVecs = D / 4, kORow = D + 8;
  const int lane = mine & 31, warp = team * TEAM + (mine >> 5);
  auto share = [&](int i) {
    return p.part + ((o0 + i) * 2 + (i == 0 ? 1 : 0)) * kRows * (D + 2);
  };
  // a thread for each row and some of the shares: the maximum, then every share's factor
  const int r = mine % kRows, k0 = mine / kRows;
  constexpr int kPer = ROWS * kVecs > crew ? ROWS * kVecs / crew : 1;
  constexpr int kParts = kPer > 1 ? 0 : 3 * crew;   // t_o's last floats: sums of other threads
  constexpr int kStep = crew / kRows, kChunk = (TEAM / 2 * kRows * kORow - kParts) / kRows;   // factors it has room for
  // with few rows several threads take shares in turn for the same elements
  const int elems = rows * kVecs, groups = kPer > 1 || 2 * elems > crew ? 1 : 4 * elems > crew ? 2 : 4;
  const int span = crew / groups, group = mine / span, mine_at = mine % span;
  float m = -INFINITY, l = 0.f;
  for (int k = k0; k < shares; k += kStep) m = fmaxf(m, __ldcg(share(k) + kRows * D + r));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, kRows));
  if (lane < kRows) s_m[warp * kRows + r] = m;
  team_sync<crew>(team);
#pragma unroll
  for (int w = 0; w < TEAM; ++w) m = fmaxf(m, s_m[(team * TEAM + w) * kRows + r]);
  float4 v[kPer];
#pragma unroll
  for (int n = 0; n < kPer; ++n) v[n] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < shares; base += kChunk) {
    const int end = min(shares, base + kChunk);
    for (int k = base + k0; k < end; k += kStep) {
      const float* q = share(k) + kRows * D + r;
      const float mk = __ldcg(q), f = mk > -INFINITY ? ex2(mk - m) : 0.f;
      l += f * __ldcg(q + kRows);
      t_o[(k - base) * kRows + r] = f;
    }
    team_sync<crew>(team);
#pragma unroll 4
    for (int k = base + group; k < end; k += groups) {
#pragma unroll
      for (int n = 0; n < kPer; ++n) {
        const int i = mine_at + n * crew;
        if (i < elems) {
          const float f = t_o[(k - base) * kRows + i / kVecs];
          const float4 x = __ldcg(reinterpret_cast<const float4*>(share(k) + 4 * i));
          v[n].x = fmaf(f, x.x, v[n].x), v[n].y = fmaf(f, x.y, v[n].y);
          v[n].z = fmaf(f, x.z, v[n].z), v[n].w = fmaf(f, x.w, v[n].w);
        }
      }
    }
    team_sync<crew>(team);
  }
  l += __shfl_xor_sync(0xffffffffu, l, kRows);
  if (lane < kRows) s_l[warp * kRows + r] = l;
  float4* parts = reinterpret_cast<float4*>(t_o + TEAM / 2 * kRows * kORow - kParts);
  if (group > 0 && mine_at < elems) parts[(group - 1) * elems + mine_at] = v[0];
  team_sync<crew>(team);
  if (group > 0) return;
  for (int n = 1; n < groups && mine_at < elems; ++n) {
    const float4 x = parts[(n - 1) * elems + mine_at];
    v[0].x += x.x, v[0].y += x.y, v[0].z += x.z, v[0].w += x.w;
  }
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    const int i = mine_at + n * crew;
    if (i >= elems) continue;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < TEAM; ++w) sum += s_l[(team * TEAM + w) * kRows + i / kVecs];
    store4<D>(p, s, row0 + i / kVecs, i % kVecs * 4, v[n], sum);
  }
}

// SPLIT: the 16 rows of an MMA tile are 8 query rows in two fp16 terms each; else 16 in one term.
// TEAM: warps that take a range of units together.
template <int D, bool SPLIT, int TEAM>
__global__ void __launch_bounds__(kThreads, 1) q4_kv_attn_split_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kE = SPLIT ? 1 : 2;             // query rows of a thread
  // what starting and ending a (sequence, tile, head) costs, in units: more where all of a CTA's warps wait for it
  // (16 / 24 / 32 / 40: 64 sequences of 50 to 8191 tokens in quarters 109 / 103 / 104 / 107 us, 12 of 700 to 5000
  // with a window of 2048 in whole CTAs 20.5 / 20.5 / 18.7 / 18.9 us)
  constexpr int kSegCost = TEAM == kWarps ? 32 : 24;
  constexpr int kTileRows = 8 * kE;             // query rows of a tile
  constexpr int KT = D / 16;                    // k steps of q . k
  constexpr int NT = D / 8;                     // column tiles of p . v
  constexpr uint32_t kStageBytes = Stage<D>::kBytes;
  constexpr uint32_t kRingAlign = kStages * kStageBytes;   // the other stage, and places in one, by exclusive or
  static_assert(kStages == 2, "stages take turns");
  constexpr int kORow = D + 8;                  // floats between rows of the warps' sums: other banks
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + kRingAlign - 1) & ~uintptr_t(kRingAlign - 1));
  float* s_o = reinterpret_cast<float*>(ring + kWarps * kStages * kStageBytes);   // [warp][row][kORow]
  float* s_m = s_o + kWarps / 2 * kRows * kORow;                                           // [warp][row]
  float* s_l = s_m + kWarps * kRows;
  float* s_scale = s_l + kWarps * kRows;                                           // [warp][stage][2]
  long long* s_cum = reinterpret_cast<long long*>(s_scale + kWarps * kStages * 2); // [B + 1] first unit of each sequence
  __shared__ int s_last[kTeams];
  __shared__ float s_rowf[kTeams][kRows];       // score of a unit product
  __shared__ int2 s_see[kTeams][kRows];         // positions a row sees: (x, y]
  __shared__ float s_tot[kTeams][2][kRows];     // maximum, weights' sum
  __shared__ long long s_warp[kWarps];
  __shared__ int s_pairs;                       // (sequence, tile, head)s; more than the grid: any such number
  __shared__ int s_longest;                     // units of the longest of them

  const KvAttnCall& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;        // MMA row (and column group), thread in group
  // the warp's team: its number, the warp's place in it, threads; its sums' slots (two warps each), which hold
  // the queries until the sums are there
  constexpr int crew = TEAM * 32;
  const int team = warp / TEAM, mate = warp % TEAM, mine = mate * 32 + lane;
  float* t_o = s_o + team * TEAM / 2 * kRows * kORow;
  uint4* s_q = reinterpret_cast<uint4*>(t_o);   // [k step][lane] A operand
  if (tid == 0) s_pairs = s_longest = 0;
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();

  // ---- the line of units ----
  const int B = a.b.B;
  {
    const int per = (B + kThreads - 1) / kThreads;
    long long sum = 0, pairs = 0;
    int longest = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < B) {
        const int nq = a.b.cu[b + 1] - a.b.cu[b];
        int lo, hi;
        seq_blocks(a, nq, a.b.kv_len[b], lo, hi);
        const long long rows = static_cast<long long>(nq) * p.group;
        const long long tiles = nq > 0 && rows <= p.max_rows ? (rows + kTileRows - 1) / kTileRows : 0;
        const long long n = tiles * a.c.heads * (hi - lo + kSegCost);
        s_cum[b + 1] = sum + n;
        sum += n;
        pairs += tiles * a.c.heads;
        if (tiles > 0) longest = max(longest, hi - lo + kSegCost);
      }
    }
    long long up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    if (lane == 31) s_warp[warp] = up;
    if (longest > 0) atomicMax(&s_longest, longest);
    if (pairs > 0) atomicAdd(&s_pairs, static_cast<int>(min(pairs, 1LL << 18)));   // kThreads of them fit an int
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
  // as many ranges as have a block for every warp of a team; where there is one for each (sequence, tile, head) and
  // these are of one length or nearly, the same number for each, so that they begin with a range and few are cut (64
  // sequences of 4096 tokens 96 us, 102 us cut anywhere; of 50 to 8191 tokens 112 us so, 103 us cut anywhere)
  const long long pairs = max(1, s_pairs), most = static_cast<long long>(gridDim.x) * (kWarps / TEAM);
  long long ranges = min(most, units / (TEAM + kSegCost));
  const bool even = pairs <= most && s_longest * pairs <= units + units / 16;
  ranges = even ? pairs * max(1LL, ranges / pairs) : max(1LL, ranges);
  auto range_of = [&](long long i) { return units * i / ranges; };
  // the range that holds unit u
  auto owner_of = [&](long long u) { return ((u + 1) * ranges - 1) / units; };
  const long long range = static_cast<long long>(team) * gridDim.x + blockIdx.x;   // few ranges: one to an SM
  const long long u0 = range < ranges ? range_of(range) : units;
  const long long u1 = range < ranges ? range_of(range + 1) : units;

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
    int b0, b1;
    seq_blocks(a, s.nq, s.len, b0, b1);
    const int nb = b1 - b0 + kSegCost;
    const long long in = u - s_cum[lo], pair = in / nb;
    s.h = static_cast<int>(pair % a.c.heads);
    s.tile = static_cast<int>(pair / a.c.heads);
    s.first = s_cum[lo] + pair * nb;
    s.last = s.first + nb;
    s.lo = b0 + max(0, static_cast<int>(u - s.first) - kSegCost);
    s.hi = b0 + max(0, static_cast<int>(min(s.last, u1) - s.first) - kSegCost);
  };

  // ---- the warp's stream of blocks: copies run kStages - 1 blocks ahead of the one in work ----
  // A block of keys (values) is consecutive; a lane copies every 32nd 16 bytes of it, to its swizzled place.
  const uint32_t my_ring = smem_u32(ring + warp * kStages * kStageBytes);
  const uint32_t my_scale = smem_u32(s_scale + warp * kStages * 2);
  const int sub_mask = (a.c.page >> 4) - 1, sub_log2 = a.c.page_log2 - 4;   // blocks of a page
  const int crow = D == 128 ? lane >> 3 : lane >> 2;
  const uint32_t cput = crow * D + (D == 128 ? ((lane & 7) ^ crow) << 4 : ((lane & 3) ^ ((crow >> 1) & 3)) << 4);
  Segment ps = {};                              // the copies' segment
  const int32_t* ptable = nullptr;              // its row of the page table
  unsigned ppages = 0;                          // pages it may have (a sequence without tokens: none)
  long long pu = u0;                            // its first unit
  int pblk = 0, ppage = -1;                     // the next block, that block's page
  bool more = u0 < u1;
  // to the warp's next block at or after pblk, through the segments
  auto settle = [&]() {
    while (pblk >= ps.hi) {
      if (pu >= u1) {
        more = false;
        return;
      }
      locate(pu, ps);
      ptable = a.b.table + ps.b * a.b.table_stride;
      ppages = ps.len > 0 ? static_cast<unsigned>(a.c.pages) : 0u;
      pu = ps.last;
      pblk = ps.lo + mate;
    }
    const int pi = pblk >> sub_log2;
    ppage = pi < a.b.table_stride ? __ldg(ptable + pi) : -1;
  };
  if (more) settle();
  uint32_t put = my_ring + cput, put_scale = my_scale + 4 * lane;   // in the stage to fill next
  // copies one block, if there is one; always closes a group, so that groups count stages
  auto produce = [&]() {
    if (more) {
      if (static_cast<unsigned>(ppage) < ppages) {
        // below 2^31: the call's checks
        const uint32_t at = (static_cast<uint32_t>(ppage * a.c.heads + ps.h) << sub_log2) + (pblk & sub_mask);
        const int8_t* k = a.c.k + static_cast<uint64_t>(at) * Stage<D>::kCodes + lane * 16;
        const int8_t* v = a.c.v + static_cast<uint64_t>(at) * Stage<D>::kCodes + lane * 16;
#pragma unroll
        for (int i = 0; i < Stage<D>::kCodes / 512; ++i) {
          const uint32_t to = (D == 128 && (i & 1) ? put ^ 64 : put) + i * 512;   // four rows on: that bit
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(k + i * 512) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + Stage<D>::kCodes), "l"(v + i * 512) : "memory");
        }
        if (lane < 2)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(put_scale), "l"((lane ? a.c.vs : a.c.ks) + at) : "memory");
      } else {                                  // no such page, or a sequence without tokens: a block nobody sees
        if (lane == 0 && ps.len > 0) atomicOr(a.err, kDevErrIndex);
        if (lane < 2) asm volatile("st.shared.f32 [%0], %1;" ::"r"(put_scale), "f"(lane ? 0.0f : -1.0f) : "memory");
      }
      put ^= kStageBytes, put_scale ^= 8;
      pblk += TEAM;
      settle();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) produce();

  // ---- segments ----
  const uint32_t qb = smem_u32(s_q + lane);
  // swizzled places of the thread's keys in a stage (plus 2 rows, the bit that differs, for the second tile) and
  // of its values (the chunk's bits change with the matrices)
  const int krow = 4 * (g >> 1) + (g & 1), vrow = lane & 15;
  const uint32_t koff = krow * D + ((D == 128 ? (2 * c) ^ (krow & 7) : c ^ ((krow >> 1) & 3)) << 4);
  const uint32_t voff = Stage<D>::kCodes + vrow * D + (((lane >> 4) ^ (D == 128 ? vrow & 7 : (vrow >> 1) & 3)) << 4);
  constexpr uint32_t kTileBit = D == 128 ? 32 : 16;   // two rows on: row bits 1 and up turn this chunk bit
  uint32_t take_k = my_ring ^ koff, take_v = my_ring ^ voff, take_scale = my_scale;   // in the stage to read next
  long long u = u0;
  while (u < u1) {
    Segment s;
    locate(u, s);
    const int row0 = s.tile * kTileRows;        // first row of the tile: row = token * group + head in group
    const int rows = min(kTileRows, s.nq * p.group - row0);
    // this thread's rows
    int qpos[2];                                // their positions
    bool have[2] = {false, false};
    long long qoff[2];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int r = g + 8 * e;
      const int j = (row0 + r) / p.group;
      qpos[e] = s.len - s.nq + j;               // below 0 (causal): it sees nothing
      have[e] = r < rows && s.c0 >= 0 && s.c0 + j < a.b.T;
      qoff[e] = (static_cast<long long>(s.c0) + j) * a.q_stride + (s.h * p.group + (row0 + r) % p.group) * D;
    }
    // queries as fp16, scaled by a power of two per row into fp16's range: the thread's
    // elements of a row are (D / 4) c + 0 .. D / 4 - 1, four for each k step
    if (mate == 0) {
      uint32_t qf[KT][4];
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        float x[D / 4];
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
        if (have[e]) {
          if (a.q_bf16) {
            const uint2* q = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + qoff[e] + c * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint2 w = __ldg(q + i);
              x[4 * i] = __uint_as_float(w.x << 16), x[4 * i + 1] = __uint_as_float(w.x & 0xffff0000u);
              x[4 * i + 2] = __uint_as_float(w.y << 16), x[4 * i + 3] = __uint_as_float(w.y & 0xffff0000u);
            }
          } else {
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + qoff[e] + c * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const float4 w = __ldg(q + i);
              x[4 * i] = w.x, x[4 * i + 1] = w.y, x[4 * i + 2] = w.z, x[4 * i + 3] = w.w;
            }
          }
        }
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) m = fmaxf(m, fabsf(x[i]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // 2^(13 - exponent of m), within fp32's normal numbers
        const int up = m > 0.f ? max(-126, min(126, 13 + 127 - static_cast<int>(__float_as_uint(m) >> 23))) : 0;
        const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        const float rowf = __uint_as_float(static_cast<uint32_t>(127 - up) << 23) * a.scale * kLog2e;
        if (c == 0) {
          const long long from = a.window > 0 && a.causal ? static_cast<long long>(qpos[e]) - a.window : -1LL;
          s_rowf[team][g + 8 * e] = rowf;
          s_see[team][g + 8 * e] = make_int2(from < -1 ? -1 : static_cast<int>(from),
                                             !have[e] ? -1 : a.causal ? qpos[e] : s.len - 1);
        }
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x0 = x[4 * t + 2 * i] * f, x1 = x[4 * t + 2 * i + 1] * f;
            qf[t][e + 2 * i] = pack_f16(x0, x1);
            if (SPLIT) qf[t][1 + 2 * i] = pack_rest(x0, x1, qf[t][2 * i], 1.0f);
          }
      }
#pragma unroll
      for (int t = 0; t < KT; ++t) s_q[t * 32 + lane] = make_uint4(qf[t][0], qf[t][1], qf[t][2], qf[t][3]);
    }
    team_sync<crew>(team);
    float rowf[2];
#pragma unroll
    for (int e = 0; e < kE; ++e) rowf[e] = s_rowf[team][g + 8 * e];
    // blocks that every row of the tile sees whole (rows are in the order of their positions)
    int inner_lo, inner_hi;
    {
      const int p0 = s.len - s.nq + row0 / p.group, p1 = s.len - s.nq + (row0 + rows - 1) / p.group;
      inner_hi = max(0, a.causal ? p0 + 1 : s.len) / kKvBlock;
      inner_lo = a.window > 0 && p1 >= a.window ? static_cast<int>((p1 - a.window + kKvBlock) / kKvBlock) : 0;
    }
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float mref[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
    float vref = 0.f, vinv = 0.f;               // value scale the sums are relative to, kUnitWeight over it

    for (int blk = s.lo + mate; blk < s.hi; blk += TEAM) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      float ks, vs;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs) : "r"(take_scale));
      // scores: column n of tile j is token 4 (n / 2) + 2 j + n % 2 of the block, so that the thread's four
      // columns are the tokens 4 c .. 4 c + 3
      uint32_t kw[2][D / 16];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint4 x = lds128(take_k ^ (2 * j * D + j * kTileBit + (i << 4)));
          kw[j][4 * i] = x.x, kw[j][4 * i + 1] = x.y, kw[j][4 * i + 2] = x.z, kw[j][4 * i + 3] = x.w;
        }
      float sc[2][4];
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const uint4 x = lds128(qb + t * 512);
        const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t b0, b1;
          widen4(kw[j][t], b0, b1);
          if (t == 0) mma_first(sc[j], q, b0, b1); else mma(sc[j], q, b0, b1);
        }
      }
      uint4 vw[D / 32];
#pragma unroll
      for (int m = 0; m < D / 32; ++m) {
        vw[m] = ldmatrix_t8(take_v ^ (m << 5));
      }
      // scaled scores of the thread's rows, four columns each
      float x[2][4];
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float f = ks * rowf[e];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[e][i] = (SPLIT ? sc[i >> 1][i & 1] + sc[i >> 1][2 + (i & 1)] : sc[i >> 1][2 * e + (i & 1)]) * f;
      }
      if (blk < inner_lo || blk >= inner_hi || ks < 0.f) {   // some row does not see all of the block
        const int pos = blk * kKvBlock + 4 * c;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const int2 see = s_see[team][g + 8 * e];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (pos + i <= see.x || pos + i > see.y || ks < 0.f) x[e][i] = -INFINITY;
        }
      }
      // the references move rarely: by a row's scores, or by the value scale
      float m[2];
      bool move = vs > kMoreScale * vref;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        m[e] = fmaxf(fmaxf(x[e][0], x[e][1]), fmaxf(x[e][2], x[e][3]));
        move |= m[e] > mref[e] + kLazy;       // also from -inf
      }
      if (__any_sync(0xffffffffu, move)) {
        const float vnew = fmaxf(vref, vs);
        const float vf = vnew > 0.f ? vref / vnew : 1.f;
        vref = vnew;
        vinv = vref > 0.f ? kUnitWeight / vref : 0.f;
        float f[2];
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], 1));
          m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], 2));
          m[e] = fmaxf(m[e], mref[e]);
          const float k = m[e] > -INFINITY ? ex2(mref[e] - m[e]) : 1.f;
          lsum[e] *= k;
          f[e] = k * vf;
          mref[e] = m[e];
        }
        if (SPLIT) f[1] = f[0];
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i][0] *= f[0], o[i][1] *= f[0], o[i][2] *= f[1], o[i][3] *= f[1];
      }
      // weights, and weights times the value scale as fp16
      const float vk = vs * vinv;
      uint32_t pf[4];
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float ref = mref[e] > -INFINITY ? mref[e] : 0.f;
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = ex2(x[e][i] - ref);
          lsum[e] += w[i];
          w[i] *= vk;
        }
        pf[e] = pack_f16(w[0], w[1]);
        pf[2 + e] = pack_f16(w[2], w[3]);
        if (SPLIT) {
          pf[1] = pack_rest(w[0], w[1], pf[0], kRestScale);
          pf[3] = pack_rest(w[2], w[3], pf[2], kRestScale);
        }
      }
      // values: column n of tile i is element 8 i + n
#pragma unroll
      for (int m = 0; m < D / 32; ++m) {
        const uint32_t w[4] = {vw[m].x, vw[m].y, vw[m].z, vw[m].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          widen4(w[i], b0, b1);
          mma(o[4 * m + i], pf, b0, b1);
        }
      }
      take_k ^= kStageBytes, take_v ^= kStageBytes, take_scale ^= 8;
      __syncwarp();
      produce();
    }

    // ---- the warps' shares ----
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      lsum[e] += __shfl_xor_sync(0xffffffffu, lsum[e], 1);
      lsum[e] += __shfl_xor_sync(0xffffffffu, lsum[e], 2);
      if (c == 0) {
        s_m[warp * kRows + g + 8 * e] = mref[e];
        s_l[warp * kRows + g + 8 * e] = lsum[e];
      }
    }
    team_sync<crew>(team);
    float top[2], fo[2];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      top[e] = -INFINITY;
#pragma unroll
      for (int w = 0; w < TEAM; ++w) top[e] = fmaxf(top[e], s_m[(warp - mate + w) * kRows + g + 8 * e]);
      fo[e] = (mref[e] > -INFINITY ? ex2(mref[e] - top[e]) : 0.f) * (vref / kUnitWeight);
    }
    // half of the warps store their sums, then the others add theirs
    auto hand_in = [&](bool add) {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        float* to_row = t_o + (mate % (TEAM / 2) * kRows + g + 8 * e) * kORow + 2 * c;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float2 y;
          y.x = (SPLIT ? fmaf(o[i][2], 1.0f / kRestScale, o[i][0]) : o[i][2 * e]) * fo[e];
          y.y = (SPLIT ? fmaf(o[i][3], 1.0f / kRestScale, o[i][1]) : o[i][2 * e + 1]) * fo[e];
          float2* to = reinterpret_cast<float2*>(to_row + 8 * i);
          if (add) {
            const float2 old = *to;
            y.x += old.x, y.y += old.y;
          }
          *to = y;
        }
      }
    };
    if (mate < TEAM / 2) hand_in(false);
    team_sync<crew>(team);
    if (mate >= TEAM / 2) hand_in(true);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      if (mate == 0 && c == 0) {
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < TEAM; ++w) {
          const float mw = s_m[(warp + w) * kRows + g + 8 * e];
          l += s_l[(warp + w) * kRows + g + 8 * e] * (mw > -INFINITY ? ex2(mw - top[e]) : 0.f);
        }
        s_tot[team][0][g + 8 * e] = top[e];
        s_tot[team][1][g + 8 * e] = l;
      }
    }
    team_sync<crew>(team);
    const bool whole = s.first >= u0 && s.last <= u1;
    // partial sums: slot 0 for a (sequence, head, tile) that began in an earlier CTA, 1 for one that begins here
    float* slot = p.part + (range * 2 + (s.first >= u0 ? 1 : 0)) * kRows * (D + 2);
    constexpr int kVecs = D / 4;
    for (int i = mine; i < rows * kVecs; i += crew) {
      const int r = i / kVecs, d = i % kVecs * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < TEAM / 2; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(t_o + (w * kRows + r) * kORow + d);
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      if (whole)
        store4<D>(p, s, row0 + r, d, v, s_tot[team][1][r]);
      else
        *reinterpret_cast<float4*>(slot + r * D + d) = v;
    }
    if (!whole) {
      if (mine < 2 * kRows) slot[kRows * D + mine] = (&s_tot[team][0][0])[mine];
      team_sync<crew>(team);
      const long long o0 = owner_of(s.first), o1 = owner_of(s.last - 1);
      if (mine == 0) {
        const unsigned old = atom_add_acq_rel_gpu(p.tickets + o0, 1u);
        s_last[team] = old == static_cast<unsigned>(o1 - o0);
        if (s_last[team]) p.tickets[o0] = 0;
      }
      team_sync<crew>(team);
      if (s_last[team])
        join<D, kTileRows, TEAM>(p, s, row0, rows, o0, static_cast<int>(o1 - o0) + 1, team, mine, t_o, s_m, s_l);
    }
    team_sync<crew>(team);   // t_o and s_m are free for the next segment
    u = min(s.last, u1);
  }

  // rows of no sequence: zeros
  const long long end = max(0, min(a.b.T, a.b.cu[B]));
  const long long row_elems = static_cast<long long>(a.Hq) * D;
  for (long long i = end * row_elems + static_cast<long long>(blockIdx.x) * kThreads + tid; i < a.b.T * row_elems;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    if (a.out_bf16)
      static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(0.f);
    else
      static_cast<float*>(a.out)[i] = 0.f;
  }
}

template <int D, bool SPLIT, int TEAM>
cudaError_t launch(const AttnParams& p, int grid, cudaStream_t st) {
  const size_t smem = smem_bytes<D>(p.a.b.B);
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(q4_kv_attn_split_kernel<D, SPLIT, TEAM>, smem_bytes<D>(kKvMaxSeqs), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_kv_attn_split_kernel<D, SPLIT, TEAM>, p);
}

template <int D, bool SPLIT>
cudaError_t launch(const AttnParams& p, int rows, int grid, cudaStream_t st) {
  // Teams of four while there are more (sequence, tile, head)s than SMs: a team's start and end then fall into the
  // others' streams (quarters / whole CTAs: 64 sequences of 50 to 8191 tokens, 8 heads, 96 / 141 us; of 4096 tokens
  // 96 / 115 us).  With fewer, whole CTAs, which leave a quarter of the shares to join (one sequence of 131,071
  // tokens 62 / 54 us, 8 of 1024 17 / 16 us).
  const long long tiles = (rows + (SPLIT ? 7 : 15)) / (SPLIT ? 8 : 16);
  return p.a.b.B * tiles * p.a.c.heads > grid ? launch<D, SPLIT, kWarps / kTeams>(p, grid, st)
                                              : launch<D, SPLIT, kWarps>(p, grid, st);
}

}  // namespace

size_t kv_attn_header_bytes() { return 4096; }   // a ticket for each range

size_t kv_attn_split_bytes(int dim, int sms) {
  return kv_attn_header_bytes() + static_cast<size_t>(sms) * kTeams * 2 * kRows * (dim + 2) * 4;
}

cudaError_t launch_kv_attn_split(const KvAttnCall& a, int max_q, int max_rows, void* ws, int sms, cudaStream_t st) {
  if (static_cast<size_t>(sms) * kTeams * sizeof(unsigned) > kv_attn_header_bytes()) return cudaErrorInvalidConfiguration;
  AttnParams p = {};
  p.a = a;
  p.group = a.Hq / a.c.heads;
  p.max_rows = max_rows;
  p.tickets = static_cast<unsigned*>(ws);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kv_attn_header_bytes());
  // fp32 in or out needs two terms; bf16 takes them too while eight rows are enough: a thread then has one row's
  // softmax instead of two (64 sequences of 50 to 8191 tokens 96 us, 106 us with rows in both halves)
  const int rows = static_cast<int>(std::min<long long>(static_cast<long long>(max_q) * p.group, max_rows));
  const bool split = !a.q_bf16 || !a.out_bf16 || rows <= 8;
  if (a.c.dim == 128) return split ? launch<128, true>(p, rows, sms, st) : launch<128, false>(p, rows, sms, st);
  return split ? launch<64, true>(p, rows, sms, st) : launch<64, false>(p, rows, sms, st);
}

}  // namespace q4
