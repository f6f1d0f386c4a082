// Leaving tokens out of the paged 8-bit cache (sm_103a): choosing those to keep
// by their weight, and moving kept tokens together.
//
// Measured (8 kv heads of 128): 48 sequences of 1500 to 8191 tokens to 2048 each,
// choice 19 us, moving into other pages 74 us (95,931 tokens, 394 MB read and
// written, 5.3 TB/s), in place 97; one of 100,003 tokens to 32,768, choice 18 us,
// moving 31 us (4.4 TB/s), in place 916: one CTA a (sequence, head) there.  The
// choice reads 4 bytes a token and head: it is bound by its passes over shared
// memory (three of 2.7 us) and what lies before and between them (length, page
// and weight one after another 5 us, five meetings of the cluster 1 us each).  Moving is bound by HBM, with a chain of
// list, page and scale before a run's first codes.
#include <algorithm>
#include <cfloat>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"

namespace q4 {
namespace {

// ---------------------------------------------------------------------------
// Choice
// ---------------------------------------------------------------------------
// A cluster of CTAs takes one (sequence, head); each a run of its tokens, whose
// weights it holds in shared memory as whole numbers in the weights' order.
// The weight down to which tokens are kept is found digit by digit (11, 11 and
// 10 bits): each CTA counts its tokens by digit among those that agree in the
// digits before, and a warp of every CTA adds the counts of all, of groups of 32
// digits first and then of the digits of one.  The list is then
// written in the tokens' order: warps count what they keep in runs of their
// own, and write it behind the counts of those before.  A thread takes four
// tokens side by side (one at a time: 35 us for the batch above, against 24).
// Counting lanes that agree first saves nothing, even where all weights are
// equal (21 us against 18): the counters of shared memory add equal addresses.
constexpr int kMostCluster = 8;        // one sequence of 100,003 tokens in L2, 8 heads, four / eight: 23 / 18 us
constexpr int kBins = 2048;
constexpr int kSelTokens = 40960;      // of a CTA in shared memory; more are read again from their pages
constexpr int kGroup = 32;             // digits whose counts are added for the peers
constexpr int kAsk = 4;                // page table entries that a thread asks for at a time
constexpr int kQuad = 4;               // tokens that a thread takes side by side: of one page

// A weight as a number in its order; NaN is the least.
__device__ __forceinline__ unsigned order_of(float w) {
  const unsigned u = __float_as_uint(w + 0.f);   // -0 becomes 0
  return w != w ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ unsigned ld_peer(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// The sum of the lanes before.
__device__ __forceinline__ unsigned scan_before(unsigned n) {
  const int lane = threadIdx.x & 31;
  unsigned up = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  return up - n;
}

// MANY: in a cluster of CTAs.  512 threads: three CTAs an SM.
template <int THREADS, bool MANY>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 3 : 1) q4_kv_select_kernel(const __grid_constant__ KvSelectParams p, int cluster, int cap) {
  constexpr int kSelThreads = THREADS, kSelWarps = THREADS / 32;
  static_assert(kGroup == 32 && kBins == 64 * kGroup && kSelThreads >= kBins / 4 && kSelWarps <= 32, "a warp finds the digit");
  extern __shared__ __align__(16) unsigned s_mem[];
  unsigned* s_hist = s_mem;                       // [3][kBins]
  unsigned* s_key = s_mem + 3 * kBins;            // [cap]
  __shared__ unsigned s_group[3][kBins / kGroup]; // sums of the counts of kGroup digits
  __shared__ unsigned s_above[kSelWarps], s_equal[kSelWarps];
  __shared__ unsigned s_digit, s_rest;            // the digit of the cut, tokens to take among those that have it
  __shared__ uint2 s_count;                       // of this CTA: tokens above the cut, at it
  // the same in all lanes, and known to be: exchanges of a warp's lanes take six times as long behind a branch that may part them
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rank = MANY ? static_cast<int>(cluster_ctarank()) : 0;
  pdl_launch_dependents();
  pdl_wait();
  const int pair = blockIdx.x / cluster, b = pair / p.c.heads, h = pair - b * p.c.heads;
  const int said = p.kv_len[b], budget = p.budget[b], len = kv_tokens(p.c, p.table_stride, said);
  if (len < said && tid == 0) atomicOr(p.err, kDevErrIndex);
  const int count = static_cast<int>(min(static_cast<long long>(max(0, min(len, budget))), p.width));
  const int head = static_cast<int>(min(static_cast<long long>(count), p.sinks));
  const int tail = static_cast<int>(min(static_cast<long long>(count - head), p.recent));
  const int most = len - head - tail;             // tokens to choose from, behind the sinks
  unsigned want = count - head - tail;            // and how many of them
  int32_t* kept = p.kept + (static_cast<long long>(b) * p.c.heads + h) * p.width;
  if (rank == 0 && h == 0 && tid == 0) p.count[b] = count;
  for (int i = rank * kSelThreads + tid; i < head; i += cluster * kSelThreads) kept[i] = i;
  for (int i = rank * kSelThreads + tid; i < tail; i += cluster * kSelThreads) kept[count - tail + i] = len - tail + i;
  const bool all = want == static_cast<unsigned>(most);   // the same for the whole cluster
  if (all || want == 0) {
    if (all)
      for (int i = rank * kSelThreads + tid; i < most; i += cluster * kSelThreads) kept[head + i] = head + i;
    return;
  }
  // tokens from a multiple of four on, the first `skip` of which are sinks; a warp's run is a number of whole steps
  constexpr int kStep = 32 * kQuad;
  const int base = head & ~(kQuad - 1), total = len - tail - base;
  const int each = static_cast<int>(min(static_cast<long long>(total),
                                        ((static_cast<long long>(total) + cluster - 1) / cluster + kQuad - 1) / kQuad * kQuad));
  const int from = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(rank) * each));
  const int mine = min(total - from, each);
  const int run = static_cast<int>((mine + kSelWarps * kStep - 1LL) / (kSelWarps * kStep) * kStep);
  const int skip = from == 0 ? head - base : 0;
  const int quads = (mine + kQuad - 1) / kQuad;
  const int32_t* table = p.table + b * p.table_stride;
  auto page_of = [&](int q) {
    const int pi = (base + from + q * kQuad) >> p.c.page_log2;
    return pi < p.table_stride ? __ldg(table + pi) : -1;
  };
  auto quad_in = [&](int q, int page) {           // weights of tokens 4 q .. 4 q + 3 of this CTA, in their order
    const int pos = base + from + q * kQuad;
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.c.pages)) {
      if (h == 0) atomicOr(p.err, kDevErrIndex);
      return make_uint4(0, 0, 0, 0);
    }
    const float4 w = __ldg(reinterpret_cast<const float4*>(
        p.weight + (((static_cast<long long>(page) * p.c.heads + h) << p.c.page_log2) + (pos & (p.c.page - 1)))));
    return make_uint4(order_of(w.x), order_of(w.y), order_of(w.z), order_of(w.w));
  };
  for (int i = tid; i < 3 * kBins; i += kSelThreads) s_hist[i] = 0;
  uint4* s_quad = reinterpret_cast<uint4*>(s_key);
  const int held = min(quads, cap / kQuad);
  for (int q0 = tid; q0 < held; q0 += kAsk * kSelThreads) {   // the pages of some, then their weights
    int page[kAsk];
#pragma unroll
    for (int i = 0; i < kAsk; ++i) page[i] = q0 + i * kSelThreads < held ? page_of(q0 + i * kSelThreads) : 0;
#pragma unroll
    for (int i = 0; i < kAsk; ++i)
      if (q0 + i * kSelThreads < held) s_quad[q0 + i * kSelThreads] = quad_in(q0 + i * kSelThreads, page[i]);
  }
  // the four weights, and which of them count
  auto keys = [&](int q, unsigned (&key)[kQuad], bool (&have)[kQuad]) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (q < quads) x = q < held ? s_quad[q] : quad_in(q, page_of(q));
    key[0] = x.x, key[1] = x.y, key[2] = x.z, key[3] = x.w;
#pragma unroll
    for (int k = 0; k < kQuad; ++k) have[k] = q * kQuad + k >= skip && q * kQuad + k < mine;
  };
  if (MANY) cluster_started();
  __syncthreads();

  // ---- the cut, digit by digit from the top ----
  unsigned cut = 0, known = 0;                    // known: bits of the cut that are found
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? kBins / 2 : kBins;
    unsigned* hist = s_hist + d * kBins;
    for (int q = tid; q - tid < quads; q += kSelThreads) {
      unsigned key[kQuad];
      bool in[kQuad];
      keys(q, key, in);
      bool any = false;
#pragma unroll
      for (int k = 0; k < kQuad; ++k) any |= in[k] = in[k] && (key[k] & known) == cut;
      if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
      for (int k = 0; k < kQuad; ++k) {
        if (in[k]) atomicAdd(hist + (key[k] >> shift & (bins - 1)), 1u);
      }
    }
    __syncthreads();
    // of each kGroup digits, so that peers read few counts: all 2048 of eight CTAs took 2 us more a digit
    if (tid < kBins / 4) {
      const uint4 x = reinterpret_cast<const uint4*>(hist)[tid];
      unsigned n = x.x + x.y + x.z + x.w;
#pragma unroll
      for (int o = 1; o < kGroup / 4; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if ((tid & (kGroup / 4 - 1)) == 0) s_group[d][tid / (kGroup / 4)] = n;
    }
    if (MANY) {
      if (d == 0) cluster_wait_started();
      cluster_sync();
    } else {
      __syncthreads();
    }
    if (warp == 0) {                              // from the largest digit down: two groups a lane, then a digit
      auto of_all = [&](const unsigned* at) {     // the sum of all CTAs' counts: all are asked for before the first is there
        if (!MANY) return *at;
        unsigned x[kMostCluster], sum = 0;
#pragma unroll
        for (int r = 0; r < kMostCluster; ++r) x[r] = ld_peer(peer_addr(at, r & (cluster - 1)));
#pragma unroll
        for (int r = 0; r < kMostCluster; ++r) sum += r < cluster ? x[r] : 0u;
        return sum;
      };
      const unsigned* at = &s_group[d][2 * (31 - lane)];
      const unsigned n[2] = {of_all(at + 1), of_all(at)};
      unsigned before = scan_before(n[0] + n[1]);
      const bool first = want - before <= n[0];
      unsigned who = __ballot_sync(0xffffffffu, before < want && want <= before + n[0] + n[1]);   // one lane
      const int group = __shfl_sync(0xffffffffu, 2 * (31 - lane) + (first ? 1 : 0), __ffs(who) - 1);
      const unsigned rest = want - __shfl_sync(0xffffffffu, first ? before : before + n[0], __ffs(who) - 1);
      const int digit = group * kGroup + 31 - lane;
      const unsigned c = of_all(hist + digit);
      before = scan_before(c);
      if (before < rest && rest <= before + c) s_digit = digit, s_rest = rest - before;   // one lane's
    }
    __syncthreads();
    cut |= s_digit << shift;
    known |= static_cast<unsigned>(bins - 1) << shift;
    want = s_rest;
  }

  // ---- the list: tokens above the cut, and the first `want` of those at it ----
  const int q0 = warp * (run / kQuad), q1 = min(quads, q0 + run / kQuad);
  unsigned above = 0, equal = 0;                  // of this warp's run
  for (int q = q0 + lane; q < q1; q += 32) {
    unsigned key[kQuad];
    bool have[kQuad];
    keys(q, key, have);
#pragma unroll
    for (int k = 0; k < kQuad; ++k) above += have[k] && key[k] > cut, equal += have[k] && key[k] == cut;
  }
  above = __reduce_add_sync(0xffffffffu, above), equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) s_above[warp] = above, s_equal[warp] = equal;
  __syncthreads();
  if (warp == 0) {
    const unsigned a = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? s_above[lane] : 0u);
    const unsigned e = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? s_equal[lane] : 0u);
    if (lane == 0) s_count = make_uint2(a, e);
  }
  unsigned taken = 0, passed = 0;                 // tokens above and at the cut before this warp's
  if (MANY) {
    cluster_sync();
    const bool earlier = lane < rank;             // a lane for each of them
    taken = __reduce_add_sync(0xffffffffu, earlier ? ld_peer(peer_addr(&s_count.x, lane)) : 0u);
    passed = __reduce_add_sync(0xffffffffu, earlier ? ld_peer(peer_addr(&s_count.y, lane)) : 0u);
  }
  taken += __reduce_add_sync(0xffffffffu, lane < warp ? s_above[lane] : 0u);
  passed += __reduce_add_sync(0xffffffffu, lane < warp ? s_equal[lane] : 0u);
  for (int q = q0 + lane; q - lane < q1; q += 32) {
    unsigned key[kQuad];
    bool have[kQuad];
    keys(q, key, have);
    if (q >= q1) have[0] = have[1] = have[2] = have[3] = false;
    unsigned mine_up = 0;                         // tokens above and, in the upper half, at the cut: of this lane's four
#pragma unroll
    for (int k = 0; k < kQuad; ++k) mine_up += (have[k] && key[k] > cut ? 1u : 0u) + (have[k] && key[k] == cut ? 0x10000u : 0u);
    unsigned up = mine_up;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    unsigned a = taken + ((up - mine_up) & 0xffffu), e = passed + ((up - mine_up) >> 16);
#pragma unroll
    for (int k = 0; k < kQuad; ++k) {
      const bool over = have[k] && key[k] > cut, at = have[k] && key[k] == cut;
      if (over || (at && e < want)) kept[head + a + min(e, want)] = base + from + q * kQuad + k;
      a += over, e += at;
    }
    const unsigned whole = __shfl_sync(0xffffffffu, up, 31);
    taken += whole & 0xffffu;
    passed += whole >> 16;
  }
  if (MANY) cluster_sync();                      // the counts are read by the peers
}

// ---------------------------------------------------------------------------
// Moving
// ---------------------------------------------------------------------------
// A CTA takes kMoveTokens consecutive places of a head at a time, keys and
// values: a thread a place finds its source and factor, then all threads move
// 16 codes at a time.  Within one page table a place may be the source of an
// earlier one (never of a later one: kept[i] >= first + i), so there a CTA takes
// all the places of a (sequence, head), in order, and writes some after all of
// their sources are in registers; into other pages every run of places has a
// CTA.  So a long sequence is cut fastest into other pages; in place is for many
// sequences, and for a few tokens each (accepted paths of 16 drafts: 3.4 us in a
// graph).
constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 128;

// Four codes times `ratio` (at most 1), each rounded: rint(code * ratio), one fp32 operation a step.  Codes become
// floats, and floats codes, by an addition that leaves the whole number in the low bits.  The product and the addition
// that rounds it are operations of one number each: those of two numbers are fused, which rounds once and moves a code
// whose product lies within half a unit of the last place of a half (one of 400,000).
__device__ __forceinline__ uint32_t scale4(uint32_t w, float ratio) {
  const uint32_t u = w ^ 0x80808080u;             // code + 128: the low byte of 2^23 + code + 128
  const f32x2 less = dup2(-8388736.f);            // -(2^23 + 128)
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float a, b;
    unpack2(add2(pack2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + 2 * i)),
                       __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441 + 2 * i))), less), a, b);
    y[2 * i] = __float_as_uint(__fadd_rn(__fmul_rn(a, ratio), 12582912.f));   // 2^23 + 2^22: no fraction is left
    y[2 * i + 1] = __float_as_uint(__fadd_rn(__fmul_rn(b, ratio), 12582912.f));
  }
  return __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) q4_kv_compact_kernel(const __grid_constant__ KvCompactParams p) {
  constexpr int kParts = D / 16, kEach = kMoveTokens * kParts / kMoveThreads;
  constexpr unsigned kNone = ~0u;
  __shared__ unsigned s_src[kMoveTokens], s_dst[kMoveTokens];   // rows of codes: fewer than 2^32 fit any GPU
  __shared__ float s_ratio[2][kMoveTokens];                // of keys and values; -1: they stay as they are
  const int tid = threadIdx.x;
  const int b = blockIdx.x / p.c.heads, h = blockIdx.x - b * p.c.heads;
  pdl_launch_dependents();
  pdl_wait();
  const int len = max(0, p.kv_len[b]), first = p.first ? max(0, p.first[b]) : 0;
  const int count = static_cast<int>(min(static_cast<long long>(max(0, p.count[b])), p.width));
  const int end = static_cast<int>(min(static_cast<long long>(first) + count, 0x7fffffffLL));
  const int32_t* kept = p.kept + (static_cast<long long>(b) * p.kept_heads + (p.kept_heads > 1 ? h : 0)) * p.width;
  const int32_t* to_table = p.to_table ? p.to_table : p.table;
  const long long to_stride = p.to_table ? p.to_stride : p.table_stride;
  // places in runs that begin with a block
  const long long step = p.to_table ? static_cast<long long>(gridDim.y) * kMoveTokens : kMoveTokens;
  for (long long t0 = first / kKvBlock * kKvBlock + static_cast<long long>(p.to_table ? blockIdx.y : 0) * kMoveTokens;
       count > 0 && t0 < end; t0 += step) {
    if (tid < kMoveTokens) {
      const int pos = static_cast<int>(min(t0 + tid, static_cast<long long>(end)));   // `end`: no place
      long long dst = -1, src = -1;
      float had[2] = {0.f, 0.f}, weight = 0.f;    // the scales that the token comes with, its weight
      const bool moves = pos >= first && pos < end;
      if (pos < end) {
        dst = kv_row(p.c, to_table, to_stride, b, pos, h);
        if (pos < first) {                        // stays where it is
          src = dst;
        } else {
          const int from = __ldg(kept + (pos - first));
          if (from >= pos && from < len) src = kv_row(p.c, p.table, p.table_stride, b, from, h);
        }
        if (src < 0 || dst < 0) atomicOr(p.err, kDevErrIndex);
        if (src >= 0) {
          had[0] = p.c.ks[src >> 4], had[1] = p.c.vs[src >> 4];
          if (p.weight && moves) weight = p.weight[src];
        }
      }
      float s[2] = {had[0], had[1]};
#pragma unroll
      for (int o = 1; o < kKvBlock; o <<= 1) {
        s[0] = fmaxf(s[0], __shfl_xor_sync(0xffffffffu, s[0], o));
        s[1] = fmaxf(s[1], __shfl_xor_sync(0xffffffffu, s[1], o));
      }
      s_src[tid] = src < 0 ? kNone : static_cast<unsigned>(src);
      s_dst[tid] = dst < 0 ? kNone : static_cast<unsigned>(dst);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float ratio = s[x] > 0.f ? __fdiv_rn(had[x], s[x]) : 0.f;
        s_ratio[x][tid] = src == dst && ratio == 1.f ? -1.f : ratio;
      }
      // all scales and weights of these places' sources have been read before the first is written
      asm volatile("bar.sync 1, %0;" ::"n"(kMoveTokens) : "memory");
      if ((tid & (kKvBlock - 1)) == 0 && dst >= 0) p.c.ks[dst >> 4] = s[0], p.c.vs[dst >> 4] = s[1];
      if (p.weight && moves && dst >= 0) p.weight[dst] = weight;
    }
    __syncthreads();
    uint4 w[2][kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int t = (i * kMoveThreads + tid) / kParts, part = (i * kMoveThreads + tid) % kParts;
      const unsigned src = s_src[t];
      const long long at = static_cast<long long>(src) * D + part * 16;
      w[0][i] = w[1][i] = make_uint4(0, 0, 0, 0);
      if (src != kNone && s_ratio[0][t] >= 0.f) w[0][i] = *reinterpret_cast<const uint4*>(p.c.k + at);
      if (src != kNone && s_ratio[1][t] >= 0.f) w[1][i] = *reinterpret_cast<const uint4*>(p.c.v + at);
    }
    if (!p.to_table) __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int t = (i * kMoveThreads + tid) / kParts, part = (i * kMoveThreads + tid) % kParts;
      const unsigned dst = s_dst[t];
      const long long at = static_cast<long long>(dst) * D + part * 16;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float ratio = s_ratio[x][t];
        if (dst == kNone || ratio < 0.f) continue;
        uint4 y = w[x][i];
        if (ratio != 1.f)
          y.x = scale4(y.x, ratio), y.y = scale4(y.y, ratio), y.z = scale4(y.z, ratio), y.w = scale4(y.w, ratio);
        *reinterpret_cast<uint4*>((x ? p.c.v : p.c.k) + at) = y;
      }
    }
    __syncthreads();
  }
}

template <typename P, typename... Args>
cudaError_t launch_pdl(void (*kernel)(P, Args...), dim3 grid, unsigned threads, size_t smem, int cluster, cudaStream_t st,
                       const P& p, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, args...);
}

template <int THREADS, bool MANY>
cudaError_t launch_select(const KvSelectParams& p, long long max_kv, int cluster, cudaStream_t st) {
  const long long each = ((max_kv + kQuad + cluster - 1) / cluster + kQuad - 1) / kQuad * kQuad;
  const int cap = static_cast<int>(std::min<long long>(each, kSelTokens));
  const size_t smem = (3 * kBins + static_cast<size_t>(cap)) * 4;
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(q4_kv_select_kernel<THREADS, MANY>, (3 * kBins + static_cast<size_t>(kSelTokens)) * 4, allowed);
  if (e != cudaSuccess) return e;
  const long long ctas = static_cast<long long>(p.B) * p.c.heads * cluster;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(q4_kv_select_kernel<THREADS, MANY>, dim3(static_cast<unsigned>(ctas)), THREADS, smem, cluster, st, p,
                    cluster, cap);
}

}  // namespace

cudaError_t launch_kv_select(const KvSelectParams& p, long long max_kv, int sms, cudaStream_t st) {
  const long long pairs = static_cast<long long>(p.B) * p.c.heads;
  // as many CTAs for a (sequence, head) as fill the GPU, or hold its tokens in shared memory, up to eight; of 1024
  // threads where each has an SM (one sequence of 100,003 tokens: 18 us against 22 of 512), else of 512 (8 of 16,000: 17
  // against 22 of 1024)
  int cluster = 1;
  while (cluster < kMostCluster && (pairs * cluster < sms || max_kv > static_cast<long long>(cluster) * kSelTokens) &&
         max_kv > cluster * 1024LL)
    cluster *= 2;
  if (cluster == 1) return launch_select<512, false>(p, max_kv, cluster, st);
  return pairs * cluster <= sms ? launch_select<1024, true>(p, max_kv, cluster, st)
                                : launch_select<512, true>(p, max_kv, cluster, st);
}

cudaError_t launch_kv_compact(const KvCompactParams& p, cudaStream_t st) {
  const long long pairs = static_cast<long long>(p.B) * p.c.heads;
  // into other pages: a CTA for each run of places, which may begin inside a block
  const long long runs = p.to_table ? std::min((p.width + kKvBlock + kMoveTokens - 1) / kMoveTokens, 65535LL) : 1;
  const dim3 grid(static_cast<unsigned>(pairs), static_cast<unsigned>(runs));
  return p.c.dim == 128 ? launch_pdl(q4_kv_compact_kernel<128>, grid, kMoveThreads, 0, 1, st, p)
                        : launch_pdl(q4_kv_compact_kernel<64>, grid, kMoveThreads, 0, 1, st, p);
}

}  // namespace q4
