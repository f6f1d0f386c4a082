// The attention weight of cached tokens on the tensor cores (sm_103a): the form
// for many queries a sequence.
//
//   weight[h, j] (+)= sum_{t, g of h} exp(scale * q[t, g] . k_j - lse[t, g])
//
// 2 D flops for each pair of a token and a query that sees it, and one
// exponential: bound by the tensor cores.  A cluster of two CTAs takes 256
// tokens of a kv head and keeps their keys in shared memory as two MMA tiles,
// and each of them takes every other tile of 256 query rows (the query heads
// that share the head, token-major).  The scores' rows are the tokens, so that
// a thread has one token's scores with all queries: it adds their exponentials
// in registers, with no exchange, and the two CTAs' sums are added at the end.
//
// * Codes are exact in bf16, as are bf16 queries: both are operands as they
//   are, queries straight from the caller's tensor by TMA.  A block's scale is
//   part of a thread's factor, -lse an addend of the exponent.
// * While the MMAs of one tile of tokens run, the other's scores are turned
//   into sums: tensor memory holds 256 columns of each.
// * The grid is as large as the GPU; clusters take pieces of work by turns
//   there and back, the largest (the first tokens, which most queries see)
//   first, so that their sums of work are nearly alike.
//
// Measured (32 query heads on 8 kv heads of 128): a prompt of 8192 tokens 231 us,
// 1190 TFLOP/s of visible products.  The tensor pipe is busy in 54% of the
// cycles, the exponentials' pipe in 55%, and neither alone is the bound: without
// exponentials it takes 209 us, with an eighth of the MMAs 229, without copies of
// queries 223, without all three 171.  A tile of 256 queries and 256 tokens takes
// 1.7 us, 1.1 of either pipe; uneven pieces add 6%, starts and ends 20 us.
// Tried, slower: keys as the operand in tensor memory (192 queries a tile) 233,
// that with scores in two halves 256, with eight more warps 237; eight more warps
// here 241; queries as the scores' rows, with the sums of 64 or 128 tokens in a
// thread's registers, 280 and more, as they spill.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"
#include "q4_kv_tc.cuh"

namespace q4 {
namespace {

using namespace gemm;

constexpr int kTile = 128;                // tokens of an MMA tile
constexpr int kTokens = 2 * kTile;        // of a cluster
constexpr int kCols = 256;                // query rows of a tile
constexpr int kStages = 2;
constexpr int kThreads = 384;             // 2 x 4 warps for the sums; a warp each for queries, MMAs and their lse; an idle one
constexpr int kTmaWarp = 8, kMmaWarp = 9, kLseWarp = 10;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMostItems = 1 << 29;

struct WeighPromptParams {
  CUtensorMap q;             // bf16 [T][Hq][D], boxes of 64 elements, the heads of a kv head, `tokens`
  KvWeighCall a;
  int group, split_rows;     // sequences with more query rows than that are this form's (0: all)
  int tokens;                // new tokens of a tile of queries
};

template <int D>
struct Cfg {
  static constexpr int kKHalf = kTile * 128, kKTile = kKHalf * (D / 64);   // 64 elements of 128 rows: a swizzled box
  static constexpr int kQHalf = kCols * 128, kQTile = kQHalf * (D / 64);
  static constexpr int kBars = 2 * kStages + 2 * kStages + 6 + 1;
  static constexpr size_t fixed() { return 1024 + 2 * kKTile + kStages * kQTile + 256 + kStages * kCols * 4 + 2 * kTokens * 4; }
  static constexpr size_t smem(int B) { return fixed() + static_cast<size_t>(B + 1) * 4; }
  static constexpr uint32_t kTmemCols = 512;
  // instruction descriptor: bf16 operands, both K-major, fp32 sums, 128 rows, 256 columns
  static constexpr uint32_t kIdescQk = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kCols >> 3) << 17) | (8u << 24);
};

// Four codes as bf16.
__device__ __forceinline__ void widen4_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  lo = *reinterpret_cast<const uint32_t*>(&a), hi = *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ int pieces_of(const WeighPromptParams& p, int b) {
  const int nq = max(0, p.a.b.cu[b + 1] - p.a.b.cu[b]), len = kv_tokens(p.a.c, p.a.b.table_stride, p.a.b.kv_len[b]);
  if (len < p.a.b.kv_len[b]) atomicOr(p.a.err, kDevErrIndex);
  if ((p.split_rows > 0 && static_cast<long long>(nq) * p.group <= p.split_rows) || len <= 0) return 0;
  return static_cast<int>(min((len + kTokens - 1LL) / kTokens * p.a.c.heads, static_cast<long long>(kMostItems)));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) q4_kv_weigh_prompt_kernel(const __grid_constant__ WeighPromptParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sk = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = sk + 2 * C::kKTile;
  uint64_t* full = reinterpret_cast<uint64_t*>(sq + kStages * C::kQTile);   // [kStages] queries are there
  uint64_t* empty = full + kStages;      // [kStages] and have been used
  uint64_t* l_full = empty + kStages;    // [kStages] their lse
  uint64_t* l_empty = l_full + kStages;
  uint64_t* k_ready = l_empty + kStages; // [2] keys of a tile of tokens
  uint64_t* d_full = k_ready + 2;        // [2] its scores
  uint64_t* d_empty = d_full + 2;        // [2] and they have been read
  uint64_t* drain = d_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  static_assert(C::kBars * 8 + 4 <= 256, "barriers");
  float* s_lse = reinterpret_cast<float*>(sq + kStages * C::kQTile + 256);   // [kStages][kCols] -lse, base 2
  float* s_peer = s_lse + kStages * kCols;                                   // [2][kTokens] the other CTA's sums
  int* s_cum = reinterpret_cast<int*>(s_peer + 2 * kTokens);                 // [B + 1] first piece of each sequence
  __shared__ int s_fail, s_odd[kStages];
  __shared__ int s_warp[kThreads / 32];

  const KvWeighCall& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.b.B;
  const int rank = static_cast<int>(cluster_ctarank());
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i)
      mbar_init(&full[i], 1), mbar_init(&empty[i], 1), mbar_init(&l_full[i], 32), mbar_init(&l_empty[i], 2 * kTile);
    for (int i = 0; i < 2; ++i) mbar_init(&k_ready[i], kTile), mbar_init(&d_full[i], 1), mbar_init(&d_empty[i], kTile);
    mbar_init(drain, 1);
    s_fail = 0;
  }
  fence_barrier_init();
  // rows of a tile of queries that no copy writes
  for (int i = tid; i < kStages * C::kQTile / 16; i += kThreads) reinterpret_cast<uint4*>(sq)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  pdl_wait();   // before tensor memory is taken: the kernel before may need this SM's
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  {             // pieces of work of each sequence
    const int per = (B + kThreads - 1) / kThreads;
    int sum = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < B) s_cum[b + 1] = sum = min(sum + pieces_of(p, b), kMostItems);
    }
    int up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up = min(up + x, kMostItems);
    }
    if (lane == 31) s_warp[warp] = up;
    int before = __shfl_up_sync(0xffffffffu, up, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    for (int i = 0; i < warp; ++i) before = min(before + s_warp[i], kMostItems);
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < B) s_cum[b + 1] = min(s_cum[b + 1] + before, kMostItems);
    }
    if (tid == 0) s_cum[0] = 0;
  }
  tc_fence_before();
  cluster_sync();               // also: the peer has started
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const int items = s_cum[B], clusters = gridDim.x / 2, me = blockIdx.x / 2;

  // counters of the barriers' phases, the same in all warps: tiles of queries that this CTA has taken, pieces with any
  int taken = 0, worked = 0, sums = 0;
  int copied = 0;               // of the copying warp: tiles whose copies have been started
  for (int turn = 0;; ++turn) {
    const long long item = static_cast<long long>(turn) * clusters + (turn & 1 ? clusters - 1 - me : me);
    if (static_cast<long long>(turn) * clusters >= items) break;
    if (item >= items) continue;
    int b = 0;
    for (int lo = 0, hi = B - 1; lo <= hi;) {   // the last b with s_cum[b] <= item
      const int mid = (lo + hi) >> 1;
      if (s_cum[mid] <= item) b = mid, lo = mid + 1; else hi = mid - 1;
    }
    const int at = static_cast<int>(item) - s_cum[b], h = at % a.c.heads, k0 = at / a.c.heads * kTokens;
    const int c0 = a.b.cu[b], nq = max(0, a.b.cu[b + 1] - c0), len = a.b.kv_len[b], base = len - nq;
    const int held = a.held ? max(0, min(a.held[b], len)) : max(0, base);
    // new tokens that may see some of the tokens: [j_lo, j_hi)
    long long j_lo = a.causal ? max(0LL, static_cast<long long>(k0) - base) : 0, j_hi = nq;
    if (a.window > 0 && k0 >= a.sinks)
      j_hi = max(0LL, min(j_hi, min(static_cast<long long>(k0) + kTokens, static_cast<long long>(len)) - 1 + a.window - base));
    j_lo = min(j_lo, j_hi);
    if (c0 < 0) j_hi = j_lo;
    const int t_lo = static_cast<int>(j_lo) / p.tokens, t_hi = j_hi > j_lo ? (static_cast<int>(j_hi) - 1) / p.tokens + 1 : t_lo;
    const bool any = t_hi > t_lo;               // the same in both CTAs
    if (!any && min(k0 + kTokens, len) <= held) continue;
    const int n = t_hi - t_lo > rank ? (t_hi - t_lo - rank + 1) / 2 : 0;   // tiles of this CTA: t_lo + rank + 2 i
    float sum = 0.f;                            // of a thread's token
    if (warp < kTmaWarp) {
      // ================= keys, then sums: a thread a token =================
      const int g = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane, pos = k0 + g * kTile + r;
      const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16, t_d = tmem + g * kCols + lanes;
      float f = 0.f;
      if (n > 0) {
        const long long row = pos < len ? kv_row(a.c, a.b.table, a.b.table_stride, b, pos, h) : -1;
        if (row >= 0) f = __ldg(a.c.ks + (row >> 4)) * a.scale * kLog2e;
        const uint4* from = reinterpret_cast<const uint4*>(a.c.k + max(row, 0LL) * D);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 w = row >= 0 ? __ldg(from + i) : make_uint4(0, 0, 0, 0);
          uint4 x, y;
          widen4_bf16(w.x, x.x, x.y), widen4_bf16(w.y, x.z, x.w);
          widen4_bf16(w.z, y.x, y.y), widen4_bf16(w.w, y.z, y.w);
          uint8_t* to = sk + g * C::kKTile + (i >> 2) * C::kKHalf + r * 128;   // 16-byte parts 2 i and 2 i + 1 of the row
          *reinterpret_cast<uint4*>(to + (((2 * i & 7) ^ (r & 7)) << 4)) = x;
          *reinterpret_cast<uint4*>(to + (((2 * i + 1 & 7) ^ (r & 7)) << 4)) = y;
        }
        fence_async_smem();
        mbar_arrive(&k_ready[g]);
      }
      const f32x2 f2 = dup2(f);
      bool ok = true;
      for (int i = 0; ok && i < n; ++i) {
        const int it = taken + i, st = it % kStages, j0 = (t_lo + rank + 2 * i) * p.tokens;
        ok = quick_wait(&l_full[st], (it / kStages) & 1, &s_fail, a.err) && quick_wait(&d_full[g], it & 1, &s_fail, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // does every query of the tile see every token of the tile?
        const long long q_lo = static_cast<long long>(base) + j0, q_hi = q_lo + p.tokens - 1, last = k0 + g * kTile + kTile - 1;
        const bool edge = s_odd[st] || (a.causal && q_lo < last) ||
                          (a.window > 0 && last >= a.sinks && q_hi - a.window >= k0 + g * kTile);
        // columns that see the token: [c_lo, c_hi)
        int c_lo = 0, c_hi = kCols;
        if (edge) {
          if (a.causal) c_lo = static_cast<int>(max(0LL, min(pos - q_lo, static_cast<long long>(kCols))) * p.group);
          if (a.window > 0 && pos >= a.sinks)
            c_hi = static_cast<int>(max(0LL, min(pos + a.window - q_lo, static_cast<long long>(kCols))) * p.group);
        }
        const uint32_t nl = smem_u32(s_lse + st * kCols);
        f32x2 part[2] = {0ull, 0ull};
        auto add_up = [&](auto on_edge) {
          uint32_t s[2][32];
          tmem_ld32_async(t_d, s[0]);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < kCols / 32; ++x) {
            const uint32_t* v = s[x & 1];
            if (x + 1 < kCols / 32) tmem_ld32_async(t_d + 32 * (x + 1), s[(x + 1) & 1]);
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              f32x2 l[2];
              lds_pairs(nl + (32 * x + c) * 4, l[0], l[1]);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float y, z;
                unpack2(fma2(pack2(__uint_as_float(v[c + 2 * k]), __uint_as_float(v[c + 2 * k + 1])), f2, l[k]), y, z);
                if (decltype(on_edge)::value) {   // a row that adds nothing may hold anything
                  float ly, lz;
                  unpack2(l[k], ly, lz);
                  const int col = 32 * x + c + 2 * k;
                  if (col < c_lo || col >= c_hi || ly == -INFINITY) y = -INFINITY;
                  if (col + 1 < c_lo || col + 1 >= c_hi || lz == -INFINITY) z = -INFINITY;
                }
                part[k] = add2(part[k], pack2(ex2(y), ex2(z)));
              }
            }
            if (x + 1 < kCols / 32) tmem_wait_ld();
            if (x + 2 == kCols / 32) {   // all columns are in registers
              tc_fence_before();
              mbar_arrive(&d_empty[g]);
            }
          }
        };
        if (edge) add_up(std::true_type{}); else add_up(std::false_type{});
        mbar_arrive(&l_empty[st]);
        float y, z;
        unpack2(add2(part[0], part[1]), y, z);
        sum += y + z;
      }
    } else if (warp == kTmaWarp) {
      if (lane == 0) {
        const uint32_t bytes = static_cast<uint32_t>(p.tokens) * p.group * D * 2;
        for (int i = 0; i < n && !s_fail; ++i) {
          const int it = taken + i, st = it % kStages;
          if (it >= kStages && !quick_wait(&empty[st], ((it / kStages) - 1) & 1, &s_fail, a.err)) break;
          mbar_arrive_expect_tx(&full[st], bytes);
          const int t = c0 + (t_lo + rank + 2 * i) * p.tokens;
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tma_load_3d(sq + st * C::kQTile + x * C::kQHalf, &p.q, x * 64, h * p.group, t, &full[st]);
          copied = it + 1;
        }
      }
    } else if (warp == kMmaWarp) {
      if (n > 0) {
        const uint32_t leader = elect_one();
        const uint64_t k_desc = smem_desc(smem_u32(sk), 16, 1024, kSwizzle128);
        const uint64_t q_desc = smem_desc(smem_u32(sq), 16, 1024, kSwizzle128);
        auto wait = [&](uint64_t* bar, uint32_t parity) { return poll_wait(bar, parity, &s_fail, a.err); };
        bool ok = wait(&k_ready[0], worked & 1) && wait(&k_ready[1], worked & 1);
        for (int i = 0; ok && i < n; ++i) {
          const int it = taken + i, st = it % kStages;
          ok = wait(&full[st], (it / kStages) & 1);
          for (int g = 0; ok && g < 2; ++g) {
            ok = it == 0 || wait(&d_empty[g], (it - 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              lead_mma(leader, tmem + g * kCols, k_desc + (g * C::kKTile >> 4) + (((kk >> 2) * C::kKHalf + (kk & 3) * 32) >> 4),
                       q_desc + (st * C::kQTile >> 4) + (((kk >> 2) * C::kQHalf + (kk & 3) * 32) >> 4), C::kIdescQk, kk > 0 ? 1u : 0u);
            lead_commit(leader, &d_full[g]);
          }
          if (ok) lead_commit(leader, &empty[st]);
        }
      }
    } else if (warp == kLseWarp) {
      // a lane's columns, and a tile's values, on their way while the tile before is in use
      float v[kCols / 32];
      auto load = [&](int i) {
        const int j0 = (t_lo + rank + 2 * i) * p.tokens;
#pragma unroll
        for (int k = 0; k < kCols / 32; ++k) {
          const int c = lane + 32 * k, j = j0 + c / p.group;
          v[k] = INFINITY;
          if (i < n && c < p.tokens * p.group && j < nq && c0 + j < a.b.T)
            v[k] = __ldg(a.lse + (static_cast<long long>(c0) + j) * a.Hq + h * p.group + c % p.group);
        }
      };
      load(0);
      for (int i = 0; i < n; ++i) {
        const int it = taken + i, st = it % kStages;
        if (it >= kStages && !__all_sync(0xffffffffu, quick_wait(&l_empty[st], ((it / kStages) - 1) & 1, &s_fail, a.err))) break;
        bool odd = false;
#pragma unroll
        for (int k = 0; k < kCols / 32; ++k) {
          const bool adds = fabsf(v[k]) <= FLT_MAX;   // a row that sees nothing, or is no number, adds nothing
          odd |= !adds;
          s_lse[st * kCols + lane + 32 * k] = adds ? -v[k] * kLog2e : -INFINITY;
        }
        odd = __any_sync(0xffffffffu, odd);
        if (lane == 0) s_odd[st] = odd;
        mbar_arrive(&l_full[st]);
        load(i + 1);
      }
    }
    __syncwarp();
    taken += n;
    worked += n > 0;
    // ---- the cluster's sums ----
    if (warp < kTmaWarp && rank == 1) st_peer(peer_addr(s_peer + (sums & 1) * kTokens + tid, 0), sum);
    cluster_sync();
    if (warp < kTmaWarp && rank == 0) {
      const int pos = k0 + tid;
      if (pos < len && (any || pos >= held)) {
        // a token that no query may see has no page to be read unless it gets its first weight
        const bool used = pos >= held || a.window == 0 || static_cast<long long>(pos) + a.window > base || pos < a.sinks;
        const long long row = used ? kv_row(a.c, a.b.table, a.b.table_stride, b, pos, h) : -1;
        if (row >= 0)
          a.weight[row] = (pos < held ? a.weight[row] : 0.f) + (sum + s_peer[(sums & 1) * kTokens + tid]);
        else if (used && (tid & (kKvBlock - 1)) == 0)
          atomicOr(a.err, kDevErrIndex);
      }
    }
    ++sums;
  }
  // no copy and no MMA may still run when their memory goes (after a failure: else all copies have been waited for)
  if (warp == kTmaWarp && lane == 0 && s_fail)
    for (int it = max(0, copied - kStages); it < copied; ++it) (void)mbar_wait(&full[it % kStages], (it / kStages) & 1);
  __syncwarp();
  if (warp == kMmaWarp) {
    lead_commit(elect_one(), drain);
    (void)mbar_wait(drain, 0);
    __syncwarp();
  }
  tc_fence_before();
  cluster_sync();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D>
cudaError_t launch(const WeighPromptParams& p, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(q4_kv_weigh_prompt_kernel<D>, Cfg<D>::smem(kKvMaxSeqs), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::smem(p.a.b.B);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, q4_kv_weigh_prompt_kernel<D>, p);
}

}  // namespace

// Query heads of a kv head that the form takes: a tile of queries has whole tokens.
int kv_weigh_prompt_group() { return kCols / 2; }

cudaError_t launch_kv_weigh_prompt(const KvWeighCall& a, int split_rows, int sms, cudaStream_t st) {
  WeighPromptParams p = {};
  p.a = a;
  p.group = a.Hq / a.c.heads;
  p.split_rows = split_rows;
  p.tokens = kCols / p.group;
  const auto encode = encoder();
  if (!encode) return cudaErrorUnknown;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.c.dim), static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.b.T)};
  const cuuint64_t strides[2] = {dims[0] * 2, static_cast<cuuint64_t>(a.q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.tokens)}, ones[3] = {1, 1, 1};
  if (encode(&p.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorUnknown;
  return a.c.dim == 128 ? launch<128>(p, sms, st) : launch<64>(p, sms, st);
}

}  // namespace q4
