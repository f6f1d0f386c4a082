// Attention of prompts over the paged 8-bit cache on the tensor cores (sm_103a):
// the form for many new tokens a sequence.
//
// 4 D flops for each query and visible key: bound by the tensor cores, and by
// the exponentials beside them.  Two launches:
//
// * q4_kv_expand_kernel turns the pages of each sequence into consecutive
//   fp16 rows (code * scale, both scaled by a power of two per sequence and
//   head so that the largest fits fp16), once for all the queries that will
//   read them: 2 bytes written for each code, against 4 D flops for each query.
//   It also writes which tokens of a 128-token tile exist.
// * q4_kv_prompt_kernel: a CTA takes 256 query rows of one kv head (the query
//   heads that share it, token-major) as two MMA tiles of 128, and walks over
//   the visible tiles of 128 tokens.  One warp copies K and V tiles with TMA
//   into a ring, one warp issues the MMAs, and four warps a tile (a thread a
//   row) take the scores from tensor memory, form the weights and put them
//   back as the fp16 A operand of the second product.  While one tile's rows
//   are in the softmax the tensor cores work on the other's.  The running
//   maximum moves only when it has grown by 2^8, so the sums in tensor memory
//   are seldom rescaled.
//
// Measured (8 kv heads of 128, 32 query heads): a prompt of 8192 tokens 406 us
// both launches, 1354 TFLOP/s of visible products (72% of the measured bf16
// peak of cuBLAS; tiles on the diagonal do up to twice the visible work); six
// pieces of up to 1537 tokens on up to 9000 cached ones 470 us, 1246 TFLOP/s.
// The tensor pipe is 62% busy by its counter: what is left is the chain of a
// tile (scores out of tensor memory, 128 exponentials a thread, weights back)
// where two tiles an SM do not cover one another, and for the pieces the last
// round of CTAs and the expansion.  The MMA warp runs its loop as a whole, with
// one lane issuing: elected before the loop, its single lane took 532 us.
#include <cfloat>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"
#include "q4_tc_core.cuh"

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
constexpr float kLog2e = 1.4426950408889634f;

struct ExpandParams {
  KvView c;
  KvBatch b;
  int group, split_rows;
  int rows_cap;              // rows of kv
  __half* kv;                // [2][heads][rows_cap][dim]
  float* factor;             // [B][heads][2]: what a row of K (V) was divided by
  uint4* seen;               // [rows_cap / 128] bit i: token i of the tile exists
  int* kv_cum;               // [B + 1] first tile of each sequence's tokens
  int* order;                // [B] sequences, the longest last
  int* q_cum;                // [B + 1] first tile of the query rows of each of those
  uint4* zeros;              // out, when rows of no sequence are this kernel's to clear, or null
  long long row_bytes;
  unsigned* err;
};

struct PromptParams {
  CUtensorMap kv;            // fp16 [2 * heads][rows_cap][dim], boxes of 64 x 128, 128-byte swizzle
  KvAttnCall a;
  int group, split_rows;
  int rows_cap;
  const float* factor;
  const uint4* seen;
  const int* kv_cum;
  const int* order;
  const int* q_cum;
};

// Sequences in this form have more query rows than the split form takes.
__device__ __forceinline__ bool is_prompt(int nq, int group, int split_rows) {
  return static_cast<long long>(nq) * group > split_rows;
}

// Exclusive prefix sums of n_of(b) into cum[0 .. B]; every thread of the block calls it.
template <int THREADS, typename F>
__device__ __forceinline__ void prefix(int B, int* cum, F n_of) {
  __shared__ int s_warp[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (B + THREADS - 1) / THREADS;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < B) {
      sum += n_of(b);
      cum[b + 1] = sum;
    }
  }
  int up = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  if (lane == 31) s_warp[warp] = up;
  __syncthreads();
  int before = up - sum;
  for (int i = 0; i < warp; ++i) before += s_warp[i];
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < B) cum[b + 1] += before;
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

__device__ __forceinline__ int kv_tiles(const KvBatch& b, int i, int group, int split_rows) {
  const int nq = b.cu[i + 1] - b.cu[i];
  return is_prompt(nq, group, split_rows) ? (max(b.kv_len[i], 0) + kTile - 1) / kTile : 0;
}

__device__ __forceinline__ int q_tiles(const KvBatch& b, int i, int group, int split_rows) {
  const int nq = b.cu[i + 1] - b.cu[i];
  return is_prompt(nq, group, split_rows)
             ? static_cast<int>((static_cast<long long>(nq) * group + kTileRows - 1) / kTileRows) : 0;
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
  __shared__ float s_max[2][kExpandThreads / 32];
  __shared__ unsigned s_seen[4];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, h = blockIdx.y, B = p.b.B;
  prefix<kExpandThreads>(B, s_cum, [&](int b) { return kv_tiles(p.b, b, p.group, p.split_rows); });
  if (p.zeros) {
    const long long from = max(0, min(p.b.T, p.b.cu[B])) * p.row_bytes / 16, all = p.b.T * p.row_bytes / 16;
    const long long at = (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * kExpandThreads + tid;
    for (long long i = from + at; i < all; i += static_cast<long long>(gridDim.x) * gridDim.y * kExpandThreads)
      p.zeros[i] = make_uint4(0, 0, 0, 0);
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
  // powers of two that bring the sequence's largest scale of this head to [2^7, 2^8)
  float km = 0.f, vm = 0.f;
  for (int i = tid; i < (len + kKvBlock - 1) / kKvBlock; i += kExpandThreads) {
    const long long row = kv_row(p.c, p.b.table, p.b.table_stride, b, i * kKvBlock, h);
    if (row >= 0) km = fmaxf(km, p.c.ks[row >> 4]), vm = fmaxf(vm, p.c.vs[row >> 4]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
    vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
  }
  if (lane == 0) s_max[0][tid >> 5] = km, s_max[1][tid >> 5] = vm;
  if (tid < 4) s_seen[tid] = 0;
  __syncthreads();
  float up[2], down[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float m = 0.f;
    for (int i = 0; i < kExpandThreads / 32; ++i) m = fmaxf(m, s_max[x][i]);
    const int e = m > 0.f ? max(-126, min(126, 7 + 127 - static_cast<int>(__float_as_uint(m) >> 23))) : 0;
    up[x] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    down[x] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  }
  if (t0 == 0 && tid < 2) p.factor[(static_cast<long long>(b) * p.c.heads + h) * 2 + tid] = down[tid];
  // 16 codes a thread
  const int D = p.c.dim, chunks = D / 16;
  for (int i = tid; i < kTile * chunks; i += kExpandThreads) {
    const int t = i / chunks, c = i % chunks, pos = t0 + t;
    long long row = -1;
    if (pos < len) {
      row = kv_row(p.c, p.b.table, p.b.table_stride, b, pos, h);
      if (c == 0 && h == 0) {
        if (row >= 0) atomicOr(&s_seen[t >> 5], 1u << (t & 31));
        else atomicOr(p.err, kDevErrIndex);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint4 w = make_uint4(0, 0, 0, 0);
      float s = 0.f;
      if (row >= 0) {
        w = *reinterpret_cast<const uint4*>((x ? p.c.v : p.c.k) + row * D + c * 16);
        s = (x ? p.c.vs : p.c.ks)[row >> 4] * up[x];
      }
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
      __half2 f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t two = q[j >> 1] >> (16 * (j & 1));
        f[j] = __floats2half2_rn(static_cast<float>(static_cast<int8_t>(two)) * s,
                                 static_cast<float>(static_cast<int8_t>(two >> 8)) * s);
      }
      uint4* to = reinterpret_cast<uint4*>(
          p.kv + ((static_cast<long long>(x) * p.c.heads + h) * p.rows_cap + static_cast<long long>(tile) * kTile + t) * D + c * 16);
      to[0] = *reinterpret_cast<uint4*>(&f[0]);
      to[1] = *reinterpret_cast<uint4*>(&f[4]);
    }
  }
  if (h == 0) {
    __syncthreads();
    if (tid == 0) p.seen[tile] = make_uint4(s_seen[0], s_seen[1], s_seen[2], s_seen[3]);
  }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 lanes x 32 columns of tensor memory to registers, without the wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// bounded_wait by the whole warp that polls instead of sleeping in the barrier: the MMA warp's waits are on the
// path between the softmax and the tensor cores, and waking up takes some 200 cycles.
__device__ __forceinline__ bool poll_wait(uint64_t* bar, uint32_t parity, volatile int* fail, unsigned* err) {
  const uint32_t at = smem_u32(bar);
  unsigned long long t0 = 0;
  for (uint32_t turn = 0;; ++turn) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(at), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
    if ((turn & 1023) == 1023) {
      if (*fail) return false;
      const unsigned long long t = globaltimer();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        *fail = 1;
        atomicOr(err, kDevErrTimeout);
        return false;
      }
    }
  }
}

// One lane of the warp, the same each time.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
// The whole warp runs the issue loop, so that descriptors stay in uniform registers (a loop of one lane took 93
// cycles an MMA, more than the 67 it runs); the instructions themselves are the leader's.
// D[tmem] (+)= A[smem desc] . B[smem desc]
__device__ __forceinline__ void lead_mma(uint32_t leader, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// D[tmem] (+)= A[tmem] . B[smem desc]
__device__ __forceinline__ void lead_mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void lead_commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}

template <int D>
struct Cfg {
  static constexpr int kHalf = kTile * 128;             // 128 rows of 64 fp16: one swizzled box
  static constexpr int kTileBytes = kHalf * (D / 64);   // a Q, K or V tile
  static constexpr int kSmem = 1024 + 2 * kTileBytes + kStages * kTileBytes + 256;
  static constexpr uint32_t kTmemCols = 512;
  // instruction descriptors: fp16 operands, fp32 sums, 128 rows; q . k: both K-major, 128 columns;
  // p . v: V MN-major, D columns
  static constexpr uint32_t kIdescQk = (1u << 4) | (static_cast<uint32_t>(kTile >> 3) << 17) | (8u << 24);
  static constexpr uint32_t kIdescPv = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (8u << 24);
};

template <int D>
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
  const int last = a.causal ? min(len - 1, len - nq + j1) : len - 1;
  int first = 0;
  if (a.window > 0) {
    const long long f = static_cast<long long>(len) - nq + j0 - a.window + 1;
    first = f > 0 ? static_cast<int>(f / kTile) : 0;
  }
  const bool fits = (static_cast<long long>(tile0) + (max(len, 0) + kTile - 1) / kTile) * kTile <= p.rows_cap;
  if (!fits && tid == 0) atomicOr(a.err, kDevErrIndex);   // longer sequences than the call said
  const int n = fits && last >= 0 ? max(0, last / kTile + 1 - first) : 0;

  if (warp >= kTmaWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kTmaWarp) {
    if (lane == 0) {
      int it = 0;
      for (; it < 2 * n && !s_fail; ++it) {
        const int st = it % kStages;
        if (it >= kStages && !gwait(&empty[st], ((it / kStages) - 1) & 1, &s_fail, a.err)) break;
        mbar_arrive_expect_tx(&full[st], C::kTileBytes);
        const int row = (tile0 + first + (it >> 1)) * kTile, z = (it & 1) * a.c.heads + h;
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
      rowc = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * fabsf(a.scale) * kLog2e *
             (n > 0 ? p.factor[(static_cast<long long>(b) * a.c.heads + h) * 2] : 0.f);
      rowc = fmaxf(rowc, 1e-30f);   // a scale of 0: scores of 0, while those of masked tokens stay -inf
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
    const int qpos = len - nq + j;
    const int to = !have ? 0x7fffffff : a.causal ? qpos : len - 1;
    const long long f = have && a.window > 0 ? static_cast<long long>(qpos) - a.window : -1LL;
    const int from = f < -1 ? -1 : static_cast<int>(f);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const uint4* seen_at = p.seen + tile0 + first;
    uint4 next_seen = n > 0 ? __ldg(seen_at) : make_uint4(0, 0, 0, 0);
    for (int i = 0; i < n; ++i) {
      const int t0 = (first + i) * kTile;
      const uint4 seen = next_seen;
      if (i + 1 < n) next_seen = __ldg(seen_at + i + 1);
      ok = gwait(&s_full[g], i & 1, &s_fail, a.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[kTile];
#pragma unroll
      for (int x = 0; x < 4; ++x) tmem_ld32_async(t_s[g] + lanes + 32 * x, s + 32 * x);
      tmem_wait_ld();
      // tiles on the edge of what a row sees, or with tokens that do not exist
      const bool edge = t0 + kTile - 1 > to || t0 <= from || (seen.x & seen.y & seen.z & seen.w) != 0xffffffffu;
      if (__any_sync(0xffffffffu, edge)) {
        const uint32_t bits[4] = {seen.x, seen.y, seen.z, seen.w};
        const int lo = from - t0, hi = to - t0;
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (c <= lo || c > hi || !((bits[c >> 5] >> (c & 31)) & 1u)) s[c] = 0xff800000u;
      }
      float mx[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) mx[x] = __uint_as_float(s[x]);
#pragma unroll
      for (int c = 4; c < kTile; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(s[c]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const float now = top > -INFINITY ? top * rowc : -INFINITY;
      if (__any_sync(0xffffffffu, now > m + kLazy)) {   // also from -inf
        const float next = fmaxf(m, now);
        const float k = next > -INFINITY ? ex2(m - next) : 1.f;
        m = next;
        l *= k;
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
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * k);
            tmem_st32(t_o[g] + lanes + 32 * x, o);
          }
        }
      }
      const float off = m > -INFINITY ? kUnit - m : 0.f;
      const f32x2 c2 = dup2(rowc), off2 = dup2(off);
      f32x2 sum2[2] = {0ull, 0ull};
      uint32_t w[kTile / 2];
#pragma unroll
      for (int c = 0; c < kTile / 2; ++c) {
        float x, y;
        unpack2(fma2(pack2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), c2, off2), x, y);
        x = ex2(x), y = ex2(y);
        sum2[c & 1] = add2(sum2[c & 1], pack2(x, y));
        const __half2 two = __floats2half2_rn(x, y);
        w[c] = *reinterpret_cast<const uint32_t*>(&two);
      }
      tmem_st32(t_s[g] + lanes, w);
      tmem_st32(t_s[g] + lanes + 32, w + 32);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_ready[g]);
      float x, y;
      unpack2(add2(sum2[0], sum2[1]), x, y);
      l += x + y;
    }
    // the rows' results
    if (n > 0 && ok) {
      ok = gwait(&o_done[g], (n - 1) & 1, &s_fail, a.err);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    if (ok) {
      const float vf = n > 0 ? p.factor[(static_cast<long long>(b) * a.c.heads + h) * 2 + 1] : 0.f;
      // a row that sees nothing: zeros; a NaN stays
      const float k = l > 0.f ? vf / l : l == 0.f ? 0.f : l;
      const long long at = ((static_cast<long long>(c0) + j) * a.Hq + h * p.group + row % p.group) * D;
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

// cuTensorMapEncodeTiled from the driver (null if unavailable).
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      fn = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  return encode;
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
  size_t factor, seen, kv_cum, order, q_cum, kv, total;
};
Layout layout(const KvView& c, int B, long long rows_cap) {
  Layout l;
  l.factor = 0;
  l.seen = up256(static_cast<size_t>(B) * c.heads * 2 * sizeof(float));
  l.kv_cum = l.seen + up256(static_cast<size_t>(rows_cap / kTile) * sizeof(uint4));
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
  x.factor = reinterpret_cast<float*>(w + l.factor);
  x.seen = reinterpret_cast<uint4*>(w + l.seen);
  x.kv_cum = reinterpret_cast<int*>(w + l.kv_cum);
  x.order = reinterpret_cast<int*>(w + l.order);
  x.q_cum = reinterpret_cast<int*>(w + l.q_cum);
  // without a split form beside it, rows of no sequence are this form's
  x.zeros = split_rows == 0 ? static_cast<uint4*>(a.out) : nullptr;
  x.row_bytes = static_cast<long long>(a.Hq) * a.c.dim * 2;
  x.err = a.err;
  PromptParams p = {};
  p.a = a;
  p.group = x.group;
  p.split_rows = split_rows;
  p.rows_cap = x.rows_cap;
  p.factor = x.factor;
  p.seen = x.seen;
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
  static std::atomic<unsigned long long> allowed[2];
  e = a.c.dim == 128 ? allow_smem(q4_kv_prompt_kernel<128>, Cfg<128>::kSmem, allowed[0])
                     : allow_smem(q4_kv_prompt_kernel<64>, Cfg<64>::kSmem, allowed[1]);
  if (e != cudaSuccess) return e;
  return a.c.dim == 128 ? launch_pdl(q4_kv_prompt_kernel<128>, grid, kThreads, Cfg<128>::kSmem, st, p)
                        : launch_pdl(q4_kv_prompt_kernel<64>, grid, kThreads, Cfg<64>::kSmem, st, p);
}

}  // namespace q4
