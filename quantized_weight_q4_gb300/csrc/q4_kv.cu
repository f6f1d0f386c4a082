// The paged 8-bit key/value cache: appending new tokens (norm, rotation and
// quantisation in one pass) and reading tokens back (sm_103a).
//
// A block is 16 consecutive tokens of one head; its codes are int8 and its
// scale s fp32, value = code * s.  Appending tokens with largest magnitude m
// to a block of scale s0 (0 for a block without earlier tokens) gives
//   s = max(s0, m * (1 / 127))   (0 below 2^-110),
//   earlier codes  c <- rint(c * (s0 / s)),
//   new codes      rint(x * (1 / s)), clamped to +-127,
// every step one fp32 operation, so that the codes are a function of the
// inputs alone, whatever the launch shape.  The norm's sum of squares is taken
// over neighbours first (a binary tree over the head's elements) for the same
// reason.
//
// Both move each byte once and are bound by HBM at best.  Measured: appending
// 21,039 tokens of 7 sequences (32 + 8 heads of 128, bf16, norms, rotation;
// 475 MB) 101 us, 4.7 TB/s; the rest is instruction issue (66% of the cycles)
// and the chain from a token's sequence to its position to its cosines.  One
// token takes 3 us.  Reading 24 sequences of 100 to 6001 tokens back to bf16
// (455 MB) 76 us, 6.0 TB/s.
#include <cfloat>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Measured with the tokens above, append and gather, an earlier step (156 us): four query heads a warp 174 us, sixteen
// 205 us; four warps a block 170 us.
constexpr int kQRows = 8;              // query heads of one token a warp takes
constexpr int kBlockWarps = 2;         // warps that share a block of keys or values
constexpr int kHeads = kWarps / (2 * kBlockWarps);   // kv heads of a CTA
constexpr int kBlockRows = kKvBlock / kBlockWarps;
constexpr float kTinyScale = 7.70371977754894341e-34f;   // 2^-110

// How heads are rotated.  kHalves: all of a head, pairs half of it apart; kPart: pairs half of the rotated part
// apart, less than the head.
enum : int { kNone = 0, kHalves = 1, kPairs = 2, kPart = 3 };

// A head's row is held by D / 8 lanes: lane l of them has elements 4 l .. 4 l + 3 and the four that lie half a head
// further on, so that kHalves turns pairs inside the lane.  A warp works on 32 / (D / 8) rows at a time.
template <int D>
struct Row {
  static constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  float x[8];
};

// A lane's elements of a row; `at`: the address of the first.
template <int D, bool BF16>
__device__ __forceinline__ void load_row(const uint8_t* at, Row<D>& r) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (BF16) {
      const uint2 w = *reinterpret_cast<const uint2*>(at + h * D);
      r.x[4 * h] = __uint_as_float(w.x << 16), r.x[4 * h + 1] = __uint_as_float(w.x & 0xffff0000u);
      r.x[4 * h + 2] = __uint_as_float(w.y << 16), r.x[4 * h + 3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      const float4 w = *reinterpret_cast<const float4*>(at + 2 * h * D);
      r.x[4 * h] = w.x, r.x[4 * h + 1] = w.y, r.x[4 * h + 2] = w.z, r.x[4 * h + 3] = w.w;
    }
  }
}

template <int D>
__device__ __forceinline__ void zero_row(Row<D>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r.x[i] = 0.f;
}

template <int D>
__device__ __forceinline__ void store_row(void* base, long long off, int bf16, int l, const Row<D>& r) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long at = off + h * (D / 2) + 4 * l;
    if (bf16) {
      __nv_bfloat162 y[2] = {__floats2bfloat162_rn(r.x[4 * h], r.x[4 * h + 1]),
                             __floats2bfloat162_rn(r.x[4 * h + 2], r.x[4 * h + 3])};
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) = *reinterpret_cast<uint2*>(y);
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(base) + at) =
          make_float4(r.x[4 * h], r.x[4 * h + 1], r.x[4 * h + 2], r.x[4 * h + 3]);
    }
  }
}

// This lane's eight weights of a norm (aligned to a float only).
template <int D>
__device__ __forceinline__ void load_weights(const float* w, int l, float (&y)[8]) {
  if (reinterpret_cast<uintptr_t>(w) & 15u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __ldg(w + (i >> 2) * (D / 2) + 4 * l + (i & 3));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(w + h * (D / 2) + 4 * l));
      y[4 * h] = u.x, y[4 * h + 1] = u.y, y[4 * h + 2] = u.z, y[4 * h + 3] = u.w;
    }
  }
}

// x <- (x * 1/sqrt(mean(x^2) + eps)) * w, one rounding a step; the sum of squares neighbours first: in the lane,
// over the row's lanes (both halves of the head), then the halves.  The 2 N sums of a lane's N rows are added
// together: at each step a lane hands half of them to its partner and keeps the others, so that a row's sum ends in
// some of the lanes, which take its square root and reciprocal.
template <int D, int N>
__device__ __forceinline__ void norm_rows(Row<D> (&r)[N], const float (&w)[8], float eps) {
  constexpr int kLanes = Row<D>::kLanes;
  static_assert((N == 2 || N == 4) && 2 * N <= kLanes, "a lane for each sum");
  const int lane = threadIdx.x & 31;
  float s[2 * N];                                 // [half][row]
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* x = r[n].x + 4 * h;
      s[h * N + n] = __fadd_rn(__fadd_rn(__fmul_rn(x[0], x[0]), __fmul_rn(x[1], x[1])),
                               __fadd_rn(__fmul_rn(x[2], x[2]), __fmul_rn(x[3], x[3])));
    }
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    const int m = N / o;                          // sums that a lane keeps
    if (m >= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < m; ++i) {
        const float keep = up ? s[i + m] : s[i], give = up ? s[i] : s[i + m];
        s[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, o));
      }
    } else {
      s[0] = __fadd_rn(s[0], __shfl_xor_sync(0xffffffffu, s[0], o));
    }
  }
  const float sum = __fadd_rn(s[0], __shfl_xor_sync(0xffffffffu, s[0], 1));   // bit 0 of the lane: the half
  const float mean = __fmul_rn(sum, 1.0f / D);    // exact: a power of two
  const float k = __frcp_rn(__fsqrt_rn(__fadd_rn(mean, eps)));
#pragma unroll
  for (int n = 0; n < N; ++n) {                   // the next bits: the row, its upper bit first
    const float f = __shfl_sync(0xffffffffu, k, N == 4 ? (n & 2) | (n & 1) << 2 : n << 1, kLanes);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[n].x[i] = __fmul_rn(__fmul_rn(r[n].x[i], f), w[i]);
  }
}

// The cosines and sines of a lane's elements (kHalves: of its four pairs; kPairs: two pairs for each four elements).
struct Turn {
  float c[8], s[8];
};

template <int D, int MODE>
__device__ __forceinline__ void load_turn(const KvAppendParams& p, int pos, int l, Turn& t) {
  const int half = p.rope_dim >> 1;
  const float* c = p.cos + static_cast<long long>(pos) * half;
  const float* s = p.sin + static_cast<long long>(pos) * half;
  if (MODE == kHalves) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(c + 4 * l)), v = __ldg(reinterpret_cast<const float4*>(s + 4 * l));
    t.c[0] = u.x, t.c[1] = u.y, t.c[2] = u.z, t.c[3] = u.w;
    t.s[0] = v.x, t.s[1] = v.y, t.s[2] = v.z, t.s[3] = v.w;
  }
#pragma unroll
  for (int h = 0; h < 2 && MODE != kHalves; ++h) {
    const int d = h * (D / 2) + 4 * l;
    if (d >= p.rope_dim) continue;
    if (MODE == kPairs) {
      const float2 u = __ldg(reinterpret_cast<const float2*>(c + d / 2)), v = __ldg(reinterpret_cast<const float2*>(s + d / 2));
      t.c[4 * h] = u.x, t.c[4 * h + 1] = u.y;
      t.s[4 * h] = v.x, t.s[4 * h + 1] = v.y;
    } else {
      const int at = d < half ? d : d - half;
#pragma unroll
      for (int i = 0; i < 4; ++i) t.c[4 * h + i] = __ldg(c + at + i), t.s[4 * h + i] = __ldg(s + at + i);
    }
  }
}

// (a, b) <- (a c - b s, b c + a s), one rounding a step.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float y = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = y;
}

// Rotates a row.  Every lane takes part.
template <int D, int MODE>
__device__ __forceinline__ void rotate_row(const KvAppendParams& p, int l, const Turn& t, Row<D>& r) {
  if (MODE == kHalves) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn(r.x[i], r.x[4 + i], t.c[i], t.s[i]);
  } else if (MODE == kPairs) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (h * (D / 2) + 4 * l < p.rope_dim) {
        turn(r.x[4 * h], r.x[4 * h + 1], t.c[4 * h], t.s[4 * h]);
        turn(r.x[4 * h + 2], r.x[4 * h + 3], t.c[4 * h + 1], t.s[4 * h + 1]);
      }
  } else if (MODE == kPart) {
    // four elements' partners are four of another lane, in its first or second half
    constexpr int kLanes = Row<D>::kLanes;
    const int half = p.rope_dim >> 1, away = half >> 2, first = (threadIdx.x & 31) - l;
    float y[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int chunk = h * kLanes + l, d = 4 * chunk;
      const int from = d < half ? chunk + away : d < p.rope_dim ? chunk - away : chunk;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = __shfl_sync(0xffffffffu, r.x[i], first + from % kLanes);
        const float v = __shfl_sync(0xffffffffu, r.x[4 + i], first + from % kLanes);
        const float o = from < kLanes ? u : v, x = r.x[4 * h + i];
        y[4 * h + i] = d < half ? __fsub_rn(__fmul_rn(x, t.c[4 * h + i]), __fmul_rn(o, t.s[4 * h + i]))
                       : d < p.rope_dim ? __fadd_rn(__fmul_rn(x, t.c[4 * h + i]), __fmul_rn(o, t.s[4 * h + i])) : x;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r.x[i] = y[i];
  }
}

// Queries: one warp takes kQRows heads of one token.
template <int D, int MODE, bool BF16>
__device__ __forceinline__ void append_queries(const KvAppendParams& p, unsigned task, int lane) {
  using R = Row<D>;
  constexpr int kSteps = kQRows / R::kRows, kSize = BF16 ? 2 : 4;
  const unsigned groups = (p.Hq + kQRows - 1) / kQRows;
  const int t = static_cast<int>(task / groups), l = lane % R::kLanes;
  const int h0 = static_cast<int>(task - t * groups) * kQRows + lane / R::kLanes;
  if (t >= p.b.T) return;
  R r[kSteps];   // on their way while the token's sequence and position are found; past the last head, that one again
  const uint8_t* src = static_cast<const uint8_t*>(p.q) + (t * p.q_stride + 4 * l) * kSize;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) load_row<D, BF16>(src + min(h0 + i * R::kRows, p.Hq - 1) * (D * kSize), r[i]);
  const int b = warp_count_le(p.b.B, t, [&](int j) { return __ldg(p.b.cu + j); });
  int pos = -1;
  if (b < p.b.B && t >= __ldg(p.b.cu + b)) pos = __ldg(p.b.kv_len + b) - (__ldg(p.b.cu + b + 1) - t);
  if (MODE != kNone && pos >= p.rope_rows) {
    if (lane == 0) atomicOr(p.err, kDevErrIndex);
    pos = -1;
  }
  Turn tn;
  if (MODE != kNone && pos >= 0) load_turn<D, MODE>(p, pos, l, tn);
  if (p.q_norm && pos >= 0) {
    float w[8];
    load_weights<D>(p.q_norm, l, w);
    norm_rows<D, kSteps>(r, w, p.eps);
  }
  const long long to = (static_cast<long long>(t) * p.Hq + h0) * D;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (pos >= 0) {
      if (MODE != kNone) rotate_row<D, MODE>(p, l, tn, r[i]);
    } else {
      zero_row(r[i]);
    }
    if (h0 + i * R::kRows < p.Hq) store_row<D>(p.q_out, to + i * R::kRows * D, p.out_bf16, l, r[i]);
  }
}

// The largest of m and eight magnitudes; a NaN stays.
__device__ __forceinline__ float largest(float m, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(x[i]), "f"(x[i + 1]));
  return m;
}

// Keys or values: kBlockWarps warps take one block of one head, eight tokens
// each (s_max: their largest magnitudes).  Slots of a sequence start at
// cu[b] / 16 + 2 b: at least as many as the blocks it touches.  Every warp of
// a unit (the block's warps) calls it and meets the others once.
template <int D, int MODE, bool BF16>
__device__ __forceinline__ void append_block(const KvAppendParams& p, int slot, int h, bool is_k, int unit, int part,
                                             int lane, float* s_max, float4* s_turn) {
  using R = Row<D>;
  constexpr int kSteps = kBlockRows / R::kRows, kSize = BF16 ? 2 : 4;
  const int l = lane % R::kLanes;
  int pos0 = 0, lo = 0, hi = 0;      // this lane's rows are at pos0 + i * kRows; those in [lo, hi) are new
  bool part_new = false;             // not all of the block is
  long long row0 = -1;
  const int b = warp_count_le(p.b.B, slot, [&](int j) { return (__ldg(p.b.cu + j) >> 4) + 2 * j; });
  R r[kSteps];
  float s0 = 0.f, m = 0.f;
  if (b < p.b.B && h < p.c.heads) {
    const int c0 = __ldg(p.b.cu + b), c1 = __ldg(p.b.cu + b + 1), len = __ldg(p.b.kv_len + b);
    const int start = len - (c1 - c0);          // position of the first new token
    const int from = max(start, 0);
    const int at = slot - ((c0 >> 4) + 2 * b), blk = (from >> 4) + at;
    if (c1 > c0 && at >= 0 && blk * kKvBlock < len) {
      // tokens past the rotation tables are not stored, neither their keys nor their values
      const int end = MODE != kNone ? min(len, p.rope_rows) : len;
      lo = max(from, blk * kKvBlock), hi = min(end, (blk + 1) * kKvBlock);
      const bool beyond = end < min(len, (blk + 1) * kKvBlock);
      part_new = hi - lo < kKvBlock;
      pos0 = blk * kKvBlock + part * kBlockRows + lane / R::kLanes;
      const long long tok0 = static_cast<long long>(c0) + (lo - start);   // packed row of position lo
      if (c0 >= 0 && lo < hi && tok0 + (hi - lo) <= p.b.T) {
        // the rows, on their way while the page is looked up; for one that is not new, the nearest that is
        const long long stride = is_k ? p.k_stride : p.v_stride;
        const uint8_t* src = static_cast<const uint8_t*>(is_k ? p.k : p.v) + (tok0 * stride + h * D + 4 * l) * kSize;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int pos = min(max(pos0 + i * R::kRows, lo), hi - 1);
          load_row<D, BF16>(src + (pos - lo) * stride * kSize, r[i]);
          if (MODE == kHalves && is_k) {        // no registers for these yet: by way of shared memory, the lane's own
            const float* c = p.cos + static_cast<long long>(pos) * (D / 2) + 4 * l;
            const float* s = p.sin + static_cast<long long>(pos) * (D / 2) + 4 * l;
            const uint32_t to = smem_u32(s_turn + 2 * 32 * i + lane);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to), "l"(c) : "memory");
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to + 32 * 16), "l"(s) : "memory");
          }
        }
        row0 = kv_row(p.c, p.b.table, p.b.table_stride, b, blk * kKvBlock, h);
      }
      if ((row0 < 0 || beyond) && lane == 0) atomicOr(p.err, kDevErrIndex);
      if (row0 < 0) {
        asm volatile("cp.async.wait_all;" ::: "memory");
      } else if (lo > blk * kKvBlock) {
        s0 = (is_k ? p.c.ks : p.c.vs)[row0 >> 4];
      }
    }
  }
  if (row0 >= 0) {
    if (is_k && p.k_norm) {
      float w[8];
      load_weights<D>(p.k_norm, l, w);
      norm_rows<D, kSteps>(r, w, p.eps);
    }
    if (is_k && MODE != kNone) {
      if (MODE == kHalves) asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        Turn tn;
        if (MODE == kHalves) {
          const float4 u = s_turn[2 * 32 * i + lane], v = s_turn[2 * 32 * i + 32 + lane];
          tn.c[0] = u.x, tn.c[1] = u.y, tn.c[2] = u.z, tn.c[3] = u.w;
          tn.s[0] = v.x, tn.s[1] = v.y, tn.s[2] = v.z, tn.s[3] = v.w;
        } else {
          load_turn<D, MODE>(p, min(max(pos0 + i * R::kRows, lo), hi - 1), l, tn);
        }
        rotate_row<D, MODE>(p, l, tn, r[i]);
      }
    }
    if (part_new) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (pos0 + i * R::kRows < lo || pos0 + i * R::kRows >= hi) zero_row(r[i]);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) m = largest(m, r[i].x);
    // a code cannot hold a NaN or an infinity: 0 and the largest number instead, and the status word says so
    if (!(m <= FLT_MAX)) {
      atomicOr(p.err, kDevErrValue);
      m = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& x = r[i].x[e];
          x = x != x ? 0.f : fminf(fmaxf(x, -FLT_MAX), FLT_MAX);
          m = fmaxf(m, fabsf(x));
        }
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));   // not negative: in the bits' order
  }
  if (lane == 0) s_max[part] = m;
  // the block's warps; also: all have read its old scale
  asm volatile("bar.sync %0, %1;" ::"r"(1 + unit), "n"(32 * kBlockWarps) : "memory");
  if (row0 < 0) return;
#pragma unroll
  for (int i = 0; i < kBlockWarps; ++i) m = fmaxf(m, s_max[i]);
  float s = fmaxf(s0, __fmul_rn(m, 1.0f / 127.0f));
  if (s < kTinyScale) s = 0.f;
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  if (part == 0 && lane == 0) (is_k ? p.c.ks : p.c.vs)[row0 >> 4] = s;
  int8_t* codes = (is_k ? p.c.k : p.c.v) + (row0 + (pos0 & (kKvBlock - 1))) * D + 4 * l;
  const auto pack = [](const float (&x)[4]) {
    uint32_t w;
    asm("{\n\t.reg .b32 t;\n\tcvt.pack.sat.s8.s32.b32 t, %4, %3, 0;\n\tcvt.pack.sat.s8.s32.b32 %0, %2, %1, t;\n\t}"
        : "=r"(w)
        : "r"(__float2int_rn(x[0])), "r"(__float2int_rn(x[1])), "r"(__float2int_rn(x[2])), "r"(__float2int_rn(x[3])));
    return w;
  };
  const float ratio = part_new && s > 0.f ? __fdiv_rn(s0, s) : 0.f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int pos = pos0 + i * R::kRows;
    if (part_new && (pos >= hi || (pos < lo && ratio == 1.f))) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t* to = reinterpret_cast<uint32_t*>(codes + i * R::kRows * D + half * (D / 2));
      float x[4];
      if (part_new && pos < lo) {
        const uint32_t old = *to;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __fmul_rn(static_cast<float>(static_cast<int8_t>(old >> (8 * e))), ratio);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __fmul_rn(r[i].x[4 * half + e], inv);   // at most 127 (1 + 2^-22)
      }
      *to = pack(x);
    }
  }
}

// Registers for four CTAs an SM, three with fp32's wider rows (five and four: 133 us for 101, fp32 the same).
template <int D, int MODE, bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? 4 : 3) q4_kv_append_kernel(const __grid_constant__ KvAppendParams p,
                                                                int kv_ctas) {
  __shared__ float s_max[kWarps];
  __shared__ float4 s_turn[MODE == kHalves ? kWarps / 2 : 1][kBlockRows * Row<D>::kLanes * 2];   // of the keys' warps
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (static_cast<int>(blockIdx.x) < kv_ctas) {   // the longer tasks first; a CTA takes keys and values of kHeads heads
    const int unit = warp / kBlockWarps, groups = (p.c.heads + kHeads - 1) / kHeads, slot = blockIdx.x / groups;
    const int h = (blockIdx.x - slot * groups) * kHeads + (unit >> 1), part = warp % kBlockWarps;
    append_block<D, MODE, BF16>(p, slot, h, (unit & 1) == 0, unit, part, lane, s_max + unit * kBlockWarps,
                                s_turn[MODE == kHalves ? (unit >> 1) * kBlockWarps + part : 0]);
  } else {
    append_queries<D, MODE, BF16>(p, (blockIdx.x - kv_ctas) * kWarps + warp, lane);
  }
}

// One thread reads 16 codes of a token's head (keys and values) and writes 16 numbers.
__device__ __forceinline__ void widen16(void* out, long long off, int bf16, const uint4& w, float s) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
  float f[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    f[i] = __fmul_rn(static_cast<float>(static_cast<int8_t>(q[i >> 2] >> (8 * (i & 3)))), s);
  if (bf16) {
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + off);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[8 * j + 2 * i], f[8 * j + 2 * i + 1]);
      o[j] = *reinterpret_cast<uint4*>(h);
    }
  } else {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + off);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
  }
}

__global__ void __launch_bounds__(kThreads) q4_kv_gather_kernel(const __grid_constant__ KvGatherParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int chunks = p.c.dim / 16;                       // per row: 4 or 8
  const long long rows = static_cast<long long>(p.T) * p.c.heads;
  const int per_warp = 32 / chunks;                      // rows of one warp
  const int lane = threadIdx.x & 31;
  const long long row0 = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * per_warp;
  if (row0 >= rows) return;
  const int t0 = static_cast<int>(row0 / p.c.heads);
  int b = warp_count_le(p.B, t0, [&](int j) { return __ldg(p.cu + j); });
  const long long row = row0 + lane / chunks;
  if (row >= rows) return;
  const int t = static_cast<int>(row / p.c.heads), h = static_cast<int>(row % p.c.heads);
  while (b < p.B && t >= __ldg(p.cu + b + 1)) ++b;       // a warp's rows may span sequences
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  float ks = 0.f, vs = 0.f;
  if (b < p.B && t >= __ldg(p.cu + b)) {
    const int pos = __ldg(p.first + b) + (t - __ldg(p.cu + b));
    const long long at = pos < 0 ? -1 : kv_row(p.c, p.table, p.table_stride, b, pos, h);
    if (at >= 0) {
      const long long off = at * p.c.dim + (lane % chunks) * 16;
      k = *reinterpret_cast<const uint4*>(p.c.k + off);
      v = *reinterpret_cast<const uint4*>(p.c.v + off);
      ks = p.c.ks[at >> 4];
      vs = p.c.vs[at >> 4];
    } else {
      atomicOr(p.err, kDevErrIndex);
    }
  }
  const long long to = row * p.c.dim + (lane % chunks) * 16;
  widen16(p.k_out, to, p.out_bf16, k, ks);
  widen16(p.v_out, to, p.out_bf16, v, vs);
}

template <typename... Args>
cudaError_t launch_pdl(void (*kernel)(Args...), unsigned grid, unsigned threads, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t st) {
  const long long slots = p.b.T / kKvBlock + 2LL * p.b.B;
  const long long kv_ctas = slots * ((p.c.heads + kHeads - 1) / kHeads);
  const long long q_tasks = p.q_out ? static_cast<long long>(p.b.T) * ((p.Hq + kQRows - 1) / kQRows) : 0;
  const long long grid = kv_ctas + (q_tasks + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL || q_tasks > 0xffffffffLL) return cudaErrorInvalidConfiguration;
  const int mode = !p.cos ? kNone : p.rope_pairs ? kPairs : p.rope_dim == p.c.dim ? kHalves : kPart;
  static void (*const kernels[2][2][4])(KvAppendParams, int) = {
      {{q4_kv_append_kernel<64, kNone, false>, q4_kv_append_kernel<64, kHalves, false>,
        q4_kv_append_kernel<64, kPairs, false>, q4_kv_append_kernel<64, kPart, false>},
       {q4_kv_append_kernel<64, kNone, true>, q4_kv_append_kernel<64, kHalves, true>,
        q4_kv_append_kernel<64, kPairs, true>, q4_kv_append_kernel<64, kPart, true>}},
      {{q4_kv_append_kernel<128, kNone, false>, q4_kv_append_kernel<128, kHalves, false>,
        q4_kv_append_kernel<128, kPairs, false>, q4_kv_append_kernel<128, kPart, false>},
       {q4_kv_append_kernel<128, kNone, true>, q4_kv_append_kernel<128, kHalves, true>,
        q4_kv_append_kernel<128, kPairs, true>, q4_kv_append_kernel<128, kPart, true>}}};
  return launch_pdl(kernels[p.c.dim == 128][p.in_bf16 != 0][mode], static_cast<unsigned>(grid), kThreads, st, p,
                    static_cast<int>(kv_ctas));
}

cudaError_t launch_kv_gather(const KvGatherParams& p, cudaStream_t st) {
  const long long per = 32 / (p.c.dim / 16) * kWarps;
  const long long grid = (static_cast<long long>(p.T) * p.c.heads + per - 1) / per;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(q4_kv_gather_kernel, static_cast<unsigned>(grid), kThreads, st, p);
}

}  // namespace q4
