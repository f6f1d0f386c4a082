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
#include <cfloat>
#include <type_traits>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kQRows = 4;              // query heads of one token a warp takes at once
constexpr int kBlockWarps = 4;         // warps that share a block of keys or values
constexpr int kBlockRows = kKvBlock / kBlockWarps;
constexpr float kTinyScale = 7.70371977754894341e-34f;   // 2^-110

// D / 32 consecutive elements of a row, as fp32.
template <int E>
__device__ __forceinline__ void load_row(const void* base, long long off, int bf16, float (&x)[E]) {
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + off;
    if (E == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      x[0] = __uint_as_float(w.x << 16);
      x[1] = __uint_as_float(w.x & 0xffff0000u);
      x[2] = __uint_as_float(w.y << 16);
      x[E - 1] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
      x[0] = __uint_as_float(w << 16);
      x[1] = __uint_as_float(w & 0xffff0000u);
    }
  } else {
    const float* p = static_cast<const float*>(base) + off;
    if (E == 4) {
      const float4 w = *reinterpret_cast<const float4*>(p);
      x[0] = w.x, x[1] = w.y, x[2] = w.z, x[E - 1] = w.w;
    } else {
      const float2 w = *reinterpret_cast<const float2*>(p);
      x[0] = w.x, x[1] = w.y;
    }
  }
}

template <int E>
__device__ __forceinline__ void store_row(void* base, long long off, int bf16, const float (&x)[E]) {
  if (bf16) {
    __nv_bfloat162 h[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    uint16_t* p = static_cast<uint16_t*>(base) + off;
    if (E == 4)
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
    else
      *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<uint32_t*>(h);
  } else {
    float* p = static_cast<float*>(base) + off;
    if (E == 4)
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[E - 1]);
    else
      *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  }
}

// x <- (x * 1/sqrt(mean(x^2) + eps)) * w, one rounding a step; the sum of
// squares neighbours first, in the lane and then over lane distances 1 to 16.
template <int E>
__device__ __forceinline__ void norm_row(float (&x)[E], const float (&w)[E], float eps) {
  float s = __fadd_rn(__fmul_rn(x[0], x[0]), __fmul_rn(x[1], x[1]));
  if (E == 4)
    s = __fadd_rn(s, __fadd_rn(__fmul_rn(x[2], x[2]), __fmul_rn(x[E - 1], x[E - 1])));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
  const float mean = __fmul_rn(s, 1.0f / (32 * E));   // exact: a power of two
  const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(mean, eps)));
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), w[i]);
}

// This lane's cosines and sines at a position: for halves the E of its own
// elements, for pairs E / 2 of them (one per pair).
template <int E>
struct Turn {
  float c[E], s[E];
};

template <int E>
__device__ __forceinline__ void load_turn(const KvAppendParams& p, int pos, int lane, Turn<E>& t) {
  const int d = lane * E, half = p.rope_dim >> 1;
  if (d >= p.rope_dim) return;
  const long long row = static_cast<long long>(pos) * half;
  if (p.rope_pairs) {
    const float* c = p.cos + row + (d >> 1);
    const float* s = p.sin + row + (d >> 1);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) t.c[i] = __ldg(c + i), t.s[i] = __ldg(s + i);
  } else {
    const int at = d < half ? d : d - half;
#pragma unroll
    for (int i = 0; i < E; ++i) t.c[i] = __ldg(p.cos + row + at + i), t.s[i] = __ldg(p.sin + row + at + i);
  }
}

// Rotates a row held across the warp.  Every lane takes part.
template <int E>
__device__ __forceinline__ void rotate_row(const KvAppendParams& p, int lane, const Turn<E>& t,
                                           float (&x)[E]) {
  const int d = lane * E, half = p.rope_dim >> 1;
  if (p.rope_pairs) {
    if (d < p.rope_dim) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
        x[2 * i + 1] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
      }
    }
    return;
  }
  const int away = half / E;
  const int from = d < half ? lane + away : d < p.rope_dim ? lane - away : lane;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float o = __shfl_sync(0xffffffffu, x[i], from);
    if (d < half)
      x[i] = __fsub_rn(__fmul_rn(x[i], t.c[i]), __fmul_rn(o, t.s[i]));
    else if (d < p.rope_dim)
      x[i] = __fadd_rn(__fmul_rn(x[i], t.c[i]), __fmul_rn(o, t.s[i]));
  }
}

// Queries: one warp takes kQRows heads of one token.
template <int E>
__device__ void append_queries(const KvAppendParams& p, long long task, int lane) {
  const int groups = (p.Hq + kQRows - 1) / kQRows;
  const int t = static_cast<int>(task / groups);
  const int h0 = static_cast<int>(task % groups) * kQRows;
  if (t >= p.b.T) return;
  constexpr int D = 32 * E;
  float x[kQRows][E];   // on their way while the token's sequence and position are found
#pragma unroll
  for (int r = 0; r < kQRows; ++r) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[r][i] = 0.f;
    if (h0 + r < p.Hq) load_row<E>(p.q, t * p.q_stride + (h0 + r) * D + lane * E, p.in_bf16, x[r]);
  }
  const int b = warp_count_le(p.b.B, t, [&](int j) { return __ldg(p.b.cu + j); });
  int pos = -1;
  if (b < p.b.B && t >= __ldg(p.b.cu + b)) pos = __ldg(p.b.kv_len + b) - (__ldg(p.b.cu + b + 1) - t);
  if (p.cos && pos >= p.rope_rows) {
    if (lane == 0) atomicOr(p.err, kDevErrIndex);
    pos = -1;
  }
  if (pos >= 0) {
    Turn<E> turn;
    float w[E];
    if (p.cos) load_turn<E>(p, pos, lane, turn);
    if (p.q_norm) {
#pragma unroll
      for (int i = 0; i < E; ++i) w[i] = __ldg(p.q_norm + lane * E + i);
    }
#pragma unroll
    for (int r = 0; r < kQRows; ++r) {
      if (p.q_norm) norm_row<E>(x[r], w, p.eps);
      if (p.cos) rotate_row<E>(p, lane, turn, x[r]);
    }
  } else {
#pragma unroll
    for (int r = 0; r < kQRows; ++r)
#pragma unroll
      for (int i = 0; i < E; ++i) x[r][i] = 0.f;
  }
#pragma unroll
  for (int r = 0; r < kQRows; ++r)
    if (h0 + r < p.Hq)
      store_row<E>(p.q_out, (static_cast<long long>(t) * p.Hq + h0 + r) * D + lane * E, p.out_bf16, x[r]);
}

// Keys or values: kBlockWarps warps take one block of one head, four tokens
// each (s_max: their largest magnitudes).  Slots of a sequence start at
// cu[b] / 16 + 2 b: at least as many as the blocks it touches.  Every thread of
// the CTA calls it and meets once.
template <int E>
__device__ void append_block(const KvAppendParams& p, long long slot, int h, bool is_k, int part, int lane,
                             float* s_max) {
  constexpr int D = 32 * E;
  int blk = 0, lo = 0, hi = 0;       // of this warp's four positions, those in [lo, hi) are new
  long long row0 = -1;
  const int b = warp_count_le(p.b.B, static_cast<int>(slot), [&](int j) { return (__ldg(p.b.cu + j) >> 4) + 2 * j; });
  float x[kBlockRows][E];
  float s0 = 0.f, m = 0.f;
  bool had = false;
  if (b < p.b.B) {
    const int c0 = __ldg(p.b.cu + b), c1 = __ldg(p.b.cu + b + 1), len = __ldg(p.b.kv_len + b);
    const int start = len - (c1 - c0);          // position of the first new token
    const int from = max(start, 0);
    const int at = static_cast<int>(slot) - ((c0 >> 4) + 2 * b);
    blk = (from >> 4) + at;
    if (c1 > c0 && at >= 0 && blk * kKvBlock < len) {
      lo = max(from, blk * kKvBlock), hi = min(len, (blk + 1) * kKvBlock);
      const long long tok0 = static_cast<long long>(c0) + (lo - start);   // packed row of position lo
      row0 = kv_row(p.c, p.b.table, p.b.table_stride, b, blk * kKvBlock, h);
      if (row0 < 0 || c0 < 0 || tok0 + (hi - lo) > p.b.T || (is_k && p.cos && hi > p.rope_rows)) {
        if (lane == 0) atomicOr(p.err, kDevErrIndex);
        row0 = -1;
      } else {
        const void* src = is_k ? p.k : p.v;
        const long long stride = is_k ? p.k_stride : p.v_stride;
#pragma unroll
        for (int r = 0; r < kBlockRows; ++r) {
#pragma unroll
          for (int i = 0; i < E; ++i) x[r][i] = 0.f;
          const int pos = blk * kKvBlock + part * kBlockRows + r;
          if (pos >= lo && pos < hi)
            load_row<E>(src, (tok0 + pos - lo) * stride + h * D + lane * E, p.in_bf16, x[r]);
        }
        had = lo > blk * kKvBlock;
        if (had) s0 = (is_k ? p.c.ks : p.c.vs)[row0 >> 4];
      }
    }
  }
  if (row0 >= 0) {
    if (is_k && (p.k_norm || p.cos)) {
      float w[E];
      if (p.k_norm) {
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = __ldg(p.k_norm + lane * E + i);
      }
#pragma unroll
      for (int r = 0; r < kBlockRows; ++r) {
        const int pos = blk * kKvBlock + part * kBlockRows + r;
        if (pos < lo || pos >= hi) continue;
        if (p.k_norm) norm_row<E>(x[r], w, p.eps);
        if (p.cos) {
          Turn<E> turn;
          load_turn<E>(p, pos, lane, turn);
          rotate_row<E>(p, lane, turn, x[r]);
        }
      }
    }
    // a code cannot hold a NaN or an infinity: 0 and the largest number instead, and the status word says so
    bool odd = false;
#pragma unroll
    for (int r = 0; r < kBlockRows; ++r)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float a = fabsf(x[r][i]);
        if (!(a <= FLT_MAX)) {
          odd = true;
          x[r][i] = x[r][i] != x[r][i] ? 0.f : copysignf(FLT_MAX, x[r][i]);
        }
        m = fmaxf(m, fabsf(x[r][i]));
      }
    if (odd) atomicOr(p.err, kDevErrValue);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (lane == 0) s_max[part] = m;
  __syncthreads();   // also: every warp has read the block's old scale
  if (row0 < 0) return;
#pragma unroll
  for (int i = 0; i < kBlockWarps; ++i) m = fmaxf(m, s_max[i]);
  float s = fmaxf(s0, __fmul_rn(m, 1.0f / 127.0f));
  if (s < kTinyScale) s = 0.f;
  const float inv = s > 0.f ? __fdiv_rn(1.0f, s) : 0.f;
  const float ratio = s > 0.f ? __fdiv_rn(s0, s) : 0.f;
  if (part == 0 && lane == 0) (is_k ? p.c.ks : p.c.vs)[row0 >> 4] = s;
  int8_t* codes = (is_k ? p.c.k : p.c.v) + (row0 + part * kBlockRows) * D + lane * E;
  using Word = typename std::conditional<E == 4, uint32_t, uint16_t>::type;   // the lane's E codes of a row
#pragma unroll
  for (int r = 0; r < kBlockRows; ++r) {
    const int pos = blk * kKvBlock + part * kBlockRows + r;
    Word* to = reinterpret_cast<Word*>(codes + r * D);
    uint32_t w = 0;
    if (pos >= lo && pos < hi) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = max(-127, min(127, __float2int_rn(__fmul_rn(x[r][i], inv))));
        w |= (static_cast<uint32_t>(c) & 0xffu) << (8 * i);
      }
    } else if (pos < lo && ratio != 1.f) {
      const uint32_t old = *to;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float c = static_cast<float>(static_cast<int8_t>(old >> (8 * i)));
        w |= (static_cast<uint32_t>(__float2int_rn(__fmul_rn(c, ratio))) & 0xffu) << (8 * i);
      }
    } else {
      continue;
    }
    *to = static_cast<Word>(w);
  }
}

template <int E>
__global__ void __launch_bounds__(kThreads) q4_kv_append_kernel(const __grid_constant__ KvAppendParams p,
                                                                int kv_ctas) {
  __shared__ float s_max[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (static_cast<int>(blockIdx.x) < kv_ctas) {   // the longer tasks first
    const int unit = warp / kBlockWarps;
    const long long task = static_cast<long long>(blockIdx.x) * (kWarps / kBlockWarps) + unit;
    const int per = 2 * p.c.heads;
    const int i = static_cast<int>(task % per);
    append_block<E>(p, task / per, i % p.c.heads, i < p.c.heads, warp % kBlockWarps, lane, s_max + unit * kBlockWarps);
  } else {
    append_queries<E>(p, static_cast<long long>(blockIdx.x - kv_ctas) * kWarps + warp, lane);
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
  const int units = kWarps / kBlockWarps;
  const long long kv_ctas = (slots * 2 * p.c.heads + units - 1) / units;
  const long long q_tasks = p.q_out ? static_cast<long long>(p.b.T) * ((p.Hq + kQRows - 1) / kQRows) : 0;
  const long long grid = kv_ctas + (q_tasks + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(p.c.dim == 128 ? q4_kv_append_kernel<4> : q4_kv_append_kernel<2>,
                    static_cast<unsigned>(grid), kThreads, st, p, static_cast<int>(kv_ctas));
}

cudaError_t launch_kv_gather(const KvGatherParams& p, cudaStream_t st) {
  const long long per = 32 / (p.c.dim / 16) * kWarps;
  const long long grid = (static_cast<long long>(p.T) * p.c.heads + per - 1) / per;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(q4_kv_gather_kernel, static_cast<unsigned>(grid), kThreads, st, p);
}

}  // namespace q4
