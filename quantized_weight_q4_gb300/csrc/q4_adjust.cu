// Logits before sampling (sm_103a): penalties for repeated tokens, biases and
// a grammar's bit masks, one pass over each row.
//
//   x = logits[t, v]; if v is in the history: x > 0 ? x / r : x * r;
//   x -= f * n; if n > 0: x -= p;  x += bias;  -inf where the mask has a 0.
//
// A CTA takes a slice of a row.  Its logits are on their way into registers
// while it looks through the row's history and biases for tokens of the slice
// and notes them in shared memory, a word a token: the last bias entry, whether
// the prompt has it, how often the answer has it.  Notes are whole numbers, so
// their order does not matter.  The slice is stored as it came, with the mask's
// -inf, and then the tokens with a note again, a thread each, from a list:
// beside their neighbours they would hold up whole warps, one after another.
// A CTA is bound by the latency of what it looks up; so all that can be is on
// its way at once, and the first part of the history before its length is known.
//
// Measured: 200 rows of 128,007 bf16 logits, histories of 2,667 to 8,000 tokens,
// 100 biases a row, grammars on half of the rows 45 us (2.3 TB/s of logits); the
// same without any of these 17 us.  What is looked up comes first and leaves HBM
// idle: of a CTA's 6.5 us, 1.8 pass until history and lengths are there and notes
// are cleared, 1.6 noting, 1.3 searching for notes, 0.9 storing, 0.7 with the list.
// Room in the list taken a quad of words at a time: 48 us; a warp at a time, by
// ballots 53.  Then (48 us) slices of 8192 logits took 52, of 4096 61; a cluster
// that shares the history by reductions in each other's shared memory 65 to 81; a
// persistent form that holds the history in registers 79.
#include <algorithm>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 512;
constexpr int kUnit = 8;                  // logits that a thread has side by side
constexpr int kUnits = 4;                 // of them
constexpr int kAhead = 4;                 // fours of the history that a thread asks for at once
constexpr int kMostSlice = kThreads * kUnit * kUnits;
constexpr unsigned kSeen = 1u << 19;      // a note: bits 0-18 how often, bit 19 in the prompt, bits 20-31 bias entry + 1
constexpr unsigned kTimes = kSeen - 1;
constexpr int kBiasShift = 20;

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, long long i) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16) : static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, long long i, float x) {
  if (BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else
    static_cast<float*>(p)[i] = x;
}

// Notes of a token, `at` in the slice of n: without a branch, as most tokens are of other slices.
__device__ __forceinline__ void note_said(uint32_t notes, unsigned at, unsigned n) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %0, %1;\n\t@p red.shared.add.u32 [%2], 1;\n\t}" ::"r"(at), "r"(n),
               "r"(notes + 4 * at) : "memory");
}
__device__ __forceinline__ void note_seen(uint32_t notes, unsigned at, unsigned n) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %0, %1;\n\t@p red.shared.or.b32 [%2], %3;\n\t}" ::"r"(at), "r"(n),
               "r"(notes + 4 * at), "r"(kSeen) : "memory");
}

// Eight logits side by side, as they lie in memory.
template <bool BF16>
struct Unit {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, long long i) {
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (BF16 ? 2 : 4));
#pragma unroll
    for (int k = 0; k < (BF16 ? 1 : 2); ++k) w[k] = at[k];
  }
  __device__ __forceinline__ void store(void* p, long long i) const {
    uint4* at = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p) + i * (BF16 ? 2 : 4));
#pragma unroll
    for (int k = 0; k < (BF16 ? 1 : 2); ++k) at[k] = w[k];
  }
  __device__ __forceinline__ void get(float (&x)[kUnit]) const {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int k = 0; k < kUnit; ++k)
      x[k] = __uint_as_float(BF16 ? (k & 1 ? v[k >> 1] & 0xffff0000u : v[k >> 1] << 16) : v[k]);
  }
  // -inf where `allowed` has a 0.
  __device__ __forceinline__ void mask(uint32_t allowed) {
    uint32_t* v = reinterpret_cast<uint32_t*>(w);
#pragma unroll
    for (int k = 0; k < (BF16 ? 4 : 8); ++k) {
      if (BF16) {
        const uint32_t two = allowed >> 2 * k, keep = (two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u);
        v[k] = (v[k] & keep) | (0xff80ff80u & ~keep);
      } else if (!(allowed >> k & 1u)) {
        v[k] = 0xff800000u;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&x)[kUnit]) {
    uint32_t* v = reinterpret_cast<uint32_t*>(w);
#pragma unroll
    for (int k = 0; k < kUnit; k += BF16 ? 2 : 1) {
      if (BF16) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(x[k], x[k + 1]);
        v[k >> 1] = *reinterpret_cast<const uint32_t*>(&y);
      } else {
        v[k] = __float_as_uint(x[k]);
      }
    }
  }
};

// IN, OUT: bf16 or fp32.  slice: logits of a CTA, a multiple of eight.
template <bool IN, bool OUT>
__global__ void __launch_bounds__(kThreads) q4_adjust_kernel(const __grid_constant__ AdjustParams p, int slice) {
  extern __shared__ __align__(16) unsigned s_mem[];     // [slice] words, [slice] halves
  const int tid = threadIdx.x, t = blockIdx.y;
  const int v0 = blockIdx.x * slice, n = min(slice, p.V - v0);
  pdl_launch_dependents();
  pdl_wait();
  const long long in = t * p.stride + v0, to = t * p.out_stride + v0;
  // eights that begin at 16 bytes in both rows, if there are such: from logit `lead` of the slice on
  constexpr int kInEach = IN ? 8 : 4, kOutEach = OUT ? 8 : 4;   // logits of 16 bytes
  const int in_at = static_cast<int>(((reinterpret_cast<uintptr_t>(p.logits) >> (IN ? 1 : 2)) + in) & (kInEach - 1));
  const int out_at = static_cast<int>(((reinterpret_cast<uintptr_t>(p.out) >> (OUT ? 1 : 2)) + to) & (kOutEach - 1));
  const int lead = IN ? (kInEach - in_at) & (kInEach - 1) : (kOutEach - out_at) & (kOutEach - 1);
  const bool wide = ((in_at + lead) & (kInEach - 1)) == 0 && ((out_at + lead) & (kOutEach - 1)) == 0;
  const int units = wide && n > lead ? (n - lead) / kUnit : 0;
  unsigned* s_note = s_mem;                             // of the slice's logits
  uint16_t* s_list = reinterpret_cast<uint16_t*>(s_note + slice);   // those with a note
  __shared__ int s_listed;
  Unit<IN> x[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    if (i * kThreads + tid < units) x[i].load(p.logits, in + lead + (i * kThreads + tid) * kUnit);
  const int req = p.request ? __ldg(p.request + t) : t;
  const int mask_row = !p.mask ? -1 : p.mask_row ? __ldg(p.mask_row + t) : t;
  const bool known = req >= 0 && req < p.requests;
  const uint32_t* mask = nullptr;
  if (mask_row >= 0 && mask_row < p.masks) mask = reinterpret_cast<const uint32_t*>(p.mask) + mask_row * ((p.V + 31LL) / 32);
  if (blockIdx.x == 0 && tid == 0 && ((p.mask && mask_row >= p.masks) || (p.request && req >= p.requests))) atomicOr(p.err, kDevErrIndex);
  const bool penalties = p.history && known;
  const float* bias = p.bias_index && known ? p.bias + static_cast<long long>(req) * p.bias_width : nullptr;
  const bool notes = penalties || bias;
  auto bits_from = [&](int v) {             // the mask's bits of tokens v .. v + 7, and more above them
    const int w = v >> 5, s = v & 31;
    const uint32_t lo = __ldg(mask + w), hi = s > 24 && v + 32 - s < p.V ? __ldg(mask + w + 1) : 0u;
    return __funnelshift_r(lo, hi, s);
  };
  uint32_t allowed[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    allowed[i] = mask && i * kThreads + tid < units ? bits_from(v0 + lead + (i * kThreads + tid) * kUnit) & 0xffu : 0xffu;
  if (notes) {
    for (int i = tid; i < slice / 4; i += kThreads) reinterpret_cast<uint4*>(s_note)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) s_listed = 0;
    const int32_t* history = p.history + static_cast<long long>(penalties ? req : 0) * p.history_width;
    // four tokens at a time from where the list begins at 16 bytes
    const int skip = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(history) & 15)) & 15) / 4;
    const int fours = penalties ? max(0, p.history_width - skip) / 4 : 0;
    const uint32_t notes_at = smem_u32(s_note);
    const int4* four = reinterpret_cast<const int4*>(history + skip);
    int4 ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      ahead[k] = k * kThreads + tid < fours ? __ldg(four + k * kThreads + tid) : make_int4(-1, -1, -1, -1);
    const int32_t* index = bias ? p.bias_index + static_cast<long long>(req) * p.bias_width : nullptr;
    const int biased = bias && tid < p.bias_width ? __ldg(index + tid) : -1;
    const int len = penalties ? min(__ldg(p.history_len + t), p.history_width) : 0;
    const int prompt = penalties && p.prompt_len ? __ldg(p.prompt_len + t) : 0;
    __syncthreads();
    if (bias) {
      auto note = [&](int token, int i) {
        const int at = token - v0;
        if (static_cast<unsigned>(at) < static_cast<unsigned>(n)) atomicMax(s_note + at, static_cast<unsigned>(i + 1) << kBiasShift);
      };
      note(biased, tid);
      for (int i = kThreads + tid; i < p.bias_width; i += kThreads) note(__ldg(index + i), i);
      if (penalties) __syncthreads();
    }
    if (penalties) {
      const int from_prompt = min(max(prompt, 0), max(len, 0));
      auto note = [&](int token, int i) {
        if (i >= len) return;
        const unsigned at = static_cast<unsigned>(token - v0);
        if (i < from_prompt) note_seen(notes_at, at, n); else note_said(notes_at, at, n);
      };
      auto note4 = [&](const int4& x, int i) {
        const int at = skip + 4 * i;
        const unsigned a[4] = {static_cast<unsigned>(x.x - v0), static_cast<unsigned>(x.y - v0),
                               static_cast<unsigned>(x.z - v0), static_cast<unsigned>(x.w - v0)};
        if (at >= from_prompt && at + 4 <= len) {
#pragma unroll
          for (int k = 0; k < 4; ++k) note_said(notes_at, a[k], n);
        } else if (at + 4 <= from_prompt) {
#pragma unroll
          for (int k = 0; k < 4; ++k) note_seen(notes_at, a[k], n);
        } else {
          note(x.x, at), note(x.y, at + 1), note(x.z, at + 2), note(x.w, at + 3);
        }
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (skip + 4 * (k * kThreads + tid) < len) note4(ahead[k], k * kThreads + tid);
#pragma unroll 4
      for (int i = kAhead * kThreads + tid; i < fours && skip + 4 * i < len; i += kThreads) note4(__ldg(four + i), i);
      if (tid < min(skip, p.history_width)) note(__ldg(history + tid), tid);
      const int rest = skip + 4 * fours + tid;
      if (rest < p.history_width) note(__ldg(history + rest), rest);   // three at most
    }
    __syncthreads();
    // a thread takes room in the list once, for all that it finds
    constexpr int kFours = kMostSlice / 4 / kThreads;
    static_assert(4 * kFours <= 32, "a bit each");
    unsigned found = 0;
#pragma unroll
    for (int k = 0; k < kFours; ++k)
      if (k * kThreads + tid < slice / 4) {
        const uint4 x = reinterpret_cast<const uint4*>(s_note)[k * kThreads + tid];
        found |= ((x.x ? 1u : 0u) | (x.y ? 2u : 0u) | (x.z ? 4u : 0u) | (x.w ? 8u : 0u)) << 4 * k;
      }
    if (found) {
      int to_list = atomicAdd(&s_listed, __popc(found));
      for (; found; found &= found - 1) {
        const int bit = __ffs(found) - 1;
        s_list[to_list++] = static_cast<uint16_t>(4 * ((bit >> 2) * kThreads + tid) + (bit & 3));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = i * kThreads + tid;
    if (u >= units) break;
    const int at = lead + u * kUnit;
    Unit<OUT> z;
    if (IN == OUT) {
      z = reinterpret_cast<const Unit<OUT>&>(x[i]);
    } else {
      float y[kUnit];
      x[i].get(y);
      z.set(y);
    }
    if (allowed[i] != 0xffu) z.mask(allowed[i]);
    z.store(p.out, to + at);
  }
  // what is outside the eights
  const int head = units > 0 ? lead : n;
  for (int i = tid; i < n - units * kUnit; i += kThreads) {
    const int at = i < head ? i : i + units * kUnit;
    store1<OUT>(p.out, to + at, mask && !(bits_from(v0 + at) & 1u) ? -INFINITY : load1<IN>(p.logits, in + at));
  }
  if (!notes) return;
  // what has a note; within one tensor these logits are still there, or -inf by the mask as they will be
  const float repetition = p.repetition ? __ldg(p.repetition + t) : 1.f, frequency = p.frequency ? __ldg(p.frequency + t) : 0.f;
  const float presence = p.presence ? __ldg(p.presence + t) : 0.f;
  __syncthreads();
  for (int i = tid; i < s_listed; i += kThreads) {
    const int at = s_list[i];
    if (mask && !(bits_from(v0 + at) & 1u)) continue;
    const unsigned note = s_note[at], times = note & kTimes;
    float y = load1<IN>(p.logits, in + at);
    if (note & (kSeen | kTimes)) y = y > 0.f ? __fdiv_rn(y, repetition) : __fmul_rn(y, repetition);
    if (times) y = __fsub_rn(__fsub_rn(y, __fmul_rn(frequency, static_cast<float>(times))), presence);
    if (note >> kBiasShift) y = __fadd_rn(y, __ldg(bias + ((note >> kBiasShift) - 1)));
    store1<OUT>(p.out, to + at, y);
  }
}

template <bool IN, bool OUT>
cudaError_t launch(const AdjustParams& p, int slice, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed;
  const cudaError_t e = allow_smem(q4_adjust_kernel<IN, OUT>, kMostSlice * 6, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.V + slice - 1) / slice), static_cast<unsigned>(p.T));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.history || p.bias_index ? static_cast<size_t>(slice) * 6 : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_adjust_kernel<IN, OUT>, p, slice);
}

}  // namespace

cudaError_t launch_adjust(const AdjustParams& p, int sms, cudaStream_t st) {
  int slice = kMostSlice;
  while (slice > 1024 && static_cast<long long>(p.T) * ((p.V + slice - 1) / slice) < 2LL * sms) slice /= 2;
  if (p.bf16) return p.out_bf16 ? launch<true, true>(p, slice, st) : launch<true, false>(p, slice, st);
  return p.out_bf16 ? launch<false, true>(p, slice, st) : launch<false, false>(p, slice, st);
}

}  // namespace q4
