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
// their order does not matter.
#include <algorithm>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 256;
constexpr int kMostSlice = 16384;         // logits of a CTA
constexpr unsigned kSeen = 1u << 19;      // a note: bits 0-18 how often, bit 19 in the prompt, bits 20-31 bias entry + 1
constexpr unsigned kTimes = kSeen - 1;
constexpr int kBiasShift = 20;

struct Row {
  bool notes, penalties;
  const float* bias;                      // of the row, or null
  const uint32_t* mask;                   // or null
  float repetition, frequency, presence;
};

__device__ __forceinline__ float adjust(float x, const Row& r, unsigned note, int v) {
  if (r.penalties) {
    const unsigned n = note & kTimes;
    if (note & (kSeen | kTimes)) x = x > 0.f ? __fdiv_rn(x, r.repetition) : __fmul_rn(x, r.repetition);
    if (n) x = __fsub_rn(__fsub_rn(x, __fmul_rn(r.frequency, static_cast<float>(n))), r.presence);
  }
  if (note >> kBiasShift) x = __fadd_rn(x, __ldg(r.bias + ((note >> kBiasShift) - 1)));
  if (r.mask && !(__ldg(r.mask + (v >> 5)) >> (v & 31) & 1u)) x = -INFINITY;
  return x;
}

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

// IN, OUT: bf16 or fp32.  slice: logits of a CTA.
template <bool IN, bool OUT>
__global__ void __launch_bounds__(kThreads) q4_adjust_kernel(const __grid_constant__ AdjustParams p, int slice) {
  extern __shared__ unsigned s_note[];    // [slice]
  const int tid = threadIdx.x, t = blockIdx.y;
  const int v0 = blockIdx.x * slice, n = min(slice, p.V - v0);
  pdl_launch_dependents();
  pdl_wait();
  const long long in = t * p.stride + v0, to = t * p.out_stride + v0;
  Row r = {};
  const int req = p.request ? __ldg(p.request + t) : t;
  const bool known = req >= 0 && req < p.requests;
  if (p.request && req >= p.requests && (p.history || p.bias_index) && blockIdx.x == 0 && tid == 0) atomicOr(p.err, kDevErrIndex);
  if (p.mask) {
    const int row = p.mask_row ? __ldg(p.mask_row + t) : t;
    if (row >= p.masks) {
      if (blockIdx.x == 0 && tid == 0) atomicOr(p.err, kDevErrIndex);
    } else if (row >= 0) {
      r.mask = reinterpret_cast<const uint32_t*>(p.mask) + row * ((p.V + 31LL) / 32);
    }
  }
  r.penalties = p.history && known;
  r.repetition = p.repetition ? __ldg(p.repetition + t) : 1.f;
  r.frequency = p.frequency ? __ldg(p.frequency + t) : 0.f;
  r.presence = p.presence ? __ldg(p.presence + t) : 0.f;
  const bool biased = p.bias_index && known;
  r.bias = biased ? p.bias + static_cast<long long>(req) * p.bias_width : nullptr;
  r.notes = r.penalties || biased;
  if (r.notes) {
    for (int i = tid; i < n; i += kThreads) s_note[i] = 0;
    __syncthreads();
    if (biased) {
      const int32_t* index = p.bias_index + static_cast<long long>(req) * p.bias_width;
      for (int i = tid; i < p.bias_width; i += kThreads) {
        const int at = __ldg(index + i) - v0;
        if (at >= 0 && at < n) atomicMax(s_note + at, static_cast<unsigned>(i + 1) << kBiasShift);
      }
      __syncthreads();
    }
    if (r.penalties) {
      const int32_t* history = p.history + static_cast<long long>(req) * p.history_width;
      const int len = min(__ldg(p.history_len + t), p.history_width), prompt = p.prompt_len ? __ldg(p.prompt_len + t) : 0;
      for (int i = tid; i < len; i += kThreads) {
        const int at = __ldg(history + i) - v0;
        if (at >= 0 && at < n) {
          if (i < prompt)
            atomicOr(s_note + at, kSeen);
          else
            atomicAdd(s_note + at, 1u);
        }
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < n; i += kThreads)
    store1<OUT>(p.out, to + i, adjust(load1<IN>(p.logits, in + i), r, r.notes ? s_note[i] : 0u, v0 + i));
}

template <bool IN, bool OUT>
cudaError_t launch(const AdjustParams& p, int slice, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(q4_adjust_kernel<IN, OUT>, kMostSlice * 4, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.V + slice - 1) / slice), static_cast<unsigned>(p.T));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(slice) * 4;
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
