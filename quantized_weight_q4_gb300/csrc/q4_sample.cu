// Sampling one token a row from logits (sm_103a).
//
// A row's definition, with l its logits, t, k, p, m its settings and u its
// uniform number:
//   z = l * (1 / t)               (t < 1e-5: z = l and k = 1; NaN counts as -inf)
//   w = floor(exp(z - max z) * 2^40)
//   ranking: z descending, equal z by index
//   kept: the first k of the ranking (k <= 0: all), of those the shortest
//         prefix whose weight reaches p * (their weight) (p >= 1: all), of
//         those the ones with exp(z - max z) >= m; the first is always kept
//   token: the first index whose kept weight, summed in index order, exceeds
//         floor(u * (all kept weight))
// Weights are whole numbers, so that no sum depends on its order.
//
// One thread-block cluster takes one row and keeps it in shared memory: the
// logits are read once.  Whether a token is kept is a comparison with one
// (z, index) cut.  The cut is found by histograms over z, coarse bins of
// 1/36 nat first, then 1/1024 of the cut's bin, then (where the cut's bin
// still holds different z) bins of the fp32 code itself; every CTA adds its
// peers' bins through distributed shared memory and scans them for itself.
#include <cfloat>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2 * kThreads;
constexpr float kPerNat = 36.0f;             // coarse bins: 1024 / 36 = 28.4 > 40 ln 2 nats
constexpr int kUnit = kWarps * 256;          // a CTA's elements are a multiple of this
constexpr int kRowCtas = 8;
constexpr int kMaxSlice = 40960;             // 160 KB of shared memory
typedef unsigned long long u64;

struct alignas(16) Shared {
  unsigned hist[2][4][kBins];                // counts and three 14-bit pieces of the weights, two turns
  float top[kRowCtas];
  u64 sums[kWarps];
  unsigned ties[kWarps];
  unsigned lo, hi;                           // range of the cut bin's codes in this CTA
  u64 scan_w[kWarps];
  unsigned scan_n[kWarps];
  float red[kWarps];
  // the bin that a search found
  int bin;
  unsigned bin_n, before_n;
  u64 bin_w, before_w;
};

static_assert(sizeof(Shared) % 16 == 0, "the elements after it are stored 16 bytes at a time");

__device__ __forceinline__ unsigned ld_peer_u32(uint32_t a) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ u64 ld_peer_u64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// Code of z that grows as z falls.
__device__ __forceinline__ unsigned falling(float z) {
  const unsigned b = __float_as_uint(z + 0.0f);           // -0 and +0 are equal
  return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}

// floor(e * 2^40) of 0 <= e <= 1.
__device__ __forceinline__ u64 weight(float e) {
  const unsigned b = __float_as_uint(e);
  const int down = 127 - static_cast<int>(b >> 23);       // e = 1.m * 2^-down
  if (down > 40) return 0;
  return (static_cast<u64>((b & 0x7fffffu) | 0x800000u) << 17) >> down;
}

__device__ __forceinline__ float clean(float l, float inv) {
  const float z = __fmul_rn(l, inv);
  return z != z ? -INFINITY : fminf(z, FLT_MAX);
}

struct Row {
  const float* z;        // this CTA's elements
  int base, n;           // this warp's: base + i, i < n (n a multiple of 32)
  float top;             // the row's largest z
};

__device__ __forceinline__ int coarse(float d) { return min(kBins - 1, static_cast<int>(d * kPerNat)); }
__device__ __forceinline__ int fine(float d, int bin) {
  return max(0, min(kBins - 1, static_cast<int>((d * kPerNat - bin) * kBins)));
}

// Two bins a thread: counts and weights of all CTAs, and those of the bins before.
struct Bins {
  unsigned n[2], before_n;
  u64 w[2], before_w;
};

// Adds bin_of(z) (negative: none) of every element into histogram `turn`, then
// all CTAs' histograms together.
template <typename F>
__device__ __forceinline__ void histogram(Shared& s, int turn, int ctas, const Row& r, F bin_of, Bins& out) {
  unsigned(*h)[kBins] = s.hist[turn];
  for (int i = threadIdx.x; i < 4 * kBins; i += kThreads) (&h[0][0])[i] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int i = lane; i < r.n; i += 32) {
    const float z = r.z[r.base + i];
    const u64 w = weight(expf(z - r.top));
    if (w == 0) continue;
    const int b = bin_of(z);
    if (b < 0) continue;
    atomicAdd(&h[0][b], 1u);
    atomicAdd(&h[1][b], static_cast<unsigned>(w) & 0x3fffu);
    atomicAdd(&h[2][b], static_cast<unsigned>(w >> 14) & 0x3fffu);
    atomicAdd(&h[3][b], static_cast<unsigned>(w >> 28));
  }
  cluster_sync();
  const int b0 = 2 * threadIdx.x;
  out.n[0] = out.n[1] = 0;
  out.w[0] = out.w[1] = 0;
  for (int c = 0; c < ctas; ++c) {
    const uint32_t a = peer_addr(&h[0][b0], c);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u64 two = ld_peer_u64(a + q * kBins * 4);
      const u64 x0 = two & 0xffffffffull, x1 = two >> 32;
      if (q == 0) {
        out.n[0] += static_cast<unsigned>(x0), out.n[1] += static_cast<unsigned>(x1);
      } else {
        out.w[0] += x0 << (14 * (q - 1)), out.w[1] += x1 << (14 * (q - 1));
      }
    }
  }
  // exclusive scan over the threads' pairs
  unsigned n = out.n[0] + out.n[1];
  u64 w = out.w[0] + out.w[1];
  unsigned sn = n;
  u64 sw = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned un = __shfl_up_sync(0xffffffffu, sn, o);
    const u64 uw = __shfl_up_sync(0xffffffffu, sw, o);
    if (lane >= o) sn += un, sw += uw;
  }
  const int warp = threadIdx.x >> 5;
  if (lane == 31) s.scan_n[warp] = sn, s.scan_w[warp] = sw;
  __syncthreads();
  unsigned pn = 0;
  u64 pw = 0;
  for (int i = 0; i < warp; ++i) pn += s.scan_n[i], pw += s.scan_w[i];
  out.before_n = pn + sn - n;
  out.before_w = pw + sw - w;
}

// The bin in which the count (or weight) reaches `target` (1 or more, at most
// the total), into s.bin and what stands beside it.
__device__ __forceinline__ void find_bin(Shared& s, const Bins& b, bool by_weight, u64 target) {
  unsigned n = b.before_n;
  u64 w = b.before_w;
  __syncthreads();   // the last search's result has been read
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const u64 at = by_weight ? w : n, to = by_weight ? w + b.w[j] : n + b.n[j];
    if (at < target && target <= to) {
      s.bin = 2 * threadIdx.x + j;
      s.before_n = n, s.bin_n = b.n[j];
      s.before_w = w, s.bin_w = b.w[j];
    }
    n += b.n[j];
    w += b.w[j];
  }
  __syncthreads();
}

// The cut: z with code below `code`, and the first `ties` (by index) with that code.
struct Cut {
  unsigned code, ties;
  u64 weight;              // of all before the cut
};

// Finds the cut at which the count (or the weight) reaches target, given the
// coarse histogram.  `turn` alternates the histograms' buffers.
__device__ __forceinline__ Cut find_cut(Shared& s, int& turn, int ctas, const Row& r, const Bins& first,
                                        bool by_weight, u64 target) {
  find_bin(s, first, by_weight, target);
  const int b1 = s.bin;
  u64 done_w = s.before_w;
  u64 left = target - (by_weight ? s.before_w : s.before_n);
  Bins bins;
  histogram(s, turn, ctas, r, [&](float z) {
    const float d = r.top - z;
    return coarse(d) == b1 ? fine(d, b1) : -1;
  }, bins);
  turn ^= 1;
  find_bin(s, bins, by_weight, left);
  const int b2 = s.bin;
  done_w += s.before_w;
  left -= by_weight ? s.before_w : s.before_n;
  // range of codes in that bin
  if (threadIdx.x == 0) s.lo = 0xffffffffu, s.hi = 0;
  __syncthreads();
  unsigned lo = 0xffffffffu, hi = 0;
  for (int i = threadIdx.x & 31; i < r.n; i += 32) {
    const float z = r.z[r.base + i], d = r.top - z;
    if (d < 32.f && coarse(d) == b1 && fine(d, b1) == b2) {
      const unsigned c = falling(z);
      lo = min(lo, c), hi = max(hi, c);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if ((threadIdx.x & 31) == 0 && lo <= hi) atomicMin(&s.lo, lo), atomicMax(&s.hi, hi);
  cluster_sync();
  lo = 0xffffffffu, hi = 0;
  for (int c = 0; c < ctas; ++c) {
    lo = min(lo, ld_peer_u32(peer_addr(&s.lo, c)));
    hi = max(hi, ld_peer_u32(peer_addr(&s.hi, c)));
  }
  // bins of the code itself until one code is left
  while (lo < hi) {
    const int shift = max(0, 32 - __clz(hi - lo) - 10);
    const unsigned l0 = lo, h0 = hi;
    histogram(s, turn, ctas, r, [&](float z) {
      const unsigned c = falling(z);
      if (c < l0 || c > h0) return -1;
      const float d = r.top - z;
      return coarse(d) == b1 && fine(d, b1) == b2 ? static_cast<int>((c - l0) >> shift) : -1;
    }, bins);
    turn ^= 1;
    find_bin(s, bins, by_weight, left);
    done_w += s.before_w;
    left -= by_weight ? s.before_w : s.before_n;
    lo = l0 + (static_cast<unsigned>(s.bin) << shift);
    hi = min(h0, lo + (1u << shift) - 1u);
  }
  // elements of one code have one weight
  const unsigned bits = (lo & 0x80000000u) ? lo : ~lo & 0x7fffffffu;
  const u64 w = weight(expf(__uint_as_float(bits) - r.top));
  Cut cut;
  cut.code = lo;
  cut.ties = static_cast<unsigned>(by_weight ? (left + w - 1) / w : left);
  cut.weight = done_w + cut.ties * w;
  return cut;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) q4_sample_kernel(const __grid_constant__ SampleParams p, int ctas,
                                                             int slice) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  float* zs = reinterpret_cast<float*>(smem + sizeof(Shared));
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x / ctas, rank = static_cast<int>(cluster_ctarank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  float t = p.temperature ? p.temperature[row] : 1.0f;
  const bool greedy = !(t >= 1e-5f);
  const float inv = greedy ? 1.0f : __fdiv_rn(1.0f, t);
  const int k = greedy ? 1 : p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.0f;
  const float min_p = p.min_p ? fminf(p.min_p[row], 1.0f) : 0.0f;   // the largest z stays

  // the CTA's elements: virtual index v = index + head, so that v = 0 is 16-byte aligned
  constexpr int kVec = BF16 ? 8 : 4, kSize = BF16 ? 2 : 4;
  const uint8_t* base = static_cast<const uint8_t*>(p.logits) + static_cast<long long>(row) * p.stride * kSize;
  const int head = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / kSize);
  base -= head * kSize;
  const int v0 = rank * slice;
  Row r;
  r.z = zs;
  r.n = slice / kWarps;
  r.base = warp * r.n;
  float top = -INFINITY;
#pragma unroll 4
  for (int i = lane * kVec; i < r.n; i += 32 * kVec) {
    const int v = v0 + r.base + i;
    float x[kVec];
    if (v >= head && v + kVec <= head + p.V) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(base + static_cast<long long>(v) * kSize));
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        x[j] = clean(BF16 ? __uint_as_float((j & 1) ? q[j / 2] & 0xffff0000u : q[j / 2] << 16) : __uint_as_float(q[j & 3]), inv);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        x[j] = -INFINITY;
        if (v + j >= head && v + j < head + p.V) {
          const uint8_t* a = base + static_cast<long long>(v + j) * kSize;
          x[j] = clean(BF16 ? bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(a)) : *reinterpret_cast<const float*>(a), inv);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kVec; j += 4) {
      *reinterpret_cast<float4*>(zs + r.base + i + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
      top = fmaxf(top, fmaxf(fmaxf(x[j], x[j + 1]), fmaxf(x[j + 2], x[j + 3])));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s.red[warp] = top;
  __syncthreads();
  if (tid < ctas) {
    float m = s.red[0];
    for (int i = 1; i < kWarps; ++i) m = fmaxf(m, s.red[i]);
    st_peer(peer_addr(&s.top[rank], tid), m);
  }
  cluster_sync();
  top = s.top[0];
  for (int i = 1; i < ctas; ++i) top = fmaxf(top, s.top[i]);
  r.top = top;
  if (top == -INFINITY) {   // nothing to choose from
    if (rank == 0 && tid == 0) {
      p.tokens[row] = -1;
      if (p.probs) p.probs[row] = 0.f;
    }
    return;   // every CTA of the cluster, and none reads a peer after this
  }

  Cut cut;
  cut.code = 0xffffffffu;    // everything
  cut.ties = 0xffffffffu;
  cut.weight = 0;
  const bool by_k = k > 0 && k < p.V, by_p = top_p < 1.0f;
  if (by_k || by_p) {
    Bins first;
    int turn = 0;
    histogram(s, turn, ctas, r, [&](float z) { return coarse(r.top - z); }, first);
    turn ^= 1;
    unsigned all_n = 0;
    u64 all_w = 0;
    for (int i = 0; i < kWarps; ++i) all_n += s.scan_n[i], all_w += s.scan_w[i];
    __syncthreads();
    if (by_k && static_cast<unsigned>(k) < all_n) {
      cut = find_cut(s, turn, ctas, r, first, false, static_cast<u64>(k));
      all_w = cut.weight;
    }
    if (by_p) {
      const double want = ceil(static_cast<double>(top_p) * static_cast<double>(all_w));
      const u64 target = want >= 1.0 ? static_cast<u64>(want) : 1ull;
      if (target < all_w) cut = find_cut(s, turn, ctas, r, first, true, target);
    }
  }

  // how many tokens with the cut's code come before each warp's
  unsigned before = 0;
  if (cut.ties != 0xffffffffu) {
    unsigned n = 0;
    for (int i = lane; i < r.n; i += 32) n += falling(zs[r.base + i]) == cut.code;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s.ties[warp] = n;
    cluster_sync();
    unsigned c = 0;
    for (int i = lane; i < rank * kWarps + warp; i += 32) c += ld_peer_u32(peer_addr(&s.ties[i % kWarps], i / kWarps));
    before = __reduce_add_sync(0xffffffffu, c);
  }
  // kept weight of element i of this warp's; `at`: tokens with the cut's code so far
  auto kept = [&](int i, unsigned& at) -> u64 {
    const float z = zs[r.base + i];
    const unsigned c = falling(z);
    bool ok = c < cut.code;
    if (cut.ties == 0xffffffffu) {
      ok = true;
    } else {
      const unsigned same = __ballot_sync(0xffffffffu, c == cut.code);
      ok = ok || (c == cut.code && at + __popc(same & ((1u << lane) - 1u)) < cut.ties);
      at += __popc(same);
    }
    const float e = expf(z - r.top);
    return ok && e >= min_p ? weight(e) : 0;
  };
  u64 sum = 0;
  {
    unsigned at = before;
    for (int i = lane; i < r.n; i += 32) sum += kept(i, at);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s.sums[warp] = sum;
  cluster_sync();
  // every warp: the weight before its own elements, and all of it
  u64 mine = 0, all = 0;
  for (int i = lane; i < ctas * kWarps; i += 32) {
    const u64 x = ld_peer_u64(peer_addr(&s.sums[i % kWarps], i / kWarps));
    all += x;
    if (i < rank * kWarps + warp) mine += x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    mine += __shfl_xor_sync(0xffffffffu, mine, o);
  }
  const double want = static_cast<double>(p.u[row]) * static_cast<double>(all);
  u64 at_w = want > 0.0 ? static_cast<u64>(want) : 0ull;
  if (all > 0 && at_w >= all) at_w = all - 1;
  if (at_w >= mine && at_w < mine + sum) {
    unsigned at = before;
    u64 done = mine;
    for (int i = lane; i < r.n; i += 32) {
      const u64 w = kept(i, at);
      u64 up = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += x;
      }
      up += done;
      const unsigned over = __ballot_sync(0xffffffffu, up > at_w);
      if (over) {
        if (lane == __ffs(over) - 1) {
          p.tokens[row] = v0 + r.base + i - head;
          if (p.probs) p.probs[row] = __fdiv_rn(__ull2float_rn(w), __ull2float_rn(all));
        }
        break;
      }
      done = __shfl_sync(0xffffffffu, up, 31);
    }
  }
  cluster_sync();   // peers may still read this CTA's sums
}

int cluster_of(int V) {
  // a cluster reads its row faster the more CTAs share it, and pays for each exchange
  int c = 1;
  while (c < kRowCtas && V > 4096 * c) c *= 2;
  return c;
}

}  // namespace

int sample_max_vocab() { return kRowCtas * kMaxSlice - 8; }

cudaError_t launch_sample(const SampleParams& p, int sms, cudaStream_t st) {
  (void)sms;
  const int ctas = cluster_of(p.V);
  const int slice = ((p.V + 7 + ctas - 1) / ctas + kUnit - 1) / kUnit * kUnit;
  const size_t smem = sizeof(Shared) + static_cast<size_t>(slice) * 4;
  auto kernel = p.bf16 ? q4_sample_kernel<true> : q4_sample_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.T) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p, ctas, slice);
}

}  // namespace q4
