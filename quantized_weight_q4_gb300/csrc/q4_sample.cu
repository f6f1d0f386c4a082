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
// logits are read once.  Whether a token is kept is a comparison with one cut,
// a z and how many tokens of that z stay (by index).  The cut is found from a
// histogram over z (bins of 1/36 nat, added over the CTAs through distributed
// shared memory) and, of the bins that matter, a list of their z that every
// CTA gathers and searches for itself; a short top-k needs no histogram of the
// row, its list is what a CTA finds above the k-th of its threads' maxima.
// Where the list would be too long (thousands of equal logits) further
// histograms narrow it down.
//
// What bounds it: for few rows the chain of barriers and exchanges between the
// CTAs (one row of 32,000 logits: 8 us greedy, 13 us top-k, 15 us top-k and
// top-p; its bytes need 0.02 us).  For many, the work on each logit whose
// weight counts: 200 rows of 128,007 bf16 logits (51 MB, 7.5 us) take 29 us
// greedy, 54 us without limits, 63 us with top-k, 73 us with top-k and top-p
// and 119 us with top-p alone, which has to weigh every logit; the issue slots
// are 55% full with the mixture that a batch of requests has (79 us).
#include <cfloat>

#include "q4_kernels.h"
#include "q4_kv_device.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kPer = kBins / kThreads;       // bins a thread
constexpr int kUnit = kWarps * 128;          // a CTA's elements are a multiple of this
constexpr float kPerNat = 36.0f;             // coarse bins: 1024 / 36 = 28.4 > 40 ln 2 nats
constexpr int kList = 2048;                  // longest list
constexpr int kListK = 1600;                 // top-k times CTAs up to which the list takes all that may be kept
constexpr int kRowCtas = 8;
constexpr int kSliceBytes = 160 * 1024;      // most elements a CTA holds
typedef unsigned long long u64;

struct alignas(16) Shared {
  unsigned hist[3][kBins];                   // this CTA's: counts, low and high words of the weights
  union {
    unsigned n[kBins];                       // all CTAs'
    unsigned list[kList];                    // this CTA's part of the list (n and w are in registers by then)
  };
  union {
    u64 w[kBins];
    unsigned all[kList];                     // the gathered list
  };
  unsigned list_n;
  unsigned lo, hi;                           // range of codes
  unsigned scan_n[kWarps];
  u64 scan_w[kWarps];
  float top[kRowCtas];
  u64 sums[kRowCtas * kWarps];               // weight before the cut, and tokens at it, of every warp's elements
  unsigned ties[kRowCtas * kWarps];
  float red[kWarps];
  u64 part[kWarps];                       // the same of the pieces of one warp's elements
  unsigned part_ties[kWarps];
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
__device__ __forceinline__ void st_peer_u32(uint32_t a, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_peer_u64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// Code of z that grows as z falls.
__device__ __forceinline__ unsigned falling(float z) {
  const unsigned b = __float_as_uint(z + 0.0f);           // -0 and +0 are equal
  return (b & 0x80000000u) ? b : ~(b | 0x80000000u);
}

// floor(e * 2^40) of 0 <= e <= 1: e's 24 significant bits at the top of a 64-bit word, shifted down.
__device__ __forceinline__ u64 weight(float e) {
  const unsigned b = __float_as_uint(e), m = b << 8 | 0x80000000u, s = 150u - (b >> 23);   // m 2^32 >> s
  unsigned lo, hi;
  asm("shf.r.clamp.b32 %0, %1, %2, %3;" : "=r"(lo) : "r"(0u), "r"(m), "r"(s));             // s >= 32: m
  asm("shr.u32 %0, %1, %2;" : "=r"(lo) : "r"(lo), "r"(max(s, 32u) - 32u));                 // 0 from 64 on
  asm("shr.u32 %0, %1, %2;" : "=r"(hi) : "r"(m), "r"(s));
  return static_cast<u64>(hi) << 32 | lo;
}

// z: a NaN becomes -inf (the maximum drops it), an infinity the largest number.
__device__ __forceinline__ float clean(float l, float inv) {
  return fminf(fmaxf(__fmul_rn(l, inv), -INFINITY), FLT_MAX);
}

// Inclusive sum over the warp's lanes.
template <typename T>
__device__ __forceinline__ T scan_up(T x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// z of a code of falling().
__device__ __forceinline__ float of_code(unsigned c) {
  return __uint_as_float((c & 0x80000000u) ? c : ~c & 0x7fffffffu);
}

// The CTA's elements as they came (fp32 or bf16; -inf where there are none).
template <bool BF16>
struct Row {
  const void* x;
  int base, n;           // this warp's: base + i, i < n (n a multiple of 128)
  float inv;             // 1 / temperature
  float top;             // the row's largest z
  int ctas, rank;

  __device__ __forceinline__ float z(int i) const {
    if (BF16) return clean(bf16_bits_to_f32(static_cast<const uint16_t*>(x)[base + i]), inv);
    return clean(static_cast<const float*>(x)[base + i], inv);
  }
};

// 16 bytes of elements, as they came.
template <bool BF16>
struct Group {
  static constexpr int kN = BF16 ? 8 : 4;
  uint4 w;

  // the largest (a NaN only if there is nothing else)
  __device__ __forceinline__ float largest() const {
    if (BF16) {
      unsigned a, b;
      asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
      asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
      asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
      return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
    }
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
  __device__ __forceinline__ float get(int j) const {
    const unsigned v = (&w.x)[BF16 ? j >> 1 : j];
    return __uint_as_float(!BF16 || (j & 1) ? (BF16 ? v & 0xffff0000u : v) : v << 16);
  }
};

// The warp's elements, 16 bytes a lane at a time: f(z) of those in groups
// whose largest z passes `want`.  z grows with the logit, so one test speaks
// for the group; most groups hold nothing that a pass looks for.  Testing
// every element instead: 200 rows of 128,007 bf16 logits 40 us greedy, 83 us
// with top-k and top-p; so 29 and 73 us.
template <bool BF16, typename W, typename F>
__device__ __forceinline__ void each(const Row<BF16>& r, W want, F f) {
  using G = Group<BF16>;
#pragma unroll 2
  for (int i = G::kN * (threadIdx.x & 31); i < r.n; i += 32 * G::kN) {
    const G g = {*reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(r.x) + (r.base + i) * (BF16 ? 2 : 4))};
    if (want(clean(g.largest(), r.inv))) {
#pragma unroll
      for (int j = 0; j < G::kN; ++j) f(clean(g.get(j), r.inv));
    }
  }
}

constexpr float kZero = 27.75f;   // weights are 0 from 40 ln 2 = 27.73 nats below the largest
__device__ __forceinline__ int coarse(float d) { return static_cast<int>(d * kPerNat); }   // d < kZero: below kBins
__device__ __forceinline__ int fine(float d, int bin) {
  return max(0, min(kBins - 1, static_cast<int>((d * kPerNat - bin) * kBins)));
}

__device__ __forceinline__ void add_bin(Shared& s, int b, u64 w, bool want_n, bool want_w) {
  if (want_n) atomicAdd(&s.hist[0][b], 1u);
  if (want_w) {
    const unsigned lo = static_cast<unsigned>(w), hi = static_cast<unsigned>(w >> 32);
    const unsigned carry = atomicAdd(&s.hist[1][b], lo) > ~lo ? 1u : 0u;
    if (hi + carry) atomicAdd(&s.hist[2][b], hi + carry);
  }
}

__device__ __forceinline__ void clear_bins(Shared& s) {
  uint4* h = reinterpret_cast<uint4*>(&s.hist[0][0]);
  for (int i = threadIdx.x; i < 3 * kBins / 4; i += kThreads) h[i] = make_uint4(0, 0, 0, 0);
}

// A thread's bins: counts and weights, and those of all bins before.
struct Bins {
  unsigned n[kPer], before_n;
  u64 w[kPer], before_w;
};

// The sums before each thread's bins; the block's totals are the sums of s.scan_*.
__device__ __forceinline__ void scan_bins(Shared& s, Bins& b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned n = 0;
  u64 w = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) n += b.n[j], w += b.w[j];
  const unsigned sn = scan_up(n);
  const u64 sw = scan_up(w);
  if (lane == 31) s.scan_n[warp] = sn, s.scan_w[warp] = sw;
  __syncthreads();
  // a lane for each warp
  unsigned pn = lane < warp ? s.scan_n[lane] : 0;
  u64 pw = lane < warp ? s.scan_w[lane] : 0;
  pn = __reduce_add_sync(0xffffffffu, pn);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) pw += __shfl_xor_sync(0xffffffffu, pw, o);
  b.before_n = pn + sn - n;
  b.before_w = pw + sw - w;
}

// The sums of all CTAs' bins in every CTA, after each has filled its own.
template <typename R>
__device__ __forceinline__ void add_up(Shared& s, const R& r, Bins& out) {
  cluster_sync();
  // each CTA adds its share of the bins and hands the sums to all
  const int share = kBins / r.ctas;
  for (int i = threadIdx.x; i < share; i += kThreads) {
    const int b = r.rank * share + i;
    unsigned n = 0;
    u64 w = 0;
    for (int c = 0; c < r.ctas; c += 4) {
      unsigned x[4][3];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < 3; ++q) x[k][q] = c + k < r.ctas ? ld_peer_u32(peer_addr(&s.hist[q][b], c + k)) : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) n += x[k][0], w += x[k][1] + (static_cast<u64>(x[k][2]) << 32);
    }
    for (int c = 0; c < r.ctas; ++c) {
      st_peer_u32(peer_addr(&s.n[b], c), n);
      st_peer_u64(peer_addr(&s.w[b], c), w);
    }
  }
  cluster_sync();
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    out.n[j] = s.n[kPer * threadIdx.x + j], out.w[j] = s.w[kPer * threadIdx.x + j];
  scan_bins(s, out);
}

// Counts and weights of bin_of(z, d) (negative: none) over the elements within
// kZero of the largest, over all CTAs.
template <typename R, typename F>
__device__ __forceinline__ void histogram(Shared& s, const R& r, bool want_n, bool want_w, F bin_of,
                                          Bins& out) {
  clear_bins(s);
  __syncthreads();
  each(r, [&](float z) { return r.top - z < kZero; }, [&](float z) {
    const float d = r.top - z;
    if (!(d < kZero)) return;
    const int b = bin_of(z, d);
    if (b >= 0) add_bin(s, b, want_w ? weight(expf(-d)) : 0, want_n, want_w);
  });
  add_up(s, r, out);
}

// The coarse bins' weights; those further than kNear from the largest together
// in the last bin: most tokens lie there and a cut seldom does, so their
// weights are added in registers instead of in shared memory.
constexpr float kNear = 14.0f;
template <typename R>
__device__ __forceinline__ void near_histogram(Shared& s, const R& r, Bins& out) {
  clear_bins(s);
  __syncthreads();
  u64 rest = 0;
  each(r, [&](float z) { return r.top - z < kZero; }, [&](float z) {
    const float d = r.top - z;
    const u64 w = weight(expf(-d));
    if (d < kNear)
      add_bin(s, coarse(d), w, false, true);
    else
      rest += w;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
  if ((threadIdx.x & 31) == 0) add_bin(s, kBins - 1, rest, false, true);
  add_up(s, r, out);
}

// Counts of this CTA's threads' largest z (theirs: its maximum), in this CTA alone: the k-th largest of those is at
// most the CTA's k-th largest z, and not much below it.
template <typename R>
__device__ __forceinline__ void top_histogram(Shared& s, const R& r, float theirs, Bins& out) {
  clear_bins(s);
  __syncthreads();
  const float d = r.top - theirs;
  if (d < kZero) add_bin(s, coarse(d), 0, true, false);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; ++j) out.n[j] = s.hist[0][kPer * threadIdx.x + j], out.w[j] = 0;
  scan_bins(s, out);
}

// The bin in which the count (or weight) reaches `target` (1 or more, at most
// the total), into s.bin and what stands beside it.
__device__ __forceinline__ void find_bin(Shared& s, const Bins& b, bool by_weight, u64 target) {
  unsigned n = b.before_n;
  u64 w = b.before_w;
  __syncthreads();   // the last search's result has been read
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const u64 at = by_weight ? w : n, to = by_weight ? w + b.w[j] : n + b.n[j];
    if (at < target && target <= to) {
      s.bin = kPer * threadIdx.x + j;
      s.before_n = n, s.bin_n = b.n[j];
      s.before_w = w, s.bin_w = b.w[j];
    }
    n += b.n[j];
    w += b.w[j];
  }
  __syncthreads();
}

// The cut: tokens with a code below `code`, and the first `ties` (by index) with that code.
struct Cut {
  unsigned code, ties;
  u64 weight;              // of all before the cut
};

// Elements of one code have one weight.
__device__ __forceinline__ Cut cut_at(unsigned code, float top, bool by_weight, u64 left, u64 done_w) {
  const u64 w = weight(expf(of_code(code) - top));
  Cut cut;
  cut.code = code;
  cut.ties = static_cast<unsigned>(by_weight ? (left + w - 1) / w : left);
  cut.weight = done_w + cut.ties * w;
  return cut;
}

// The range of the codes that `f` hands out, in s.lo and s.hi.
template <typename F>
__device__ __forceinline__ void code_range(Shared& s, F f) {
  if (threadIdx.x == 0) s.lo = 0xffffffffu, s.hi = 0;
  __syncthreads();
  unsigned lo = 0xffffffffu, hi = 0;
  f([&](unsigned c) { lo = min(lo, c), hi = max(hi, c); });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if ((threadIdx.x & 31) == 0 && lo <= hi) atomicMin(&s.lo, lo), atomicMax(&s.hi, hi);
  __syncthreads();
}

// The cut of the list in s.all at which its count (or weight) reaches target.
// before_w: weight of the tokens that come before the list.
__device__ __forceinline__ Cut cut_of_list(Shared& s, int n, float top, bool by_weight, u64 target, u64 before_w) {
  unsigned code[kList / kThreads];
  u64 w[kList / kThreads];
#pragma unroll
  for (int k = 0; k < kList / kThreads; ++k) {
    const int i = threadIdx.x + k * kThreads;
    code[k] = i < n ? s.all[i] : 0xffffffffu;
    w[k] = i < n ? weight(expf(of_code(code[k]) - top)) : 0;
  }
  code_range(s, [&](auto see) {
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k)
      if (static_cast<int>(threadIdx.x) + k * kThreads < n) see(code[k]);
  });
  unsigned lo = s.lo, hi = s.hi;
  u64 left = target, done_w = before_w;
  while (lo < hi) {
    const int shift = max(0, 32 - __clz(hi - lo) - 10);
    clear_bins(s);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k)
      if (static_cast<int>(threadIdx.x) + k * kThreads < n && code[k] >= lo && code[k] <= hi)
        add_bin(s, static_cast<int>((code[k] - lo) >> shift), w[k], true, true);
    __syncthreads();
    Bins b;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = kPer * threadIdx.x + j;
      b.n[j] = s.hist[0][i];
      b.w[j] = s.hist[1][i] + (static_cast<u64>(s.hist[2][i]) << 32);
    }
    scan_bins(s, b);
    find_bin(s, b, by_weight, left);
    done_w += s.before_w;
    left -= by_weight ? s.before_w : s.before_n;
    const unsigned end = hi;
    lo += static_cast<unsigned>(s.bin) << shift;
    hi = min(end, lo + (1u << shift) - 1u);
    if (s.bin_n == 1 && lo < hi) {   // one token: its code is the cut
      const unsigned l0 = lo, h0 = hi;
      code_range(s, [&](auto see) {
#pragma unroll
        for (int k = 0; k < kList / kThreads; ++k)
          if (static_cast<int>(threadIdx.x) + k * kThreads < n && code[k] >= l0 && code[k] <= h0) see(code[k]);
      });
      lo = hi = s.lo;
    }
  }
  return cut_at(lo, top, by_weight, left, done_w);
}

// The codes of all elements in the coarse bins first .. last into s.all of
// every CTA; returns how many there are, more than kList: too many for the list.
template <typename R>
__device__ __forceinline__ unsigned gather_list(Shared& s, const R& r, int first, int last) {
  if (threadIdx.x == 0) s.list_n = 0;
  __syncthreads();
  const auto reach = [&](float z) { return r.top - z < kZero && coarse(r.top - z) <= last; };
  each(r, reach, [&](float z) {
    if (reach(z) && coarse(r.top - z) >= first) {
      const unsigned at = atomicAdd(&s.list_n, 1u);
      if (at < kList) s.list[at] = falling(z);
    }
  });
  cluster_sync();
  // each warp reads every part's length, and copies from the CTAs that fall to it
  const int lane = threadIdx.x & 31;
  const unsigned mine = lane < r.ctas ? ld_peer_u32(peer_addr(&s.list_n, lane)) : 0;
  unsigned up = mine;
#pragma unroll
  for (int o = 1; o < kRowCtas; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  const unsigned n = __shfl_sync(0xffffffffu, up, r.ctas - 1);
  if (n <= kList) {
    const int warp = threadIdx.x >> 5, c = warp % r.ctas, share = kWarps / r.ctas;   // share: warps a part
    const unsigned here = __shfl_sync(0xffffffffu, mine, c), at = __shfl_sync(0xffffffffu, up, c) - here;
    for (unsigned i = (warp / r.ctas) * 32 + lane; i < here; i += 32 * share)
      s.all[at + i] = ld_peer_u32(peer_addr(&s.list[i], c));
  }
  __syncthreads();
  return n;
}

// The cut inside coarse bin b1, whose list would be too long: `left` of the
// count (or weight) is to be reached in it.  Finer bins, then bins of the code.
template <typename R>
__device__ __noinline__ Cut cut_by_bins(Shared& s, const R& r, int b1, bool by_weight, u64 left, u64 done_w) {
  Bins bins;
  histogram(s, r, true, true, [&](float z, float d) { return coarse(d) == b1 ? fine(d, b1) : -1; }, bins);
  find_bin(s, bins, by_weight, left);
  const int b2 = s.bin;
  done_w += s.before_w;
  left -= by_weight ? s.before_w : s.before_n;
  code_range(s, [&](auto see) {
    each(r, [&](float z) { return r.top - z < kZero; }, [&](float z) {
      const float d = r.top - z;
      if (d < kZero && coarse(d) == b1 && fine(d, b1) == b2) see(falling(z));
    });
  });
  cluster_sync();
  unsigned lo = 0xffffffffu, hi = 0;
  for (int c = 0; c < r.ctas; ++c) {
    lo = min(lo, ld_peer_u32(peer_addr(&s.lo, c)));
    hi = max(hi, ld_peer_u32(peer_addr(&s.hi, c)));
  }
  while (lo < hi) {
    const int shift = max(0, 32 - __clz(hi - lo) - 10);
    const unsigned l0 = lo, h0 = hi;
    histogram(s, r, true, true, [&](float z, float d) {
      const unsigned c = falling(z);
      return c >= l0 && c <= h0 && coarse(d) == b1 && fine(d, b1) == b2 ? static_cast<int>((c - l0) >> shift) : -1;
    }, bins);
    find_bin(s, bins, by_weight, left);
    done_w += s.before_w;
    left -= by_weight ? s.before_w : s.before_n;
    lo = l0 + (static_cast<unsigned>(s.bin) << shift);
    hi = min(h0, lo + (1u << shift) - 1u);
  }
  cluster_sync();   // peers have read s.lo and s.hi
  return cut_at(lo, r.top, by_weight, left, done_w);
}

// The cut in coarse bin s.bin (just found).
template <typename R>
__device__ __forceinline__ Cut cut_in_bin(Shared& s, const R& r, bool by_weight, u64 target) {
  const int b = s.bin;
  const u64 done_w = s.before_w, left = target - (by_weight ? s.before_w : s.before_n);
  const unsigned n = gather_list(s, r, b, b);
  if (n <= kList) return cut_of_list(s, static_cast<int>(n), r.top, by_weight, left, done_w);
  return cut_by_bins(s, r, b, by_weight, left, done_w);
}

// The weight that top-p asks for, of `all` (at least 1).
__device__ __forceinline__ u64 part_of(float top_p, u64 all) {
  const double want = ceil(static_cast<double>(top_p) * static_cast<double>(all));
  return want >= 1.0 ? static_cast<u64>(want) : 1ull;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) q4_sample_kernel(const __grid_constant__ SampleParams p, int ctas,
                                                             int slice) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  uint8_t* xs = smem + sizeof(Shared);
  cluster_started();         // waited for before the first store to a peer
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
  Row<BF16> r;
  r.x = xs;
  r.n = slice / kWarps;
  r.base = warp * r.n;
  r.inv = inv;
  r.ctas = ctas, r.rank = rank;
  // asynchronous copies, so that all of a thread's are on their way together; the row's edges by element
#pragma unroll 4
  for (int i = lane * kVec; i < r.n; i += 32 * kVec) {
    const int v = v0 + r.base + i;
    uint8_t* to = xs + static_cast<size_t>(r.base + i) * kSize;
    if (v >= head && v + kVec <= head + p.V) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)),
                   "l"(base + static_cast<long long>(v) * kSize)
                   : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const bool in = v + j >= head && v + j < head + p.V;
        const uint8_t* a = base + static_cast<long long>(v + j) * kSize;
        if (BF16)
          reinterpret_cast<uint16_t*>(to)[j] = in ? *reinterpret_cast<const uint16_t*>(a) : 0xff80;   // -inf
        else
          reinterpret_cast<uint32_t*>(to)[j] = in ? *reinterpret_cast<const uint32_t*>(a) : 0xff800000u;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();   // a warp reads its own elements only
  if (inv == 0.f) {   // an infinite temperature: z of +inf is a NaN, below those beside it; as -inf it is passed over alike
    for (int i = r.base + lane; i < r.base + r.n; i += 32) {
      if (BF16) {
        uint16_t& x = reinterpret_cast<uint16_t*>(xs)[i];
        if (x == 0x7f80) x = 0xff80;
      } else {
        uint32_t& x = reinterpret_cast<uint32_t*>(xs)[i];
        if (x == 0x7f800000u) x = 0xff800000u;
      }
    }
    __syncwarp();
  }
  float top = -INFINITY;
  each(r, [&](float z) { top = fmaxf(top, z); return false; }, [](float) {});
  const float theirs = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s.red[warp] = top;
  __syncthreads();
  cluster_wait_started();
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
  cut.code = 0;
  cut.ties = 0;              // no cut: everything is kept
  const bool by_k = k > 0 && k < p.V, by_p = top_p < 1.0f;
  if (k == 1) {
    cut.code = falling(top);
    cut.ties = 1;
  } else if (by_k || by_p) {
    Bins bins;
    bool done = false;
    if (by_k && k * ctas <= kListK) {
      // a short top-k: every token that may be kept goes on the list.  The row's first k are among the CTAs' first
      // k, so each CTA finds for itself how far down it has to look
      top_histogram(s, r, theirs, bins);
      unsigned tops = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) tops += s.scan_n[i];
      int last = kBins;                     // fewer threads than k have an element: all elements
      if (tops >= static_cast<unsigned>(k)) {
        find_bin(s, bins, false, static_cast<u64>(k));
        last = s.bin;
      }
      const int n = static_cast<int>(gather_list(s, r, 0, last));
      if (n <= kList) {
        cut = cut_of_list(s, n, r.top, false, static_cast<u64>(min(k, n)), 0);
        if (by_p) {
          const u64 part = part_of(top_p, cut.weight);
          if (part < cut.weight) cut = cut_of_list(s, n, r.top, true, part, 0);
        }
        done = true;
      }
    }
    if (!done) {
      // by the bins of all elements; a top-k needs their counts, a top-p their weights
      const auto bin_of = [&](float, float d) { return coarse(d); };
      if (by_k) histogram(s, r, true, by_p, bin_of, bins);
      else near_histogram(s, r, bins);
      unsigned all_n = 0;
      u64 all_w = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) all_n += s.scan_n[i], all_w += s.scan_w[i];
      const bool cut_k = by_k && static_cast<unsigned>(k) < all_n;
      if (cut_k) {
        find_bin(s, bins, false, static_cast<u64>(k));
        cut = cut_in_bin(s, r, false, static_cast<u64>(k));
        all_w = cut.weight;
      }
      if (by_p) {
        const u64 part = part_of(top_p, all_w);
        if (part < all_w) {
          if (cut_k) cluster_sync();   // peers have read this CTA's part of the last list
          find_bin(s, bins, true, part);
          if (!by_k && s.bin == kBins - 1) {   // a flat row: its cut lies among the far ones
            histogram(s, r, false, true, bin_of, bins);
            find_bin(s, bins, true, part);
          }
          cut = cut_in_bin(s, r, true, part);
        }
      }
    }
  }

  // kept weight of each warp's elements before the cut, and tokens at it
  const bool has_cut = cut.ties > 0;
  const float cut_z = has_cut ? of_code(cut.code) : -INFINITY;
  // below `low` a weight is 0 or, by min-p, not kept (the slack is far above the rounding of logf and expf)
  const float low = r.top - fminf(kZero, min_p > 0.f ? 0.001f - 1.001f * logf(min_p) : kZero);
  u64 sum = 0;
  unsigned same = 0;
  each(r, [&](float z) { return z >= cut_z && z >= low; }, [&](float z) {
    if (z > cut_z) {
      const float e = expf(z - r.top);
      if (e >= min_p) sum += weight(e);
    } else {
      same += z == cut_z;
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  same = __reduce_add_sync(0xffffffffu, same);
  // to every CTA: none reads another's shared memory after this, so that each may leave when it is done
  if (lane < ctas) {
    st_peer_u64(peer_addr(&s.sums[rank * kWarps + warp], lane), sum);
    st_peer_u32(peer_addr(&s.ties[rank * kWarps + warp], lane), same);
  }
  cluster_sync();
  // every warp: the weight before its own elements, and all of it
  const float tie_e = expf(cut_z - r.top);
  const u64 tie_w = has_cut && tie_e >= min_p ? weight(tie_e) : 0;
  // weight of warp i's kept tokens, i = 32 q + lane, and of all before; tokens at the cut before it
  constexpr int kQ = kRowCtas * kWarps / 32;
  u64 x[kQ], upto[kQ], all = 0;
  unsigned at[kQ], ties = 0;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int i = 32 * q + lane;
    const bool have = i < ctas * kWarps;
    x[q] = have ? s.sums[i] : 0;
    at[q] = have ? s.ties[i] : 0;
  }
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    if (32 * q >= ctas * kWarps) break;
    const unsigned t = at[q];
    at[q] = ties + scan_up(t) - t;
    ties = __shfl_sync(0xffffffffu, at[q] + t, 31);
    x[q] += tie_w * (at[q] < cut.ties ? min(t, cut.ties - at[q]) : 0u);
    upto[q] = all + scan_up(x[q]);
    all = __shfl_sync(0xffffffffu, upto[q], 31);
  }
  const double want = static_cast<double>(p.u[row]) * static_cast<double>(all);
  u64 at_w = want > 0.0 ? static_cast<u64>(want) : 0ull;
  if (all > 0 && at_w >= all) at_w = all - 1;
  // the warp whose elements hold it, the weight and the tokens at the cut before them
  int owner = -1;
  u64 done = 0;
  unsigned before = 0;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    if (32 * q >= ctas * kWarps) break;
    const unsigned over = __ballot_sync(0xffffffffu, upto[q] > at_w);
    if (owner < 0 && over) {
      const int l = __ffs(over) - 1;
      owner = 32 * q + l;
      done = __shfl_sync(0xffffffffu, upto[q] - x[q], l);
      before = __shfl_sync(0xffffffffu, at[q], l);
    }
  }
  if (owner >= 0 && owner / kWarps == rank) {
    // that CTA's warps take a piece of those elements each
    r.base = (owner % kWarps) * r.n;
    const int piece = r.n / kWarps, from = warp * piece;   // a multiple of 4
    u64 sum = 0;
    unsigned same = 0;
    for (int i = from + lane; i < from + piece; i += 32) {
      const float z = r.z(i), e = expf(z - r.top);
      same += z == cut_z;
      if (z > cut_z && e >= min_p) sum += weight(e);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    same = __reduce_add_sync(0xffffffffu, same);
    if (lane == 0) s.part[warp] = sum, s.part_ties[warp] = same;
    __syncthreads();
    const unsigned t = lane < kWarps ? s.part_ties[lane] : 0;
    unsigned at1 = before + scan_up(t) - t;
    const u64 w1 = (lane < kWarps ? s.part[lane] : 0) + tie_w * (at1 < cut.ties ? min(t, cut.ties - at1) : 0u);
    const u64 up1 = done + scan_up(w1);
    const int l = __ffs(__ballot_sync(0xffffffffu, up1 > at_w)) - 1;
    if (l == warp) {
      done = __shfl_sync(0xffffffffu, up1 - w1, l);
      before = __shfl_sync(0xffffffffu, at1, l);
      for (int i0 = from; i0 < from + piece; i0 += 32) {
        const int i = i0 + lane;
        const float z = i < from + piece ? r.z(i) : -INFINITY, e = expf(z - r.top);
        const unsigned tied = __ballot_sync(0xffffffffu, z == cut_z);
        const bool ok = z > cut_z || (z == cut_z && before + __popc(tied & ((1u << lane) - 1u)) < cut.ties);
        before += __popc(tied);
        const u64 w = ok && e >= min_p ? weight(e) : 0;
        const u64 up = done + scan_up(w);
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
  }
}

// CTAs of a row: up to four while each has 4096 elements or more, and eight where four would leave room for
// only one CTA an SM (80 KB of elements each).  Measured with 512 threads each, top-k and top-p on: 200 rows of
// 128,007 bf16 logits 73 us with two, 75 us with four, 133 us with eight (clusters of eight seldom fit the SMs
// that are free), with top-p alone 146 / 123 / 162 us; one row of 32,000 logits 20 / 16.5 / 15.3 / 15.5 us with
// one / two / four / eight; 64 rows of 32,000 20 / 21 / 20 / 37 us.  128,007 fp32 logits, four and eight: one
// row 16 and 14 us, 200 rows 113 and 130 us, with top-p alone 171 and 164 us.
int ctas_of(const SampleParams& p) {
  const int size = p.bf16 ? 2 : 4;
  int c = 1;
  while (c < 4 && p.V > 4096 * c) c *= 2;
  while (c < kRowCtas && static_cast<long long>(p.V) * size > 80 * 1024 * c) c *= 2;
  return c;
}

template <bool BF16>
cudaError_t launch(const SampleParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> allowed;
  cudaError_t e = allow_smem(q4_sample_kernel<BF16>, sizeof(Shared) + kSliceBytes, allowed);
  if (e != cudaSuccess) return e;
  const int ctas = ctas_of(p), slice = ((p.V + 7 + ctas - 1) / ctas + kUnit - 1) / kUnit * kUnit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.T) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared) + static_cast<size_t>(slice) * (BF16 ? 2 : 4);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, q4_sample_kernel<BF16>, p, ctas, slice);
}

}  // namespace

int sample_max_vocab() { return kRowCtas * (kSliceBytes / 4 / kUnit * kUnit) - 8; }

cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  return p.bf16 ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace q4
