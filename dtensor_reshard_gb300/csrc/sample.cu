// sample.cu -- reshard_sample: one token a row of logits, with temperature, top-k,
// top-p and min-p, from one given uniform number a row.
//
// A cluster of CTAs takes a row and keeps it in shared memory (a slice a CTA), so that
// the row is read from HBM once however many questions are asked of it:
//   1. the largest logit;
//   2. the weights' sum, and for top-k and top-p a histogram of how far below the
//      largest each token lies: counts and weights in 512 bins of ln p (for top-p of 1/64,
//      8 nats at a time: few tokens lie so high, which keeps atomics rare; for top-k of 1/16,
//      without the tokens that the lanes' largest logits rule out);
//   3. the bin in which the last kept token lies, from the histograms' sums.  Where no more
//      than 256 tokens lie as high, these are listed and the first CTA finishes the row
//      with them; else the tokens of that one bin are listed and ranked by (logit, index),
//      which gives the last kept token exactly, and
//   4. the kept weights' sums, and the token whose running sum passes the target, come from
//      one more pass over the slices.
// Weights are whole numbers (2^-40 of the largest), so sums are exact and neither the
// order of atomics nor the split over warps and CTAs can change a result.
#include <type_traits>

#include "operators.cuh"
#include "tensor_core.cuh"

namespace rs {
namespace {

using namespace op;
using staging::smem_addr;
using tc::cluster_sync;
using tc::in_cta;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 512;
// Bins of 1/64 nat, a histogram of 8 nats at a time, for top-p alone; bins of 1/16 nat, all
// 32 nats beyond which every weight is 0, for top-k, whose histogram leaves out most tokens.
constexpr int kBinsPerNat = 64, kWideBinsPerNat = 16;
constexpr int kNats = 32;
static_assert(kBins == kNats * kWideBinsPerNat, "one histogram for top-k");
constexpr uint32_t kFew = kThreads;  // tokens with which the first CTA finishes a row on its own
constexpr uint64_t kOne = uint64_t(1) << 40;           // weight of the most likely token

struct SampleArgs {
  const void* logits;
  int64_t vocab, ld;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t* token;
  float* logprob;
};

// A logit as it is ranked: NaN as -inf, -0 as +0.
__device__ __forceinline__ float clean(float l) { return l == l ? l + 0.0f : -INFINITY; }
// Whole numbers in the order of the floats, and back.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// Two float32 operations at once, each rounded on its own (and never contracted).
__device__ __forceinline__ float2 add2(float2 a, float b) {
  uint64_t d, x = tc::pack2(__float_as_uint(a.x), __float_as_uint(a.y));
  const uint64_t y = tc::pack2(__float_as_uint(b), __float_as_uint(b));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return tc::unpack2(d);
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  uint64_t d;
  const uint64_t x = tc::pack2(__float_as_uint(a.x), __float_as_uint(a.y));
  const uint64_t y = tc::pack2(__float_as_uint(-b.x), __float_as_uint(-b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return tc::unpack2(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float b) {
  uint64_t d, x = tc::pack2(__float_as_uint(a.x), __float_as_uint(a.y));
  const uint64_t y = tc::pack2(__float_as_uint(b), __float_as_uint(b));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return tc::unpack2(d);
}

// The row's scale: z = ln of a token's probability relative to the largest.  top is
// finite, and so is inv; z of -inf, of a difference that overflows and of NaN has weight 0
// (-inf, or NaN where inv is 0).
struct Scale {
  float top, inv;
  __device__ float2 z(float l0, float l1) const { return mul2(add2(make_float2(l0, l1), -top), inv); }
  __device__ float z(float l) const { return z(l, l).x; }
  __device__ static float e(float z) { return fmaxf(expf(z), 0.0f); }
};

// round(2^40 e), e in [0, 1], as high * 2^22 + low: adding 48 = 1.5 * 2^5 leaves e's
// multiples of 2^-18 in the sum's low bits, adding 1.5 * 2^-17 to what is left those of
// 2^-40.  The bits of both sums are added up as they are, in 32 bits (both halves of 256
// weights fit), and their constant parts taken off at the end.
struct Weights {
  uint32_t high = 0, low = 0, n = 0;
  __device__ void add(float e0, float e1) {
    const float2 a = add2(make_float2(e0, e1), 48.0f);
    const float2 b = add2(sub2(make_float2(e0, e1), add2(a, -48.0f)), 0x1.8p-17f);
    high += __float_as_uint(a.x) + __float_as_uint(a.y);
    low += __float_as_uint(b.x) + __float_as_uint(b.y);
    n += 2;
  }
  __device__ uint64_t sum() const {
    const int h = int(high - n * __float_as_uint(48.0f));
    const int l = int(low - n * __float_as_uint(0x1.8p-17f));
    return uint64_t((int64_t(h) << 22) + l);
  }
};
__device__ __forceinline__ uint64_t weight_of(float e) {
  Weights w;
  w.add(e, 0.0f);
  return w.sum();
}

// The histogram bin of a token, from 0 at the largest logit on, in whole steps of
// 1 / per_nat: the low bits of 2^23 + steps.  Grows as the logit falls; beyond any
// histogram for weight 0.
__device__ __forceinline__ uint32_t bin_of(float z, float per_nat) {
  return __float_as_uint(__fmaf_rn(z, -per_nat, 8388608.0f)) - 0x4b000000u;
}

// The smallest whole number that is not below x as a float64 (above: that is above x).
// Comparing sums with it replaces comparing their float64s with x.
__device__ uint64_t threshold(double x, bool above) {
  if (!(x < 0x1p60)) return ~uint64_t(0);
  uint64_t s = __double2ull_ru(x) + 64;  // sums below 2^60 round by at most 64
  for (uint64_t o = 64; o; o >>= 1)
    if (s >= o && (above ? double(s - o) > x : double(s - o) >= x)) s -= o;
  return s;
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan64(uint64_t v, int lane) {  // inclusive
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

__device__ __forceinline__ int cdiv_int(int a, int b) { return (a - 1) / b + 1; }

template <typename T>
__device__ __forceinline__ void store_cluster(T* at, uint32_t rank, T value) {
  const uint32_t to = in_cta(smem_addr(at), rank);
  if (sizeof(T) == 8)
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(uint64_t(value)) : "memory");
  else
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to), "r"(uint32_t(value)) : "memory");
}
__device__ __forceinline__ uint2 load_cluster8(const void* at, uint32_t rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(in_cta(smem_addr(at), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void sum_cluster(uint64_t* at, uint32_t rank, uint64_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(in_cta(smem_addr(at), rank)),
               "l"(v)
               : "memory");
}
__device__ __forceinline__ void sum_cluster(uint32_t* at, uint32_t rank, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(in_cta(smem_addr(at), rank)),
               "r"(v)
               : "memory");
}
__device__ __forceinline__ void max_cluster(uint32_t* at, uint32_t rank, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(in_cta(smem_addr(at), rank)),
               "r"(v)
               : "memory");
}
__device__ __forceinline__ uint32_t add_cluster(uint32_t* at, uint32_t rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(old)
               : "r"(in_cta(smem_addr(at), rank)), "r"(v)
               : "memory");
  return old;
}

// The last kept token: those with a larger key are kept, and with this key those up to
// this index.
struct Cut {
  uint32_t key, index;
};

enum Step : uint32_t { kList, kListFew, kHistogram, kBisect, kCut };
// What every CTA does next, as the first one has decided.
struct Order {
  uint32_t step, bin;  // kList: that bin's tokens; kListFew: up to it; kHistogram: from it on
  Cut cut;
};

constexpr int kListMost = 512;  // listed tokens, in the histogram's place

struct SampleSmem {
  union {
    struct {
      alignas(16) uint32_t mass[3][kBins];  // 14 bits of the weights each
      alignas(16) uint32_t counts[kBins];
    };
    struct {
      uint32_t key[kListMost], index[kListMost];
      uint64_t weight[kListMost];
    };
  };
  uint64_t warp_mass[kWarps];
  uint64_t cta_mass[2][kMaxCluster];  // added to by every warp of the cluster: each CTA's
  uint32_t count[2];                  // sums of a pass, and the cluster's count
  uint32_t top_key;                   // the largest logit
  uint32_t rising;                    // ~ the lowest index of the largest logit
  uint32_t below;                     // ~ the key below which no token is among the top k
  uint64_t scan_mass[kWarps];
  uint32_t scan_count[kWarps];
  uint32_t listed;
  Order order;
  uint64_t limit, best_mass;
};
static_assert(16 * kListMost <= 16 * kBins, "the list lies in the histogram");

// This CTA's slice of a row, in granules of 16 aligned bytes; what lies outside the row
// in the first and last granule reads as -inf.
template <typename T, bool RESIDENT>
struct Slice {
  static constexpr int kPer = 16 / int(sizeof(T));
  const T* row;
  unsigned char* smem;
  int vocab, skew;  // elements of the first granule that lie before the row
  int g0, g1;       // granules of the CTA
  int w0, w1;       // granules of the warp
  bool infinite;    // the largest logit is +inf: only such tokens have a weight

  __device__ int first(int g) const { return g * kPer - skew; }  // index of its first element
  __device__ uint4 fetch(int g) const {
    const int i = first(g);
    if (i >= 0 && i + kPer <= vocab) return __ldg(reinterpret_cast<const uint4*>(row + i));
    __align__(16) T v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      v[j] = i + j >= 0 && i + j < vocab ? row[i + j] : from_float<T>(-INFINITY);
    return *reinterpret_cast<const uint4*>(v);
  }
  __device__ uint4* place(int g) const { return reinterpret_cast<uint4*>(smem + size_t(g - g0) * 16); }
  // +inf as 0, all others as -inf
  __device__ static uint4 flattened(uint4 v) {
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int j = 0; j < kPer; ++j) e[j] = from_float<T>(to_float(e[j]) == INFINITY ? 0.0f : -INFINITY);
    return v;
  }
  __device__ uint4 granule(int g) const {
    if (RESIDENT) return *place(g);
    return infinite ? flattened(fetch(g)) : fetch(g);
  }
  __device__ static float largest(const uint4& v) { return op::largest_of(reinterpret_cast<const T(&)[kPer]>(v)); }
  __device__ static float at(const uint4& v, int j) { return to_float(reinterpret_cast<const T*>(&v)[j]); }
};

template <typename T, bool RESIDENT>
__global__ void __launch_bounds__(kThreads, 5) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  SampleSmem& sm = *reinterpret_cast<SampleSmem*>(dynamic);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const uint32_t rank = tc::cluster_rank();
  const int64_t r = blockIdx.x / ctas;
  if (tid < 2 * kMaxCluster) sm.cta_mass[tid / kMaxCluster][tid % kMaxCluster] = 0;
  if (tid < 2) sm.count[tid] = 0;
  if (tid == 0) sm.top_key = 0, sm.rising = 0, sm.below = 0;
  tc::cluster_arrive();  // before another CTA adds to these

  Slice<T, RESIDENT> s;
  constexpr int kPer = s.kPer;
  s.row = static_cast<const T*>(a.logits) + r * a.ld;
  s.smem = dynamic + (sizeof(SampleSmem) + 15) / 16 * 16;
  s.vocab = int(a.vocab);
  s.skew = int(reinterpret_cast<uintptr_t>(s.row) % 16 / sizeof(T));
  const int granules = (s.vocab + s.skew + kPer - 1) / kPer;
  s.g0 = int(int64_t(granules) * rank / ctas);
  s.g1 = int(int64_t(granules) * (rank + 1) / ctas);
  const int per_warp = (s.g1 - s.g0 + kWarps - 1) / kWarps;
  s.w0 = min(s.g1, s.g0 + warp * per_warp);
  s.w1 = min(s.g1, s.w0 + per_warp);

  // 1. the slice, and the largest logit
  float top = -INFINITY;
#pragma unroll 4
  for (int g = s.w0 + lane; g < s.w1; g += 32) {
    const uint4 v = s.fetch(g);
    if (RESIDENT) *s.place(g) = v;
    top = fmaxf(top, s.largest(v));
  }
  const float temperature = a.temperature ? a.temperature[r] : 1.0f;
  const bool greedy = !(temperature > 0.0f);
  float p = a.top_p ? a.top_p[r] : 1.0f;
  int k = a.top_k ? a.top_k[r] : 0;
  const float floor_e = fminf(a.min_p ? a.min_p[r] : 0.0f, 1.0f);
  const float u = fmaxf(a.u[r], 0.0f);  // NaN: 0
  if (!(p > 0.0f)) k = 1, p = 1.0f;     // only the first
  const bool by_count = !greedy && k > 0 && k < s.vocab;
  const bool by_mass = !greedy && p < 1.0f;
  if (by_count || by_mass)
    for (int i = tid; i < kBins; i += kThreads) sm.mass[0][i] = sm.mass[1][i] = sm.mass[2][i] = 0, sm.counts[i] = 0;
  const float mine_top = top;
  top = warp_max(top + 0.0f);
  tc::cluster_wait();  // the other CTAs have set their sums to 0
  if (lane < int(ctas)) max_cluster(&sm.top_key, lane, key_of(top));
  if (by_count) {
    // If each of the cluster's warps holds `most` tokens not below a logit, at least k tokens
    // are not: the least over the warps of the most-th largest of their lanes' largest ones.
    const int most = int(cdiv_int(k, kWarps * int(ctas)));
    uint32_t left = key_of(mine_top + 0.0f), bound = 0;
    for (int i = 0; i < most && most <= 32; ++i) {
      bound = __reduce_max_sync(0xffffffffu, left);
      if (lane == __ffs(int(__ballot_sync(0xffffffffu, left == bound))) - 1) left = 0;
    }
    if (lane < int(ctas)) max_cluster(&sm.below, lane, ~bound);
  }
  cluster_sync();
  const uint32_t top_key = sm.top_key;
  Scale scale;
  scale.top = logit_of(top_key);
  scale.inv = greedy ? 1.0f : fminf(1.0f / temperature, 0x1.fffffep127f);
  if (scale.top == -INFINITY) {
    if (rank == 0 && tid == 0) {
      a.token[r] = -1;
      if (a.logprob) a.logprob[r] = -INFINITY;
    }
    return;
  }
  s.infinite = scale.top == INFINITY;
  const bool holds_top = mine_top == scale.top;
  if (s.infinite) {
    scale.top = 0.0f;
    if (RESIDENT)
      for (int g = s.w0 + lane; g < s.w1; g += 32) *s.place(g) = s.flattened(*s.place(g));
  }

  // 2. weights, and the histogram of the nats below the largest
  const float per_nat = float(by_count ? kWideBinsPerNat : kBinsPerNat);
  // top-k: the bins of tokens that may be among the k
  uint32_t bins = kBins;
  if (by_count && ~sm.below != 0 && !s.infinite)
    bins = min(bins, bin_of(scale.z(logit_of(~sm.below)), per_nat) + 1);
  auto tally = [&](float z, float e, uint32_t begin) {
    const uint32_t bin = bin_of(z, per_nat) - begin;
    if (bin < bins) {
      atomicAdd(&sm.counts[bin], 1u);
      const uint64_t w = weight_of(e);
      atomicAdd(&sm.mass[0][bin], uint32_t(w) & 0x3fffu);
      atomicAdd(&sm.mass[1][bin], uint32_t(w >> 14) & 0x3fffu);
      atomicAdd(&sm.mass[2][bin], uint32_t(w >> 28));
    }
  };
  Weights sums;
  uint32_t lowest = 0xffffffffu;
  if (by_count || by_mass) {
    for (int g = s.w0 + lane; g < s.w1; g += 32) {
      const uint4 v = s.granule(g);
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        const float2 z = scale.z(s.at(v, j), s.at(v, j + 1));
        const float e0 = scale.e(z.x), e1 = scale.e(z.y);
        sums.add(e0, e1);
        tally(z.x, e0, 0);
        tally(z.y, e1, 0);
      }
    }
  } else {
    for (int g = s.w0 + lane; g < s.w1; g += 32) {
      const uint4 v = s.granule(g);
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        const float2 z = scale.z(s.at(v, j), s.at(v, j + 1));
        sums.add(scale.e(z.x), scale.e(z.y));
      }
    }
    if (greedy && holds_top)
      for (int g = s.w0 + lane; g < s.w1 && lowest == 0xffffffffu; g += 32) {
        const uint4 v = s.granule(g);
        for (int j = kPer - 1; j >= 0; --j)
          if (s.at(v, j) == scale.top) lowest = uint32_t(s.first(g) + j);
      }
  }
  // Adds the threads' values to every CTA's sums (of the given slot, which are 0 before).
  uint32_t slot = 0;
  auto publish = [&](uint64_t mass, uint32_t count) {
    mass = warp_sum64(mass);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) sm.warp_mass[warp] = mass;
    if (lane < int(ctas)) {
      sum_cluster(&sm.cta_mass[slot][rank], lane, mass);
      if (count) sum_cluster(&sm.count[slot], lane, count);
    }
    cluster_sync();
  };
  auto cluster_mass = [&] {
    uint64_t m = 0;
    for (uint32_t i = 0; i < ctas; ++i) m += sm.cta_mass[slot][i];
    return m;
  };
  // The other slot, for the next sums; the one just read is set to 0 for those after them
  // (their CTAs add to it only after the cluster has met once more).
  auto next_slot = [&] {
    __syncthreads();
    if (tid < kMaxCluster) sm.cta_mass[slot][tid] = 0;
    if (tid == 0) sm.count[slot] = 0;
    slot ^= 1;
  };
  if (greedy) {
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    if (lane == 0 && lowest != 0xffffffffu) max_cluster(&sm.rising, 0, ~lowest);
  }
  publish(sums.sum(), 0);
  const uint64_t total = cluster_mass();
  auto answer = [&](int i, float l) {
    a.token[r] = i;
    if (a.logprob)
      a.logprob[r] = scale.z(l) - log1pf(float(double(total - kOne) / double(kOne)));
  };
  if (greedy) {
    if (rank == 0 && tid == 0) answer(int(~sm.rising), scale.top);
    return;
  }

  // 3. the last kept token
  Cut cut = {0, 0xffffffffu};
  auto kept = [&](uint32_t key, int i) {
    return key > cut.key || (key == cut.key && uint32_t(i) <= cut.index);
  };
  if (by_count || by_mass) {
    // The first CTA's view: the histograms' sums (two bins a thread) and what lies before.
    static_assert(kBins == 2 * kThreads, "two bins a thread");
    uint32_t counts[2] = {}, count_before = 0;
    uint64_t masses[2] = {}, mass_before = 0;
    uint32_t skipped_count = 0;   // tokens above the histogram's range
    uint64_t skipped_mass = 0;
    uint32_t begin = 0;           // the histogram's first bin
    bool count_open = by_count;   // top-k still to be resolved, else top-p
    uint64_t kept_mass = total;   // of the tokens that top-k keeps
    uint32_t bin_count = 0;       // tokens and weights before the listed bin
    uint64_t bin_mass = 0;
    auto gather = [&] {
      counts[0] = counts[1] = 0, masses[0] = masses[1] = 0;
#pragma unroll 4
      for (uint32_t c = 0; c < ctas; ++c) {
        const uint2 n = load_cluster8(&sm.counts[2 * tid], c);
        const uint2 m0 = load_cluster8(&sm.mass[0][2 * tid], c);
        const uint2 m1 = load_cluster8(&sm.mass[1][2 * tid], c);
        const uint2 m2 = load_cluster8(&sm.mass[2][2 * tid], c);
        counts[0] += n.x, counts[1] += n.y;
        masses[0] += m0.x + (uint64_t(m1.x) << 14) + (uint64_t(m2.x) << 28);
        masses[1] += m0.y + (uint64_t(m1.y) << 14) + (uint64_t(m2.y) << 28);
      }
      const uint32_t cn = counts[0] + counts[1];
      const uint64_t mn = masses[0] + masses[1];
      uint64_t ci = warp_scan64(cn, lane), mi = warp_scan64(mn, lane);
      __syncthreads();
      if (lane == 31) sm.scan_count[warp] = uint32_t(ci), sm.scan_mass[warp] = mi;
      __syncthreads();
      count_before = skipped_count + uint32_t(ci) - cn;
      mass_before = skipped_mass + mi - mn;
      for (int i = 0; i < warp; ++i)
        count_before += sm.scan_count[i], mass_before += sm.scan_mass[i];
    };
    // Orders the bin in which the last kept token lies to be listed; where it lies beyond
    // the histogram, a histogram of the next nats.
    auto decide = [&] {
      if (tid == 0) {
        sm.order.step = kHistogram;
        sm.limit = threshold(double(p) * double(kept_mass), false);
      }
      __syncthreads();
      const uint64_t limit = sm.limit;
      uint32_t c = count_before;
      uint64_t m = mass_before;
      for (int j = 0; j < 2; ++j) {
        const bool inside = count_open ? c < uint32_t(k) && c + counts[j] >= uint32_t(k)
                                       : m < limit && m + masses[j] >= limit;
        if (inside) {
          sm.order.step = c + counts[j] <= kFew ? kListFew : kList;
          sm.order.bin = begin + 2 * tid + j;
          sm.scan_count[0] = c;
          sm.scan_mass[0] = m;
        }
        c += counts[j], m += masses[j];
      }
      if (tid == kThreads - 1) sm.scan_count[1] = c, sm.scan_mass[1] = m;
      __syncthreads();
      if (sm.order.step != kHistogram) {
        bin_count = sm.scan_count[0], bin_mass = sm.scan_mass[0];
        if (tid == 0) sm.listed = 0;
        return;
      }
      skipped_count = sm.scan_count[1], skipped_mass = sm.scan_mass[1];
      __syncthreads();
      if (begin + kBins < uint32_t(kNats) * uint32_t(per_nat)) {
        begin += kBins;
      } else if (count_open && by_mass) {
        count_open = false;
        begin = 0, skipped_count = 0, skipped_mass = 0;
      } else if (tid == 0) {
        sm.order.step = kCut, sm.order.cut = {0, 0xffffffffu};
      }
      if (tid == 0) sm.order.bin = begin;
    };
    // Ranks the listed tokens by (logit, index) and takes the last kept one.
    auto resolve = [&] {
      const uint32_t n = sm.listed;
      if (n > uint32_t(kListMost)) {
        if (tid == 0) sm.order.step = kBisect;
        return;
      }
      const uint64_t limit = sm.limit;
      for (uint32_t i = tid; i < n; i += kThreads)
        sm.weight[i] = weight_of(scale.e(scale.z(logit_of(sm.key[i]))));
      __syncthreads();
      for (uint32_t i = tid; i < n; i += kThreads) {
        const uint32_t key = sm.key[i], index = sm.index[i];
        uint32_t before = bin_count;
        const uint64_t own = sm.weight[i];
        uint64_t m = bin_mass;
        for (uint32_t j = 0; j < n; ++j) {
          const uint32_t kj = sm.key[j];
          if (kj > key || (kj == key && sm.index[j] < index)) ++before, m += sm.weight[j];
        }
        if (count_open ? before + 1 == uint32_t(k) : m < limit && m + own >= limit) {
          sm.order.cut = {key, index};
          sm.best_mass = m + own;
        }
      }
      __syncthreads();
      if (!(count_open && by_mass)) {
        if (tid == 0) sm.order.step = kCut;
        return;
      }
      kept_mass = sm.best_mass;  // now top-p among what top-k keeps
      count_open = false;
      if (begin == 0) {          // its bin is in the histogram that the registers still hold
        decide();
      } else {
        begin = 0, skipped_count = 0, skipped_mass = 0;
        if (tid == 0) sm.order.step = kHistogram, sm.order.bin = 0;
      }
    };
    // The whole rest, with all tokens that may be kept in the list: a token a thread.
    auto finish_few = [&] {
      const uint32_t n = sm.listed;
      const bool mine = tid < int(n);
      const uint32_t key = mine ? sm.key[tid] : 0, index = mine ? sm.index[tid] : 0;
      const float e = mine ? scale.e(scale.z(logit_of(key))) : 0.0f;
      const uint64_t own = weight_of(e);
      sm.weight[tid] = own;
      __syncthreads();
      uint32_t before = 0;
      uint64_t m = 0;
      for (uint32_t j = 0; mine && j < n; ++j) {
        const uint32_t kj = sm.key[j];
        if (kj > key || (kj == key && sm.index[j] < index)) ++before, m += sm.weight[j];
      }
      Cut last = {0, 0xffffffffu};
      if (count_open) {  // else top-k has been resolved, or keeps all that has a weight
        if (mine && before + 1 == uint32_t(k)) sm.order.cut = {key, index}, sm.best_mass = m + own;
        __syncthreads();
        last = sm.order.cut, kept_mass = sm.best_mass;
        __syncthreads();
      }
      if (by_mass) {
        if (tid == 0) sm.limit = threshold(double(p) * double(kept_mass), false);
        __syncthreads();
        if (mine && m < sm.limit && m + own >= sm.limit) sm.order.cut = {key, index};
        __syncthreads();
        last = sm.order.cut;
      }
      const bool kept = mine && !(e < floor_e) &&
                        (key > last.key || (key == last.key && index <= last.index));
      sm.weight[tid] = kept ? own : 0;
      __syncthreads();
      uint64_t all = 0, upto = 0;
      for (uint32_t j = 0; j < n; ++j) {
        const uint64_t w = sm.weight[j];
        all += w;
        if (sm.index[j] <= index) upto += w;
      }
      if (tid == 0) sm.limit = min(threshold(double(u) * double(all), true), all);
      __syncthreads();
      if (kept && upto >= sm.limit && upto - own < sm.limit) answer(int(index), logit_of(key));
    };
    auto send = [&] {  // sm.order to every CTA
      __syncthreads();
      if (tid < int(ctas) && tid > 0) {
        store_cluster(&sm.order.step, tid, sm.order.step);
        store_cluster(&sm.order.bin, tid, sm.order.bin);
        store_cluster(&sm.order.cut.key, tid, sm.order.cut.key);
        store_cluster(&sm.order.cut.index, tid, sm.order.cut.index);
      }
    };

    bool fresh = true;  // the histograms have just been made
    Order order;
    for (;;) {
      if (rank == 0) {
        if (fresh) {
          gather();
          decide();
        } else {
          resolve();
        }
        send();
      }
      cluster_sync();
      order = sm.order;
      if (order.step == kCut || order.step == kBisect) break;
      fresh = order.step == kHistogram;
      const uint32_t lowest_bin = order.step == kListFew ? 0 : order.bin;
      if (fresh) {
        for (int i = tid; i < kBins; i += kThreads) sm.mass[0][i] = sm.mass[1][i] = sm.mass[2][i] = 0, sm.counts[i] = 0;
        __syncthreads();
      }
      if (fresh) {
        for (int g = s.w0 + lane; g < s.w1; g += 32) {
          const uint4 v = s.granule(g);
#pragma unroll
          for (int j = 0; j < kPer; j += 2) {
            const float2 z = scale.z(s.at(v, j), s.at(v, j + 1));
            tally(z.x, scale.e(z.x), order.bin);
            tally(z.y, scale.e(z.y), order.bin);
          }
        }
      } else {
        // no token of these bins lies below this (all rounding goes that way)
        const float lowest_logit = __fsub_rd(
            scale.top, __fdiv_ru(__fdiv_ru(float(order.bin + 1), per_nat), scale.inv));
        for (int g = s.w0 + lane; g < s.w1; g += 32) {
          const uint4 v = s.granule(g);
          if (!(s.largest(v) >= lowest_logit)) continue;
#pragma unroll 1
          for (int j = 0; j < kPer; ++j) {
            const float l = clean(s.at(v, j));
            const uint32_t bin = bin_of(scale.z(l), per_nat);
            if (bin < lowest_bin || bin > order.bin) continue;
            const uint32_t to = add_cluster(&sm.listed, 0, 1);
            if (to >= uint32_t(kListMost)) continue;
            store_cluster(&sm.key[to], 0, key_of(l));
            store_cluster(&sm.index[to], 0, uint32_t(s.first(g) + j));
          }
        }
      }
      cluster_sync();
      if (order.step == kListFew) {
        if (rank == 0) finish_few();
        return;
      }
    }
    if (order.step == kCut) {
      cut = order.cut;
    } else {
      // Too many tokens in one bin, as where logits are alike: the cut's key by bisection over
      // its bits, every CTA over its slice, then its index by counting the tokens with it.
      uint64_t mass;   // of the tokens inside the cut with at least
      uint32_t count;  // this key
      auto sums_to = [&](uint32_t key) {
        uint64_t m = 0;
        uint32_t c = 0;
#pragma unroll 1
        for (int g = s.w0 + lane; g < s.w1; g += 32) {
          const uint4 v = s.granule(g);
#pragma unroll 1
          for (int j = 0; j < kPer; ++j) {
            const int i = s.first(g) + j;
            const float l = clean(s.at(v, j));
            const uint32_t q = key_of(l);
            if (uint32_t(i) >= uint32_t(s.vocab) || !kept(q, i)) continue;
            if (q < key) continue;
            m += weight_of(scale.e(scale.z(l))), ++c;
          }
        }
        next_slot();
        publish(m, c);
        mass = cluster_mass(), count = sm.count[slot];
      };
      constexpr uint32_t kAll = 0xffffffffu;
      // bits of a key that are alike in all positive and in all negative logits of the type
      constexpr int kLowBits = sizeof(T) == 4 ? 0 : std::is_same<T, __half>::value ? 13 : 16;
      bool open = by_count;
      uint64_t limit = by_count ? uint64_t(k) : threshold(double(p) * double(total), false);
#pragma unroll 1
      for (;;) {
        uint32_t key = 0;  // the largest for which the sum reaches the limit
#pragma unroll 1
        for (int b = 31; b >= kLowBits; --b) {
          sums_to(key | 1u << b);
          if ((open ? uint64_t(count) : mass) >= limit) key |= 1u << b;
        }
        if (!(key >> 31)) key |= (1u << kLowBits) - 1;
        // the ties at this key that are kept, and the index of the last of them
        const uint64_t w = weight_of(scale.e(scale.z(logit_of(key))));
        if (key == kAll) mass = 0, count = 0;
        else sums_to(key + 1);
        const uint64_t ties = open ? limit - count : (limit - mass + w - 1) / w;
        const uint64_t upto = mass + ties * w;
        auto ties_of = [&](const uint4& v, int g) {
          uint32_t n = 0;
          for (int j = 0; j < kPer; ++j) {
            const int i = s.first(g) + j;
            n += key_of(clean(s.at(v, j))) == key && uint32_t(i) < uint32_t(s.vocab) && kept(key, i);
          }
          return n;
        };
        uint64_t mine = 0;
        for (int g = s.w0 + lane; g < s.w1; g += 32) mine += ties_of(s.granule(g), g);
        next_slot();
        publish(mine, 0);
        uint64_t run = 0;
        for (uint32_t i = 0; i < rank; ++i) run += sm.cta_mass[slot][i];
        for (int i = 0; i < warp; ++i) run += sm.warp_mass[i];
        if (run < ties && run + sm.warp_mass[warp] >= ties) {
          for (int g = s.w0 + lane;; g += 32) {  // ends: the warp has the last of them
            uint4 v = make_uint4(0, 0, 0, 0);
            uint64_t n = 0;
            if (g < s.w1) {
              v = s.granule(g);
              n = ties_of(v, g);
            }
            const uint64_t through = run + warp_scan64(n, lane);
            const uint32_t found = __ballot_sync(0xffffffffu, through >= ties);
            if (found) {
              if (lane == __ffs(int(found)) - 1) {
                uint64_t left = ties - (through - n);
                int i = s.first(g);
                for (int j = 0; left > 0; ++j, ++i)
                  if (key_of(clean(s.at(v, j))) == key && uint32_t(i) < uint32_t(s.vocab) && kept(key, i))
                    if (--left == 0) break;
                for (uint32_t c = 0; c < ctas; ++c) store_cluster(&sm.order.cut.index, c, uint32_t(i));
              }
              break;
            }
            run = __shfl_sync(0xffffffffu, through, 31);
          }
        }
        cluster_sync();
        cut = {key, sm.order.cut.index};
        if (!open || !by_mass) break;
        open = false;
        limit = threshold(double(p) * double(upto), false);
      }
    }
  }

  // 4. the token
  const float cut_logit = cut.key == 0 ? -INFINITY : logit_of(cut.key);
  auto chance = [&](float l, float z, int i) {  // 0 for a token that is not kept
    const float e = scale.e(z);
    if (!(l >= cut_logit) || (l == cut_logit && uint32_t(i) > cut.index) || e < floor_e) return 0.0f;
    return e;
  };
  auto granule_sum = [&](const uint4& v, int g) {
    Weights w;
#pragma unroll
    for (int j = 0; j < kPer; j += 2) {
      const float l0 = s.at(v, j), l1 = s.at(v, j + 1);
      const float2 z = scale.z(l0, l1);
      w.add(chance(l0, z.x, s.first(g) + j), chance(l1, z.y, s.first(g) + j + 1));
    }
    return w.sum();
  };
  uint64_t all = total;
  if (by_count || by_mass || floor_e > 0.0f) {
    uint64_t mine = 0;
    for (int g = s.w0 + lane; g < s.w1; g += 32) {
      const uint4 v = s.granule(g);
      if (s.largest(v) >= cut_logit) mine += granule_sum(v, g);
    }
    next_slot();
    publish(mine, 0);
    all = cluster_mass();
  }
  // the first token at which the sum passes u times all; none does for u >= 1: the last
  // one with a weight, at which the sum is complete
  if (tid == 0) sm.limit = min(threshold(double(u) * double(all), true), all);
  __syncthreads();
  const uint64_t limit = sm.limit;
  uint64_t run = 0;
  for (uint32_t i = 0; i < rank; ++i) run += sm.cta_mass[slot][i];
  for (int i = 0; i < warp; ++i) run += sm.warp_mass[i];
  if (run >= limit || run + sm.warp_mass[warp] < limit) return;
  for (int g = s.w0 + lane;; g += 32) {  // ends: the warp's sum reaches the limit
    uint4 v = make_uint4(0, 0, 0, 0);
    uint64_t mine = 0;
    if (g < s.w1) {
      v = s.granule(g);
      mine = granule_sum(v, g);
    }
    const uint64_t upto = run + warp_scan64(mine, lane);
    const uint32_t found = __ballot_sync(0xffffffffu, upto >= limit);
    if (found) {
      if (lane == __ffs(int(found)) - 1) {
        uint64_t sum = upto - mine;
        for (int j = 0; j < kPer; ++j) {
          const int i = s.first(g) + j;
          const float l = s.at(v, j), z = scale.z(l);
          sum += weight_of(chance(l, z, i));
          if (sum >= limit) {
            answer(i, l);
            break;
          }
        }
      }
      return;
    }
    run = __shfl_sync(0xffffffffu, upto, 31);
  }
}

template <typename T>
reshard_status_t launch_sample(const SampleArgs& a, int64_t rows, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(ce));
  const int64_t bytes = (a.vocab + 16 / int64_t(sizeof(T))) * int64_t(sizeof(T));
  // CTAs a row: slices of at most 32 KiB; smaller ones while SMs would stay without a CTA
  int ctas = 1;
  while (ctas < kMaxCluster && (bytes > ctas * 32768 || (rows * ctas < sms && bytes > ctas * 4096)))
    ctas *= 2;
  const int64_t slice = (cdiv(cdiv(bytes, 16) + 1, ctas) + 1) * 16;
  const size_t fixed = (sizeof(SampleSmem) + 15) / 16 * 16;
  const bool resident = fixed + size_t(slice) <= 227 * 1024;
  const size_t smem = fixed + (resident ? size_t(slice) : 0);
  const void* kernel = resident ? reinterpret_cast<const void*>(sample_kernel<T, true>)
                                : reinterpret_cast<const void*>(sample_kernel<T, false>);
  ce = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (ce == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(rows * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {unsigned(ctas), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<SampleArgs*>(&a)};
    ce = cudaLaunchKernelExC(&cfg, kernel, args);
  }
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string("reshard_sample: ") + cudaGetErrorString(ce));
  return RESHARD_OK;
}

}  // namespace
}  // namespace rs

using rs::fail;

extern "C" reshard_status_t reshard_sample(const void* logits, int32_t dtype, int64_t rows,
                                           int64_t vocab, int64_t ld, const float* temperature,
                                           const int32_t* top_k, const float* top_p,
                                           const float* min_p, const float* u, int32_t* token,
                                           float* logprob, void* stream) {
  rs::TraceRange trace("op.sample");
  if (!rs::op::float_dtype(dtype))
    return fail(RESHARD_ERR_INVALID_ARG, "dtype must be BF16, FP16 or FP32");
  if (rows < 0 || vocab < 0) return fail(RESHARD_ERR_INVALID_ARG, "negative size");
  if (vocab > RESHARD_MAX_VOCAB) return fail(RESHARD_ERR_UNSUPPORTED, "vocabulary too large");
  if (rows >= int64_t(1) << 28) return fail(RESHARD_ERR_UNSUPPORTED, "2^28 rows or more");
  if (rows == 0 || vocab == 0) return RESHARD_OK;
  if (ld < vocab) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!logits || !u || !token) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(logits, rs::op::dtype_size(dtype)) || !rs::op::aligned(temperature, 4) ||
      !rs::op::aligned(top_k, 4) || !rs::op::aligned(top_p, 4) || !rs::op::aligned(min_p, 4) ||
      !rs::op::aligned(u, 4) || !rs::op::aligned(token, 4) || !rs::op::aligned(logprob, 4))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  rs::SampleArgs a = {logits, vocab, ld, temperature, top_p, min_p, u, top_k, token, logprob};
  return rs::op::by_dtype(dtype, [&](auto t) {
    return rs::launch_sample<decltype(t)>(a, rows, static_cast<cudaStream_t>(stream));
  });
}
