// sample.cu -- reshard_sample: one token a row of logits, with temperature, top-k,
// top-p and min-p, from one given uniform number a row.
//
// With e_i = exp((l_i - max l) / T), top-k keeps the k first by (logit, index), top-p of these
// the shortest run whose e reach p times their sum, min-p those with e_i >= min_p; the token is
// the first kept index whose running sum of e passes u times the kept sum, and its log-
// probability (l_i - max l) / T - ln(sum of all e).
// A cluster of CTAs takes a row and keeps it in shared memory (a slice a CTA), so that
// the row is read from HBM once however many questions are asked of it:
//   1. the largest logit;
//   2. the weights' sum, and for top-k and top-p a histogram of how far below the
//      largest each token lies: counts and weights in 512 bins of ln p (for top-p of 1/48,
//      10.7 nats: few tokens lie so high, which keeps atomics rare; for top-k of 1/16, without
//      the tokens that the lanes' largest logits rule out);
//   3. the bin in which the last kept token lies: each CTA sends the sums of its groups of 32
//      bins to the others, which then read that one group's bins, and all decide alike (one
//      CTA that read all histograms and told the others took 11 000 clocks of a row's 37 000,
//      this 4 000).  Where no more than 256 tokens lie as high, these are listed and the
//      first CTA finishes the row with them; else the tokens of that one bin are listed and
//      ranked by (logit, index), which gives the last kept token exactly (a bin of more than
//      384 tokens is bisected over the logits' bits instead), and
//   4. the kept weights' sums, and the token whose running sum passes the target, come from
//      one more pass over the slices.
// Weights are whole numbers (2^-40 of the largest), so sums are exact and neither the
// order of atomics nor the split over warps and CTAs can change a result.
//
// Bound by instructions (about 23 a token of a warp's 32) and by the cluster's meetings, not by
// HBM: 256 rows of 131072 bf16 logits take 35 us greedy, 42 us whole, 76 us with top-p 0.95,
// 60 to 71 us mixed, by the set (67 MB, 10 us of HBM; all with a few likely tokens a row); one row
// 12 to 15 us, 37 rows of 50021 float32 14.4 to 17 us.
// Where a bin is bisected it takes 16 (16-bit logits) to 32 passes over the row.  That is where
// logits are alike (256 equal rows of 131072: bf16 1.3 ms, float32 2.8 ms) and where top-p ends
// among very many tokens: 256 rows of 131072 normal logits of deviation 0.5 to 2, top-p 0.95, take
// 1.4 ms in bf16 and 3.5 ms in float32, of deviation 3 0.3 and 0.46 ms; of 32000 60 to 210 us.
#include <type_traits>

#include "operators.cuh"
#include "tensor_core.cuh"

namespace rs {
namespace {

using namespace op;
using staging::smem_addr;
using tc::cluster_sync;
using tc::in_cta;

constexpr int kFewThreads = 256, kManyThreads = 512;  // of a CTA
constexpr int kMaxCluster = 8;
constexpr int kBins = 512;
// Bins of 1/48 nat, 10.7 nats first, for top-p alone (256 rows of 131072 with top-p 0.95, ten
// sets: 75.7 us on average; 1/64 79.6 us, 1/40 84.7 us); bins of 1/16 nat, all 32 nats beyond
// which every weight is 0, for top-k, whose histogram leaves out most tokens.
constexpr int kBinsPerNat = 48, kWideBinsPerNat = 16;
constexpr int kNats = 32;
// Where top-p goes beyond those it seldom goes far, and ever more tokens lie there (256 mixed
// rows of 131072, one set: 71 us in steps of 2 nats, 74 of 1, 72 of 4, 77 of 8).
constexpr int kNextBins = 128;
static_assert(kBins == kNats * kWideBinsPerNat, "one histogram for top-k");
constexpr int kFew = 256;  // tokens with which the first CTA finishes a row on its own
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

__device__ __forceinline__ uint64_t pack(float2 v) {
  return tc::pack2(__float_as_uint(v.x), __float_as_uint(v.y));
}
__device__ __forceinline__ uint64_t pack(float v) { return pack(make_float2(v, v)); }
// Two float32 operations at once, each rounded on its own (and never contracted).
__device__ __forceinline__ float2 add2(float2 a, float b) {
  uint64_t d, x = tc::pack2(__float_as_uint(a.x), __float_as_uint(a.y));
  const uint64_t y = tc::pack2(__float_as_uint(b), __float_as_uint(b));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return tc::unpack2(d);
}
// (a product with -1 is exact, and needs no change of signs beforehand)
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  return tc::unpack2(tc::fma2(pack(b), pack(-1.0f), pack(a)));
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
  // e^z for z <= 0, and what has the weight 0 for what lies 40 below, -inf and NaN.  After
  // Cody and Waite: z log2(e) = n + f with n whole (the sum with 1.5 * 2^23 rounds to it), f
  // from log2(e) in two parts, and 2^n added to the exponent of 2^f.
  __device__ static float2 e(float2 z) {
    constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f, kWhole = 0x1.8p23f;
    const uint64_t x = pack(make_float2(fmaxf(z.x, -40.0f), fmaxf(z.y, -40.0f)));
    const uint64_t t = tc::fma2(x, pack(kLog2e), pack(kWhole));
    const uint64_t minus_n = pack(sub2(make_float2(kWhole, kWhole), tc::unpack2(t)));
    const float2 f = tc::unpack2(tc::fma2(x, pack(kRest), tc::fma2(x, pack(kLog2e), minus_n)));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(f.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(f.y));
    return make_float2(__uint_as_float(__float_as_uint(e.x) + (uint32_t(t) << 23)),
                       __uint_as_float(__float_as_uint(e.y) + (uint32_t(t >> 32) << 23)));
  }
  __device__ static float e(float z) { return e(make_float2(z, z)).x; }
};

// round(2^40 e), e in [0, 1], as high * 2^22 + low: adding 48 = 1.5 * 2^5 leaves e's
// multiples of 2^-18 in the sum's low bits, adding 1.5 * 2^-17 to what is left those of
// 2^-40.  The bits of both sums are added up as they are, in 32 bits (the low halves lie
// within 2^21 either way, so that 1023 weights fit; a thread has 520 at most, of a row of
// RESHARD_MAX_VOCAB by eight CTAs of 256 threads), and their constant parts taken off at the end.
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
  if (x < 0x1p53) return above ? __double2ull_rd(x) + 1 : __double2ull_ru(x);  // sums are exact
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
__device__ __forceinline__ uint32_t warp_scan32(uint32_t v, int lane) {  // inclusive
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
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
__device__ __forceinline__ uint32_t load_cluster(const uint32_t* at, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(in_cta(smem_addr(at), rank)) : "memory");
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

constexpr int kGroup = 32;  // bins of which a CTA sends the sums to the others
constexpr int kGroups = kBins / kGroup;
static_assert(kGroups <= 32, "a group a lane");
constexpr int kListMost = 384;  // listed tokens: with slices of 32 KiB, five CTAs an SM

struct Entry {  // a listed token as the first CTA compares it
  uint64_t rank, weight;
};

template <int kWarps>
struct SampleSmem {
  union {
    struct {
      alignas(16) uint32_t mass[3][kBins];  // 14 bits of the weights each
      uint32_t counts[kBins];
    };
    uint64_t weight[kListMost];  // of the first CTA's list
    alignas(16) Entry entry[kFew];
  };
  uint32_t key[kListMost], index[kListMost];  // the list, in the first CTA
  uint64_t group_mass[2][kGroups], bin_mass[kGroup];
  uint64_t warp_mass[kWarps];
  uint64_t cta_mass[2][kMaxCluster];  // added to by every warp of the cluster: each CTA's
  uint64_t limit, best_mass;          // sums of a pass, and the cluster's count
  uint32_t group_count[2][kGroups], bin_count[kGroup];
  uint32_t count[2];
  uint32_t top_key;                   // the largest logit
  uint32_t rising;                    // ~ the lowest index of the largest logit
  uint32_t below;                     // ~ the key below which no token is among the top k
  uint32_t listed;
  Cut cut;
  uint32_t bisect;                    // the bin held too many tokens to list
};

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
  // element j of granule g, which v holds, j known at run time only
  __device__ float element(const uint4& v, int g, int j) const {
    if (RESIDENT) return to_float(reinterpret_cast<const T*>(place(g))[j]);
    const uint32_t w = j * int(sizeof(T)) / 4;
    uint32_t word = w < 2 ? (w < 1 ? v.x : v.y) : (w < 3 ? v.z : v.w);
    if (sizeof(T) == 2 && (j & 1)) word >>= 16;
    return to_float(reinterpret_cast<const T&>(word));
  }
  __device__ static float at(const uint4& v, int j) { return to_float(reinterpret_cast<const T*>(&v)[j]); }
};

template <typename T, bool RESIDENT, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == kFewThreads ? 5 : 1) sample_kernel(const SampleArgs a) {
  constexpr int kWarps = kThreads / 32;
  using Smem = SampleSmem<kWarps>;
  extern __shared__ __align__(16) unsigned char dynamic[];
  Smem& sm = *reinterpret_cast<Smem*>(dynamic);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const uint32_t rank = tc::cluster_rank();
  const int64_t r = blockIdx.x / ctas;
  if (tid < 2 * kMaxCluster) sm.cta_mass[tid / kMaxCluster][tid % kMaxCluster] = 0;
  if (tid < 2) sm.count[tid] = 0;
  if (tid < 2 * kGroups) sm.group_mass[0][tid] = 0, sm.group_count[0][tid] = 0;
  if (tid == 0) sm.top_key = 0, sm.rising = 0, sm.below = 0, sm.listed = 0;
  tc::cluster_arrive();  // before another CTA adds to these

  Slice<T, RESIDENT> s;
  constexpr int kPer = s.kPer;
  s.row = static_cast<const T*>(a.logits) + r * a.ld;
  s.smem = dynamic + sizeof(Smem);
  s.vocab = int(a.vocab);
  s.skew = int(reinterpret_cast<uintptr_t>(s.row) % 16 / sizeof(T));
  const int granules = (s.vocab + s.skew + kPer - 1) / kPer;
  s.g0 = int(int64_t(granules) * rank / ctas);
  s.g1 = int(int64_t(granules) * (rank + 1) / ctas);
  const int per_warp = (s.g1 - s.g0 + kWarps - 1) / kWarps;
  s.w0 = min(s.g1, s.g0 + warp * per_warp);
  s.w1 = min(s.g1, s.w0 + per_warp);

  const float temperature = a.temperature ? a.temperature[r] : 1.0f;
  float p = a.top_p ? a.top_p[r] : 1.0f;
  int k = a.top_k ? a.top_k[r] : 0;
  const float min_p = a.min_p ? a.min_p[r] : 0.0f, given_u = a.u[r];
  auto clear = [&] {  // the histogram
    uint4* to = reinterpret_cast<uint4*>(sm.mass);
    for (int i = tid; i < kBins; i += kThreads) to[i] = make_uint4(0, 0, 0, 0);
  };
  static_assert(offsetof(Smem, key) == 16 * kBins, "masses and counts in a row");
  clear();

  // 1. the slice, and the largest logit
  float top = -INFINITY;
  auto take = [&](int g, const uint4& v) {
    if (RESIDENT) *s.place(g) = v;
    top = fmaxf(top, s.largest(v));
  };
  // whole granules first, four loads in flight
  const int whole0 = max(s.w0, int(s.skew > 0)), whole1 = min(s.w1, (s.vocab + s.skew) / kPer);
  for (int g = s.w0 + lane; g < whole1; g += 4 * 32) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (g + 32 * i >= whole0 && g + 32 * i < whole1) v[i] = __ldg(reinterpret_cast<const uint4*>(s.row + s.first(g + 32 * i)));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (g + 32 * i >= whole0 && g + 32 * i < whole1) take(g + 32 * i, v[i]);
  }
  // the row's ends
  if (lane == 0 && s.w0 < min(s.w1, whole0)) take(s.w0, s.fetch(s.w0));
  if (lane == ((s.w1 - 1 - s.w0) & 31) && max(s.w0, max(whole0, whole1)) < s.w1) take(s.w1 - 1, s.fetch(s.w1 - 1));
  const bool greedy = !(temperature > 0.0f);
  const float floor_e = fminf(min_p, 1.0f);
  const float u = fmaxf(given_u, 0.0f);  // NaN: 0
  if (!(p > 0.0f)) k = 1, p = 1.0f;      // only the first
  const bool by_count = !greedy && k > 0 && k < s.vocab;
  const bool by_mass = !greedy && p < 1.0f;
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
  // The tokens of a granule in the histogram's bins, from the given one on.  Those that may be
  // are marked first, z - histogram_z having no sign, the first element highest; then each
  // lane takes its next one at a time, so that a warp makes as many rounds as its fullest
  // lane needs.
  float histogram_z = by_count || by_mass ? -float(bins) / per_nat : 0.0f;  // none lies below
  auto mark = [&](uint32_t& below, float2 z) {
    const float2 d = add2(z, -histogram_z);
    below = __funnelshift_l(__float_as_uint(d.x), below, 1);
    below = __funnelshift_l(__float_as_uint(d.y), below, 1);
  };
  auto tally = [&](uint32_t below, const uint4& v, int g, uint32_t begin) {
    for (uint32_t hits = ~below << (32 - kPer); hits;) {
      const int j = __clz(int(hits));
      hits &= ~(0x80000000u >> j);
      const float z = scale.z(s.element(v, g, j));
      const uint32_t bin = bin_of(z, per_nat) - begin;
      if (bin >= bins) continue;
      atomicAdd(&sm.counts[bin], 1u);
      const uint64_t w = weight_of(scale.e(z));
      atomicAdd(&sm.mass[0][bin], uint32_t(w) & 0x3fffu);
      atomicAdd(&sm.mass[1][bin], uint32_t(w >> 14) & 0x3fffu);
      atomicAdd(&sm.mass[2][bin], uint32_t(w >> 28));
    }
  };
  uint32_t turn = 0;  // histograms take turns with the sums of their groups
  auto send_groups = [&] {
    __syncthreads();
    // for the next one, before any CTA can be there
    if (tid < kGroups) sm.group_mass[turn ^ 1][tid] = 0, sm.group_count[turn ^ 1][tid] = 0;
    for (int i = warp; i < kGroups; i += kWarps) {
      const int bin = i * kGroup + lane;
      const uint32_t n = __reduce_add_sync(0xffffffffu, sm.counts[bin]);
      const uint32_t m0 = __reduce_add_sync(0xffffffffu, sm.mass[0][bin]);
      const uint32_t m1 = __reduce_add_sync(0xffffffffu, sm.mass[1][bin]);
      const uint32_t m2 = __reduce_add_sync(0xffffffffu, sm.mass[2][bin]);
      if (n && lane < int(ctas)) {
        sum_cluster(&sm.group_count[turn][i], lane, n);
        sum_cluster(&sm.group_mass[turn][i], lane, m0 + (uint64_t(m1) << 14) + (uint64_t(m2) << 28));
      }
    }
  };
  Weights sums;
  uint32_t lowest = 0xffffffffu;
  if (by_count || by_mass) {
    for (int g = s.w0 + lane; g < s.w1; g += 32) {
      const uint4 v = s.granule(g);
      uint32_t below = 0;
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        const float2 z = scale.z(s.at(v, j), s.at(v, j + 1)), e = scale.e(z);
        sums.add(e.x, e.y);
        mark(below, z);
      }
      tally(below, v, g, 0);
    }
  } else {
#pragma unroll 2
    for (int g = s.w0 + lane; g < s.w1; g += 32) {
      const uint4 v = s.granule(g);
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        const float2 e = scale.e(scale.z(s.at(v, j), s.at(v, j + 1)));
        sums.add(e.x, e.y);
      }
    }
  }
  if (by_count || by_mass) send_groups();
  if (greedy && holds_top)
    for (int g = s.w0 + lane; g < s.w1 && lowest == 0xffffffffu; g += 32) {
      const uint4 v = s.granule(g);
      for (int j = kPer - 1; j >= 0; --j)
        if (s.at(v, j) == scale.top) lowest = uint32_t(s.first(g) + j);
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
    // Every CTA decides, alike, from the sums of the cluster's histograms.
    uint32_t skipped_count = 0;   // tokens above the histogram's range
    uint64_t skipped_mass = 0;
    uint32_t begin = 0;           // the histogram's first bin
    bool count_open = by_count;   // top-k still to be resolved, else top-p
    uint64_t kept_mass = total;   // of the tokens that top-k keeps
    uint32_t bin = 0;             // the bin in which the last kept token lies
    uint32_t bin_count = 0, through = 0;  // tokens before it, and with it
    uint64_t bin_mass = 0;                // weights before it
    // Finds that bin; false where it lies beyond the histogram.
    auto decide = [&] {
      if (tid == 0 && !count_open) sm.limit = threshold(double(p) * double(kept_mass), false);
      if (tid < kGroup) sm.bin_mass[tid] = 0, sm.bin_count[tid] = 0;
      __syncthreads();
      const uint64_t limit = count_open ? uint64_t(k) : sm.limit;
      // the lane's share of a scan: whether the limit is reached in it, and what lies before
      auto search = [&](uint32_t n, uint64_t m, uint32_t& count, uint64_t& mass) {
        const uint32_t to_count = count + warp_scan32(n, lane);
        const uint64_t to_mass = mass + warp_scan64(m, lane);
        const uint64_t to = count_open ? to_count : to_mass;
        const uint32_t found = __ballot_sync(0xffffffffu, to >= limit && to - (count_open ? n : m) < limit);
        const int i = found ? __ffs(int(found)) - 1 : 31;
        through = __shfl_sync(0xffffffffu, to_count, i);
        count = found ? through - __shfl_sync(0xffffffffu, n, i) : through;
        mass = __shfl_sync(0xffffffffu, found ? to_mass - m : to_mass, i);
        return found ? i : -1;
      };
      const int group = search(lane < kGroups ? sm.group_count[turn][lane] : 0,
                               lane < kGroups ? sm.group_mass[turn][lane] : 0, skipped_count, skipped_mass);
      if (group < 0) return false;
      if (warp < int(ctas)) {  // the group's bins from every CTA
        const int i = group * kGroup + lane;
        const uint32_t n = load_cluster(&sm.counts[i], warp);
        const uint32_t m0 = load_cluster(&sm.mass[0][i], warp);
        const uint32_t m1 = load_cluster(&sm.mass[1][i], warp);
        const uint32_t m2 = load_cluster(&sm.mass[2][i], warp);
        if (n) {
          atomicAdd(&sm.bin_count[lane], n);
          sum_cluster(&sm.bin_mass[lane], rank, m0 + (uint64_t(m1) << 14) + (uint64_t(m2) << 28));
        }
      }
      __syncthreads();
      bin_count = skipped_count, bin_mass = skipped_mass;
      bin = begin + group * kGroup + search(sm.bin_count[lane], sm.bin_mass[lane], bin_count, bin_mass);
      return true;
    };
    // Ranks the listed tokens by (logit, index) and takes the last kept one.
    auto resolve = [&] {
      const uint32_t n = sm.listed;
      if (tid == 0) sm.bisect = n > uint32_t(kListMost);
      if (n > uint32_t(kListMost)) return;
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
          sm.cut = {key, index};
          sm.best_mass = m + own;
        }
      }
    };
    // The whole rest, with all tokens that may be kept in the list: `per` threads a token,
    // which compare it with the others.
    auto finish_few = [&] {
      const int n = int(sm.listed);
      int per = 1;
      while (per < 32 && 2 * per * n <= kThreads) per *= 2;
      const int i = tid / per, part = tid % per;
      const bool mine = i < n;
      const uint32_t key = mine ? sm.key[i] : 0, index = mine ? sm.index[i] : 0;
      const float e = mine ? scale.e(scale.z(logit_of(key))) : 0.0f;
      const uint64_t own = weight_of(e), place = uint64_t(key) << 32 | uint32_t(~index);
      if (mine && part == 0) sm.entry[i] = {place, own};
      __syncthreads();
      uint32_t before = 0;
      uint64_t m = 0;
#pragma unroll 4
      for (int j = part; j < n; j += per) {
        const ulonglong2 other = reinterpret_cast<const ulonglong2*>(sm.entry)[j];
        if (other.x > place) ++before, m += other.y;
      }
      for (int o = 1; o < per; o *= 2) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        m += __shfl_xor_sync(0xffffffffu, m, o);
      }
      Cut last = {0, 0xffffffffu};
      if (count_open) {  // else top-k has been resolved, or keeps all that has a weight
        if (mine && before + 1 == uint32_t(k)) sm.cut = {key, index}, sm.best_mass = m + own;
        __syncthreads();
        last = sm.cut, kept_mass = sm.best_mass;
      }
      if (by_mass) {
        __syncthreads();
        if (tid == 0) sm.limit = threshold(double(p) * double(kept_mass), false);
        __syncthreads();
        if (mine && m < sm.limit && m + own >= sm.limit) sm.cut = {key, index};
        __syncthreads();
        last = sm.cut;
      }
      const bool kept = mine && !(e < floor_e) &&
                        (key > last.key || (key == last.key && index <= last.index));
      __syncthreads();
      if (mine && part == 0) sm.entry[i] = {index, kept ? own : 0};
      __syncthreads();
      uint64_t all = 0, upto = 0;
#pragma unroll 4
      for (int j = part; j < n; j += per) {
        const ulonglong2 other = reinterpret_cast<const ulonglong2*>(sm.entry)[j];
        all += other.y;
        if (other.x <= index) upto += other.y;
      }
      for (int o = 1; o < per; o *= 2) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        upto += __shfl_xor_sync(0xffffffffu, upto, o);
      }
      if (tid == 0) sm.limit = min(threshold(double(u) * double(all), true), all);
      __syncthreads();
      if (kept && part == 0 && upto >= sm.limit && upto - own < sm.limit) answer(int(index), logit_of(key));
    };
    bool found;
    for (;;) {
      found = decide();
      if (!found) {
        begin += bins;
        bins = kNextBins;
        if (by_count || begin >= kNats * kBinsPerNat) {  // every token with a weight is kept
          if (!(count_open && by_mass)) break;
          count_open = false;  // (top-k's histogram is all there is: it serves top-p too)
          bins = kBins, begin = 0, skipped_count = 0, skipped_mass = 0;
          continue;
        }
      } else {
        // no token of these bins lies below this (all rounding goes that way)
        const float lowest_logit =
            __fsub_rd(scale.top, __fdiv_ru(__fdiv_ru(float(bin + 1), per_nat), scale.inv));
        const bool few = through <= uint32_t(kFew);
        const uint32_t lowest_bin = few ? 0 : bin;
        for (int g = s.w0 + lane; g < s.w1; g += 32) {
          const uint4 v = s.granule(g);
          if (!(s.largest(v) >= lowest_logit)) continue;
          uint32_t hits = 0;
#pragma unroll
          for (int j = 0; j < kPer; ++j) hits |= uint32_t(s.at(v, j) >= lowest_logit) << j;
          for (; hits; hits &= hits - 1) {
            const int j = __ffs(int(hits)) - 1;
            const float l = clean(s.element(v, g, j));
            const uint32_t b = bin_of(scale.z(l), per_nat);
            if (b < lowest_bin || b > bin) continue;
            const uint32_t to = add_cluster(&sm.listed, 0, 1);
            if (to >= uint32_t(kListMost)) continue;
            store_cluster(&sm.key[to], 0, key_of(l));
            store_cluster(&sm.index[to], 0, uint32_t(s.first(g) + j));
          }
        }
        cluster_sync();
        if (few) {
          if (rank == 0) finish_few();
          return;
        }
        if (rank == 0) {
          resolve();
          __syncthreads();
          if (tid == 0) sm.listed = 0;
          if (tid > 0 && tid < int(ctas)) {
            store_cluster(&sm.bisect, tid, sm.bisect);
            store_cluster(&sm.cut.key, tid, sm.cut.key);
            store_cluster(&sm.cut.index, tid, sm.cut.index);
            store_cluster(&sm.best_mass, tid, sm.best_mass);
          }
        }
        cluster_sync();
        if (sm.bisect || !(count_open && by_mass)) break;
        kept_mass = sm.best_mass;  // now top-p among what top-k keeps, by a new histogram
        count_open = false;
        begin = 0, skipped_count = 0, skipped_mass = 0;
      }
      clear();
      __syncthreads();
      histogram_z = -float(begin + bins) / per_nat;
      for (int g = s.w0 + lane; g < s.w1; g += 32) {
        const uint4 v = s.granule(g);
        uint32_t below = 0;
#pragma unroll
        for (int j = 0; j < kPer; j += 2) mark(below, scale.z(s.at(v, j), s.at(v, j + 1)));
        tally(below, v, g, begin);
      }
      turn ^= 1;
      send_groups();
      cluster_sync();
    }
    if (found && !sm.bisect) {
      cut = sm.cut;
    } else if (found) {
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
                for (uint32_t c = 0; c < ctas; ++c) store_cluster(&sm.cut.index, c, uint32_t(i));
              }
              break;
            }
            run = __shfl_sync(0xffffffffu, through, 31);
          }
        }
        cluster_sync();
        cut = {key, sm.cut.index};
        if (!open || !by_mass) break;
        open = false;
        limit = threshold(double(p) * double(upto), false);
      }
    }
  }

  // 4. the token
  const float cut_logit = cut.key == 0 ? -INFINITY : logit_of(cut.key);
  auto chance = [&](float l, float e, int i) {  // 0 for a token that is not kept
    if (!(l >= cut_logit) || (l == cut_logit && uint32_t(i) > cut.index) || e < floor_e) return 0.0f;
    return e;
  };
  auto granule_sum = [&](const uint4& v, int g) {
    Weights w;
#pragma unroll
    for (int j = 0; j < kPer; j += 2) {
      const float l0 = s.at(v, j), l1 = s.at(v, j + 1);
      const float2 e = scale.e(scale.z(l0, l1));
      w.add(chance(l0, e.x, s.first(g) + j), chance(l1, e.y, s.first(g) + j + 1));
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
          const float l = s.at(v, j);
          sum += weight_of(chance(l, scale.e(scale.z(l)), i));
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
  // 512 threads a CTA while each has an SM to itself (4 mixed rows of 131072: 13.5 us, with
  // 256 threads 14.4 us, with 1024 14.9 us), else 256 and five CTAs an SM (37 rows of 50021
  // float32: 14.4 us, with 512 threads 15.5 us)
  const bool many = rows * ctas <= sms;
  const size_t fixed = many ? sizeof(SampleSmem<kManyThreads / 32>) : sizeof(SampleSmem<kFewThreads / 32>);
  const bool resident = fixed + size_t(slice) <= kSmemMost;
  const size_t smem = fixed + (resident ? size_t(slice) : 0);
  const Launch l = {rows * ctas, many ? kManyThreads : kFewThreads, smem, ctas, stream};
  void* args[] = {const_cast<SampleArgs*>(&a)};
  const char* what = "reshard_sample";
  if (many)
    return resident ? launch<sample_kernel<T, true, kManyThreads>, kSmemMost>(what, dev, l, args)
                    : launch<sample_kernel<T, false, kManyThreads>, kSmemMost>(what, dev, l, args);
  return resident ? launch<sample_kernel<T, true, kFewThreads>, kSmemMost>(what, dev, l, args)
                  : launch<sample_kernel<T, false, kFewThreads>, kSmemMost>(what, dev, l, args);
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
