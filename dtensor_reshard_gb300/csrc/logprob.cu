// logprob.cu -- reshard_logprob: the log-probability of a given token, the entropy and the most
// likely tokens of each row of logits; reshard_logprob_grad: the gradient in the logits.
//
// With z = (l - m) / T, S = sum e^z and U = sum e^z z: logprob = z_t - ln S, entropy =
// ln S - U / S.  One pass: a thread carries its own largest logit with S and U relative to it, in
// float32; differences of logits and 1 / T are rounded once each, exponentials are powers of 2.
//
// The pass is bound by HBM: 4096 rows of 131072 bf16, a tenth of which do not count, take 141 us (6.8 TB/s;
// 30000 instructions a row, 61% of the issue slots), and so is the gradient, 148 us for 2048 such rows, read
// and written (6.9 TB/s).
//
// The most likely tokens: with the pass done, the k-th largest of the threads' own largest logits is
// reached by k tokens, and by few others (77 of 131072 for k = 64); the groups of granules that reach it,
// which each thread noted, are read again, their tokens listed, and the list is ranked exactly by
// comparing all with all.  Nothing of the row's size is sorted or kept.  2048 such rows with 64 tokens: 97 us
// (71 of HBM alone: 70% of the issue slots, and a fifth of a row's time at barriers and the list), with 1
// token 90, with none 79; with 128 114, with 256 189: the more of the threads have to reach the threshold, the lower
// it lies and the more is listed and ranked.  (A threshold from the first granules alone listed 512 tokens for
// 64: 245 us.)  A row whose list overflows, as one of equal logits, goes through the histograms of list_again:
// 2048 such rows 0.79 ms.  (61 to 64 registers; float32 with alternatives spills 24 bytes.)
#include <type_traits>

#include "vocab_row.cuh"

namespace rs {
namespace {

using namespace vocab;

constexpr int kMany = 512, kSome = 256, kFewest = 128;  // threads of a CTA
constexpr int kVecs = 4;          // granules that a thread has on their way
constexpr int kMaxCluster = 8;
constexpr int kCap = 1024;        // tokens that may be among the most likely, of a CTA
constexpr int kFew = 256;         // of which so many are ranked at once
constexpr int kGroups = 32;       // groups of granules whose largest logits a thread notes
static_assert(RESHARD_MAX_TOP <= kFew && kCap >= kFew && kCap % kMany == 0, "lists");

struct LogprobArgs {
  const void* logits;
  int64_t vocab, ld, ldtop;
  const float* temperature;
  const int32_t* target;
  float *logprob, *entropy;
  int32_t* top_token;
  float* top_logprob;
  float4* state;
  int32_t ntop;
};

// What a CTA tells the others of its cluster.
struct Part {
  float top, sum, moment;  // its largest logit, S and U (in powers of 2) relative to it
  uint32_t listed;         // its most likely tokens, in order in TopSmem::best
};
struct TopSmem {
  union {
    struct {
      uint64_t listed[kCap];  // key, then ~index: the largest first
      uint32_t hit[kCap];     // groups with such tokens
    };
    uint64_t other[kMaxCluster][RESHARD_MAX_TOP];  // in the end: the lists of the cluster's CTAs
  };
  uint64_t best[RESHARD_MAX_TOP];  // the most likely of them in order
  uint32_t rank[RESHARD_MAX_TOP];  // how many tokens of other CTAs come before each
  uint32_t hist[256], count[32];
  uint32_t n, n2, digit, hits;
  uint32_t either[kMany / 32], common[kMany / 32];
};

__device__ __forceinline__ uint64_t place_of(uint32_t key, uint32_t index) {
  return uint64_t(key) << 32 | uint32_t(~index);
}
template <typename T>
__device__ __forceinline__ T load_far(const T* at, uint32_t rank) {
  const uint32_t from = tc::in_cta(staging::smem_addr(at), rank);
  if (sizeof(T) == 8) {
    uint64_t v;
    asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(from) : "memory");
    return T(v);
  }
  uint32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(from) : "memory");
  return reinterpret_cast<const T&>(v);
}

// An arrival at the cluster's barrier that orders nothing: what was read is in registers.
__device__ __forceinline__ void arrive_read() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
// Brings `bytes` (a multiple of 16) at `at`, 16-byte aligned, to the L2 cache.
__device__ __forceinline__ void prefetch(const void* at, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}

// Places for `count` entries of each lane of a warp behind the `taken` ones: one atomic a warp.
__device__ __forceinline__ uint32_t claim(uint32_t count, uint32_t* taken) {
  const int lane = threadIdx.x & 31;
  uint32_t upto = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  uint32_t base = 0;
  if (lane == 31 && upto) base = atomicAdd(taken, upto);
  return __shfl_sync(0xffffffffu, base, 31) + upto - count;
}

// Adds a token to the list; beyond its end it is only counted.
__device__ __forceinline__ void append(TopSmem& sm, float l, int index) {
  const uint32_t at = atomicAdd(&sm.n, 1u);
  if (at < uint32_t(kCap)) sm.listed[at] = place_of(key_of(l), uint32_t(index));
}
// The same for a granule of each lane of a warp (or none): its tokens that reach the threshold.
template <typename T>
__device__ __forceinline__ void append_reaching(TopSmem& sm, const uint4& v, bool there, int first, float threshold) {
  const T* e = reinterpret_cast<const T*>(&v);
  uint32_t reaching = 0;
#pragma unroll
  for (int j = 0; j < Slice<T>::kPer; ++j) reaching |= uint32_t(to_float(e[j]) >= threshold) << j;
  if (!there) reaching = 0;
  uint32_t at = claim(__popc(reaching), &sm.n);
  for (; reaching; reaching &= reaching - 1, ++at) {
    const uint32_t j = __ffs(int(reaching)) - 1, w = j * sizeof(T) / 4;
    uint32_t word = w < 2 ? (w < 1 ? v.x : v.y) : (w < 3 ? v.z : v.w);
    if (sizeof(T) == 2 && (j & 1)) word >>= 16;
    const float l = clean<T>(to_float(reinterpret_cast<const T&>(word)));
    if (at < uint32_t(kCap)) sm.listed[at] = place_of(key_of(l), uint32_t(first) + j);
  }
}

// A logit's bucket: the upper 16 bits of its key, 0 for -inf.
__device__ __forceinline__ uint32_t bucket_of(float l) { return l > -INFINITY ? key_of(l + 0.0f) >> 16 : 0; }

// A logit that at least k threads' largest reach, so that at least k tokens do: the lowest one whose
// key has the upper 16 bits that k threads' have at least, which are found bit by bit (none that all
// have alike); the lowest finite one where fewer threads have any.
template <int kThreads>
__device__ float shared_threshold(uint32_t mine, int k, uint32_t* either, uint32_t* common) {
  const uint32_t any = __reduce_or_sync(0xffffffffu, mine), all = __reduce_and_sync(0xffffffffu, mine);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) either[warp] = any, common[warp] = all;
  __syncthreads();
  const uint32_t some = __reduce_or_sync(0xffffffffu, lane < kThreads / 32 ? either[lane] : 0);
  uint32_t bucket = __reduce_and_sync(0xffffffffu, lane < kThreads / 32 ? common[lane] : 0xffffu);
  const uint32_t open = some & ~bucket;
  bucket &= ~((2u << (31 - __clz(int(open | 1)))) - 1);  // of the bits above the highest open one
#pragma unroll 1
  for (int b = 31 - __clz(int(open | 1)); b >= 0; --b)
    if (__syncthreads_count(mine >= (bucket | 1u << b)) >= k) bucket |= 1u << b;
  return bucket < 0x80 ? -kLargest : logit_of(bucket << 16);
}

// Lists the tokens that reach the threshold: of the groups that do, which are read again.  Groups are
// of 2^log2_per rounds each.  Returns whether all are listed.
template <typename T, int kThreads>
__device__ bool list_reaching(TopSmem& sm, const uint16_t* noted, const Slice<T>& row, int rounds, int log2_per,
                              float threshold) {
  const int tid = threadIdx.x, groups = rounds > 0 ? ((rounds - 1) >> log2_per) + 1 : 0;
  const uint32_t bucket = bucket_of(threshold);
  uint32_t reaching = 0;  // a bit a group
#pragma unroll 4
  for (int i = 0; i < groups; ++i) reaching |= uint32_t(noted[i * kThreads + tid] >= bucket) << i;
  uint32_t at = claim(__popc(reaching), &sm.hits);
  for (; reaching; reaching &= reaching - 1, ++at)
    if (at < uint32_t(kCap)) sm.hit[at] = uint32_t((__ffs(int(reaching)) - 1) * kThreads + tid);
  __syncthreads();
  const uint32_t hits = sm.hits;
  static_assert(kVecs == 4 && kGroups <= 32, "of a round; bits");
  const int log2_granules = log2_per + 2;  // of a group
  if (hits > uint32_t(kCap)) return false;
  const uint32_t all = hits << log2_granules;
#pragma unroll 1
  for (uint32_t w = tid; (w & ~31) < all; w += kThreads) {  // (a warp at a time)
    const uint32_t h = w < all ? sm.hit[w >> log2_granules] : 0, q = w & ((1u << log2_granules) - 1);
    const int round = (int(h / kThreads) << log2_per) + int(q / kVecs);
    const int g = (round * kVecs + int(q % kVecs)) * kThreads + int(h % kThreads);
    const bool there = w < all && round < rounds && g < row.n;
    uint4 v = Slice<T>::nothing();
    if (there) v = row.granules()[g];
    append_reaching<T>(sm, v, there, row.first + g * Slice<T>::kPer, threshold);
  }
  __syncthreads();
  return sm.n <= uint32_t(kCap);
}

// Puts the k largest of the n listed tokens (or all, if fewer) in order into sm.best.
template <int kThreads>
__device__ void rank_listed(TopSmem& sm, int n, int k) {
  const int tid = threadIdx.x;
  if (n > kFew) {
    // the k-th largest key, by its bits; what reaches it goes to the front of the list
    uint64_t mine[kCap / kThreads];
#pragma unroll
    for (int i = 0; i < kCap / kThreads; ++i) mine[i] = i * kThreads + tid < n ? sm.listed[i * kThreads + tid] : 0;
    if (tid < 32) sm.count[tid] = 0;
    if (tid == 0) sm.n2 = 0;
    __syncthreads();
    uint32_t cut = 0;
#pragma unroll 1
    for (int b = 31; b >= 0; --b) {
      const uint32_t at_least = cut | 1u << b;
      int c = 0;
#pragma unroll
      for (int i = 0; i < kCap / kThreads; ++i) c += uint32_t(mine[i] >> 32) >= at_least;
      c = __reduce_add_sync(0xffffffffu, c);
      if (tid % 32 == 0 && c) atomicAdd(&sm.count[b], uint32_t(c));
      __syncthreads();
      if (sm.count[b] >= uint32_t(k)) cut = at_least;
    }
#pragma unroll
    for (int i = 0; i < kCap / kThreads; ++i)
      if (uint32_t(mine[i] >> 32) >= cut) sm.listed[atomicAdd(&sm.n2, 1u)] = mine[i];
    __syncthreads();
    n = int(sm.n2);
  }
  // a token's rank is the number of tokens before it
  int per = 1;
  while (per < 32 && 2 * per * n <= kThreads) per *= 2;
  for (int base = 0; base < n; base += kThreads / per) {
    const int i = base + tid / per;
    if (base + (tid & ~31) / per >= n) break;  // a warp without any
    const uint64_t own = i < n ? sm.listed[i] : ~uint64_t(0);
    int before = 0;
#pragma unroll 4
    for (int j = tid % per; j < n; j += per) before += sm.listed[j] > own;
    for (int o = 1; o < per; o *= 2) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (i < n && tid % per == 0 && before < k) sm.best[before] = own;
  }
  __syncthreads();
}

// More tokens reach the threshold than the list holds, as where logits are alike: the k-th largest key
// eight bits at a time, by histograms of the CTA's tokens, and then the list anew, of tokens that
// share that key those of lowest index.
template <typename T, int kThreads>
__device__ __noinline__ void list_again(TopSmem& sm, const Slice<T> row, bool edges, int k) {
  constexpr int kPer = Slice<T>::kPer, kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The tokens in order, kThreads granules at a time: those before the first granule, the granules,
  // those behind the last.  f(index of the first, their logits) says whether that was enough.
  const int steps = (row.n + kThreads - 1) / kThreads;
  auto each = [&](auto&& f) {
#pragma unroll 1
    for (int b = edges ? -1 : 0; b < (edges ? steps + 1 : steps); ++b) {
      float l[kPer];
      int index = 0, count = 0;
      const int g = b * kThreads + tid;
      if (b < 0 || b == steps) {
        const int from = b < 0 ? 0 : row.last, to = b < 0 ? row.head : row.vocab;
        index = from + tid;
        count = index < to;
        if (count) l[0] = row.at(index);
      } else if (g < row.n) {
        const uint4 v = row.granules()[g];
        const T* e = reinterpret_cast<const T*>(&v);
        index = row.first + g * kPer;
        count = kPer;
#pragma unroll
        for (int j = 0; j < kPer; ++j) l[j] = clean<T>(to_float(e[j]));
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j >= count) l[j] = -INFINITY;
      if (f(index, l)) return;
    }
  };
  uint32_t prefix = 0, need = uint32_t(k);
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) sm.hist[i] = 0;
    __syncthreads();
    each([&](int, const float(&l)[kPer]) {
      // a warp whose tokens are all alike adds them up at once
      bool alike = true;
#pragma unroll
      for (int j = 1; j < kPer; ++j) alike = alike && l[j] == l[0];
      const float one = __shfl_sync(0xffffffffu, l[0], 0);
      if (__all_sync(0xffffffffu, alike && l[0] == one)) {
        const uint32_t key = key_of(one);
        if (lane == 0 && one > -INFINITY && (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8)))
          atomicAdd(&sm.hist[key >> shift & 255], 32u * kPer);
        return false;
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t key = key_of(l[j]);
        if (l[j] > -INFINITY && (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8)))
          atomicAdd(&sm.hist[key >> shift & 255], 1u);
      }
      return false;
    });
    __syncthreads();
    if (tid == 0) {
      uint32_t above = 0;
      int d = 255;
      while (d > 0 && above + sm.hist[d] < need) above += sm.hist[d--];
      sm.digit = uint32_t(d);
      sm.n2 = need - above;
    }
    __syncthreads();
    prefix |= sm.digit << shift;
    need = sm.n2;
    __syncthreads();
  }
  if (tid == 0) sm.n = 0;
  __syncthreads();
  uint32_t ties = 0;  // of the tokens before
  each([&](int index, const float(&l)[kPer]) {
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t key = key_of(l[j]);
      if (!(l[j] > -INFINITY)) continue;
      if (key > prefix) append(sm, l[j], index + j);
      mine += key == prefix;
    }
    uint32_t upto = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t w = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += w;
    }
    if (lane == 31) sm.hist[warp] = upto;
    __syncthreads();
    uint32_t before = ties + upto - mine;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.hist[w];
      ties += sm.hist[w];
    }
    if (mine && before < need) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (l[j] > -INFINITY && key_of(l[j]) == prefix && before++ < need) append(sm, l[j], index + j);
    }
    __syncthreads();
    const bool enough = sm.n == uint32_t(k);
    __syncthreads();
    return enough;
  });
}

template <typename T, bool TOP, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logprob_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int kPer = Slice<T>::kPer, kWarps = kThreads / 32;
  extern __shared__ __align__(16) unsigned char dynamic[];
  TopSmem& sm = *reinterpret_cast<TopSmem*>(dynamic);  // (TOP)
  __shared__ float warp_top[kWarps], warp_s[kWarps], warp_u[kWarps];
  __shared__ Part part;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const uint32_t rank = tc::cluster_rank();
  const int64_t r = blockIdx.x / ctas;
  const Slice<T> row(a.logits, r, a.ld, a.vocab, int(rank), int(ctas));
  const int k = a.ntop;
  // rounds of kVecs granules a thread, the next one's on their way while one is worked on; the first
  // CTA also has what is left at the row's ends
  constexpr int kRound = kVecs * kThreads;
  const int rounds = (row.n + kRound - 1) / kRound;
  const uint4* from = row.granules() + tid;
  auto load = [&](uint4(&v)[kVecs], int i) {
    if (i >= rounds) return;
    const uint4* p = from + i * kRound;
    if ((i + 1) * kRound <= row.n) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) v[j] = TOP ? p[j * kThreads] : __ldcs(p + j * kThreads);
    } else {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        v[j] = Slice<T>::nothing();
        if (i * kRound + j * kThreads + tid < row.n) v[j] = p[j * kThreads];
      }
    }
  };
  let_next_start();
  wait_for_previous();
  uint4 v[kVecs], w[kVecs];
  load(v, 0);
  const int target = a.target ? a.target[r] : 0;
  const float inverse = inverse_of(a.temperature, r), c = log2_scale(inverse);
  const int edge = rank == 0 ? row.edge() : -1;
  const float at_edge = edge >= 0 ? row.at(edge) : -INFINITY;
  if (uint32_t(target) >= uint32_t(row.vocab)) {  // a row that does not count
    if (rank != 0) return;
    if (tid == 0) {
      if (a.logprob) a.logprob[r] = 0.0f;
      if (a.entropy) a.entropy[r] = 0.0f;
      if (a.state) a.state[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    if (TOP)
      for (int i = tid; i < k; i += kThreads) {
        a.top_token[r * a.ldtop + i] = -1;
        a.top_logprob[r * a.ldtop + i] = -INFINITY;
      }
    return;
  }
  const uint64_t c2 = both(c);
  T chosen = from_float<T>(0.0f);  // on its way until it is used
  if (rank == 0 && tid == 0 && a.logprob) chosen = row.row[target];
  uint16_t* noted = reinterpret_cast<uint16_t*>(dynamic + sizeof(TopSmem));  // [groups][kThreads]
  int log2_per = 0;
  while (kGroups << log2_per < rounds) ++log2_per;
  uint32_t group = 0;
  int in_group = 0;
  uint16_t* note = noted + tid;
  if (TOP) {
    if (tid == 0) sm.n = sm.hits = 0;
    for (int i = tid; i < k; i += kThreads) sm.rank[i] = 0;
  }
  float m = at_edge, s = at_edge > -INFINITY ? 1.0f : 0.0f, u = 0.0f;
  auto work = [&](uint4(&g)[kVecs]) {
    float largest = largest_in<T>(g);
    if (largest == INFINITY) {
      make_finite<T>(g);
      largest = largest_finite<T>();
    }
    if (TOP) {  // what the group has reached so far
      group = max(group, bucket_of(largest));
      *note = uint16_t(group);
      if (++in_group == 1 << log2_per) in_group = 0, group = 0, note += kThreads;
    }
    const float top = fmaxf(m, largest);
    const float shift = exponent(m, top, c), factor = exp2_of(shift);
    uint64_t s2 = 0, u2 = 0;
    const uint64_t minus = both(-top);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const T* e = reinterpret_cast<const T*>(&g[j]);
#pragma unroll
      for (int q = 0; q < kPer; q += 2) {
        const uint64_t z = exponents(pair(pair_of(e + q)), minus, c2), x = exp2_both(z);
        s2 = add2(s2, x);
        u2 = tc::fma2(x, z, u2);
      }
    }
    u = fmaf(fmaf(s, shift, u), factor, sum2(u2));
    s = fmaf(s, factor, sum2(s2));
    m = top;
  };
  // Where the most likely tokens are wanted, two more rounds are on their way to the L2: while a CTA
  // ranks, the others of its SM would load too little (2048 rows of 131072 bf16 with 64 tokens: 100 us,
  // without 103.5, four rounds 106; without alternatives it costs 2%).
  auto ahead = [&](int i) {
    if (TOP && tid == 0 && (i + 3) * kRound <= row.n) prefetch(row.granules() + (i + 2) * kRound, 16 * kRound);
  };
  ahead(-1), ahead(0);
#pragma unroll 1
  for (int i = 0; i < rounds; i += 2) {
    load(w, i + 1);
    ahead(i + 1);
    work(v);
    load(v, i + 2);
    ahead(i + 2);
    if (i + 1 < rounds) work(w);
  }
  // the CTA's sums
  float top = warp_max(m);
  if (lane == 0) warp_top[warp] = top;
  __syncthreads();
  top = warp_top[0];
  for (int i = 1; i < kWarps; ++i) top = fmaxf(top, warp_top[i]);
  {
    const float shift = exponent(m, top, c), factor = exp2_of(shift);
    u = warp_sum(fmaf(s, shift, u) * factor);
    s = warp_sum(s * factor);
    if (lane == 0) warp_s[warp] = s, warp_u[warp] = u;
  }
  if (TOP) {
    const float threshold = shared_threshold<kThreads>(bucket_of(m), k, sm.either, sm.common);
    if (at_edge >= threshold) append(sm, at_edge, edge);
    if (!list_reaching<T, kThreads>(sm, noted, row, rounds, log2_per, threshold))
      list_again<T, kThreads>(sm, row, rank == 0, k);
    rank_listed<kThreads>(sm, int(sm.n), k);
  } else {
    __syncthreads();
  }
  if (tid == 0) {
    s = warp_s[0], u = warp_u[0];
    for (int i = 1; i < kWarps; ++i) s += warp_s[i], u += warp_u[i];
    part = {top, s, u, TOP ? min(sm.n, uint32_t(k)) : 0};
  }
  __syncthreads();
  // the row's
  int theirs = 0;  // the most likely tokens of CTA `lane`
  if (ctas == 1) {
    s = part.sum, u = part.moment;
  } else {
    tc::cluster_sync();
    m = -INFINITY, s = u = 0.0f;
    if (lane < int(ctas)) {
      m = load_far(&part.top, lane);
      s = load_far(&part.sum, lane);
      u = load_far(&part.moment, lane);
      if (TOP) theirs = int(load_far(&part.listed, lane));
    }
    top = warp_max(m);
    const float shift = exponent(m, top, c), factor = exp2_of(shift);
    u = warp_sum(fmaf(s, shift, u) * factor);
    s = warp_sum(s * factor);
    if (!TOP) arrive_read();
  }
  const bool empty = !(top > -INFINITY);
  const float normal = empty ? 0.0f : logf(s);
  if (rank == 0 && tid == 0) {
    const float entropy = empty ? 0.0f : fmaxf(normal - u / s * kLn2, 0.0f);
    if (a.logprob) {
      const float l = clean<T>(to_float(chosen));
      a.logprob[r] = empty || l == -INFINITY ? -INFINITY : (l == top ? 0.0f : (l - top) * inverse) - normal;
    }
    if (a.entropy) a.entropy[r] = entropy;
    if (a.state) a.state[r] = make_float4(empty ? 0.0f : top, empty ? 0.0f : 1.0f / s, normal, entropy);
  }
  if (TOP) {
    const int listed = int(part.listed);
    int all = listed;
    if (ctas > 1) {
      // a warp a list of another CTA: it is fetched, and counted before each token of this one
      all = __reduce_add_sync(0xffffffffu, theirs);
      for (int o = warp; o < int(ctas); o += kWarps) {
        const int n = __shfl_sync(0xffffffffu, theirs, o);
        if (o == int(rank)) continue;
        for (int i = lane; i < n; i += 32) sm.other[o][i] = load_far(&sm.best[i], o);
        __syncwarp();
        for (int i = lane; i < listed; i += 32) {
          const uint64_t own = sm.best[i];
          int lo = 0, hi = n;
          while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (sm.other[o][mid] > own) lo = mid + 1;
            else hi = mid;
          }
          if (lo) atomicAdd(&sm.rank[i], uint32_t(lo));
        }
      }
      arrive_read();  // this CTA has read what it needs of the others
      __syncthreads();
    }
    for (int i = tid; i < listed; i += kThreads) {
      const uint64_t own = sm.best[i];
      const int at = i + int(sm.rank[i]);
      if (at >= k) continue;
      const float l = logit_of(uint32_t(own >> 32));
      a.top_token[r * a.ldtop + at] = int32_t(~uint32_t(own));
      a.top_logprob[r * a.ldtop + at] = (l == top ? 0.0f : (l - top) * inverse) - normal;
    }
    if (rank == 0)
      for (int i = all + tid; i < k; i += kThreads) {
        a.top_token[r * a.ldtop + i] = -1;
        a.top_logprob[r * a.ldtop + i] = -INFINITY;
      }
  }
  if (ctas > 1) tc::cluster_wait();  // no CTA's shared memory goes away under a reader
}

// --------------------------------------------------------------------------- gradient
struct GradArgs {
  const void* logits;
  int64_t vocab, ld;
  const float* temperature;
  const int32_t* target;
  const float4* state;
  const float *dlogprob, *dentropy;
  void* dlogits;
  int32_t chunks;  // CTAs of a row
};

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;
// The most that A and B are, so that A + B z, z down to kLeast, is finite (1 / T can be as large as a float32).
constexpr float kMostA = 0.75f * kLargest, kMostB = kLargest / 1024;
static_assert(kMostA - kLeast * kMostB < kLargest, "A + B z");

// dl = g / T (1[target] - p) - h / T p (ln p + H), p = e^z / S: e^z times (A + B z).
template <typename T, bool ALIKE>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_kernel(const __grid_constant__ GradArgs a) {
  constexpr int kPer = Slice<T>::kPer;
  constexpr int kRound = kGradThreads * kGradVecs;
  const int64_t r = blockIdx.x / a.chunks;
  const int chunk = int(blockIdx.x % a.chunks), tid = int(threadIdx.x);
  const Slice<T> row(a.logits, r, a.ld, a.vocab, 0, 1);
  T* to = static_cast<T*>(a.dlogits) + r * a.ld;
  const int g0 = chunk * kRound + tid;
  const bool full = (chunk + 1) * kRound <= row.n;
  const int edge = chunk == 0 ? row.edge() : -1;
  let_next_start();
  wait_for_previous();
  const int target = a.target ? a.target[r] : -1;
  const float4 state = a.state[r];  // largest logit, 1 / S, ln S, entropy
  float g = a.dlogprob && a.target ? a.dlogprob[r] : 0.0f, h = a.dentropy ? a.dentropy[r] : 0.0f;
  if (state.y == 0.0f) g = h = 0.0f;  // no logit of the row counts, or the row does not
  if (g == 0.0f && h == 0.0f) {
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
      const int at = g0 + i * kGradThreads;
      if (at < row.n) store_granule<ALIKE>(to + row.first + at * kPer, make_uint4(0, 0, 0, 0));
    }
    if (edge >= 0) to[edge] = from_float<T>(0.0f);
    return;
  }
  uint4 v[kGradVecs];
  const uint4* from = row.granules() + g0;
#pragma unroll
  for (int i = 0; i < kGradVecs; ++i)
    v[i] = full || g0 + i * kGradThreads < row.n ? __ldcs(from + i * kGradThreads) : Slice<T>::nothing();
  const float at_edge = edge >= 0 ? row.at(edge) : 0.0f;
  if (largest_in<T>(v) == INFINITY) make_finite<T>(v);
  const float inverse = inverse_of(a.temperature, r), c = log2_scale(inverse);
  const float both_of = g + h;  // (NaN or infinite where one of them is)
  const float slope = inverse * state.y, onehot = factor_of(g * inverse, g, kMostA);
  const float a0 = factor_of(-(g + h * (state.w - state.z)) * slope, both_of, kMostA);
  const float b0 = factor_of(-h * slope * kLn2, h, kMostB);
  auto one = [&](float l) {
    const float z = exponent(l, state.x, c);
    return exp2_of(z) * fmaf(z, b0, a0);
  };
  const uint64_t A = both(a0), B = both(b0), minus = both(-state.x), c2 = both(c);
#pragma unroll
  for (int i = 0; i < kGradVecs; ++i) {
    const int at = g0 + i * kGradThreads;
    if (!full && at >= row.n) break;
    T* e = reinterpret_cast<T*>(&v[i]);
    const int index = row.first + at * kPer, of_target = target - index;
    float chosen = 0.0f;
    if (uint32_t(of_target) < uint32_t(kPer)) chosen = one(row.at(target)) + onehot;
#pragma unroll
    for (int q = 0; q < kPer; q += 2) {
      const uint64_t z = exponents(pair(pair_of(e + q)), minus, c2), w = exp2_both(z);
      set_pair(e + q, tc::unpack2(mul2(w, tc::fma2(z, B, A))));
    }
    if (uint32_t(of_target) < uint32_t(kPer)) {
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        if (of_target == q) e[q] = from_float<T>(chosen);
    }
    if (full) store_granules<ALIKE>(to + index, v[i]);
    else store_granule<ALIKE>(to + index, v[i]);
  }
  if (edge >= 0) to[edge] = from_float<T>(one(at_edge) + (edge == target ? onehot : 0.0f));
}

// ---------------------------------------------------------------------------- launches
template <typename T, bool TOP, int kThreads>
reshard_status_t launch_threads(const LogprobArgs& a, int64_t rows, int ctas, int dev, cudaStream_t stream) {
  const int64_t granules = a.vocab * int64_t(sizeof(T)) / 16;
  const int64_t rounds = cdiv(cdiv(granules, ctas), kVecs * kThreads);
  const size_t smem = sizeof(TopSmem) + size_t(2 * kThreads * (rounds < kGroups ? rounds : kGroups));
  void* args[] = {const_cast<LogprobArgs*>(&a)};
  return launch<logprob_kernel<T, TOP, kThreads>, TOP ? sizeof(TopSmem) + 2 * kThreads * kGroups : 0>(
      "reshard_logprob", dev, {rows * ctas, kThreads, TOP ? smem : 0, ctas, stream, true}, args);
}

template <typename T>
reshard_status_t launch_logprob(const LogprobArgs& a, int64_t rows, int dev, int sms, cudaStream_t stream) {
  // CTAs a row: more than one while an eighth of the SMs would stay without one (61 rows of 50021
  // float32, with the gradient: two CTAs a row 12.3 us, four 10.2; 37 rows with alternatives: four, for
  // 148 SMs, 9.6, eight 10.7), and a slice has 32 KiB or more (16 rows of 9000 float32: 2.9 us, with slices
  // of 8 KiB 4.1)
  const int64_t bytes = a.vocab * int64_t(sizeof(T));
  int ctas = 1;
  while (ctas < kMaxCluster && rows * ctas * 8 < int64_t(sms) * 7 && bytes > ctas * 32768) ctas *= 2;
  // short rows in small CTAs, of which an SM has more (4000 rows of 300 bf16: 10.2 us, with 20
  // alternatives 24.7; in CTAs of 256 threads 18.1 and 43.4)
  const bool is_short = bytes <= 16 * kVecs * kFewest * 2;
  if (a.ntop == 0)
    return is_short ? launch_threads<T, false, kFewest>(a, rows, ctas, dev, stream)
                    : launch_threads<T, false, kSome>(a, rows, ctas, dev, stream);
  // the most likely tokens are told apart from the others by the threads' largest logits: with
  // twice as many threads as tokens wanted, few others reach the last of those
  if (is_short && a.ntop <= kFewest / 2) return launch_threads<T, true, kFewest>(a, rows, ctas, dev, stream);
  return a.ntop <= kSome / 2 ? launch_threads<T, true, kSome>(a, rows, ctas, dev, stream)
                             : launch_threads<T, true, kMany>(a, rows, ctas, dev, stream);
}

constexpr int64_t kMostRows = int64_t(1) << 28;

// What both calls check.
reshard_status_t check(int32_t dtype, int64_t rows, int64_t vocab, int64_t ld) {
  if (!float_dtype(dtype)) return fail(RESHARD_ERR_INVALID_ARG, "dtype must be BF16, FP16 or FP32");
  if (rows < 0 || vocab < 0) return fail(RESHARD_ERR_INVALID_ARG, "negative size");
  if (vocab > RESHARD_MAX_VOCAB) return fail(RESHARD_ERR_UNSUPPORTED, "vocabulary too large");
  if (rows >= kMostRows) return fail(RESHARD_ERR_UNSUPPORTED, "2^28 rows or more");
  if (ld < vocab) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  return RESHARD_OK;
}

}  // namespace
}  // namespace rs

using rs::fail;

extern "C" reshard_status_t reshard_logprob(const void* logits, int32_t dtype, int64_t rows,
                                            int64_t vocab, int64_t ld, const float* temperature,
                                            const int32_t* target, float* logprob, float* entropy,
                                            int32_t ntop, int32_t* top_token, float* top_logprob,
                                            int64_t ldtop, float* state, void* stream) {
  rs::TraceRange trace("op.logprob");
  const reshard_status_t ok = rs::check(dtype, rows, vocab, ld);
  if (ok != RESHARD_OK) return ok;
  if (ntop < 0) return fail(RESHARD_ERR_INVALID_ARG, "negative size");
  if (ntop > RESHARD_MAX_TOP) return fail(RESHARD_ERR_UNSUPPORTED, "more alternatives than RESHARD_MAX_TOP");
  if (rows == 0) return RESHARD_OK;
  if (ntop > 0 && ldtop < ntop) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!logprob && !entropy && ntop == 0 && !state) return RESHARD_OK;
  // (without a vocabulary no row counts, and none is read)
  if ((!logits && vocab > 0) || (logprob && !target) || (ntop > 0 && (!top_token || !top_logprob)))
    return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(logits, rs::op::dtype_size(dtype)) || !rs::op::aligned(temperature, 4) ||
      !rs::op::aligned(target, 4) || !rs::op::aligned(logprob, 4) || !rs::op::aligned(entropy, 4) ||
      !rs::op::aligned(top_token, 4) || !rs::op::aligned(top_logprob, 4) || !rs::op::aligned(state, 16))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type, or state to 16 bytes");
  int dev = 0, sms = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(ce));
  const rs::LogprobArgs a = {logits,    vocab,       ld,   ldtop, temperature, target, logprob, entropy,
                             top_token, top_logprob, reinterpret_cast<float4*>(state), ntop};
  return rs::op::by_dtype(dtype, [&](auto t) {
    return rs::launch_logprob<decltype(t)>(a, rows, dev, sms, static_cast<cudaStream_t>(stream));
  });
}

extern "C" reshard_status_t reshard_logprob_grad(const void* logits, int32_t dtype, int64_t rows,
                                                 int64_t vocab, int64_t ld, const float* temperature,
                                                 const int32_t* target, const float* state,
                                                 const float* dlogprob, const float* dentropy,
                                                 void* dlogits, void* stream) {
  rs::TraceRange trace("op.logprob_grad");
  const reshard_status_t ok = rs::check(dtype, rows, vocab, ld);
  if (ok != RESHARD_OK) return ok;
  if (rows == 0 || vocab == 0) return RESHARD_OK;
  if (!logits || !state || !dlogits || (dlogprob && !target))
    return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  const int64_t size = rs::op::dtype_size(dtype);
  if (!rs::op::aligned(logits, size) || !rs::op::aligned(dlogits, size) || !rs::op::aligned(temperature, 4) ||
      !rs::op::aligned(target, 4) || !rs::op::aligned(dlogprob, 4) || !rs::op::aligned(dentropy, 4) ||
      !rs::op::aligned(state, 16))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type, or state to 16 bytes");
  rs::GradArgs a = {logits,   vocab,    ld,      temperature, target, reinterpret_cast<const float4*>(state),
                    dlogprob, dentropy, dlogits, 0};
  const bool alike = (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(dlogits)) % 16 == 0;
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    // (one at least, which has what lies at the row's ends)
    const int64_t chunks = rs::op::cdiv(vocab / rs::vocab::Slice<T>::kPer, rs::kGradThreads * rs::kGradVecs);
    a.chunks = int32_t(chunks > 1 ? chunks : 1);
    const int64_t grid = rows * a.chunks;
    if (grid >= int64_t(1) << 31) return fail(RESHARD_ERR_UNSUPPORTED, "2^31 pieces of rows or more");
    void* args[] = {&a};
    const rs::op::Launch l = {grid, rs::kGradThreads, 0, 0, static_cast<cudaStream_t>(stream)};
    const char* what = "reshard_logprob_grad";
    return alike ? rs::op::launch<rs::logprob_grad_kernel<T, true>, 0>(what, 0, l, args)
                 : rs::op::launch<rs::logprob_grad_kernel<T, false>, 0>(what, 0, l, args);
  });
}
