// balance.cu -- reshard_balance_loss: the router's load-balance loss, the tokens each
// expert got, and the gradient in the router's logits.
//
// The loss is linear in each token's scores with weights f that depend on the choices
// alone, so with d_t = sum_e f_e p_te it is a sum of d_t, and the gradient needs d_t and
// the token's own scores: once the choices are counted, one pass over the logits gives
// both, and nothing of the size of the experts is summed over tokens.  Two kernels: the
// counts (a cluster a sequence, or several), and the pass, whose first logits are loaded
// while the counts are still being made.
//
// Bound by instructions (18 for the 32 logits of a warp, 70% of the issue slots) before
// HBM: 64 sequences of 8192 tokens and 256 experts in bf16 take 110 us (4.9 TB/s, reads and
// writes), 16 of them 37 us, 35 us with padding; of that the counts are 7 us.  In float32 16 of
// them take 59 us (4.6 TB/s).
#include <type_traits>

#include "operators.cuh"
#include "tensor_core.cuh"

namespace rs {
namespace {

using namespace op;

constexpr int kChunk = 8;           // a pass's CTA takes whole multiples of this many tokens
constexpr int kCountCluster = 8;
constexpr int kCountThreads = 1024;

struct BalanceArgs {
  const void* logits;
  int64_t ld;
  const int32_t* experts;
  const uint8_t* mask;
  const float* grad;
  float* loss;
  int32_t* counts;
  void* dlogits;
  int32_t* tokens;  // workspace: [nseq] tokens with mask
  float* parts;     // [nseq * chunks] the pass's sums over tokens
  uint32_t* done;   // CTAs of the pass that have written theirs
  int32_t* live;    // sequences that have tokens, where there are many, else NULL
  int32_t nseq, seqlen, topk;
  int32_t chunk, chunks;            // tokens of a pass's CTA, CTAs of a sequence
  int32_t clusters;                 // of the counts of a sequence
  int32_t nexperts;
  float coef;
};

// Counts a sequence's choices: every CTA of a cluster counts its share of the tokens in
// shared memory, then adds up the cluster's counts of its share of the experts.  With one
// cluster a sequence the sums are the result; several add theirs to zeros.
__global__ void __launch_bounds__(kCountThreads) count_kernel(const __grid_constant__ BalanceArgs a) {
  extern __shared__ int32_t counted[];  // [nexperts + 1]: the last one counts tokens
  let_next_start();
  const int bins = a.nexperts + 1;
  for (int i = threadIdx.x; i < bins; i += kCountThreads) counted[i] = 0;
  __syncthreads();
  const uint32_t rank = tc::cluster_rank();
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int part = blockIdx.x % (ctas * a.clusters), s = blockIdx.x / (ctas * a.clusters);
  const int parts = int(ctas) * a.clusters;
  const uint32_t t0 = uint32_t(int64_t(a.seqlen) * part / parts);
  const uint32_t t1 = uint32_t(int64_t(a.seqlen) * (part + 1) / parts);
  const bool fours = a.topk % 4 == 0 && reinterpret_cast<uintptr_t>(a.experts) % 16 == 0;
  auto count = [&](int e) {
    if (uint32_t(e) < uint32_t(a.nexperts)) atomicAdd(&counted[e], 1);
  };
  int live = 0;
  // (unsigned: a step beyond the last of nearly 2^31 tokens)
  for (uint32_t i = t0 + threadIdx.x; i < t1; i += kCountThreads) {
    const int64_t t = int64_t(s) * a.seqlen + i;
    const int32_t* e = a.experts + t * a.topk;
    int4 first = {}, second = {};  // on their way while the mask is
    if (fours) {
      first = __ldg(reinterpret_cast<const int4*>(e));
      if (a.topk > 4) second = __ldg(reinterpret_cast<const int4*>(e + 4));
    }
    if (a.mask && !a.mask[t]) continue;
    ++live;
    if (fours) {
      count(first.x), count(first.y), count(first.z), count(first.w);
      if (a.topk > 4) count(second.x), count(second.y), count(second.z), count(second.w);
      for (int j = 8; j < a.topk; j += 4) {
        const int4 v = __ldg(reinterpret_cast<const int4*>(e + j));
        count(v.x), count(v.y), count(v.z), count(v.w);
      }
    } else {
      for (int j = 0; j < a.topk; ++j) count(e[j]);
    }
  }
  live = __reduce_add_sync(0xffffffffu, live);
  if (threadIdx.x % 32 == 0) atomicAdd(&counted[a.nexperts], live);
  __syncthreads();
  tc::cluster_sync();
  for (int i = int(rank * kCountThreads + threadIdx.x); i < bins; i += int(ctas) * kCountThreads) {
    const uint32_t at = staging::smem_addr(&counted[i]);
    int sum = 0;
    for (uint32_t r = 0; r < ctas; ++r)
      sum += __float_as_int(tc::load_cluster(tc::in_cta(at, r)));
    int32_t* to = i < a.nexperts ? &a.counts[int64_t(s) * a.nexperts + i] : &a.tokens[s];
    if (a.live && i == a.nexperts && sum) atomicAdd(a.live, 1);
    if (a.clusters == 1) *to = sum;
    else if (sum) atomicAdd(to, sum);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
  __syncthreads();
  tc::cluster_sync();  // no CTA's shared memory goes away under a reader
}

// A token's scores before they are divided by their sum, two at a time: exp(l - top), or
// 1 / (1 + exp(-l)).  Exponentials are 2^x, x = log2(e) z rounded to float32, which alone would put
// them off by up to 2^-24 |z| beside the 2 units in the last place of 2^x.  For float32 logits 2^x is
// multiplied by 1 + t, t = z - x ln 2 what the rounding left: then it is off by 5 units in the last
// place at most.  For 16-bit logits it is not: their gradients are rounded to 2^-9 or 2^-12, and the
// loss is a mean over tokens of errors of either sign.  Scores below 2^-126 are 0.
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t both(float v) {
  return tc::pack2(__float_as_uint(v), __float_as_uint(v));
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  return tc::pack2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum2(uint64_t v) {
  const float2 f = tc::unpack2(v);
  return f.x + f.y;
}
// z within bounds outside which e^z is 0, or 1 / (1 + e^z) below 2^-126 (a NaN stays one), so
// that x and t are finite.
__device__ __forceinline__ float at_least(float z, float low) {
  float v;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(z), "f"(low));
  return v;
}
__device__ __forceinline__ float at_most(float z, float high) {
  float v;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(z), "f"(high));
  return v;
}
template <int SCORE, bool FLOAT32>
struct Score {
  __device__ static uint64_t exp_of(uint64_t z) {
    if (FLOAT32) {
      float2 v = tc::unpack2(z);
      if (SCORE == RESHARD_SCORE_SIGMOID) v = make_float2(at_most(v.x, 88.0f), at_most(v.y, 88.0f));
      z = pair(at_least(v.x, -200.0f), at_least(v.y, -200.0f));
    }
    const uint64_t x = mul2(z, both(kLog2E));
    const float2 f = tc::unpack2(x);
    const uint64_t e = pair(exp2_of(f.x), exp2_of(f.y));
    return FLOAT32 ? tc::fma2(e, tc::fma2(x, both(-kLn2), z), e) : e;
  }
  __device__ static uint64_t inverse(uint64_t v) {
    const float2 d = tc::unpack2(v);
    float r0, r1;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d.y));
    return pair(r0, r1);
  }
  // What is kept of two logits: their scores, or exp(-l), from which a score a = 1 / (1 + exp(-l))
  // and 1 - a = exp(-l) a are made without the digits that 1 - a loses where a is nearly 1
  // (16-bit gradients have not got them).
  static constexpr bool kExp = SCORE == RESHARD_SCORE_SIGMOID && FLOAT32;
  __device__ static uint64_t of(float l0, float l1, float top) {
    if (SCORE == RESHARD_SCORE_SOFTMAX) return exp_of(add2(pair(l0, l1), both(-top)));
    const uint64_t e = exp_of(pair(-l0, -l1));
    return kExp ? e : inverse(add2(e, both(1.0f)));
  }
  __device__ static uint64_t score(uint64_t v) { return kExp ? inverse(add2(v, both(1.0f))) : v; }
  // the score's own slope: p (softmax) or p (1 - a)
  __device__ static uint64_t slope(uint64_t v) {
    const uint64_t a = score(v);
    if (SCORE == RESHARD_SCORE_SOFTMAX) return a;
    return mul2(a, kExp ? mul2(v, a) : tc::fma2(a, both(-1.0f), both(1.0f)));
  }
};

// Sequences of which each CTA of the pass counts those with tokens by itself (up to four loads a
// thread); for more the counting kernel does (262144 sequences of a token: 103 ms when each
// CTA went through all of them).
constexpr int kManySequences = 1024;

// What a CTA of the pass needs of the counts: f[e] in shared memory, and the loss's share
// of a token.
struct Weighting {
  float share, inv_tokens;
  int sequences;  // that have tokens
  __device__ void make(const BalanceArgs& a, int s, float* f) {
    __shared__ int live;
    if (threadIdx.x == 0) live = 0;
    const int n = max(a.tokens[s], 1);
    const int32_t* counts = a.counts + int64_t(s) * a.nexperts;
    const int first = int(threadIdx.x) < a.nexperts ? counts[threadIdx.x] : 0;
    __syncthreads();
    int mine = 0;
    if (!a.live)
      for (int i = threadIdx.x; i < a.nseq; i += blockDim.x) mine += a.tokens[i] > 0;
    else if (threadIdx.x == 0)
      mine = *a.live;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (threadIdx.x % 32 == 0 && mine) atomicAdd(&live, mine);
    const float per_count = float(a.nexperts) / (float(a.topk) * float(n));
    if (int(threadIdx.x) < a.nexperts) f[threadIdx.x] = float(first) * per_count;
    for (int e = threadIdx.x + blockDim.x; e < a.nexperts; e += blockDim.x)
      f[e] = float(counts[e]) * per_count;
    __syncthreads();
    inv_tokens = 1.0f / float(n);
    sequences = live;
    share = a.coef / float(max(live, 1)) / float(n) * (a.grad ? *a.grad : 1.0f);
  }
};

// The CTA's sum over its tokens, and in the last CTA of the launch the loss: all parts in
// one fixed order.
__device__ void finish(const BalanceArgs& a, float sum, float inv_tokens, int live) {
  __shared__ float sums[8];
  __shared__ double total[8];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += sums[w];
    a.parts[blockIdx.x] = sum * inv_tokens;
    __threadfence();
    last = atomicAdd(a.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last || !a.loss) return;
  __threadfence();
  double mine = 0.0;
  for (uint32_t i = threadIdx.x; i < gridDim.x; i += 256) mine += double(__ldcg(a.parts + i));
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) total[warp] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) mine += total[w];
    *a.loss = float(mine * double(a.coef) / double(max(live, 1)));
  }
}

// Two values at once.
__device__ __forceinline__ void set_pair(float* to, float2 x) { to[0] = x.x, to[1] = x.y; }
__device__ __forceinline__ void set_pair(__nv_bfloat16* to, float2 x) {
  *reinterpret_cast<__nv_bfloat162*>(to) = __float22bfloat162_rn(x);
}
__device__ __forceinline__ void set_pair(__half* to, float2 x) {
  *reinterpret_cast<__half2*>(to) = __float22half2_rn(x);
}

// A token's logits as a lane holds them: N values, read 16 bytes at a time (VEC: every row
// starts on 16 bytes and ends with a vector) or element by element, neighbouring lanes
// next to each other either way.  Values beyond the experts, and all of a token that does
// not count, are -inf: scores and gradients 0.
template <typename T, bool VEC, int N>
struct Logits {
  static constexpr int kPer = VEC ? 16 / int(sizeof(T)) : 1;
  alignas(16) T v[N];
  // the expert of value i
  __device__ static int expert(int i, int lane, int lanes) {
    return (lane + i / kPer * lanes) * kPer + i % kPer;
  }
  __device__ void load(const T* row, bool on, int lane, int lanes, int experts) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = expert(i, lane, lanes);
      if (on && e < experts) v[i] = row[e];
    }
  }
  __device__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = from_float<T>(-INFINITY);
  }
  __device__ float largest() const { return largest_of(v); }
  __device__ void set(int i, float2 x) { set_pair(v + i, x); }  // values i and i + 1
  __device__ void store(T* row, int lane, int lanes, int experts) const {
#pragma unroll
    for (int i = 0; i < N; i += kPer) {
      const int e = expert(i, lane, lanes);
      if (e >= experts) continue;
      if (VEC) __stcs(reinterpret_cast<uint4*>(row + e), *reinterpret_cast<const uint4*>(v + i));
      else row[e] = v[i];
    }
  }
};

// The pass: a token a group of `lanes` lanes, N logits a lane in registers.  While a token
// is worked on the kAhead next ones are on their way (32 KiB a CTA: registers alone kept
// too little of the memory busy), one where rows are not aligned.
constexpr int kAhead = 4;
template <typename T, int SCORE, bool VEC, int N>
__global__ void __launch_bounds__(256, N <= 16 ? 3 : 2)
    balance_kernel(const __grid_constant__ BalanceArgs a, const int lanes) {
  using L = Logits<T, VEC, N>;
  using S = Score<SCORE, std::is_same<T, float>::value>;
  const int s = blockIdx.x / a.chunks;
  // tokens are unsigned: the last chunk's end, and those fetched ahead, may lie beyond 2^31
  const uint32_t first = blockIdx.x % a.chunks * a.chunk;
  const uint32_t end = min(uint32_t(a.seqlen), first + a.chunk);
  const int lane = threadIdx.x & (lanes - 1), groups = 256 / lanes;
  const int64_t row0 = int64_t(s) * a.seqlen;
  const T* logits = static_cast<const T*>(a.logits) + row0 * a.ld;
  T* dlogits = a.dlogits ? static_cast<T*>(a.dlogits) + row0 * a.ld : nullptr;
  auto live = [&](uint32_t t) { return t < end && (!a.mask || a.mask[row0 + t] != 0); };
  uint32_t t = first + threadIdx.x / lanes;
  // VEC: a ring of kAhead tokens' vectors in shared memory, each thread's own
  extern __shared__ __align__(16) float dynamic[];
  constexpr int kVectors = VEC ? N / L::kPer : 1;
  uint4* ring = reinterpret_cast<uint4*>(dynamic) + threadIdx.x;  // [kAhead][kVectors][256]
  float* f_smem = dynamic + (VEC ? kAhead * kVectors * 256 * 4 : 0);
  // (zeros for a token that does not count; what lies beyond the experts stays -inf)
  auto fetch = [&](uint32_t t, bool on, int slot) {
    const T* row = logits + int64_t(on ? t : first) * a.ld;
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const int e = L::expert(i * L::kPer, lane, lanes);
      if (e < a.nexperts)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         staging::smem_addr(ring + (slot * kVectors + i) * 256)),
                     "l"(row + e), "r"(on ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  L next;
  next.clear();
  if (VEC && lanes * N > a.nexperts) {
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
      if (L::expert(i * L::kPer, lane, lanes) >= a.nexperts)
        for (int d = 0; d < kAhead; ++d)
          ring[(d * kVectors + i) * 256] = *reinterpret_cast<const uint4*>(next.v + i * L::kPer);
  }
  bool on = live(t);       // whether token t counts, and (VEC) the kAhead ones after it
  uint32_t ahead = 0;
  bool coming = false;     // the one after those: read an iteration before it is needed
  if (VEC) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const bool counts = live(t + d * groups);
      ahead |= uint32_t(counts) << d;
      fetch(t + d * groups, counts, d);
    }
    coming = live(t + kAhead * groups);
  } else {
    next.load(logits + int64_t(t) * a.ld, on, lane, lanes, a.nexperts);
  }
  wait_for_previous();
  Weighting w;
  w.make(a, s, f_smem);
  uint64_t f[N / 2];
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const int e0 = L::expert(i, lane, lanes), e1 = L::expert(i + 1, lane, lanes);
    f[i / 2] = pair(e0 < a.nexperts ? f_smem[e0] : 0.0f, e1 < a.nexperts ? f_smem[e1] : 0.0f);
  }
  float sum = 0.0f;
  int slot = 0;
  // the groups of a warp walk together: the shuffles need all lanes
  for (uint32_t base = first; base < end; base += groups, t += groups) {
    L now;
    bool counts = on;
    if (VEC) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      counts = ahead & 1;
#pragma unroll
      for (int i = 0; i < kVectors; ++i)
        *reinterpret_cast<uint4*>(now.v + i * L::kPer) = ring[(slot * kVectors + i) * 256];
      fetch(t + kAhead * groups, coming, slot);
      ahead = ahead >> 1 | uint32_t(coming) << (kAhead - 1);
      coming = live(t + (kAhead + 1) * groups);
      slot = slot + 1 == kAhead ? 0 : slot + 1;
    } else {
      now = next;
      on = live(t + groups);
      next.clear();
      next.load(logits + int64_t(t + groups) * a.ld, on, lane, lanes, a.nexperts);
    }
    L grad;
    if (__any_sync(0xffffffffu, counts)) {
      uint64_t p[N / 2], total2 = both(0.0f), dot2 = both(0.0f);
      float top = 0.0f;
      if (SCORE == RESHARD_SCORE_SOFTMAX) {
        top = now.largest();
        for (int o = lanes / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top == -INFINITY) top = 0.0f;  // all scores 0
      }
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        p[i / 2] = S::of(to_float(now.v[i]), to_float(now.v[i + 1]), top);
        const uint64_t score = S::score(p[i / 2]);
        total2 = add2(total2, score);
        dot2 = tc::fma2(score, f[i / 2], dot2);
      }
      float total = sum2(total2), dot = sum2(dot2);
      for (int o = lanes / 2; o; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      dot *= inv;
      if (counts && lane == 0) sum += dot;
      const float each = counts ? w.share * inv : 0.0f;
      const uint64_t scale = both(each), minus_dot = both(-each * dot);
#pragma unroll
      for (int i = 0; i < N; i += 2)
        grad.set(i, tc::unpack2(mul2(S::slope(p[i / 2]), tc::fma2(f[i / 2], scale, minus_dot))));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) grad.v[i] = from_float<T>(0.0f);
    }
    if (dlogits && t < end) grad.store(dlogits + int64_t(t) * a.ld, lane, lanes, a.nexperts);
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  finish(a, sum, w.inv_tokens, w.sequences);
}

// A token's loss (before its sequence's share) and gradient by a warp, the row read again for
// each question; f_of(e) is the weight f of expert e.
template <typename T, int SCORE, typename F>
__device__ __forceinline__ float token_by_warp(const T* l, T* d, int experts, float share, F&& f_of) {
  using S = Score<SCORE, std::is_same<T, float>::value>;
  const int lane = threadIdx.x & 31;
  float top = 0.0f, total = 0.0f, dot = 0.0f;
  if (SCORE == RESHARD_SCORE_SOFTMAX) {
    top = -INFINITY;
    for (int e = lane; e < experts; e += 32) top = fmaxf(top, to_float(l[e]));
    top = warp_max(top);
    if (top == -INFINITY) top = 0.0f;  // all scores 0
  }
  for (int e = lane; e < experts; e += 32) {
    const float v = tc::unpack2(S::score(S::of(to_float(l[e]), 0.0f, top))).x;
    total += v;
    dot = fmaf(v, f_of(e), dot);
  }
  total = warp_sum(total);
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  dot = warp_sum(dot) * inv;
  if (d != nullptr)
    for (int e = lane; e < experts; e += 32) {
      const uint64_t v = S::of(to_float(l[e]), 0.0f, top);
      d[e] = from_float<T>(share * inv * tc::unpack2(S::slope(v)).x * (f_of(e) - dot));
    }
  return dot;
}

// The pass for more experts than a warp's registers hold: a warp a token, which reads the row two
// or three times (the later ones from L1) and waits for each: 16 x 8192 tokens of 1100 experts in bf16
// take 292 us, of 1000 experts in registers 113 us.
template <typename T, int SCORE>
__global__ void __launch_bounds__(256) balance_many_kernel(const __grid_constant__ BalanceArgs a) {
  extern __shared__ float f_smem[];
  const int s = blockIdx.x / a.chunks;
  const int first = blockIdx.x % a.chunks * a.chunk;
  const int end = min(a.seqlen, first + a.chunk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_previous();
  Weighting w;
  w.make(a, s, f_smem);
  float sum = 0.0f;
  for (int i = first + warp; i < end; i += 8) {
    const int64_t t = int64_t(s) * a.seqlen + i;
    T* d = a.dlogits ? static_cast<T*>(a.dlogits) + t * a.ld : nullptr;
    if (a.mask && !a.mask[t]) {
      if (d)
        for (int e = lane; e < a.nexperts; e += 32) d[e] = from_float<T>(0.0f);
      continue;
    }
    sum += token_by_warp<T, SCORE>(static_cast<const T*>(a.logits) + t * a.ld, d, a.nexperts, w.share,
                                   [&](int e) { return f_smem[e]; });
  }
  finish(a, lane == 0 ? sum : 0.0f, w.inv_tokens, w.sequences);
}

// Counts, loss and gradient of few tokens by one CTA, a warp a token: one launch instead of
// two, the second of which waits for the first (61 tokens of 19 experts: 12.3 -> 6.3 us).
constexpr int kSmallThreads = 1024;
constexpr int64_t kSmallCounts = 4096, kSmallChoices = 8192;
// The CTA's warps go through the tokens in rounds, each as long as 3 + experts / 32 steps:
// 61 tokens of 19 experts (8 steps) take 6.3 us, 128 of 64 (20) 10.3 us, 128 of 256 (44) 12.4
// us; the two kernels 10.3 us and more.
inline bool small_enough(int64_t tokens, int64_t experts) {
  return cdiv(tokens, kSmallThreads / 32) * (cdiv(experts, 32) + 3) <= 16;
}

template <typename T, int SCORE>
__global__ void __launch_bounds__(kSmallThreads) balance_small_kernel(const __grid_constant__ BalanceArgs a) {
  extern __shared__ int32_t counted[];  // [nseq][nexperts], then the tokens of each sequence
  __shared__ float sums[kSmallThreads / 32];
  __shared__ int live;
  int32_t* tokens = counted + a.nseq * a.nexperts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bins = a.nseq * a.nexperts, count = a.nseq * a.seqlen;
  for (int i = threadIdx.x; i < bins + a.nseq; i += kSmallThreads) counted[i] = 0;
  if (threadIdx.x == 0) live = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < count * a.topk; i += kSmallThreads) {
    const int t = i / a.topk, s = t / a.seqlen;
    if (a.mask && !a.mask[t]) continue;
    const int e = a.experts[i];
    if (uint32_t(e) < uint32_t(a.nexperts)) atomicAdd(&counted[s * a.nexperts + e], 1);
    if (i == t * a.topk) atomicAdd(&tokens[s], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < bins; i += kSmallThreads) a.counts[i] = counted[i];
  for (int i = threadIdx.x; i < a.nseq; i += kSmallThreads)
    if (tokens[i] > 0) atomicAdd(&live, 1);
  __syncthreads();
  const float share = a.coef / float(max(live, 1)) * (a.grad ? *a.grad : 1.0f);
  float sum = 0.0f;
  for (int t = warp; t < count; t += kSmallThreads / 32) {
    const int s = t / a.seqlen;
    T* d = a.dlogits ? static_cast<T*>(a.dlogits) + t * a.ld : nullptr;
    if (a.mask && !a.mask[t]) {
      if (d)
        for (int e = lane; e < a.nexperts; e += 32) d[e] = from_float<T>(0.0f);
      continue;
    }
    const float n = float(tokens[s]);
    const float per_count = float(a.nexperts) / (float(a.topk) * n);
    sum += token_by_warp<T, SCORE>(
               static_cast<const T*>(a.logits) + t * a.ld, d, a.nexperts, share / n,
               [&](int e) { return float(counted[s * a.nexperts + e]) * per_count; }) /
           n;
  }
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0 && a.loss) {
    for (int w = 1; w < kSmallThreads / 32; ++w) sum += sums[w];
    *a.loss = sum * a.coef / float(max(live, 1));
  }
}

int64_t header_bytes(int64_t nseq) { return cdiv(nseq * 4 + 8, 16) * 16; }  // tokens, done, live

template <typename T, int SCORE>
reshard_status_t launch_small(BalanceArgs& a, cudaStream_t stream) {
  balance_small_kernel<T, SCORE>
      <<<1, kSmallThreads, sizeof(int32_t) * size_t(a.nseq) * size_t(a.nexperts + 1), stream>>>(a);
  return launched("reshard_balance_loss");
}

constexpr const char* kWhat = "reshard_balance_loss";

template <typename T, int SCORE, bool VEC, int N>
reshard_status_t launch_values(BalanceArgs& a, int dev, int lanes, cudaStream_t stream) {
  constexpr size_t kRing = VEC ? kAhead * sizeof(T) * 256 * N : 0;
  void* args[] = {&a, &lanes};
  return launch<balance_kernel<T, SCORE, VEC, N>, kRing + sizeof(float) * 32 * N>(
      kWhat, dev, {int64_t(a.nseq) * a.chunks, 256, kRing + sizeof(float) * size_t(a.nexperts), 0, stream},
      args);
}

template <typename T, int SCORE, bool VEC>
reshard_status_t launch_lanes(BalanceArgs& a, int dev, int lanes, int values, cudaStream_t stream) {
  return values <= 8    ? launch_values<T, SCORE, VEC, 8>(a, dev, lanes, stream)
         : values <= 16 ? launch_values<T, SCORE, VEC, 16>(a, dev, lanes, stream)
                        : launch_values<T, SCORE, VEC, 32>(a, dev, lanes, stream);
}

template <typename T, int SCORE>
reshard_status_t launch_pass(BalanceArgs& a, int dev, int64_t sms, cudaStream_t stream) {
  constexpr int kPer = 16 / int(sizeof(T));
  const bool vec = a.nexperts % kPer == 0 && a.ld % kPer == 0 && aligned(a.logits, 16) &&
                   aligned(a.dlogits, 16);
  // 16 logits a lane while a warp is enough: half the shuffles a logit of 8 a lane; up to 32
  int lanes = 1;
  while (lanes < 32 && lanes * 16 < a.nexperts) lanes *= 2;
  const int values = int(cdiv(cdiv(a.nexperts, vec ? kPer : 1), lanes)) * (vec ? kPer : 1);
  // as many CTAs as are on the GPU at a time
  const int64_t target = sms * (values > 32 ? 8 : values > 16 ? 2 : 3);
  const int64_t per_seq = target / a.nseq > 1 ? target / a.nseq : 1;
  a.chunk = int32_t(cdiv(cdiv(a.seqlen, per_seq), kChunk) * kChunk);
  a.chunks = int32_t(cdiv(a.seqlen, a.chunk));
  if (values <= 32)
    return vec ? launch_lanes<T, SCORE, true>(a, dev, lanes, values, stream)
               : launch_lanes<T, SCORE, false>(a, dev, lanes, values, stream);
  void* args[] = {&a};
  return launch<balance_many_kernel<T, SCORE>, sizeof(float) * RESHARD_MAX_EXPERTS>(
      kWhat, dev, {int64_t(a.nseq) * a.chunks, 256, sizeof(float) * size_t(a.nexperts), 0, stream}, args);
}

}  // namespace
}  // namespace rs

using rs::fail;

extern "C" int64_t reshard_balance_loss_workspace(int64_t nseq, int64_t seqlen, int64_t nexperts) {
  constexpr int64_t kMost = int64_t(1) << 31;
  if (nseq < 0 || seqlen < 0 || nexperts < 0 || nseq >= kMost || seqlen >= kMost || nseq * seqlen >= kMost)
    return 0;
  return rs::header_bytes(nseq) + 4 * nseq * rs::op::cdiv(seqlen, rs::kChunk);
}

extern "C" reshard_status_t reshard_balance_loss(
    const void* logits, int32_t dtype, int64_t nseq, int64_t seqlen, int64_t nexperts, int64_t ld,
    const int32_t* experts, int64_t topk, const uint8_t* mask, int32_t score, float coef,
    const float* grad, float* loss, int32_t* counts, void* dlogits, void* workspace,
    int64_t workspace_bytes, void* stream) {
  rs::TraceRange trace("op.balance_loss");
  if (!rs::op::float_dtype(dtype))
    return fail(RESHARD_ERR_INVALID_ARG, "dtype must be BF16, FP16 or FP32");
  if (score != RESHARD_SCORE_SOFTMAX && score != RESHARD_SCORE_SIGMOID)
    return fail(RESHARD_ERR_INVALID_ARG, "unknown score");
  if (nseq < 0 || seqlen < 0 || nexperts < 0 || topk < 1)
    return fail(RESHARD_ERR_INVALID_ARG, "negative size or topk < 1");
  if (nexperts > RESHARD_MAX_EXPERTS) return fail(RESHARD_ERR_UNSUPPORTED, "too many experts");
  constexpr int64_t kMost = int64_t(1) << 31;
  if (nseq >= kMost || seqlen >= kMost || topk >= kMost || nseq * seqlen >= kMost ||
      nseq * seqlen * topk >= kMost)
    return fail(RESHARD_ERR_UNSUPPORTED, "nseq * seqlen * topk of 2^31 or more");
  if (ld < nexperts) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  const bool none = nseq == 0 || seqlen == 0 || nexperts == 0;
  if ((nseq > 0 && nexperts > 0 && !counts) || (!none && (!logits || !experts)))
    return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  const int64_t need = reshard_balance_loss_workspace(nseq, seqlen, nexperts);
  if (workspace_bytes < need || (need > 0 && (!workspace || !rs::op::aligned(workspace, 16))))
    return fail(RESHARD_ERR_INVALID_ARG, "workspace too small or not 16-byte aligned");
  if (!rs::op::aligned(logits, rs::op::dtype_size(dtype)) ||
      !rs::op::aligned(dlogits, rs::op::dtype_size(dtype)) || !rs::op::aligned(experts, 4) ||
      !rs::op::aligned(counts, 4) || !rs::op::aligned(loss, 4) || !rs::op::aligned(grad, 4))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (none) {
    cudaError_t ce = cudaSuccess;
    if (nseq > 0 && nexperts > 0) ce = cudaMemsetAsync(counts, 0, size_t(4 * nseq * nexperts), st);
    if (ce == cudaSuccess && loss) ce = cudaMemsetAsync(loss, 0, 4, st);
    if (ce != cudaSuccess)
      return fail(RESHARD_ERR_CUDA, std::string("reshard_balance_loss: ") + cudaGetErrorString(ce));
    return RESHARD_OK;
  }
  int dev = 0, sms = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(ce));
  rs::BalanceArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.experts = experts;
  a.mask = mask;
  a.grad = grad;
  a.loss = loss;
  a.counts = counts;
  a.dlogits = dlogits;
  a.tokens = static_cast<int32_t*>(workspace);
  a.done = static_cast<uint32_t*>(workspace) + nseq;
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + rs::header_bytes(nseq));
  a.nseq = int32_t(nseq);
  a.seqlen = int32_t(seqlen);
  a.topk = int32_t(topk);
  a.nexperts = int32_t(nexperts);
  a.coef = coef;
  if (rs::small_enough(nseq * seqlen, nexperts) && nseq * (nexperts + 1) <= rs::kSmallCounts &&
      nseq * seqlen * topk <= rs::kSmallChoices)
    return rs::op::by_dtype(dtype, [&](auto t) {
      using T = decltype(t);
      return score == RESHARD_SCORE_SOFTMAX ? rs::launch_small<T, RESHARD_SCORE_SOFTMAX>(a, st)
                                            : rs::launch_small<T, RESHARD_SCORE_SIGMOID>(a, st);
    });
  // the counts: a cluster a sequence, more of them for choices beyond 4096 a CTA while there
  // are SMs for them; a short sequence takes one CTA
  const int64_t choices = seqlen * topk;
  const int cluster = choices <= 2048 ? 1 : rs::kCountCluster;
  const int64_t useful = rs::op::cdiv(choices, 4096 * cluster), room = sms / (nseq * cluster);
  a.clusters = int32_t(useful < 1 || room < 1 ? 1 : useful < room ? useful : room);
  if (nseq > rs::kManySequences) {  // (a cluster a sequence then)
    a.live = static_cast<int32_t*>(workspace) + nseq + 1;
    ce = cudaMemsetAsync(a.live, 0, 4, st);
    if (ce != cudaSuccess)
      return fail(RESHARD_ERR_CUDA, std::string("reshard_balance_loss: ") + cudaGetErrorString(ce));
  }
  if (a.clusters > 1) {
    ce = cudaMemsetAsync(counts, 0, size_t(4 * nseq * nexperts), st);
    if (ce == cudaSuccess) ce = cudaMemsetAsync(a.tokens, 0, size_t(4 * nseq), st);
    if (ce != cudaSuccess)
      return fail(RESHARD_ERR_CUDA, std::string("reshard_balance_loss: ") + cudaGetErrorString(ce));
  }
  void* args[] = {&a};
  const reshard_status_t status =
      rs::op::launch<rs::count_kernel, sizeof(int32_t) * (RESHARD_MAX_EXPERTS + 1)>(
          rs::kWhat, dev,
          {nseq * a.clusters * cluster, rs::kCountThreads, sizeof(int32_t) * size_t(nexperts + 1), cluster, st},
          args);
  if (status != RESHARD_OK || !(loss || dlogits)) return status;
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return score == RESHARD_SCORE_SOFTMAX ? rs::launch_pass<T, RESHARD_SCORE_SOFTMAX>(a, dev, sms, st)
                                          : rs::launch_pass<T, RESHARD_SCORE_SIGMOID>(a, dev, sms, st);
  });
}
