// distill.cu -- reshard_distill_loss: the divergence of the student's distribution from a teacher's
// most likely tokens, and its gradient in the student's logits.
//
// With q the teacher's probabilities of its listed tokens, q_R what is left of 1 (or 0), p the
// student's and p_R its probability of all other tokens: loss = sum q_j ln(q_j / p_j) + q_R ln(q_R /
// p_R), dl = p - q for listed tokens and p (1 - q_R / p_R) for others.  A row needs the sum over its
// logits before the first gradient: it is read twice, the second time from the L2 cache, which holds
// the rows that are on the SMs (two of 256 KB each).  The second pass goes backwards through what the
// first was told to keep there, and tells it to drop what it has read.
//
// Where the rest counts, the sum R over the other tokens is held relative to their own largest logit m_R: a
// student that is sure of the listed tokens leaves the others a probability below float32's range, but
// ln p_R = (m_R - m) / T + ln R - ln S is an ordinary number, and so are the others' gradients,
// e^((l - m_R) / T) times (p_R - q_R) / R.
//
// Bound by HBM, and by the tenth of the rows that the L2 has lost by the second pass: 2048 rows of
// 131072 bf16 with 64 tokens take 191 us (158 of HBM alone, each logit read and written once; 621 MB
// read where 509 would do, 5.7 TB/s), with the rest as an outcome 204 us.  Measured and dropped: a row
// held in the shared memory of four CTAs (291 us) or two (286), whose fixed costs weigh more than a
// second read; a part of it held in one CTA's (244: it leaves the loads too little of the L1).
// 64 registers: 16-bit rows with the rest spill 16 bytes, gradients that lie otherwise on 16 bytes than
// the logits 124 to 160 (317 us, with the rest 341).
#include "vocab_row.cuh"

namespace rs {
namespace {

using namespace vocab;

constexpr int kMany = 512, kFew = 128;     // threads of a CTA: for long rows, and for short ones
constexpr int kWarpsMost = kMany / 32;
constexpr int kVecs = 4;                  // granules that a thread has on their way
constexpr int kTable = 512;               // of the list's tokens, half full at most
constexpr int kMarked = 64 * 1024;        // granules of a slice whose listed elements can be marked
constexpr int kMaxCluster = 8;
constexpr int kListWarps = RESHARD_MAX_TOP / 32;
constexpr float kShrunk = 0x1p-10f;       // of the loss's terms: they and their sum stay in float32's range
constexpr float kFarthest = 32768.0f;     // T between the row's largest logit and the others' beyond which p_R is 0
static_assert(RESHARD_MAX_TOP <= kMany && 2 * RESHARD_MAX_TOP <= kTable, "an entry a thread");

struct DistillArgs {
  const void* logits;
  int64_t vocab, ld, ldtop;
  const float* temperature;
  const int32_t* top_token;
  const float* top_logprob;
  const float* grad;
  float* loss;
  void* dlogits;
  int32_t ntop;
};

// A number as the sum of two float32, the second what the first's rounding left: 48 bits or so in
// operations that these SMs have many of, where those on float64 take a warp 16 clocks each.  Sums by
// Knuth's exact addition (The Art of Computer Programming 2, 4.2.2), combined as Dekker does (Numerische
// Mathematik 18, 1971), products with the remainder from one fused operation.  What they are made of here, S, p_R,
// a probability, 1 / T, is float32: the pairs keep the small difference of the loss's large terms.
struct Two {
  float high, low;
};
__device__ __forceinline__ Two sum_of(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  const Two s = sum_of(a.high, b.high);
  return sum_of(s.high, __fadd_rn(s.low, __fadd_rn(a.low, b.low)));
}
__device__ __forceinline__ Two operator-(Two a) { return {-a.high, -a.low}; }
__device__ __forceinline__ Two operator*(Two a, float b) {
  const float p = __fmul_rn(a.high, b);
  return sum_of(p, fmaf(a.low, b, fmaf(a.high, b, -p)));
}
// The warp's sum.
__device__ __forceinline__ Two sum_of_warp(Two v) {
  for (int o = 16; o; o >>= 1)
    v = v + Two{__shfl_xor_sync(0xffffffffu, v.high, o), __shfl_xor_sync(0xffffffffu, v.low, o)};
  return v;
}
// ln x for a positive finite x: of x = m 2^n, m from sqrt(1/2) to sqrt(2) (the usual reduction, as in Cody and
// Waite, Software Manual for the Elementary Functions, 1980), by float32's logf and n ln 2, so that it is off
// by 2^-24 of ln m and not of ln x.
__device__ __forceinline__ Two log_of(float x) {
  int n = 0;
  if (x < 0x1p-126f) x *= 0x1p32f, n = -32;
  const uint32_t b = __float_as_uint(x) - 0x3f3504f3u;  // (sqrt(1/2))
  n += int(b) >> 23;
  const float m = __uint_as_float((b & 0x7fffffu) + 0x3f3504f3u);
  return Two{0x1.62e430p-1f, -0x1.05c610p-29f} * float(n) + Two{logf(m), 0.0f};  // ln 2
}

// e^y within 2^-42 of itself, 0 below e^-87.  With y = n ln 2 + 16 s, ln 2 and 1 / 6 as pairs: e^s - 1 = s +
// s^2 / 2 + s^3 / 6 + s^4 (1 / 24 + s / 120 + ...), of which the last is 2^-21 of the whole at most and needs
// float32's digits alone, and four times e^2s - 1 = 2 (e^s - 1) + (e^s - 1)^2.
// (Float64's exponential takes a call of 37 rows of 50021 float32 0.1 to 0.3 us longer.)
__device__ __forceinline__ Two exp_of(float y) {
  if (!(y < 88.0f)) return {expf(y), 0.0f};
  if (y < -87.0f) return {0.0f, 0.0f};
  const float n = rintf(y * 1.44269504f);
  Two s = Two{y, 0.0f} + -(Two{0x1.62e430p-1f, -0x1.05c610p-29f} * n);
  s = {s.high * 0.0625f, s.low * 0.0625f};
  const float t = s.high;
  const Two square = s * t + Two{t * s.low, 0.0f}, cube = square * t + Two{square.high * s.low, 0.0f};
  const float most = square.high * square.high * fmaf(t, fmaf(t, 1.0f / 720.0f, 1.0f / 120.0f), 1.0f / 24.0f);
  const Two sixth = cube * 0x1.555556p-3f + Two{cube.high * -0x1.555556p-28f, 0.0f};
  Two e = (s + square * 0.5f) + (sixth + Two{most, 0.0f});
#pragma unroll
  for (int i = 0; i < 4; ++i) e = Two{2.0f * e.high, 2.0f * e.low} + (e * e.high + Two{e.high * e.low, 0.0f});
  e = e + Two{1.0f, 0.0f};
  const float scale = __uint_as_float(uint32_t(int(n) + 127) << 23);  // (n from -126 to 127)
  return {e.high * scale, e.low * scale};
}

// What the threads of a CTA, and the CTAs of a cluster, tell each other.
struct Shared {
  int32_t token[RESHARD_MAX_TOP];  // the teacher's list, -1 for what is no entry
  float q[RESHARD_MAX_TOP];        // its probabilities, not yet scaled to 1
  Two list_q[kListWarps];          // sums of the list's warps
  Two list_term[kListWarps];
  int32_t table[kTable];           // its tokens, by a hash: a token that stands there twice meets itself
  float list_top[kListWarps], list_e[kListWarps];
  float warp_top[kWarpsMost], warp_other[kWarpsMost];
  float part_top, part_other;      // of the CTA: its largest logit, its sum (TAIL: of other tokens)
  float rest;                      // q_R
  uint32_t again;                  // whether one does
  uint32_t endless;                // whether the loss is infinite
  uint32_t edges;                  // listed tokens among those at the row's ends, a bit a thread
};

__device__ __forceinline__ float load_far(const float* at, uint32_t rank) {
  return tc::load_cluster(tc::in_cta(staging::smem_addr(at), rank));
}
// The largest of the warp's `top`, and the sum of its `other`, each relative to its lane's top.
__device__ __forceinline__ void join(float& top, float& other, float c) {
  const float own = top;
  top = warp_max(top);
  other = warp_sum(other * exp2_of(exponent(own, top, c)));
}

static_assert(kVecs == 4, "marks of a round in a word");
// The elements of a granule that `bits` name, as -inf.
template <typename T>
__device__ __forceinline__ void hide(uint4& v, uint32_t bits) {
  T* e = reinterpret_cast<T*>(&v);
#pragma unroll
  for (int i = 0; i < Slice<T>::kPer; ++i)
    if (bits >> i & 1) e[i] = from_float<T>(-INFINITY);
}

// Dynamic shared memory (TAIL): a byte a granule whose bits say which of its elements are listed.
__device__ __forceinline__ uint64_t keep_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t drop_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint4 load_with(const uint4* at, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at), "l"(policy) : "memory");
  return v;
}

template <typename T, bool TAIL, bool ALIKE, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int kPer = Slice<T>::kPer, kWarps = kThreads / 32, kRound = kVecs * kThreads;
  extern __shared__ uint32_t marks[];
  const uint8_t* listed = reinterpret_cast<const uint8_t*>(marks);
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const uint32_t rank = tc::cluster_rank();
  const int64_t r = blockIdx.x / ctas;
  const Slice<T> row(a.logits, r, a.ld, a.vocab, int(rank), int(ctas));
  T* to = a.dlogits ? static_cast<T*>(a.dlogits) + r * a.ld : nullptr;
  const int edge = rank == 0 ? row.edge() : -1;
  // rounds of kVecs granules a thread, the next one's on their way while one is worked on
  const int rounds = (row.n + kRound - 1) / kRound;
  const uint4* from = row.granules() + tid;
  uint64_t policy;
  auto load = [&](uint4(&v)[kVecs], int i) {
    if (uint32_t(i) >= uint32_t(rounds)) return;
    const uint4* p = from + i * kRound;
    if ((i + 1) * kRound <= row.n) {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) v[j] = load_with(p + j * kThreads, policy);
    } else {
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        v[j] = Slice<T>::nothing();
        if (i * kRound + j * kThreads + tid < row.n) v[j] = load_with(p + j * kThreads, policy);
      }
    }
  };
  uint4 v[kVecs], w[kVecs];
  for (int i = tid; i < kTable; i += kThreads) sh.table[i] = -1;
  let_next_start();
  wait_for_previous();
  policy = drop_policy();  // (a row that does not count is not read again)
  load(v, 0);
  if (to) policy = keep_policy();
  if (tid == 0) sh.again = sh.edges = sh.endless = 0;
  __syncthreads();
  // the teacher's list, an entry a thread: tokens outside the vocabulary, and NaN, are none.  Every
  // warp looks for an entry by itself, so that none waits for another.
  const int k = a.ntop, list_warps = (k + 31) / 32;
  int mine = -1;
  float y = -INFINITY, y_top = -INFINITY;
  for (int i = 0; i < list_warps; ++i) {
    const int at = i * 32 + lane;
    int token = -1;
    float value = -INFINITY;
    if (at < k) {
      token = a.top_token[r * a.ldtop + at];
      value = a.top_logprob[r * a.ldtop + at];
      if (uint32_t(token) >= uint32_t(row.vocab) || !(value == value)) token = -1, value = -INFINITY;
    }
    if (i == warp) mine = token, y = value;
    y_top = fmaxf(y_top, value);
  }
  y_top = warp_max(y_top);
  auto put_zeros = [&] {
    for (int g = tid; g < row.n; g += kThreads) store_granule<ALIKE>(to + row.first + g * kPer, make_uint4(0, 0, 0, 0));
    if (edge >= 0) to[edge] = from_float<T>(0.0f);
  };
  if (!(y_top > -INFINITY)) {  // a row that does not count
    if (rank == 0 && tid == 0 && a.loss) a.loss[r] = 0.0f;
    if (to) put_zeros();
    return;
  }
  const float inverse = inverse_of(a.temperature, r), c = log2_scale(inverse);
  const uint64_t c2 = both(c);
  const int place = mine - row.first;
  const bool at_end = rank == 0 && mine >= 0 && (mine < row.head || mine >= row.last);
  const bool inside = mine >= 0 && place >= 0 && place < row.n * kPer;
  T student = from_float<T>(-INFINITY);  // its logit of this thread's entry, on its way until it is used
  if (mine >= 0) student = row.row[mine];
  const float at_edge = edge >= 0 ? row.at(edge) : -INFINITY;
  bool edge_counts = at_edge > -INFINITY;
  if (TAIL) {
    for (int i = tid; i < (row.n + 3) / 4; i += kThreads) marks[i] = 0;
    __syncthreads();
    if (inside) atomicOr(&marks[place / kPer / 4], 1u << (place / kPer % 4 * 8 + place % kPer));
    if (at_end) atomicOr(&sh.edges, 1u << (mine < row.head ? mine : mine - row.last + row.head));
    __syncthreads();
    edge_counts = edge_counts && !(sh.edges >> (tid & 31) & 1);
  }
  float q = 0.0f;
  if (warp < list_warps) {
    sh.token[tid] = mine;
    Two all = {0.0f, 0.0f};
    if (mine >= 0) {
      for (uint32_t at = uint32_t(mine) * 2654435761u >> 23;; at = (at + 1) % kTable) {  // half full at most
        const int other = atomicCAS(&sh.table[at], -1, mine);
        if (other == mine) sh.again = 1;
        if (other == mine || other == -1) break;
      }
      all = TAIL ? exp_of(y) : Two{expf(y - y_top), 0.0f};
      q = all.high;
    }
    sh.q[tid] = q;
    // in pairs where what is left of 1 counts, which can be small
    if (TAIL) all = sum_of_warp(all);
    else all.high = warp_sum(q);
    if (lane == 0) sh.list_q[warp] = all;
  }
  // the sum over all tokens, or (TAIL) those that are not listed, relative to each thread's own
  // largest logit of them
  float m = edge_counts ? at_edge : -INFINITY, other = edge_counts ? 1.0f : 0.0f;
  bool unclean = false;
  auto add = [&](uint4(&v)[kVecs], int round) {
    if (TAIL) {
      uint32_t bits = 0;  // a byte a granule
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const int g = round * kRound + j * kThreads + tid;
        if (g < row.n) bits |= uint32_t(listed[g]) << 8 * j;
      }
      if (bits)
#pragma unroll
        for (int j = 0; j < kVecs; ++j) hide<T>(v[j], bits >> 8 * j);
    }
    float largest = largest_or_nan<T>(v);
    if (!(largest < INFINITY)) {
      unclean = true;
      make_clean<T>(v);
      largest = largest_in<T>(v);
    }
    const float top = fmaxf(m, largest);
    const uint64_t minus = both(top > -INFINITY ? -top : 0.0f);
    uint64_t s2 = 0;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const T* e = reinterpret_cast<const T*>(&v[j]);
      uint64_t w[kPer / 2];
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) w[i] = exp2_both(mul2(add2(pair(pair_of(e + 2 * i)), minus), c2));
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) s2 = add2(s2, w[i]);
    }
    other = fmaf(other, exp2_of(exponent(m, top, c)), sum2(s2));
    m = top;
  };
#pragma unroll 1
  for (int i = 0; i < rounds; i += 2) {
    load(w, i + 1);
    add(v, i);
    load(v, i + 2);
    if (i + 1 < rounds) add(w, i + 1);
  }
  // the gradient goes through the row backwards: what was read last is the likeliest to be in the L2
  policy = drop_policy();
  if (to) load(v, rounds - 1);
  join(m, other, c);
  if (lane == 0) sh.warp_top[warp] = m, sh.warp_other[warp] = other;
  if (TAIL && warp < list_warps) {
    const float list_top = warp_max(clean<T>(to_float(student)));
    if (lane == 0) sh.list_top[warp] = list_top;
  }
  __syncthreads();
  const bool again = sh.again != 0;  // tokens stand there twice: what to do once, the first of them does
  bool first = mine >= 0;
  if (again)
    for (int j = 0; first && j < tid; ++j) first = sh.token[j] != mine;
  float top = lane < kWarps ? sh.warp_top[lane] : -INFINITY;
  other = lane < kWarps ? sh.warp_other[lane] : 0.0f;
  join(top, other, c);
  if (ctas > 1) {
    if (tid == 0) sh.part_top = top, sh.part_other = other;
    tc::cluster_sync();
    top = -INFINITY, other = 0.0f;
    if (lane < int(ctas)) top = load_far(&sh.part_top, lane), other = load_far(&sh.part_other, lane);
    join(top, other, c);
    tc::cluster_arrive();  // this CTA has read the others' parts
  }
  const float base = top;  // what `other` is relative to
  if (TAIL) top = fmaxf(top, warp_max(lane < list_warps ? sh.list_top[lane] : -INFINITY));
  const float x = clean<T>(to_float(student));
  const bool empty = !(top > -INFINITY);
  float sum = other, lead = 0.0f, rest = 0.0f;  // S; (p_R - q_R) / R; q_R
  if (TAIL) {
    if (warp < list_warps) {
      const float e = warp_sum(first ? exp2_of(exponent(x, top, c)) : 0.0f);
      if (lane == 0) sh.list_e[warp] = e;
    }
    if (tid == 0) {
      Two left = {1.0f, 0.0f};
      for (int i = 0; i < list_warps; ++i) left = left + -sh.list_q[i];
      // (without other tokens it has nowhere to be)
      sh.rest = left.high > 0.0f && (base - top) * inverse >= -kFarthest ? left.high + left.low : 0.0f;
    }
    __syncthreads();
    const float factor = exp2_of(exponent(base, top, c));
    sum *= factor;
    for (int i = 0; i < list_warps; ++i) sum += sh.list_e[i];
    rest = sh.rest;
    lead = factor / sum;
    if (rest > 0.0f) lead -= rest / other;
  }
  if (to && empty) {
    put_zeros();
  } else if (to) {
    const float g = a.grad ? a.grad[r] : 1.0f;
    const float slope = factor_of(g * inverse, g), scale = factor_of(TAIL ? slope * lead : slope / sum, g);
    const float from_top = base > -INFINITY ? -base : 0.0f;  // (listed tokens are written behind it, whatever comes out)
    const uint64_t A = both(scale), minus = both(from_top);
    T* begin = to + row.first;
    auto put = [&](uint4(&v)[kVecs], int round) {
      if (unclean) make_clean<T>(v);
      T* e = reinterpret_cast<T*>(v);
#pragma unroll
      for (int i = 0; i < kVecs * kPer; i += 2)
        set_pair(e + i, tc::unpack2(mul2(exp2_both(mul2(add2(pair(pair_of(e + i)), minus), c2)), A)));
      const int g0 = round * kRound + tid;
      if ((round + 1) * kRound <= row.n) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) store_granules<ALIKE>(begin + (g0 + j * kThreads) * kPer, v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          const int g = g0 + j * kThreads;
          if (g < row.n) store_granule<ALIKE>(begin + g * kPer, v[j]);
        }
      }
    };
#pragma unroll 1
    for (int i = rounds - 1; i >= 0; i -= 2) {
      load(w, i - 1);
      put(v, i);
      load(v, i - 2);
      if (i > 0) put(w, i - 1);
    }
    if (edge >= 0) to[edge] = from_float<T>(exp2_of(exponent(at_edge, -from_top, c)) * scale);
    __syncthreads();
  }
  if (warp < list_warps) {
    float all = 1.0f;  // the list's sum where it is scaled to 1
    if (!TAIL) {
      all = sh.list_q[0].high;
      for (int i = 1; i < list_warps; ++i) all += sh.list_q[i].high;
    }
    const float inv_q = 1.0f / all;
    // the CTA's listed tokens, behind what was just written for them as for others
    if (to && !empty && first && (inside || at_end)) {
      const float g = a.grad ? a.grad[r] : 1.0f;
      const float slope = factor_of(g * inverse, g);
      float mass = q;
      if (again)
        for (int j = tid + 1; j < k; ++j)
          if (sh.token[j] == mine) mass += sh.q[j];
      const float p = exp2_of(exponent(x, top, c)) / sum;
      to[mine] = from_float<T>(slope * (p - mass * inv_q));
    }
    if (rank == 0 && a.loss) {
      // q (ln q - ln p) = q ((y - ln of the list's sum) - (z - ln S))
      Two term = {0.0f, 0.0f};
      const float scaled = q * inv_q;
      if (mine >= 0 && !(scaled <= 0.0f)) {
        const Two z = sum_of(x, -top) * inverse, ln_q = sum_of(y, TAIL ? 0.0f : -y_top);
        if (z.high > -INFINITY) term = ((ln_q + -z) + (log_of(sum) + -log_of(all))) * (scaled * kShrunk);
        else sh.endless = 1;
      }
      term = sum_of_warp(term);
      if (lane == 0) sh.list_term[warp] = term;
    }
  }
  if (ctas > 1) tc::cluster_wait();
  if (rank != 0 || !a.loss) return;
  __syncthreads();
  if (tid == 0) {
    Two loss = sh.list_term[0];
    for (int i = 1; i < list_warps; ++i) loss = loss + sh.list_term[i];
    if (rest > 0.0f)
      loss = loss + (log_of(rest) + (log_of(sum) + -log_of(other)) + -(sum_of(base, -top) * inverse)) * (rest * kShrunk);
    a.loss[r] = empty || sh.endless ? INFINITY : (loss.high + loss.low) * (1.0f / kShrunk);
  }
}

template <typename T, int kThreads>
reshard_status_t launch_threads(const DistillArgs& a, bool tail, int64_t rows, int ctas, int dev, cudaStream_t stream) {
  const int64_t granules = a.vocab * int64_t(sizeof(T)) / 16;
  void* args[] = {const_cast<DistillArgs*>(&a)};
  const char* what = "reshard_distill_loss";
  const size_t smem = tail ? size_t(cdiv(cdiv(granules, ctas), 4) * 4) : 0;
  const Launch l = {rows * ctas, kThreads, smem, ctas, stream, true};
  // whether logits and gradients lie alike on 16 bytes
  if ((reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.dlogits)) % 16 == 0 || !a.dlogits)
    return tail ? launch<distill_kernel<T, true, true, kThreads>, kMarked>(what, dev, l, args)
                : launch<distill_kernel<T, false, true, kThreads>, 0>(what, dev, l, args);
  return tail ? launch<distill_kernel<T, true, false, kThreads>, kMarked>(what, dev, l, args)
              : launch<distill_kernel<T, false, false, kThreads>, 0>(what, dev, l, args);
}

template <typename T>
reshard_status_t launch_distill(const DistillArgs& a, bool tail, int64_t rows, int dev, int sms,
                                cudaStream_t stream) {
  // CTAs a row: more than one while an eighth of the SMs would stay without one, and a slice has 32 KiB
  // or more (64 rows of 9000 bf16: 4.9 us, with slices of 8 KiB 6.8); or where one could not mark its
  // elements
  const int64_t granules = a.vocab * int64_t(sizeof(T)) / 16;
  int ctas = 1;
  while (ctas < kMaxCluster && (granules > ctas * int64_t(kMarked) ||
                                (rows * ctas * 8 < int64_t(sms) * 7 && granules > ctas * 2048)))
    ctas *= 2;
  static_assert(RESHARD_MAX_VOCAB / 4 <= kMaxCluster * kMarked, "marks of a slice");
  // short rows in small CTAs, of which an SM has more (4000 rows of 300 bf16: 21 us, in CTAs of 512
  // threads 70)
  return granules <= kVecs * kFew * 2 && a.ntop <= kFew
             ? launch_threads<T, kFew>(a, tail, rows, ctas, dev, stream)
             : launch_threads<T, kMany>(a, tail, rows, ctas, dev, stream);
}

}  // namespace
}  // namespace rs

using rs::fail;

extern "C" reshard_status_t reshard_distill_loss(const void* logits, int32_t dtype, int64_t rows,
                                                 int64_t vocab, int64_t ld, const float* temperature,
                                                 const int32_t* top_token, const float* top_logprob,
                                                 int32_t ntop, int64_t ldtop, int32_t tail,
                                                 const float* grad, float* loss, void* dlogits,
                                                 void* stream) {
  rs::TraceRange trace("op.distill_loss");
  if (!rs::op::float_dtype(dtype))
    return fail(RESHARD_ERR_INVALID_ARG, "dtype must be BF16, FP16 or FP32");
  if (rows < 0 || vocab < 0 || ntop < 1) return fail(RESHARD_ERR_INVALID_ARG, "negative size or ntop < 1");
  if (vocab > RESHARD_MAX_VOCAB) return fail(RESHARD_ERR_UNSUPPORTED, "vocabulary too large");
  if (ntop > RESHARD_MAX_TOP) return fail(RESHARD_ERR_UNSUPPORTED, "more tokens than RESHARD_MAX_TOP");
  if (rows >= int64_t(1) << 28) return fail(RESHARD_ERR_UNSUPPORTED, "2^28 rows or more");
  if (ld < vocab || ldtop < ntop) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (rows == 0) return RESHARD_OK;
  if (vocab == 0) {
    if (!loss) return RESHARD_OK;
    if (!rs::op::aligned(loss, 4)) return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
    const cudaError_t ce = cudaMemsetAsync(loss, 0, size_t(4 * rows), static_cast<cudaStream_t>(stream));
    return ce == cudaSuccess
               ? RESHARD_OK
               : fail(RESHARD_ERR_CUDA, std::string("reshard_distill_loss: ") + cudaGetErrorString(ce));
  }
  if (!logits || !top_token || !top_logprob) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  const int64_t size = rs::op::dtype_size(dtype);
  if (!rs::op::aligned(logits, size) || !rs::op::aligned(dlogits, size) || !rs::op::aligned(temperature, 4) ||
      !rs::op::aligned(top_token, 4) || !rs::op::aligned(top_logprob, 4) || !rs::op::aligned(grad, 4) ||
      !rs::op::aligned(loss, 4))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  if (!loss && !dlogits) return RESHARD_OK;
  int dev = 0, sms = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(ce));
  const rs::DistillArgs a = {
      logits, vocab, ld, ldtop, temperature, top_token, top_logprob, grad, loss, dlogits, ntop};
  return rs::op::by_dtype(dtype, [&](auto t) {
    return rs::launch_distill<decltype(t)>(a, tail != 0, rows, dev, sms, static_cast<cudaStream_t>(stream));
  });
}
