// logprob.cu -- reshard_logprob: the log-probability of a given token, the entropy and the most
// likely tokens of each row of logits; reshard_logprob_grad: the gradient in the logits.
//
// With z = (l - m) / T, S = sum e^z and U = sum e^z z: logprob = z_t - ln S, entropy =
// ln S - U / S.  One pass: a thread carries its own largest logit with S and U relative to it.
#include <type_traits>

#include "vocab_row.cuh"

namespace rs {
namespace {

using namespace vocab;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;          // granules that a thread has on their way
constexpr int kMaxCluster = 8;
constexpr int kCap = 4096;        // tokens that may be among the most likely, of a CTA
constexpr int kFew = 256;         // of which so many are ranked at once
static_assert(RESHARD_MAX_TOP <= kFew && kCap >= kFew, "lists");

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
  uint32_t key[kCap], index[kCap];
  uint64_t best[RESHARD_MAX_TOP];  // key, then ~index: the largest first
  uint32_t hist[256], count[32];
  uint32_t n, n2, digit;
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

// Adds a token to the list; beyond its end it is only counted.
__device__ __forceinline__ void append(TopSmem& sm, float l, int index) {
  const uint32_t at = atomicAdd(&sm.n, 1u);
  if (at < uint32_t(kCap)) sm.key[at] = key_of(l), sm.index[at] = uint32_t(index);
}

// The lowest logit of a bucket (of the upper 16 bits of a key) that at least k threads' largest
// logits reach, so that at least k tokens do; all finite logits reach the lowest.
__device__ float first_threshold(float largest, int k) {
  const uint32_t mine = largest > -INFINITY ? key_of(largest + 0.0f) >> 16 : 0;
  uint32_t bucket = 0;
#pragma unroll 1
  for (int b = 15; b >= 0; --b)
    if (__syncthreads_count(mine >= (bucket | 1u << b)) >= k) bucket |= 1u << b;
  return logit_of(max(bucket, 0x80u) << 16);
}

// Puts the k largest of the n listed tokens (or all, if fewer) in order into sm.best.
__device__ void rank_listed(TopSmem& sm, int n, int k) {
  const int tid = threadIdx.x;
  if (n > kFew) {
    // the k-th largest key, by its bits; what reaches it goes to the front of the list
    uint32_t key[kCap / kThreads], index[kCap / kThreads];
#pragma unroll
    for (int i = 0; i < kCap / kThreads; ++i) {
      const int at = i * kThreads + tid;
      key[i] = at < n ? sm.key[at] : 0;
      index[i] = at < n ? sm.index[at] : 0;
    }
    if (tid < 32) sm.count[tid] = 0;
    if (tid == 0) sm.n2 = 0;
    __syncthreads();
    uint32_t cut = 0;
#pragma unroll 1
    for (int b = 31; b >= 0; --b) {
      const uint32_t at_least = cut | 1u << b;
      int c = 0;
#pragma unroll
      for (int i = 0; i < kCap / kThreads; ++i) c += key[i] >= at_least;
      c = __reduce_add_sync(0xffffffffu, c);
      if (tid % 32 == 0 && c) atomicAdd(&sm.count[b], uint32_t(c));
      __syncthreads();
      if (sm.count[b] >= uint32_t(k)) cut = at_least;
    }
#pragma unroll
    for (int i = 0; i < kCap / kThreads; ++i) {
      if (key[i] < cut || i * kThreads + tid >= n) continue;
      const uint32_t at = atomicAdd(&sm.n2, 1u);
      sm.key[at] = key[i], sm.index[at] = index[i];
    }
    __syncthreads();
    n = int(sm.n2);
  }
  // a token's rank is the number of tokens before it
  int per = 1;
  while (per < 32 && 2 * per * n <= kThreads) per *= 2;
  for (int base = 0; base < n; base += kThreads / per) {
    const int i = base + tid / per;
    const uint64_t own = i < n ? place_of(sm.key[i], sm.index[i]) : 0;
    int before = 0;
    for (int j = tid % per; j < n; j += per) before += place_of(sm.key[j], sm.index[j]) > own;
    for (int o = 1; o < per; o *= 2) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (i < n && tid % per == 0 && before < k) sm.best[before] = own;
  }
  __syncthreads();
}

// More tokens reach the threshold than the list holds, as where a row's logits rise: the k-th
// largest key eight bits at a time, by histograms of the CTA's granules g0 to g1, and then the
// list anew, of tokens that share that key those of lowest index.
template <typename T>
__device__ void list_again(TopSmem& sm, const Row<T>& row, int g0, int g1, int k) {
  constexpr int kPer = Row<T>::kPer;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t prefix = 0, need = uint32_t(k);
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) sm.hist[tid] = 0;
    __syncthreads();
    for (int g = g0 + tid; g < g1; g += kThreads) {
      const uint4 v = row.fetch(g);
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float l = clean<T>(to_float(e[j]));
        const uint32_t key = key_of(l);
        if (l > -INFINITY && (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8)))
          atomicAdd(&sm.hist[key >> shift & 255], 1u);
      }
    }
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
  uint32_t ties = 0;  // of the granules before
  for (int b = g0; b < g1; b += kThreads) {
    const int g = b + tid;
    const uint4 v = g < g1 ? row.fetch(g) : Row<T>::nothing();
    const T* e = reinterpret_cast<const T*>(&v);
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float l = clean<T>(to_float(e[j]));
      const uint32_t key = key_of(l);
      if (!(l > -INFINITY)) continue;
      if (key > prefix) append(sm, l, row.first(g) + j);
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
      for (int j = 0; j < kPer; ++j) {
        const float l = clean<T>(to_float(e[j]));
        if (l > -INFINITY && key_of(l) == prefix && before++ < need) append(sm, l, row.first(g) + j);
      }
    }
    __syncthreads();
  }
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 2) logprob_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int kPer = Row<T>::kPer;
  extern __shared__ __align__(16) unsigned char dynamic[];
  TopSmem& sm = *reinterpret_cast<TopSmem*>(dynamic);  // (TOP)
  __shared__ float warp_top[kWarps], warp_s[kWarps], warp_u[kWarps];
  __shared__ Part part;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const uint32_t rank = tc::cluster_rank();
  const int64_t r = blockIdx.x / ctas;
  const Row<T> row(a.logits, r, a.ld, a.vocab);
  const int k = a.ntop;
  const int target = a.target ? __ldg(a.target + r) : 0;
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
  const float inverse = inverse_of(a.temperature, r), c = log2_scale(inverse);
  const uint64_t c2 = both(c);
  float chosen = 0.0f;
  if (rank == 0 && tid == 0 && a.logprob) chosen = to_float(row.row[target]);
  const int granules = row.granules();
  const int g0 = int(int64_t(granules) * rank / ctas), g1 = int(int64_t(granules) * (rank + 1) / ctas);
  // rounds of kVecs granules a thread, a round's spread evenly over the slice: the first tells
  // what the most likely tokens reach wherever they are
  const int blocks = (g1 - g0 + kThreads - 1) / kThreads, rounds = (blocks + kVecs - 1) / kVecs;
  if (TOP && tid == 0) sm.n = 0;
  float m = -INFINITY, s = 0.0f, u = 0.0f, threshold = 0.0f;
  for (int i = 0; i < rounds; ++i) {
    uint4 v[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int g = g0 + (j * rounds + i) * kThreads + tid;
      v[j] = g < g1 ? row.fetch(g) : Row<T>::nothing();
    }
    float largest = largest_in<T>(v);
    if (largest == INFINITY) {
      make_finite<T>(v);
      largest = largest_finite<T>();
    }
    if (TOP) {
      if (i == 0) threshold = first_threshold(largest, k);
      if (largest >= threshold) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          const uint4(&one)[1] = reinterpret_cast<const uint4(&)[1]>(v[j]);
          if (!(largest_in<T>(one) >= threshold)) continue;
          const T* e = reinterpret_cast<const T*>(&v[j]);
          const int at = row.first(g0 + (j * rounds + i) * kThreads + tid);
#pragma unroll
          for (int q = 0; q < kPer; ++q)
            if (to_float(e[q]) >= threshold) append(sm, to_float(e[q]) + 0.0f, at + q);
        }
      }
    }
    const float top = fmaxf(m, largest);
    const float shift = exponent(m, top, c), factor = exp2_of(shift);
    uint64_t s2 = 0, u2 = 0;
    const uint64_t minus = both(-top);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const T* e = reinterpret_cast<const T*>(&v[j]);
#pragma unroll
      for (int q = 0; q < kPer; q += 2) {
        const uint64_t z = exponents(pair(pair_of(e + q)), minus, c2), w = exp2_both(z);
        s2 = add2(s2, w);
        u2 = tc::fma2(w, z, u2);
      }
    }
    u = fmaf(fmaf(s, shift, u), factor, sum2(u2));
    s = fmaf(s, factor, sum2(s2));
    m = top;
  }
  // the CTA's sums
  float top = warp_max(m);
  if (lane == 0) warp_top[warp] = top;
  __syncthreads();
  top = warp_top[0];
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, warp_top[w]);
  {
    const float shift = exponent(m, top, c), factor = exp2_of(shift);
    u = warp_sum(fmaf(s, shift, u) * factor);
    s = warp_sum(s * factor);
    if (lane == 0) warp_s[warp] = s, warp_u[warp] = u;
  }
  if (TOP) {
    __syncthreads();
    if (sm.n > uint32_t(kCap)) list_again(sm, row, g0, g1, k);
    rank_listed(sm, int(sm.n), k);
  } else {
    __syncthreads();
  }
  if (tid == 0) {
    s = warp_s[0], u = warp_u[0];
    for (int w = 1; w < kWarps; ++w) s += warp_s[w], u += warp_u[w];
    part = {top, s, u, TOP ? min(sm.n, uint32_t(k)) : 0};
  }
  __syncthreads();
  // the row's
  if (ctas == 1) {
    s = part.sum, u = part.moment;
  } else {
    tc::cluster_sync();
    for (uint32_t o = 0; o < ctas; ++o) top = fmaxf(top, load_far(&part.top, o));
    s = u = 0.0f;
    for (uint32_t o = 0; o < ctas; ++o) {
      const float shift = exponent(load_far(&part.top, o), top, c), factor = exp2_of(shift);
      const float so = load_far(&part.sum, o);
      u = fmaf(fmaf(so, shift, load_far(&part.moment, o)), factor, u);
      s = fmaf(so, factor, s);
    }
  }
  const bool empty = !(top > -INFINITY);
  const float normal = empty ? 0.0f : logf(s);
  if (rank == 0 && tid == 0) {
    const float entropy = empty ? 0.0f : fmaxf(normal - u / s * kLn2, 0.0f);
    if (a.logprob) {
      const float l = clean<T>(chosen);
      a.logprob[r] = empty || l == -INFINITY ? -INFINITY : (l == top ? 0.0f : (l - top) * inverse) - normal;
    }
    if (a.entropy) a.entropy[r] = entropy;
    if (a.state) a.state[r] = make_float4(empty ? 0.0f : top, empty ? 0.0f : 1.0f / s, normal, entropy);
  }
  if (TOP) {
    const int listed = int(part.listed);
    int all = listed;
    if (ctas > 1) {
      all = 0;
      for (uint32_t o = 0; o < ctas; ++o) all += int(load_far(&part.listed, o));
    }
    for (int i = tid; i < listed; i += kThreads) {
      const uint64_t own = sm.best[i];
      int at = i;
      if (ctas > 1) {
        for (uint32_t o = 0; o < ctas; ++o) {
          if (o == rank) continue;
          int lo = 0, hi = int(load_far(&part.listed, o));  // tokens of that CTA before this one
          while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (load_far(&sm.best[mid], o) > own) lo = mid + 1;
            else hi = mid;
          }
          at += lo;
        }
      }
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
  if (ctas > 1) tc::cluster_sync();  // no CTA's shared memory goes away under a reader
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
  bool alike;      // logits and gradients lie alike on 16 bytes
};

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;

// dl = g / T (1[target] - p) - h / T p (ln p + H), p = e^z / S: e^z times (A + B z).
template <typename T>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_kernel(const __grid_constant__ GradArgs a) {
  constexpr int kPer = Row<T>::kPer;
  const int64_t r = blockIdx.x / a.chunks;
  const int chunk = int(blockIdx.x % a.chunks);
  const Row<T> row(a.logits, r, a.ld, a.vocab);
  T* to = static_cast<T*>(a.dlogits) + r * a.ld;
  const int first = chunk * kGradThreads * kGradVecs + int(threadIdx.x), granules = row.granules();
  const int target = a.target ? __ldg(a.target + r) : -1;
  const float4 state = __ldg(a.state + r);  // largest logit, 1 / S, ln S, entropy
  float g = a.dlogprob && a.target ? __ldg(a.dlogprob + r) : 0.0f, h = a.dentropy ? __ldg(a.dentropy + r) : 0.0f;
  if (state.y == 0.0f) g = h = 0.0f;  // no logit of the row counts, or the row does not
  if (g == 0.0f && h == 0.0f) {
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
      const int at = first + i * kGradThreads;
      if (at < granules) row.store(to, at, make_uint4(0, 0, 0, 0), a.alike);
    }
    return;
  }
  uint4 v[kGradVecs];
#pragma unroll
  for (int i = 0; i < kGradVecs; ++i) {
    const int at = first + i * kGradThreads;
    v[i] = at < granules ? row.fetch(at) : Row<T>::nothing();
  }
  if (largest_in<T>(v) == INFINITY) make_finite<T>(v);
  const float inverse = inverse_of(a.temperature, r), c = log2_scale(inverse);
  // (finite, so that 0 times one is 0)
  auto finite = [](float x) { return fmaxf(fminf(x, 3.402823466e38f), -3.402823466e38f); };
  const float slope = finite(inverse * state.y), onehot = finite(g * inverse);
  const uint64_t B = both(finite(-h * slope) * kLn2);
  const uint64_t A = both(finite(-(g + h * (state.w - state.z)) * slope));
  const uint64_t minus = both(-state.x), c2 = both(c);
#pragma unroll
  for (int i = 0; i < kGradVecs; ++i) {
    const int at = first + i * kGradThreads;
    if (at >= granules) break;
    T* e = reinterpret_cast<T*>(&v[i]);
    const int of_target = target - row.first(at);
#pragma unroll
    for (int q = 0; q < kPer; q += 2) {
      const uint64_t z = exponents(pair(pair_of(e + q)), minus, c2), w = exp2_both(z);
      float2 d = tc::unpack2(mul2(w, tc::fma2(z, B, A)));
      if (of_target == q) d.x += onehot;
      if (of_target == q + 1) d.y += onehot;
      set_pair(e + q, d);
    }
    row.store(to, at, v[i], a.alike);
  }
}

// ---------------------------------------------------------------------------- launches
template <typename T>
reshard_status_t launch_logprob(const LogprobArgs& a, int64_t rows, int dev, int sms, cudaStream_t stream) {
  // CTAs a row: more than one while SMs would stay without one, and a slice has 4 KiB or more
  const int64_t bytes = a.vocab * int64_t(sizeof(T));
  int ctas = 1;
  while (ctas < kMaxCluster && rows * ctas < sms && bytes > ctas * 8192) ctas *= 2;
  void* args[] = {const_cast<LogprobArgs*>(&a)};
  const char* what = "reshard_logprob";
  if (a.ntop > 0)
    return launch<logprob_kernel<T, true>, sizeof(TopSmem)>(
        what, dev, {rows * ctas, kThreads, sizeof(TopSmem), ctas, stream}, args);
  return launch<logprob_kernel<T, false>, 0>(what, dev, {rows * ctas, kThreads, 0, ctas, stream}, args);
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
  if (rows == 0 || vocab == 0) return RESHARD_OK;
  if (ntop > 0 && ldtop < ntop) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!logits || (logprob && !target) || (ntop > 0 && (!top_token || !top_logprob)))
    return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(logits, rs::op::dtype_size(dtype)) || !rs::op::aligned(temperature, 4) ||
      !rs::op::aligned(target, 4) || !rs::op::aligned(logprob, 4) || !rs::op::aligned(entropy, 4) ||
      !rs::op::aligned(top_token, 4) || !rs::op::aligned(top_logprob, 4) || !rs::op::aligned(state, 16))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type, or state to 16 bytes");
  if (!logprob && !entropy && ntop == 0 && !state) return RESHARD_OK;
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
                    dlogprob, dentropy, dlogits, 0,
                    (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(dlogits)) % 16 == 0};
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    // (a row that starts inside a granule may end in one more)
    const bool inside = !rs::op::aligned(logits, 16) || ld * size % 16 != 0;
    a.chunks = int32_t(rs::op::cdiv(rs::op::cdiv(vocab, rs::vocab::Row<T>::kPer) + inside,
                                    rs::kGradThreads * rs::kGradVecs));
    const int64_t grid = rows * a.chunks;
    if (grid >= int64_t(1) << 31) return fail(RESHARD_ERR_UNSUPPORTED, "2^31 pieces of rows or more");
    rs::logprob_grad_kernel<T><<<unsigned(grid), rs::kGradThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return rs::op::launched("reshard_logprob_grad");
  });
}
