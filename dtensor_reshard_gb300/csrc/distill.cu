// distill.cu -- reshard_distill_loss: the divergence of the student's distribution from a teacher's
// most likely tokens, and its gradient in the student's logits.
//
// With q the teacher's probabilities of its listed tokens, q_R what is left of 1 (or 0), p the
// student's and p_R its probability of all other tokens: loss = sum q_j ln(q_j / p_j) + q_R ln(q_R /
// p_R), dl = p - q for listed tokens and p (1 - q_R / p_R) for others.  A row needs the sum over its
// logits before the first gradient, so a cluster of CTAs keeps it in registers between the two: it
// is read once and written once.
#include "vocab_row.cuh"

namespace rs {
namespace {

using namespace vocab;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 8;         // granules that a thread keeps; a slice's others are read again
constexpr int kMaxCluster = 8;
constexpr int kListWarps = RESHARD_MAX_TOP / 32;

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
  bool tail;   // the teacher's remaining probability is one more outcome
  bool alike;  // logits and gradients lie alike on 16 bytes
};

// What the threads of a CTA, and the CTAs of a cluster, tell each other.
struct Shared {
  int32_t token[RESHARD_MAX_TOP];  // the teacher's list, -1 for what is no entry
  double q[RESHARD_MAX_TOP];       // its probabilities
  double list_q[kListWarps];       // sums of the list's warps
  float list_e[kListWarps], list_top[kListWarps];
  float warp_top[kWarps], warp_other[kWarps];
  float part_top, part_other;      // of the CTA: its largest logit, its sum over other tokens
  float top, other;                // of the row
  float outside;                   // 1 - q_R / p_R
  double rest, inv_q;              // q_R, 1 / sum of the list
};

__device__ __forceinline__ float load_far(const float* at, uint32_t rank) {
  return tc::load_cluster(tc::in_cta(staging::smem_addr(at), rank));
}
// (top, other) of two parts as one: a sum is relative to its part's largest logit.
__device__ __forceinline__ void join(float& top, float& other, float c, int from) {
  for (int o = from; o; o >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, other, o);
    const float both_top = fmaxf(top, t);
    other = other * exp2_of(exponent(top, both_top, c)) + s * exp2_of(exponent(t, both_top, c));
    top = both_top;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) distill_kernel(const __grid_constant__ DistillArgs a) {
  constexpr int kPer = Row<T>::kPer;
  extern __shared__ uint32_t listed_bits[];  // of the slice's elements
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const uint32_t rank = tc::cluster_rank();
  const int64_t r = blockIdx.x / ctas;
  const Row<T> row(a.logits, r, a.ld, a.vocab);
  T* to = a.dlogits ? static_cast<T*>(a.dlogits) + r * a.ld : nullptr;
  const int granules = row.granules();
  const int g0 = int(int64_t(granules) * rank / ctas), g1 = int(int64_t(granules) * (rank + 1) / ctas);
  const int elements = (g1 - g0) * kPer;
  // the teacher's list, an entry a thread: tokens outside the vocabulary, and NaN, are none
  const int k = a.ntop, list_warps = (k + 31) / 32;
  int mine = -1;
  float y = -INFINITY;
  if (warp < list_warps) {
    if (tid < k) {
      mine = __ldg(a.top_token + r * a.ldtop + tid);
      y = __ldg(a.top_logprob + r * a.ldtop + tid);
      if (uint32_t(mine) >= uint32_t(row.vocab) || !(y == y)) mine = -1, y = -INFINITY;
    }
    if (tid < RESHARD_MAX_TOP) sh.token[tid] = mine;
    const float most = warp_max(y);
    if (lane == 0) sh.list_top[warp] = most;
  }
  for (int i = tid; i <= elements / 32; i += kThreads) listed_bits[i] = 0;
  __syncthreads();
  float y_top = sh.list_top[0];
  for (int w = 1; w < list_warps; ++w) y_top = fmaxf(y_top, sh.list_top[w]);
  if (!(y_top > -INFINITY)) {  // a row that does not count
    if (rank == 0 && tid == 0 && a.loss) a.loss[r] = 0.0f;
    if (to)
      for (int g = g0 + tid; g < g1; g += kThreads) row.store(to, g, make_uint4(0, 0, 0, 0), a.alike);
    return;
  }
  // the slice, on its way while the list is worked on
  uint4 v[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int g = g0 + i * kThreads + tid;
    v[i] = g < g1 ? row.fetch(g) : Row<T>::nothing();
  }
  const float inverse = inverse_of(a.temperature, r), c = log2_scale(inverse);
  const uint64_t c2 = both(c);
  float x = -INFINITY;     // the student's logit of this thread's entry
  bool first = mine >= 0;  // of the entries with this token
  const int place = mine + row.skew - g0 * kPer;
  const bool here = mine >= 0 && place >= 0 && place < elements;
  if (first) {
    x = clean<T>(to_float(row.row[mine]));
    for (int j = 0; j < tid; ++j) first = first && sh.token[j] != mine;
    if (here) atomicOr(&listed_bits[place / 32], 1u << (place % 32));
  }
  const bool again = __syncthreads_or(mine >= 0 && !first);  // some token stands there twice
  // the sum over tokens that are not listed, relative to each thread's own largest logit
  float m = -INFINITY, other = 0.0f;
  auto add = [&](uint4& granule, int g) {
    uint4(&one)[1] = reinterpret_cast<uint4(&)[1]>(granule);
    float largest = largest_in<T>(one);
    if (largest == INFINITY) {
      make_finite<T>(one);
      largest = largest_finite<T>();
    }
    const float top = fmaxf(m, largest);
    const uint64_t minus = both(-top);
    const int at = (g - g0) * kPer;
    const uint32_t bits = g < g1 ? listed_bits[at / 32] >> (at % 32) & ((1u << kPer) - 1) : 0;
    const T* e = reinterpret_cast<const T*>(&granule);
    uint64_t s2 = 0;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      uint64_t w = exp2_both(exponents(pair(pair_of(e + i)), minus, c2));
      if (bits) {
        float2 f = tc::unpack2(w);
        if (bits >> i & 1) f.x = 0.0f;
        if (bits >> (i + 1) & 1) f.y = 0.0f;
        w = pair(f);
      }
      s2 = add2(s2, w);
    }
    other = fmaf(other, exp2_of(exponent(m, top, c)), sum2(s2));
    m = top;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) add(v[i], g0 + i * kThreads + tid);
  for (int g = g0 + kHeld * kThreads + tid; g < g1; g += kThreads) {
    uint4 w = row.fetch(g);
    add(w, g);
  }
  join(m, other, c, 16);
  if (lane == 0) sh.warp_top[warp] = m, sh.warp_other[warp] = other;
  __syncthreads();
  if (warp == 0) {
    float top = lane < kWarps ? sh.warp_top[lane] : -INFINITY, sum = lane < kWarps ? sh.warp_other[lane] : 0.0f;
    join(top, sum, c, 16);
    if (lane == 0) sh.part_top = top, sh.part_other = sum;
  }
  if (ctas > 1) tc::cluster_sync();
  else __syncthreads();
  // the row's sums, and the list's: of the student over its different tokens, of the teacher over
  // its entries.  The teacher's are in 64 bits: what is left of 1 can be small.
  double q = 0.0;
  if (warp < list_warps) {
    float top = -INFINITY;
    other = 0.0f;
    if (lane < int(ctas)) top = load_far(&sh.part_top, lane), other = load_far(&sh.part_other, lane);
    join(top, other, c, 4);
    m = top;  // (lanes 0 to 7 have it)
    m = __shfl_sync(0xffffffffu, m, 0);
    other = __shfl_sync(0xffffffffu, other, 0);
    const float e = warp_sum(first ? exp2_of(exponent(x, m, c)) : 0.0f);
    if (mine >= 0) q = a.tail ? exp(double(y)) : double(expf(y - y_top));
    double all = q;
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    sh.q[tid] = q;
    if (lane == 0) {
      sh.list_e[warp] = e, sh.list_q[warp] = all;
      if (warp == 0) sh.top = m, sh.other = other;
    }
  }
  if (ctas > 1) tc::cluster_arrive();  // this CTA has read the others' parts
  __syncthreads();
  const float top = sh.top;
  const bool empty = !(top > -INFINITY);
  float sum = sh.other;
  for (int w = 0; w < list_warps; ++w) sum += sh.list_e[w];
  if (tid == 0) {
    double all = sh.list_q[0];
    for (int w = 1; w < list_warps; ++w) all += sh.list_q[w];
    sh.rest = 0.0, sh.outside = 1.0f, sh.inv_q = a.tail ? 1.0 : 1.0 / all;
    if (a.tail && all < 1.0 && sh.other > 0.0f) {  // (else it has nowhere to be)
      sh.rest = 1.0 - all;
      sh.outside = float(1.0 - sh.rest * (double(sum) / double(sh.other)));
    }
  }
  __syncthreads();
  if (to && empty) {
    for (int g = g0 + tid; g < g1; g += kThreads) row.store(to, g, make_uint4(0, 0, 0, 0), a.alike);
  } else if (to) {
    const float g = a.grad ? __ldg(a.grad + r) : 1.0f;
    const float slope = fmaxf(fminf(g * inverse, 3.402823466e38f), -3.402823466e38f);
    const uint64_t A = both(slope / sum * sh.outside), minus = both(-top);
    auto put = [&](uint4& granule, int at) {
      T* e = reinterpret_cast<T*>(&granule);
#pragma unroll
      for (int i = 0; i < kPer; i += 2)
        set_pair(e + i, tc::unpack2(mul2(exp2_both(exponents(pair(pair_of(e + i)), minus, c2)), A)));
      row.store(to, at, granule, a.alike);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int at = g0 + i * kThreads + tid;
      if (at < g1) put(v[i], at);
    }
    for (int at = g0 + kHeld * kThreads + tid; at < g1; at += kThreads) {
      uint4 w = row.fetch(at);
      uint4(&one)[1] = reinterpret_cast<uint4(&)[1]>(w);
      if (largest_in<T>(one) == INFINITY) make_finite<T>(one);
      put(w, at);
    }
    // the slice's listed tokens, behind what was just written for them as for others
    __syncthreads();
    if (first && here) {
      double all = q;
      if (again)
        for (int j = tid + 1; j < k; ++j)
          if (sh.token[j] == mine) all += sh.q[j];
      const float p = exp2_of(exponent(x, top, c)) / sum;
      to[mine] = from_float<T>(slope * (p - float(all * sh.inv_q)));
    }
  }
  if (rank == 0 && a.loss && warp < list_warps) {
    double term = 0.0;
    q *= sh.inv_q;
    if (!(q <= 0.0)) {
      const double z = x == top ? 0.0 : double(x - top) * double(inverse);
      term = q * ((double(y) - z) + (a.tail ? 0.0 : log(sh.inv_q) - double(y_top)) + log(double(sum)));
    }
    for (int o = 16; o; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
    if (lane == 0) sh.list_q[warp] = term;
  }
  if (ctas > 1) tc::cluster_wait();
  __syncthreads();
  if (rank == 0 && a.loss && tid == 0) {
    double loss = sh.list_q[0];
    for (int w = 1; w < list_warps; ++w) loss += sh.list_q[w];
    if (sh.rest > 0.0) loss += sh.rest * log(sh.rest * (double(sum) / double(sh.other)));
    a.loss[r] = empty ? INFINITY : float(loss);
  }
}

template <typename T>
reshard_status_t launch_distill(const DistillArgs& a, int64_t rows, int dev, int sms, cudaStream_t stream) {
  // CTAs a row: so many that they hold it; more while SMs would stay without one, and a slice
  // has 4 KiB or more
  const int64_t bytes = a.vocab * int64_t(sizeof(T));
  int ctas = 1;
  while (ctas < kMaxCluster && (bytes > ctas * int64_t(kHeld * kThreads * 16) ||
                                (rows * ctas < sms && bytes > ctas * 8192)))
    ctas *= 2;
  const int64_t slice = cdiv(cdiv(bytes, 16) + 1, ctas) + 1;  // granules
  const size_t smem = size_t(slice * (16 / int64_t(sizeof(T))) / 32 + 1) * 4;
  constexpr size_t kMost = RESHARD_MAX_VOCAB / kMaxCluster / 8 + 64;
  void* args[] = {const_cast<DistillArgs*>(&a)};
  return launch<distill_kernel<T>, kMost>("reshard_distill_loss", dev, {rows * ctas, kThreads, smem, ctas, stream},
                                          args);
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
      logits, vocab, ld, ldtop, temperature, top_token, top_logprob, grad, loss, dlogits, ntop, tail != 0,
      (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(dlogits)) % 16 == 0};
  return rs::op::by_dtype(dtype, [&](auto t) {
    return rs::launch_distill<decltype(t)>(a, rows, dev, sms, static_cast<cudaStream_t>(stream));
  });
}
