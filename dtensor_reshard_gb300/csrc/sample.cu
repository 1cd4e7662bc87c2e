// sample.cu -- reshard_sample: one token a row of logits, with temperature, top-k,
// top-p and min-p, from one given uniform number a row.
#include "operators.cuh"

namespace rs {
namespace {

using namespace op;

constexpr int kThreads = 1024;
constexpr uint64_t kOne = uint64_t(1) << 40;  // weight of the most likely token

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
// Whole numbers in the order of the floats.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float scaled(float l, float top, float inv) {
  return l == top ? 0.0f : (l - top) * inv;
}
__device__ __forceinline__ float prob_of(float l, float top, float inv) {
  return l == top ? 1.0f : l - top == -INFINITY ? 0.0f : expf((l - top) * inv);
}
__device__ __forceinline__ uint64_t weight_of(float e) {
  return uint64_t(__float2ll_rn(e * float(kOne)));
}

__device__ uint64_t block_sum(uint64_t v, uint64_t* part) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < kThreads / 32; ++i) v += part[i];
  return v;
}
// Sum over the threads before this one.
__device__ uint64_t block_before(uint64_t v, uint64_t* part) {
  uint64_t run = v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t w = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += w;
  }
  __syncthreads();
  if (lane == 31) part[warp] = run;
  __syncthreads();
  for (int i = 0; i < warp; ++i) run += part[i];
  return run - v;
}

// One CTA a row; the row is read again for every question asked of it.
template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a) {
  __shared__ uint64_t part[kThreads / 32];
  __shared__ float tops[kThreads / 32];
  __shared__ int32_t found;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  const int vocab = int(a.vocab), tid = threadIdx.x;
  // every thread owns consecutive tokens
  const int each = (vocab + kThreads - 1) / kThreads;
  const int i0 = min(vocab, tid * each), i1 = min(vocab, i0 + each);

  float top = -INFINITY;
  for (int i = tid; i < vocab; i += kThreads) top = fmaxf(top, clean(to_float(x[i])));
  top = warp_max(top);
  if ((tid & 31) == 0) tops[tid >> 5] = top;
  if (tid == 0) found = vocab;
  __syncthreads();
  for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, tops[i]);
  if (top == -INFINITY) {
    if (tid == 0) {
      a.token[row] = -1;
      if (a.logprob) a.logprob[row] = -INFINITY;
    }
    return;
  }
  const float temp = a.temperature ? a.temperature[row] : 1.0f;
  const bool greedy = !(temp > 0.0f);
  const float inv = greedy ? 1.0f : 1.0f / temp;
  auto weight = [&](float l) { return weight_of(prob_of(l, top, inv)); };
  uint64_t total = 0;
  for (int i = tid; i < vocab; i += kThreads) total += weight(clean(to_float(x[i])));
  total = block_sum(total, part);

  if (greedy) {
    for (int i = i0; i < i1; ++i)
      if (clean(to_float(x[i])) == top) {
        atomicMin(&found, i);
        break;
      }
  } else {
    // kept so far: keys above `cut`, and the first `ties` tokens with that key
    uint32_t cut = 0;
    uint64_t ties = uint64_t(vocab);
    auto sum_from = [&](uint32_t key, bool mass) {
      uint64_t v = 0;
      for (int i = tid; i < vocab; i += kThreads) {
        const float l = clean(to_float(x[i]));
        if (key_of(l) >= key) v += mass ? weight(l) : 1;
      }
      return block_sum(v, part);
    };
    const int k = a.top_k ? a.top_k[row] : 0;
    if (k > 0 && k < vocab) {
      for (int b = 31; b >= 0; --b)
        if (sum_from(cut | (1u << b), false) >= uint64_t(k)) cut |= 1u << b;
      ties = uint64_t(k) - (cut == 0xffffffffu ? 0 : sum_from(cut + 1, false));
    }
    auto tie_weight = [&](uint32_t key) {
      const float l = __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
      return key == 0 ? 0 : weight(l);
    };
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    if (!(p >= 1.0f)) {
      // the weights of the kept tokens with at least this key
      auto mass_from = [&](uint32_t key) {
        if (key <= cut && ties < uint64_t(vocab))
          return sum_from(cut + 1, true) + ties * tie_weight(cut);
        return sum_from(key, true);
      };
      const double mass = double(p) * double(mass_from(0));
      uint32_t pcut = 0;
      for (int b = 31; b >= 0; --b)
        if (double(mass_from(pcut | (1u << b))) >= mass) pcut |= 1u << b;
      const uint32_t first = key_of(top);
      if (!(mass > 0.0) || pcut > first) pcut = first;
      const uint64_t above = pcut == first ? 0 : mass_from(pcut + 1);
      const uint64_t w = tie_weight(pcut);
      uint64_t most = pcut == cut ? ties : sum_from(pcut, false) - sum_from(pcut + 1, false);
      uint64_t lo = pcut == first ? 1 : 0, hi = most;  // ties kept: the largest t with
      while (lo < hi) {                                // double(above + (t - 1) w) < mass
        const uint64_t t = (lo + hi + 1) / 2;
        if (double(above + (t - 1) * w) < mass) lo = t;
        else hi = t - 1;
      }
      cut = pcut;
      ties = lo;
    }
    const float floor_p = fminf(a.min_p ? a.min_p[row] : 0.0f, 1.0f);
    uint64_t tied = 0;
    for (int i = i0; i < i1; ++i) tied += key_of(clean(to_float(x[i]))) == cut;
    const uint64_t tied_before = block_before(tied, part);
    auto walk = [&](auto&& visit) {
      uint64_t seen = tied_before;
      for (int i = i0; i < i1; ++i) {
        const float l = clean(to_float(x[i]));
        const uint32_t key = key_of(l);
        const bool in = key > cut || (key == cut && seen < ties);
        seen += key == cut;
        const float e = prob_of(l, top, inv);
        if (in && !(e < floor_p)) {
          if (visit(i, weight_of(e))) return;
        }
      }
    };
    uint64_t mine = 0;
    walk([&](int, uint64_t w) {
      mine += w;
      return false;
    });
    uint64_t run = block_before(mine, part);
    const uint64_t all = block_sum(mine, part);
    const double target = double(fmaxf(a.u[row], 0.0f)) * double(all);
    // the first token at which the sum passes the target; if none does, the last one
    // with a weight
    if (double(run + mine) > target || (run + mine == all && mine > 0)) {
      int at = vocab;
      walk([&](int i, uint64_t w) {
        run += w;
        if (w > 0) at = i;
        return double(run) > target;
      });
      atomicMin(&found, at);
    }
  }
  __syncthreads();
  if (tid == 0) {
    a.token[row] = found;
    if (a.logprob)
      a.logprob[row] = scaled(clean(to_float(x[found])), top, inv) -
                       log1pf(float(double(total - kOne) / double(kOne)));
  }
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
  if (rows >= int64_t(1) << 31) return fail(RESHARD_ERR_UNSUPPORTED, "2^31 rows or more");
  if (rows == 0 || vocab == 0) return RESHARD_OK;
  if (ld < vocab) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!logits || !u || !token) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(logits, rs::op::dtype_size(dtype)) || !rs::op::aligned(temperature, 4) ||
      !rs::op::aligned(top_k, 4) || !rs::op::aligned(top_p, 4) || !rs::op::aligned(min_p, 4) ||
      !rs::op::aligned(u, 4) || !rs::op::aligned(token, 4) || !rs::op::aligned(logprob, 4))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  rs::SampleArgs a = {logits, vocab, ld, temperature, top_p, min_p, u, top_k, token, logprob};
  return rs::op::by_dtype(dtype, [&](auto t) {
    rs::sample_kernel<decltype(t)>
        <<<unsigned(rows), rs::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return rs::op::launched("reshard_sample");
  });
}
