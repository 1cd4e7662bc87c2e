// balance.cu -- reshard_balance_loss: the router's load-balance loss, the tokens each
// expert got, and the gradient in the router's logits.
#include "operators.cuh"

namespace rs {
namespace {

using namespace op;

constexpr int kChunk = 64;  // tokens of one CTA

struct BalanceArgs {
  const void* logits;
  int64_t ld;
  const int32_t* experts;
  const uint8_t* mask;
  const float* grad;
  float* loss;
  int32_t* counts;
  void* dlogits;
  int32_t* tokens;  // [nseq]: tokens with mask (workspace)
  float* parts;     // [nseq * chunks]: sums over tokens (workspace)
  int64_t nseq, seqlen, topk, chunks;
  int32_t nexperts, score;
  float coef;
};

__global__ void __launch_bounds__(256) count_kernel(BalanceArgs a) {
  const int64_t s = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
  const int64_t t0 = c * kChunk, t1 = t0 + kChunk < a.seqlen ? t0 + kChunk : a.seqlen;
  for (int64_t i = t0 * a.topk + threadIdx.x; i < t1 * a.topk; i += blockDim.x) {
    const int64_t t = s * a.seqlen + i / a.topk;
    if (a.mask && !a.mask[t]) continue;
    if (i % a.topk == 0) atomicAdd(&a.tokens[s], 1);
    const int32_t e = a.experts[s * a.seqlen * a.topk + i];
    if (e >= 0 && e < a.nexperts) atomicAdd(&a.counts[s * a.nexperts + e], 1);
  }
}

__device__ __forceinline__ float score_of(float l, float top, int score) {
  return score == RESHARD_SCORE_SOFTMAX ? expf(l - top) : 1.0f / (1.0f + expf(-l));
}

// One warp a token.
template <typename T>
__global__ void __launch_bounds__(256) balance_kernel(BalanceArgs a) {
  __shared__ float sums[8];
  __shared__ int live_s;
  const int64_t s = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) live_s = 0;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < a.nseq; i += blockDim.x)
    if (a.tokens[i] > 0) atomicAdd(&live_s, 1);
  __syncthreads();
  const float n = float(a.tokens[s] > 0 ? a.tokens[s] : 1);
  const float per_count = float(a.nexperts) / (float(a.topk) * n);
  const float share = a.coef / float(live_s > 0 ? live_s : 1) / n * (a.grad ? *a.grad : 1.0f);
  const int32_t* counts = a.counts + s * a.nexperts;
  const T* logits = static_cast<const T*>(a.logits);
  T* dlogits = static_cast<T*>(a.dlogits);
  float sum = 0.0f;
  for (int64_t i = c * kChunk + warp; i < (c + 1) * kChunk && i < a.seqlen; i += 8) {
    const int64_t t = s * a.seqlen + i;
    const T* l = logits + t * a.ld;
    T* d = dlogits ? dlogits + t * a.ld : nullptr;
    if (a.mask && !a.mask[t]) {
      if (d)
        for (int e = lane; e < a.nexperts; e += 32) d[e] = from_float<T>(0.0f);
      continue;
    }
    float top = -INFINITY, total = 0.0f, dot = 0.0f;
    for (int e = lane; e < a.nexperts; e += 32) top = fmaxf(top, to_float(l[e]));
    top = warp_max(top);
    const bool none = top == -INFINITY;
    for (int e = lane; e < a.nexperts; e += 32) {
      const float v = none ? 0.0f : score_of(to_float(l[e]), top, a.score);
      total += v;
      dot += v * (float(counts[e]) * per_count);
    }
    total = warp_sum(total);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    dot = warp_sum(dot) * inv;
    sum += dot;
    if (!d) continue;
    for (int e = lane; e < a.nexperts; e += 32) {
      const float v = none ? 0.0f : score_of(to_float(l[e]), top, a.score);
      const float slope = v * inv * (a.score == RESHARD_SCORE_SOFTMAX ? 1.0f : 1.0f - v);
      d[e] = from_float<T>(share * slope * (float(counts[e]) * per_count - dot));
    }
  }
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += sums[w];
    a.parts[blockIdx.x] = sum / n;
  }
}

__global__ void __launch_bounds__(256) loss_kernel(BalanceArgs a) {
  __shared__ double sums[256];
  __shared__ int live_s;
  if (threadIdx.x == 0) live_s = 0;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < a.nseq; i += 256)
    if (a.tokens[i] > 0) atomicAdd(&live_s, 1);
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < a.nseq * a.chunks; i += 256) sum += double(a.parts[i]);
  sums[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 256; ++i) sum += sums[i];
    *a.loss = float(sum * double(a.coef) / double(live_s > 0 ? live_s : 1));
  }
}

int64_t tokens_bytes(int64_t nseq) { return cdiv(nseq * 4, 16) * 16; }

}  // namespace
}  // namespace rs

using rs::fail;

extern "C" int64_t reshard_balance_loss_workspace(int64_t nseq, int64_t seqlen, int64_t nexperts) {
  if (nseq < 0 || seqlen < 0 || nexperts < 0) return 0;
  return rs::tokens_bytes(nseq) + 4 * nseq * rs::op::cdiv(seqlen, rs::kChunk);
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
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + rs::tokens_bytes(nseq));
  a.nseq = nseq;
  a.seqlen = seqlen;
  a.topk = topk;
  a.chunks = rs::op::cdiv(seqlen, rs::kChunk);
  a.nexperts = int32_t(nexperts);
  a.score = score;
  a.coef = coef;
  cudaError_t ce = cudaMemsetAsync(counts, 0, size_t(4 * nseq * nexperts), st);
  if (ce == cudaSuccess) ce = cudaMemsetAsync(a.tokens, 0, size_t(4 * nseq), st);
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string("reshard_balance_loss: ") + cudaGetErrorString(ce));
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const unsigned grid = none ? 0 : unsigned(a.nseq * a.chunks);
    if (none) a.chunks = 0;
    if (grid > 0) {
      rs::count_kernel<<<grid, 256, 0, st>>>(a);
      if (loss || dlogits) rs::balance_kernel<T><<<grid, 256, 0, st>>>(a);
    }
    if (loss) rs::loss_kernel<<<1, 256, 0, st>>>(a);
    return rs::op::launched("reshard_balance_loss");
  });
}
