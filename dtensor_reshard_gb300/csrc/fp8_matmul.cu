// fp8_matmul.cu -- reshard_fp8_matmul: the product of e4m3 matrices with a float32
// scale for each block of 128, dense or one weight matrix for each expert.
#include "operators.cuh"

namespace rs {
namespace {

using namespace op;

__device__ __forceinline__ float e4m3(uint8_t v) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

// One warp an output: lanes share each block's products.
template <typename Y>
__global__ void __launch_bounds__(256)
    matmul_kernel(const uint8_t* x, int64_t ldx, const float* xs, int64_t ldxs, const uint8_t* w,
                  int64_t ldw, const float* ws, int64_t ldws, const int32_t* offsets,
                  int64_t nexperts, int64_t tokens, int64_t n, int64_t k, Y* y, int64_t ldy) {
  const int64_t o = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (o >= tokens * n) return;
  const int64_t t = o / n, j = o % n;
  int64_t e = 0;
  if (offsets != nullptr) {
    while (e < nexperts && !(offsets[e] <= t && t < offsets[e + 1])) ++e;
    if (e == nexperts) return;
  }
  const uint8_t* xr = x + t * ldx;
  const uint8_t* wr = w + (e * n + j) * ldw;
  const float* wsr = ws + (e * ((n + 127) / 128) + j / 128) * ldws;
  float sum = 0.0f;
  for (int64_t b = 0; b * 128 < k; ++b) {
    float part = 0.0f;
    for (int64_t i = b * 128 + lane; i < k && i < b * 128 + 128; i += 32)
      part += e4m3(xr[i]) * e4m3(wr[i]);
    sum += warp_sum(part) * (xs[t * ldxs + b] * wsr[b]);
  }
  if (lane == 0) y[t * ldy + j] = from_float<Y>(sum);
}

}  // namespace
}  // namespace rs

using rs::fail;

extern "C" reshard_status_t reshard_fp8_matmul(const void* x, int64_t ldx, const float* xs,
                                               int64_t ldxs, const void* w, int64_t ldw,
                                               const float* ws, int64_t ldws,
                                               const int32_t* offsets, int64_t nexperts,
                                               int64_t tokens, int64_t n, int64_t k, void* y,
                                               int32_t ydtype, int64_t ldy, void* stream) {
  rs::TraceRange trace("op.fp8_matmul");
  if (!rs::op::float_dtype(ydtype))
    return fail(RESHARD_ERR_INVALID_ARG, "ydtype must be BF16, FP16 or FP32");
  if (tokens < 0 || n < 0 || k < 0 || nexperts < 1)
    return fail(RESHARD_ERR_INVALID_ARG, "negative size");
  if (!offsets && nexperts != 1)
    return fail(RESHARD_ERR_INVALID_ARG, "several experts need offsets");
  if (nexperts > RESHARD_MAX_EXPERTS) return fail(RESHARD_ERR_UNSUPPORTED, "too many experts");
  constexpr int64_t kMost = int64_t(1) << 31;
  if (tokens >= kMost || n >= kMost || k >= kMost || nexperts * n >= kMost)
    return fail(RESHARD_ERR_UNSUPPORTED, "size of 2^31 or more");
  if (tokens == 0 || n == 0) return RESHARD_OK;
  const int64_t blocks = rs::op::cdiv(k, 128);
  if (ldx < k || ldw < k || ldxs < blocks || ldws < blocks || ldy < n)
    return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!y || (k > 0 && (!x || !xs || !w || !ws)))
    return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(x, 16) || !rs::op::aligned(w, 16) || ldx % 16 != 0 || ldw % 16 != 0)
    return fail(RESHARD_ERR_INVALID_ARG, "x, w and their row pitches must be multiples of 16 bytes");
  if (!rs::op::aligned(xs, 4) || !rs::op::aligned(ws, 4) || !rs::op::aligned(offsets, 4) ||
      !rs::op::aligned(y, rs::op::dtype_size(ydtype)))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  return rs::op::by_dtype(ydtype, [&](auto t) {
    using Y = decltype(t);
    rs::matmul_kernel<Y><<<unsigned(rs::op::cdiv(tokens * n, 8)), 256, 0,
                           static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint8_t*>(x), ldx, xs, ldxs, static_cast<const uint8_t*>(w), ldw, ws,
        ldws, offsets, nexperts, tokens, n, k, static_cast<Y*>(y), ldy);
    return rs::op::launched("reshard_fp8_matmul");
  });
}
