// fp8_quantize.cu -- reshard_fp8_quantize: e4m3 values with one float32 scale for
// each block of 1x128 or 128x128.
#include "operators.cuh"

namespace rs {
namespace {

using namespace op;

constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: a block of zeros

// One CTA a block: the largest magnitude, then the quotients.
template <typename T>
__global__ void __launch_bounds__(256) quantize_kernel(const T* x, int64_t rows, int64_t cols,
                                                       int64_t ldx, int block_rows, uint8_t* q,
                                                       int64_t ldq, float* scale, int64_t lds,
                                                       int64_t col_blocks, int64_t row_blocks) {
  __shared__ float part[8];
  const int64_t cb = blockIdx.x % col_blocks, rb = blockIdx.x / col_blocks;
  const int64_t mat = rb / row_blocks, band = rb % row_blocks;
  const int64_t r0 = band * block_rows, c0 = cb * 128;
  const int nr = int(rows - r0 < block_rows ? rows - r0 : block_rows);
  const int nc = int(cols - c0 < 128 ? cols - c0 : 128);
  const T* xb = x + (mat * rows + r0) * ldx + c0;
  uint8_t* qb = q + (mat * rows + r0) * ldq + c0;
  float most = 0.0f;
  for (int i = threadIdx.x; i < nr * nc; i += blockDim.x)
    most = fmaxf(most, fabsf(to_float(xb[int64_t(i / nc) * ldx + i % nc])));
  most = warp_max(most);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = most;
  __syncthreads();
  for (int i = 0; i < 8; ++i) most = fmaxf(most, part[i]);
  const float s = fmaxf(most / kE4m3Max, kScaleMin);
  if (threadIdx.x == 0) scale[rb * lds + cb] = s;
  for (int i = threadIdx.x; i < nr * nc; i += blockDim.x)
    qb[int64_t(i / nc) * ldq + i % nc] = __nv_cvt_float_to_fp8(
        to_float(xb[int64_t(i / nc) * ldx + i % nc]) / s, __NV_SATFINITE, __NV_E4M3);
}

}  // namespace
}  // namespace rs

using rs::fail;

extern "C" reshard_status_t reshard_fp8_quantize(const void* x, int32_t dtype, int64_t nmat,
                                                 int64_t rows, int64_t cols, int64_t ldx,
                                                 int32_t block_rows, void* q, int64_t ldq,
                                                 float* scale, int64_t lds, void* stream) {
  rs::TraceRange trace("op.fp8_quantize");
  if (!rs::op::float_dtype(dtype))
    return fail(RESHARD_ERR_INVALID_ARG, "dtype must be BF16, FP16 or FP32");
  if (block_rows != 1 && block_rows != 128)
    return fail(RESHARD_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  if (nmat < 0 || rows < 0 || cols < 0) return fail(RESHARD_ERR_INVALID_ARG, "negative size");
  if (nmat == 0 || rows == 0 || cols == 0) return RESHARD_OK;
  const int64_t col_blocks = rs::op::cdiv(cols, 128), row_blocks = rs::op::cdiv(rows, block_rows);
  if (ldx < cols || ldq < cols || lds < col_blocks)
    return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!x || !q || !scale) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (!rs::op::aligned(x, sizeof(T)) || !rs::op::aligned(scale, 4))
      return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
    rs::quantize_kernel<T><<<unsigned(nmat * row_blocks * col_blocks), 256, 0,
                             static_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(x), rows, cols, ldx, block_rows, static_cast<uint8_t*>(q), ldq, scale,
        lds, col_blocks, row_blocks);
    return rs::op::launched("reshard_fp8_quantize");
  });
}
