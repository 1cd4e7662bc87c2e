// fp8_quantize.cu -- reshard_fp8_quantize: e4m3 values with one float32 scale for
// each block of 1x128 or 128x128.
//
// scale = max(largest magnitude / 448, 2^-126), value = the nearest e4m3 to x / scale.  Read
// once, 2 or 4 bytes a value, written once, 1 byte: bound by HBM for blocks of 128x128 (16
// matrices of [2048, 7168] in bf16: 124 us, 5.7 TB/s) and nearly so for 1x128, where the
// quotients' instructions fill 73% of the issue slots (8192 rows of 7168: 37 us, 4.8 TB/s).
// Rows off 16 bytes cost the shifts that align them and narrow stores at both ends, 35 instructions
// for 32 values: 8192 x 14335 in bf16 take 129 us in 1x128 (82% of the issue slots) and 182 us in
// 128x128, where the registers of a block leave 16 warps an SM to hide them.
#include "fp8_block.cuh"

namespace rs {
namespace {

using namespace op;

struct QuantizeArgs {
  const void* x;
  uint8_t* q;
  float* scale;
  int64_t rows, cols, ldx, ldq, lds;
  int64_t col_blocks, row_blocks, mat_blocks;  // row_blocks: of all matrices, mat_blocks: of one
};

// 1 x 128: sixteen lanes a block, eight values a lane; a lane has its values of N rows in
// flight.  VEC: every row of x starts on 16 bytes, of q on 8.
template <typename T, bool VEC, int N>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __grid_constant__ QuantizeArgs a) {
  const uint32_t group = blockIdx.x * 16 + threadIdx.x / 16;
  const uint32_t rows = uint32_t(a.row_blocks);  // of all matrices
  const uint32_t bands = (rows + N - 1) / N;
  const uint32_t block = group % uint32_t(a.col_blocks), band = group / uint32_t(a.col_blocks);
  const int c = threadIdx.x % 16 * 8;
  const int64_t col = int64_t(block) * 128 + c;
  const uint32_t row0 = min(band, bands) * N;  // bands beyond the last have no rows
  const int left = int(min(max(a.cols - col, int64_t(0)), int64_t(8)));
  const T* x = static_cast<const T*>(a.x) + col;
  Eight<T> e[N];
  const bool whole = __all_sync(0xffffffffu, VEC && left == 8 && row0 + N <= rows);
  if (whole) {
#pragma unroll
    for (int i = 0; i < N; ++i) e[i].load(x + (row0 + i) * a.ldx);
  } else if (VEC) {
#pragma unroll
    for (int i = 0; i < N; ++i) e[i].load(x + (row0 + i) * a.ldx, row0 + i < rows ? left : 0);
  } else {
    const T* begin = static_cast<const T*>(a.x);
    const T* end = begin + (rows - 1) * a.ldx + a.cols;
    const T* last = Eight<T>::granule_of(x + (row0 + N - 1) * a.ldx);
    if (__all_sync(0xffffffffu, row0 + N <= rows && Eight<T>::granule_of(x + row0 * a.ldx) >= begin &&
                                    last + 16 + Eight<T>::kPer <= end)) {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i].template load_granules<true>(x + (row0 + i) * a.ldx, begin, end);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i].template load_granules<false>(x + (row0 + i) * a.ldx, begin, end);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) e[i].align(x + (row0 + i) * a.ldx, row0 + i < rows ? left : 0);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float m = e[i].largest();
    for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = scale_of(m);
    if (c == 0 && row0 + i < rows) a.scale[(row0 + i) * a.lds + block] = s;
    const uint2 q = e[i].quotients(s);
    uint8_t* to = a.q + (row0 + i) * a.ldq + col;
    if (whole) *reinterpret_cast<uint2*>(to) = q;
    else store_row(to - c, q, row0 + i < rows ? int(min(a.cols - (col - c), int64_t(128))) : 0);
  }
}

// 128 x 128: a CTA a block, 64 values a thread kept in registers between the maximum and
// the quotients, so that the block is read once (read twice, a value at a time: 785 us for
// the 16 matrices above).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const __grid_constant__ QuantizeArgs a) {
  __shared__ float part[8];
  const uint32_t cb = blockIdx.x % uint32_t(a.col_blocks), rb = blockIdx.x / uint32_t(a.col_blocks);
  const uint32_t mat = rb / uint32_t(a.mat_blocks);
  const int64_t band = int64_t(rb - mat * uint32_t(a.mat_blocks)) * 128;
  const int64_t row0 = mat * a.rows + band;  // over all matrices
  const int c = threadIdx.x % 16 * 8;
  const int64_t col = int64_t(cb) * 128 + c;
  const int r0 = threadIdx.x / 16;
  const int rows = int(min(a.rows - band, int64_t(128)));
  const int left = int(min(max(a.cols - col, int64_t(0)), int64_t(8)));
  const bool whole = __all_sync(0xffffffffu, VEC && rows == 128 && left == 8);
  const T* x = static_cast<const T*>(a.x) + row0 * a.ldx + col;
  Eight<T> e[8];
  if (whole) {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i].load(x + (r0 + 16 * i) * a.ldx);
  } else if (VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i].load(x + (r0 + 16 * i) * a.ldx, r0 + 16 * i < rows ? left : 0);
  } else {
    const T* begin = static_cast<const T*>(a.x);
    const T* end = begin + (a.row_blocks / a.mat_blocks * a.rows - 1) * a.ldx + a.cols;
    const T* last = Eight<T>::granule_of(x + (r0 + 16 * 7) * a.ldx);
    if (__all_sync(0xffffffffu, rows == 128 && Eight<T>::granule_of(x + r0 * a.ldx) >= begin &&
                                    last + 16 + Eight<T>::kPer <= end)) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        e[i].template load_granules<true>(x + (r0 + 16 * i) * a.ldx, begin, end);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        e[i].template load_granules<false>(x + (r0 + 16 * i) * a.ldx, begin, end);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      e[i].align(x + (r0 + 16 * i) * a.ldx, r0 + 16 * i < rows ? left : 0);
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, e[i].largest());
  m = warp_max(m);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i]);
  const float s = scale_of(m);
  if (threadIdx.x == 0) a.scale[rb * a.lds + cb] = s;
  uint8_t* q = a.q + row0 * a.ldq + col;
  const int count = int(min(a.cols - (col - c), int64_t(128)));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint2 v = e[i].quotients(s);
    uint8_t* to = q + (r0 + 16 * i) * a.ldq;
    if (whole) *reinterpret_cast<uint2*>(to) = v;
    else store_row(to - c, v, r0 + 16 * i < rows ? count : 0);
  }
}

template <typename T>
reshard_status_t launch_quantize(const QuantizeArgs& a, int block_rows, cudaStream_t stream) {
  const bool vec = aligned(a.x, 16) && a.ldx * sizeof(T) % 16 == 0 && aligned(a.q, 8) && a.ldq % 8 == 0;
  if (block_rows == 128) {
    const unsigned grid = unsigned(a.col_blocks * a.row_blocks);
    if (vec) quantize_tiles_kernel<T, true><<<grid, 256, 0, stream>>>(a);
    else quantize_tiles_kernel<T, false><<<grid, 256, 0, stream>>>(a);
  } else if (a.col_blocks * a.row_blocks < 64 * 1024) {
    const unsigned grid = unsigned(cdiv(a.col_blocks * a.row_blocks, 16));
    if (vec) quantize_rows_kernel<T, true, 1><<<grid, 256, 0, stream>>>(a);
    else quantize_rows_kernel<T, false, 1><<<grid, 256, 0, stream>>>(a);
  } else {  // four rows a lane once every SM has a few CTAs
    const unsigned grid = unsigned(cdiv(a.col_blocks * cdiv(a.row_blocks, 4), 16));
    if (vec) quantize_rows_kernel<T, true, 4><<<grid, 256, 0, stream>>>(a);
    else quantize_rows_kernel<T, false, 4><<<grid, 256, 0, stream>>>(a);
  }
  return launched("reshard_fp8_quantize");
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
  const int64_t col_blocks = rs::op::cdiv(cols, 128), mat_blocks = rs::op::cdiv(rows, block_rows);
  constexpr int64_t kMost = int64_t(1) << 31;  // of each first: the products fit 64 bits then
  if (col_blocks >= kMost || nmat >= kMost || mat_blocks >= kMost || nmat * mat_blocks >= kMost ||
      nmat * mat_blocks * col_blocks >= kMost)
    return fail(RESHARD_ERR_UNSUPPORTED, "2^31 blocks or more");
  if (ldx < cols || ldq < cols || lds < col_blocks)
    return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!x || !q || !scale) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (!rs::op::aligned(x, sizeof(T)) || !rs::op::aligned(scale, 4))
      return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
    const rs::QuantizeArgs a = {x,   static_cast<uint8_t*>(q), scale,      rows,       cols,
                                ldx, ldq,                      lds,        col_blocks, nmat * mat_blocks,
                                mat_blocks};
    return rs::launch_quantize<T>(a, block_rows, static_cast<cudaStream_t>(stream));
  });
}
