// experts.cu -- a router's choices sorted by expert (reshard_expert_sort), the rows of tokens
// at the places of their experts, as they are or in 8 bits (reshard_expert_dispatch), and back
// with weights (reshard_expert_combine, reshard_expert_combine_grad).
#include "fp8_block.cuh"

namespace rs {
namespace {

using namespace op;

// ------------------------------------------------------------------------------- sort
constexpr int kSortCluster = 8;
constexpr size_t kSortSmem = 200 * 1024;

struct SortArgs {
  const int32_t* experts;
  int32_t *slot, *offsets;
  uint32_t n;
  int32_t nexperts;
};

// A stable counting sort.  The choices go in order to the warps of a cluster (CTA by CTA); each
// warp counts its own for every expert, the counts become each warp's first place of every
// expert, and each warp goes through its choices again, 32 at a time, and gives them their
// places: the expert's next one, and within the 32 by the lanes before with the same expert.
__global__ void __launch_bounds__(1024) sort_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ int32_t counted[];  // [warps][nexperts], total [nexperts], first [nexperts]
  __shared__ int32_t warp_sum[32];
  const int E = a.nexperts, warps = blockDim.x / 32, threads = blockDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* total = counted + warps * E;
  int32_t* first = total + E;
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const uint32_t rank = tc::cluster_rank();
  for (int i = tid; i < warps * E; i += threads) counted[i] = 0;
  const uint64_t batches = (uint64_t(a.n) + 31) / 32;
  const uint32_t part = rank * warps + warp, parts = ctas * warps;
  const uint32_t b0 = uint32_t(batches * part / parts), b1 = uint32_t(batches * (part + 1) / parts);
  int32_t* mine = counted + warp * E;
  auto choice = [&](uint32_t b) {
    const uint64_t i = uint64_t(b) * 32 + lane;
    const int e = b < b1 && i < a.n ? __ldg(a.experts + i) : -1;
    return uint32_t(e) < uint32_t(E) ? e : -1;
  };
  __syncthreads();
  for (uint32_t b = b0; b < b1; ++b) {
    const int e = choice(b);
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < E; e += threads) {
    int sum = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = counted[w * E + e];
      counted[w * E + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
  tc::cluster_sync();
  int carry = 0;  // choices of the experts before
  for (int base = 0; base < E; base += threads) {
    const int e = base + tid;
    int before = 0, all = 0;
    if (e < E) {
      const uint32_t at = staging::smem_addr(&total[e]);
      for (uint32_t r = 0; r < ctas; ++r) {
        const int c = __float_as_int(tc::load_cluster(tc::in_cta(at, r)));
        before += r < rank ? c : 0;
        all += c;
      }
    }
    int to = all;  // inclusive scan over the CTA
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, to, o);
      if (lane >= o) to += v;
    }
    if (lane == 31) warp_sum[warp] = to;
    __syncthreads();
    int chunk = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) to += warp_sum[w];
      chunk += warp_sum[w];
    }
    if (e < E) {
      first[e] = carry + to - all + before;
      if (rank == 0) a.offsets[e] = carry + to - all;
    }
    carry += chunk;
    __syncthreads();
  }
  if (rank == 0 && tid == 0) a.offsets[E] = carry;
  tc::cluster_arrive();  // this CTA has read the others' totals
  for (uint32_t b = b0; b < b1; ++b) {
    const int e = choice(b);
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int before = __popc(same & ((1u << lane) - 1));
    int place = -1;
    if (e >= 0) place = first[e] + mine[e] + before;
    __syncwarp();
    if (e >= 0 && before == 0) mine[e] += __popc(same);
    __syncwarp();
    const uint64_t i = uint64_t(b) * 32 + lane;
    if (i < a.n) a.slot[i] = place;
  }
  tc::cluster_wait();
}

// --------------------------------------------------------------------------- dispatch
struct DispatchArgs {
  const unsigned char* x;
  unsigned char* rows;
  float* scale;
  const int32_t* slot;
  int64_t ldx, ldr, lds;  // bytes; floats
  int64_t tokens, cols;
  int64_t vecs, chunks;   // accesses of a row; CTAs that share one
  uint32_t nrows;
  int32_t topk, lanes;    // lanes of a token
};

// Each row is read once and written to all of its places.
constexpr int kDispatchVecs = 4;  // of a thread
template <typename V>
__global__ void __launch_bounds__(256) dispatch_kernel(const __grid_constant__ DispatchArgs a) {
  const int lane = threadIdx.x & (a.lanes - 1);
  const int64_t group = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  const int64_t t = group * (256 / a.lanes) + threadIdx.x / a.lanes;
  if (t >= a.tokens) return;
  const int64_t c0 = chunk * kDispatchVecs * a.lanes + lane;
  const V* x = reinterpret_cast<const V*>(a.x + t * a.ldx);
  V v[kDispatchVecs];
#pragma unroll
  for (int i = 0; i < kDispatchVecs; ++i)
    if (c0 + i * a.lanes < a.vecs) v[i] = __ldcs(x + c0 + i * a.lanes);
  const int32_t* slot = a.slot + t * a.topk;
#pragma unroll 4
  for (int j = 0; j < a.topk; ++j) {
    const uint32_t s = uint32_t(__ldg(slot + j));
    if (s >= a.nrows) continue;
    V* to = reinterpret_cast<V*>(a.rows + int64_t(s) * a.ldr);
#pragma unroll
    for (int i = 0; i < kDispatchVecs; ++i)
      if (c0 + i * a.lanes < a.vecs) to[c0 + i * a.lanes] = v[i];
  }
}

// The same in 8 bits: sixteen lanes a block of 128 values, quantised once.  VEC: every row of x
// starts on 16 bytes, of the 8-bit rows on 8.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) dispatch_fp8_kernel(const __grid_constant__ DispatchArgs a) {
  const uint64_t group = uint64_t(blockIdx.x) * 16 + threadIdx.x / 16;
  const int64_t blocks = a.chunks, tt = int64_t(group / uint64_t(blocks));
  const int64_t block = int64_t(group % uint64_t(blocks)), t = tt < a.tokens ? tt : a.tokens - 1;
  const int c = threadIdx.x % 16 * 8;
  const int64_t col = block * 128 + c;
  const int inside = int(min(max(a.cols - col, int64_t(0)), int64_t(8)));
  const int left = tt < a.tokens ? inside : 0;
  const T* x = reinterpret_cast<const T*>(a.x + t * a.ldx) + col;
  Eight<T> e;
  const bool whole = __all_sync(0xffffffffu, VEC && left == 8);
  if (whole) {
    e.load(x);
  } else if (VEC) {
    e.load(x, left);
  } else {
    const T* begin = reinterpret_cast<const T*>(a.x);
    const T* end = reinterpret_cast<const T*>(a.x + (a.tokens - 1) * a.ldx) + a.cols;
    e.template load_granules<false>(x, begin, end);
    e.align(x, left);
  }
  float m = e.largest();
  for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float s = scale_of(m);
  const uint2 q = e.quotients(s);
  const int count = tt < a.tokens ? int(min(a.cols - (col - c), int64_t(128))) : 0;
  const int32_t* slot = a.slot + t * a.topk;
#pragma unroll 4
  for (int j = 0; j < a.topk; ++j) {
    const uint32_t to = uint32_t(__ldg(slot + j));
    const bool on = to < a.nrows && tt < a.tokens;
    uint8_t* row = a.rows + (on ? int64_t(to) * a.ldr + (col - c) : 0);
    if (on && c == 0) a.scale[int64_t(to) * a.lds + block] = s;
    if (whole) {
      if (on) *reinterpret_cast<uint2*>(row + c) = q;
    } else {
      store_row(row, q, on ? count : 0);
    }
  }
}

// ---------------------------------------------------------------------------- combine
struct CombineArgs {
  const void *rows, *dout;
  void *out, *drows;
  const int32_t* slot;
  const float* weight;
  float* dweight;
  int64_t ldr, ldo;     // elements
  int64_t tokens, vecs, chunks;
  uint32_t nrows;
  int32_t topk, lanes;
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Values {
  T v[N];
};

constexpr int kTogether = 8;  // choices whose rows are on their way at a time

// out = sum of weight x row over a token's choices, in float32 in the order of the choices.
template <typename T, int N>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ CombineArgs a) {
  using V = Values<T, N>;
  const int lane = threadIdx.x & (a.lanes - 1);
  const int64_t group = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  const int64_t t = group * (256 / a.lanes) + threadIdx.x / a.lanes;
  const int64_t c = chunk * a.lanes + lane;
  if (t >= a.tokens || c >= a.vecs) return;
  float sum[N];
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0.0f;
  for (int j0 = 0; j0 < a.topk; j0 += kTogether) {
    V v[kTogether];
    float w[kTogether];
    bool on[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int64_t at = t * a.topk + j0 + j;
      const uint32_t s = j0 + j < a.topk ? uint32_t(__ldg(a.slot + at)) : 0xffffffffu;
      on[j] = s < a.nrows;
      w[j] = on[j] && a.weight ? __ldg(a.weight + at) : 1.0f;
      if (on[j]) v[j] = *(reinterpret_cast<const V*>(static_cast<const T*>(a.rows) + int64_t(s) * a.ldr) + c);
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      if (!on[j]) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] = fmaf(w[j], to_float(v[j].v[i]), sum[i]);
    }
  }
  V out;
#pragma unroll
  for (int i = 0; i < N; ++i) out.v[i] = from_float<T>(sum[i]);
  *(reinterpret_cast<V*>(static_cast<T*>(a.out) + t * a.ldo) + c) = out;
}

// drows = weight x dout at the places of a token's choices; dweight = the products of dout with
// its rows.  LANES: of a token, a warp or a CTA.
template <typename T, int N, int LANES, bool DOT>
__global__ void __launch_bounds__(256) combine_grad_kernel(const __grid_constant__ CombineArgs a) {
  using V = Values<T, N>;
  __shared__ float part[8][kTogether];
  const int lane = threadIdx.x % LANES, warp = threadIdx.x / 32;
  const int64_t t = int64_t(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
  if (t >= a.tokens) return;  // (whole warps, and with a CTA a token none)
  const V* dout = reinterpret_cast<const V*>(static_cast<const T*>(a.dout) + t * a.ldo);
  for (int j0 = 0; j0 < a.topk; j0 += kTogether) {
    const int together = min(kTogether, a.topk - j0);
    uint32_t s[kTogether];
    float w[kTogether], dot[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const int64_t at = t * a.topk + j0 + j;
      s[j] = j < together ? uint32_t(__ldg(a.slot + at)) : 0xffffffffu;
      w[j] = j < together && a.weight ? __ldg(a.weight + at) : 1.0f;
      dot[j] = 0.0f;
    }
    for (int64_t c = lane; c < a.vecs; c += LANES) {
      const V d = dout[c];
      V r[kTogether];
      if (DOT) {
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
          if (s[j] < a.nrows)
            r[j] = *(reinterpret_cast<const V*>(static_cast<const T*>(a.rows) + int64_t(s[j]) * a.ldr) + c);
      }
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        if (s[j] >= a.nrows) continue;
        if (DOT) {
#pragma unroll
          for (int i = 0; i < N; ++i) dot[j] = fmaf(to_float(d.v[i]), to_float(r[j].v[i]), dot[j]);
        }
        if (!a.drows) continue;
        V g;
#pragma unroll
        for (int i = 0; i < N; ++i) g.v[i] = from_float<T>(w[j] * to_float(d.v[i]));
        *(reinterpret_cast<V*>(static_cast<T*>(a.drows) + int64_t(s[j]) * a.ldr) + c) = g;
      }
    }
    if (!DOT) continue;
#pragma unroll
    for (int j = 0; j < kTogether; ++j) dot[j] = warp_sum(dot[j]);
    float* to = a.dweight + t * a.topk + j0;
    if (LANES == 32) {
      if (lane == 0)
        for (int j = 0; j < kTogether; ++j)
          if (j < together) to[j] = dot[j];
    } else {
      if (threadIdx.x % 32 == 0)
        for (int j = 0; j < kTogether; ++j) part[warp][j] = dot[j];
      __syncthreads();
      if (int(threadIdx.x) < together) {
        float sum = 0.0f;
        for (int i = 0; i < 8; ++i) sum += part[i][threadIdx.x];
        to[threadIdx.x] = sum;
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------- launches
constexpr int64_t kMost = int64_t(1) << 31;

// Whether every address that a call forms is a multiple of `to` bytes.
bool all_aligned(int64_t to, std::initializer_list<const void*> pointers, std::initializer_list<int64_t> bytes) {
  for (const void* p : pointers)
    if (!aligned(p, uintptr_t(to))) return false;
  for (int64_t b : bytes)
    if (b % to != 0) return false;
  return true;
}

// f(std::integral_constant<int, W>()) with W the widest access, 16 bytes at most.
template <typename F>
reshard_status_t by_width(int64_t least, std::initializer_list<const void*> pointers,
                          std::initializer_list<int64_t> bytes, F&& f) {
  if (all_aligned(16, pointers, bytes)) return f(std::integral_constant<int, 16>());
  if (all_aligned(8, pointers, bytes)) return f(std::integral_constant<int, 8>());
  if (least == 4 || all_aligned(4, pointers, bytes)) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 2>());
}
template <int W>
struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = unsigned short; };

// Lanes of a token: a power of two, 256 at most, no more than a row has accesses for.
int lanes_of(int64_t vecs) {
  int lanes = 1;
  while (lanes < 256 && lanes < vecs) lanes *= 2;
  return lanes;
}

reshard_status_t too_many(int64_t grid) {
  return grid < kMost ? RESHARD_OK : fail(RESHARD_ERR_UNSUPPORTED, "2^31 pieces of rows or more");
}

// What the calls on rows have in common.
reshard_status_t check(int32_t dtype, int64_t tokens, int64_t topk, int64_t cols, int64_t nrows) {
  if (!float_dtype(dtype)) return fail(RESHARD_ERR_INVALID_ARG, "dtype must be BF16, FP16 or FP32");
  if (tokens < 0 || topk < 0 || cols < 0 || nrows < 0) return fail(RESHARD_ERR_INVALID_ARG, "negative size");
  if (tokens >= kMost || topk >= kMost || cols >= kMost || nrows >= kMost || tokens * topk >= kMost)
    return fail(RESHARD_ERR_UNSUPPORTED, "a size, or tokens * topk, of 2^31 or more");
  return RESHARD_OK;
}

}  // namespace
}  // namespace rs

using rs::fail;

extern "C" reshard_status_t reshard_expert_sort(const int32_t* experts, int64_t tokens, int64_t topk,
                                                int64_t nexperts, int32_t* slot, int32_t* offsets,
                                                void* stream) {
  rs::TraceRange trace("op.expert_sort");
  if (tokens < 0 || topk < 0 || nexperts < 0) return fail(RESHARD_ERR_INVALID_ARG, "negative size");
  if (nexperts > RESHARD_MAX_EXPERTS) return fail(RESHARD_ERR_UNSUPPORTED, "too many experts");
  if (tokens >= rs::kMost || topk >= rs::kMost || tokens * topk >= rs::kMost)
    return fail(RESHARD_ERR_UNSUPPORTED, "tokens * topk of 2^31 or more");
  const int64_t n = tokens * topk;
  if (!offsets || (n > 0 && (!experts || !slot))) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(experts, 4) || !rs::op::aligned(slot, 4) || !rs::op::aligned(offsets, 4))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce == cudaSuccess && n == 0) ce = cudaMemsetAsync(offsets, 0, size_t(4 * (nexperts + 1)), st);
  if (ce != cudaSuccess)
    return fail(RESHARD_ERR_CUDA, std::string("reshard_expert_sort: ") + cudaGetErrorString(ce));
  if (n == 0) return RESHARD_OK;
  rs::SortArgs a = {experts, slot, offsets, uint32_t(n), int32_t(nexperts)};
  int64_t warps = 32;
  while ((warps + 2) * nexperts * 4 > int64_t(rs::kSortSmem)) warps /= 2;
  const int ctas = n <= 8192 ? 1 : rs::kSortCluster;
  void* args[] = {&a};
  return rs::op::launch<rs::sort_kernel, rs::kSortSmem>(
      "reshard_expert_sort", dev,
      {ctas, int(32 * warps), size_t((warps + 2) * nexperts * 4), ctas, st}, args);
}

extern "C" reshard_status_t reshard_expert_dispatch(const void* x, int32_t dtype, int64_t tokens,
                                                    int64_t topk, int64_t cols, int64_t ldx,
                                                    const int32_t* slot, int64_t nrows, void* rows,
                                                    int64_t ldr, float* scale, int64_t lds,
                                                    void* stream) {
  rs::TraceRange trace("op.expert_dispatch");
  const reshard_status_t ok = rs::check(dtype, tokens, topk, cols, nrows);
  if (ok != RESHARD_OK) return ok;
  if (tokens == 0 || topk == 0 || cols == 0 || nrows == 0) return RESHARD_OK;
  const int64_t size = rs::op::dtype_size(dtype), blocks = rs::op::cdiv(cols, 128);
  if (ldx < cols || ldr < cols || (scale && lds < blocks))
    return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!x || !slot || !rows) return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(x, size) || !rs::op::aligned(slot, 4) || !rs::op::aligned(scale, 4) ||
      (!scale && !rs::op::aligned(rows, size)))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rs::DispatchArgs a = {};
  a.x = static_cast<const unsigned char*>(x);
  a.rows = static_cast<unsigned char*>(rows);
  a.scale = scale;
  a.slot = slot;
  a.ldx = ldx * size;
  a.ldr = scale ? ldr : ldr * size;
  a.lds = lds;
  a.tokens = tokens;
  a.cols = cols;
  a.nrows = uint32_t(nrows);
  a.topk = int32_t(topk);
  if (scale) {
    a.chunks = blocks;
    const int64_t grid = rs::op::cdiv(tokens * blocks, 16);
    if (const reshard_status_t s = rs::too_many(grid); s != RESHARD_OK) return s;
    const bool vec = rs::all_aligned(16, {x}, {a.ldx}) && rs::all_aligned(8, {rows}, {a.ldr});
    return rs::op::by_dtype(dtype, [&](auto t) {
      using T = decltype(t);
      if (vec) rs::dispatch_fp8_kernel<T, true><<<unsigned(grid), 256, 0, st>>>(a);
      else rs::dispatch_fp8_kernel<T, false><<<unsigned(grid), 256, 0, st>>>(a);
      return rs::op::launched("reshard_expert_dispatch");
    });
  }
  return rs::by_width(size, {x, rows}, {a.ldx, a.ldr, cols * size}, [&](auto w) {
    a.vecs = cols * size / w;
    a.lanes = rs::lanes_of(a.vecs);
    a.chunks = rs::op::cdiv(a.vecs, rs::kDispatchVecs * a.lanes);
    const int64_t grid = rs::op::cdiv(tokens, 256 / a.lanes) * a.chunks;
    if (const reshard_status_t s = rs::too_many(grid); s != RESHARD_OK) return s;
    rs::dispatch_kernel<typename rs::Word<w>::type><<<unsigned(grid), 256, 0, st>>>(a);
    return rs::op::launched("reshard_expert_dispatch");
  });
}

extern "C" reshard_status_t reshard_expert_combine(const void* rows, int32_t dtype, int64_t tokens,
                                                   int64_t topk, int64_t cols, int64_t nrows,
                                                   int64_t ldr, const int32_t* slot,
                                                   const float* weight, void* out, int64_t ldo,
                                                   void* stream) {
  rs::TraceRange trace("op.expert_combine");
  const reshard_status_t ok = rs::check(dtype, tokens, topk, cols, nrows);
  if (ok != RESHARD_OK) return ok;
  if (tokens == 0 || cols == 0) return RESHARD_OK;
  const int64_t size = rs::op::dtype_size(dtype);
  if (ldo < cols || ldr < cols) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!out || (topk > 0 && !slot) || (topk > 0 && nrows > 0 && !rows))
    return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(rows, size) || !rs::op::aligned(out, size) || !rs::op::aligned(slot, 4) ||
      !rs::op::aligned(weight, 4))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  rs::CombineArgs a = {};
  a.rows = rows;
  a.out = out;
  a.slot = slot;
  a.weight = weight;
  a.ldr = ldr;
  a.ldo = ldo;
  a.tokens = tokens;
  a.nrows = uint32_t(nrows);
  a.topk = int32_t(topk);
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return rs::by_width(size, {rows, out}, {ldr * size, ldo * size, cols * size}, [&](auto w) {
      constexpr int N = w / int(sizeof(T)) > 0 ? w / int(sizeof(T)) : 1;
      a.vecs = cols / N;
      a.lanes = rs::lanes_of(a.vecs);
      a.chunks = rs::op::cdiv(a.vecs, a.lanes);
      const int64_t grid = rs::op::cdiv(tokens, 256 / a.lanes) * a.chunks;
      if (const reshard_status_t s = rs::too_many(grid); s != RESHARD_OK) return s;
      rs::combine_kernel<T, N><<<unsigned(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
      return rs::op::launched("reshard_expert_combine");
    });
  });
}

extern "C" reshard_status_t reshard_expert_combine_grad(const void* dout, int32_t dtype, int64_t tokens,
                                                        int64_t topk, int64_t cols, int64_t ldo,
                                                        const int32_t* slot, int64_t nrows,
                                                        const void* rows, int64_t ldr,
                                                        const float* weight, void* drows,
                                                        float* dweight, void* stream) {
  rs::TraceRange trace("op.expert_combine_grad");
  const reshard_status_t ok = rs::check(dtype, tokens, topk, cols, nrows);
  if (ok != RESHARD_OK) return ok;
  if (tokens == 0 || topk == 0 || !(drows || dweight)) return RESHARD_OK;
  const int64_t size = rs::op::dtype_size(dtype);
  if (ldo < cols || ldr < cols) return fail(RESHARD_ERR_INVALID_ARG, "row pitch smaller than a row");
  if (!slot || (cols > 0 && (!dout || (dweight && nrows > 0 && !rows))))
    return fail(RESHARD_ERR_INVALID_ARG, "null pointer");
  if (!rs::op::aligned(rows, size) || !rs::op::aligned(dout, size) || !rs::op::aligned(drows, size) ||
      !rs::op::aligned(slot, 4) || !rs::op::aligned(weight, 4) || !rs::op::aligned(dweight, 4))
    return fail(RESHARD_ERR_INVALID_ARG, "pointer not aligned to its element type");
  rs::CombineArgs a = {};
  a.rows = rows;
  a.dout = dout;
  a.drows = drows;
  a.slot = slot;
  a.weight = weight;
  a.dweight = dweight;
  a.ldr = ldr;
  a.ldo = ldo;
  a.tokens = tokens;
  a.nrows = uint32_t(nrows);
  a.topk = int32_t(topk);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const void* read = dweight ? rows : nullptr;
    return rs::by_width(size, {dout, read, drows}, {ldr * size, ldo * size, cols * size}, [&](auto w) {
      constexpr int N = w / int(sizeof(T)) > 0 ? w / int(sizeof(T)) : 1;
      a.vecs = cols / N;
      const bool cta = a.vecs > 128;  // a CTA a token, else a warp
      const int64_t grid = cta ? tokens : rs::op::cdiv(tokens, 8);
      if (const reshard_status_t s = rs::too_many(grid); s != RESHARD_OK) return s;
      const unsigned g = unsigned(grid);
      if (dweight && cta) rs::combine_grad_kernel<T, N, 256, true><<<g, 256, 0, st>>>(a);
      else if (dweight) rs::combine_grad_kernel<T, N, 32, true><<<g, 256, 0, st>>>(a);
      else if (cta) rs::combine_grad_kernel<T, N, 256, false><<<g, 256, 0, st>>>(a);
      else rs::combine_grad_kernel<T, N, 32, false><<<g, 256, 0, st>>>(a);
      return rs::op::launched("reshard_expert_combine_grad");
    });
  });
}
