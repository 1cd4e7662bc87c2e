// experts.cu -- a router's choices sorted by expert (reshard_expert_sort), the rows of tokens
// at the places of their experts, as they are or in 8 bits (reshard_expert_dispatch), and back
// with weights (reshard_expert_combine, reshard_expert_combine_grad).
//
// Beside the sort all of them move rows, each once, and are bound by HBM: 4096 tokens of 7168 bf16 with
// 8 choices take 80 us to their places (6.6 TB/s), 49 us in 8 bits, 79 us back (6.7 TB/s), and 150 us
// for both gradients (6.7 TB/s).  Rows that do not start on 16 bytes go in narrower accesses, or those of
// 16-bit elements in shifted granules (shifted_rows.cuh): to their places unless 8 bytes fit them (7170
// columns 102 us, 7169 105), back and in gradients unless 4 bytes do (7170 in accesses of 4 bytes 103 and
// 199 us, 7169 in granules 119 and 229).  float32 rows off 16 bytes go in accesses of 4: 7169 columns 208,
// 196 and 381 us, 7168 157, 150 and 291.  In 8 bits, columns that are no multiple of 8 take 117 to 124 us.
#include <type_traits>

#include "fp8_block.cuh"
#include "shifted_rows.cuh"

namespace rs {
namespace {

using namespace op;

// ------------------------------------------------------------------------------- sort
constexpr int kSortCluster = 8;
constexpr size_t kSortSmem = 200 * 1024;
constexpr int kKept = 8;

struct SortArgs {
  const int32_t* experts;
  int32_t *slot, *offsets;
  uint32_t n;
  int32_t nexperts;
};

// A stable counting sort.  The choices go in order to the warps of a cluster (CTA by CTA); each
// warp counts its own for every expert, the counts become each warp's first place of every
// expert, and each warp goes through its choices again, 32 at a time, and gives them their
// places: the expert's next one, and within the 32 by the lanes before with the same expert.  That takes
// 180 instructions for 32 choices (finding equal experts by a vote a bit no less), which fill one
// cluster's SMs: several clusters count all of them, and each gives some warps' choices their places
// (65536 choices of 256 experts: one cluster 13.9 us, eight 7.9, behind another call 5.8; 256 choices 2.5).
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
  const int copy = blockIdx.x / ctas, copies = gridDim.x / ctas;
  let_next_start();
  for (int i = tid; i < warps * E; i += threads) counted[i] = 0;
  const uint64_t batches = (uint64_t(a.n) + 31) / 32;
  const uint32_t part = rank * warps + warp, parts = ctas * warps;
  const uint32_t b0 = uint32_t(batches * part / parts), b1 = uint32_t(batches * (part + 1) / parts);
  int32_t* mine = counted + warp * E;
  // 32 choices of the warp, the first kKept of them kept; others are read again
  auto choice = [&](uint32_t b) {
    const uint64_t i = uint64_t(b) * 32 + lane;
    const int e = b < b1 && i < a.n ? a.experts[i] : -1;
    return uint32_t(e) < uint32_t(E) ? e : -1;
  };
  wait_for_previous();
  int kept[kKept];
#pragma unroll
  for (int i = 0; i < kKept; ++i) kept[i] = choice(b0 + i);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (kept[i] >= 0) atomicAdd(&mine[kept[i]], 1);
#pragma unroll 4
  for (uint32_t b = b0 + kKept; b < b1; ++b) {
    const int e = choice(b);
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();
  // each warp's first place of an expert among the CTA's
  for (int e = tid; e < E; e += threads) {
    int sum = 0;
    for (int w = 0; w < warps; w += 8) {  // (eight warps at least)
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = counted[(w + i) * E + e];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        counted[(w + i) * E + e] = sum;
        sum += c[i];
      }
    }
    total[e] = sum;
  }
  if (ctas > 1) tc::cluster_sync();
  else __syncthreads();
  int carry = 0;  // choices of the experts before
  for (int base = 0; base < E; base += threads) {
    const int e = base + tid;
    int before = 0, all = 0;
    if (e < E) {
      const uint32_t at = staging::smem_addr(&total[e]);
      int c[kSortCluster];
#pragma unroll
      for (uint32_t r = 0; r < kSortCluster; ++r)
        c[r] = r < ctas ? __float_as_int(tc::load_cluster(tc::in_cta(at, r))) : 0;
#pragma unroll
      for (uint32_t r = 0; r < kSortCluster; ++r) {
        before += r < rank ? c[r] : 0;
        all += c[r];
      }
    }
    int to = all;  // inclusive scan over the CTA
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, to, o);
      if (lane >= o) to += v;
    }
    if (lane == 31) warp_sum[warp] = to;
    __syncthreads();
    const int of_warp = lane < warps ? warp_sum[lane] : 0;
    to += __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0);
    const int chunk = __reduce_add_sync(0xffffffffu, of_warp);
    if (e < E) {
      first[e] = carry + to - all + before;
      if (rank == 0 && copy == 0) a.offsets[e] = carry + to - all;
    }
    carry += chunk;
    __syncthreads();
  }
  if (rank == 0 && copy == 0 && tid == 0) a.offsets[E] = carry;
  if (ctas > 1) tc::cluster_arrive();  // this CTA has read the others' totals
  auto give = [&](uint32_t b, int e) {
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int before = __popc(same & ((1u << lane) - 1));
    int place = -1;
    if (e >= 0) place = first[e] + mine[e] + before;
    __syncwarp();
    if (e >= 0 && before == 0) mine[e] += __popc(same);
    __syncwarp();
    const uint64_t i = uint64_t(b) * 32 + lane;
    if (b < b1 && i < a.n) a.slot[i] = place;
  };
  // (in a loop of few instructions: unrolled, fetching them costs more than running them)
  const bool ours = warp * copies / warps == copy;
#pragma unroll 1
  for (uint32_t b = b0; ours && b < b1; b += kKept) {
    if (b != b0)
#pragma unroll
      for (int i = 0; i < kKept; ++i) kept[i] = choice(b + i);
#pragma unroll 1
    for (uint32_t i = 0; i < kKept && b + i < b1; ++i) {
      give(b + i, kept[0]);
#pragma unroll
      for (int j = 1; j < kKept; ++j) kept[j - 1] = kept[j];
    }
  }
  if (ctas > 1) tc::cluster_wait();
}

// --------------------------------------------------------------------------- dispatch
struct DispatchArgs {
  const unsigned char* x;
  unsigned char* rows;
  float* scale;
  const int32_t* slot;
  int64_t ldx, ldr, lds;  // bytes; floats
  uint32_t tokens, cols;
  uint32_t vecs, chunks;  // accesses of a row; CTAs that share one
  uint32_t nrows;
  uint32_t topk, lanes;    // lanes (in 8 bits: sixteens of lanes) of a token
};

// Each row is read once and written to all of its places.  A thread has four accesses of its row on
// their way, and makes a place's address once for them.
constexpr int kDispatchVecs = 4;    // of a thread
constexpr int kDispatchBlocks = 4;  // of a lane, in 8 bits
template <typename V>
__global__ void __launch_bounds__(256) dispatch_kernel(const __grid_constant__ DispatchArgs a) {
  const uint32_t lane = threadIdx.x & (a.lanes - 1);
  const uint32_t t = blockIdx.x / a.chunks * (256 / a.lanes) + threadIdx.x / a.lanes;
  if (t >= a.tokens) return;
  const uint32_t c0 = blockIdx.x % a.chunks * (kDispatchVecs * a.lanes) + lane;
  let_next_start();
  wait_for_previous();
  const V* x = reinterpret_cast<const V*>(a.x + t * a.ldx) + c0;
  V v[kDispatchVecs];
#pragma unroll
  for (uint32_t i = 0; i < kDispatchVecs; ++i)
    if (c0 + i * a.lanes < a.vecs) v[i] = __ldcs(x + i * a.lanes);
  const int32_t* slot = a.slot + int64_t(t) * a.topk;
  uint32_t s[kPlaces];
  load_places(s, slot, 0, a.topk);
  for (uint32_t j0 = 0; j0 < a.topk; j0 += kPlaces) {
    if (j0) load_places(s, slot, j0, a.topk);
#pragma unroll
    for (uint32_t j = 0; j < kPlaces; ++j) {
      if (s[j] >= a.nrows) continue;
      V* to = reinterpret_cast<V*>(a.rows + s[j] * a.ldr) + c0;
#pragma unroll
      for (uint32_t i = 0; i < kDispatchVecs; ++i)
        if (c0 + i * a.lanes < a.vecs) to[i * a.lanes] = v[i];
    }
  }
}

// The same in 8 bits: sixteen lanes a block of 128 values, which is quantised once; a lane has B
// blocks of its token, so that a place's address is made once for all of them (8192 tokens of 7168
// bf16, 8 choices: 90 us, 6.5 TB/s, against 116 with one block and a 64-bit division for it).  Lane i
// stores the scale of the i-th.  VEC: every row of x starts on 16 bytes, of the 8-bit rows on 8.
template <typename T, bool VEC, int B>
__global__ void __launch_bounds__(256) dispatch_fp8_kernel(const __grid_constant__ DispatchArgs a) {
  const uint32_t sixteenth = threadIdx.x / 16, l = threadIdx.x % 16;
  const uint32_t tt = blockIdx.x / a.chunks * (16 / a.lanes) + sixteenth / a.lanes;
  const bool there = tt < a.tokens;
  const uint32_t t = there ? tt : a.tokens - 1;
  const uint32_t block0 = blockIdx.x % a.chunks * (B * a.lanes) + sixteenth % a.lanes;
  const uint32_t step = a.lanes * 128, col0 = block0 * 128;
  const T* x = reinterpret_cast<const T*>(a.x + t * a.ldx) + col0 + 8 * l;
  const int32_t* slot = a.slot + int64_t(t) * a.topk;
  const uint32_t my_block = block0 + l * a.lanes;
  const bool scales = l < B && there && my_block * 128 < a.cols;
  let_next_start();
  wait_for_previous();
  Eight<T> e[B];
  uint2 q[B];
  float scale = 0.0f;
  auto quantise = [&] {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      float m = e[i].largest();
      for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = scale_of(m);
      if (l == i) scale = s;
      q[i] = e[i].quotients(s);
    }
  };
  // blocks that lie inside the row
  const uint32_t blocks = there && col0 < a.cols ? (a.cols - col0 + step - 1) / step : 0;
  if (VEC && a.cols % 8 == 0) {  // each lane has eight values of a block, or none of the last
    const uint32_t to0 = col0 + 8 * l;
    const uint32_t mine = there && to0 < a.cols ? (a.cols - to0 + step - 1) / step : 0;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (i < mine) e[i].load(x + i * step);
      else if (a.cols % 128 != 0) e[i].load(x, 0);  // zeros beside values
    }
    uint32_t s[kPlaces];
    load_places(s, slot, 0, a.topk);
    quantise();
    for (uint32_t j0 = 0; j0 < a.topk; j0 += kPlaces) {
      if (j0) load_places(s, slot, j0, a.topk);
#pragma unroll
      for (uint32_t j = 0; j < kPlaces; ++j) {
        const uint32_t to = s[j];
        if (to >= a.nrows) continue;
        uint8_t* row = a.rows + to * a.ldr + to0;
        if (scales) a.scale[to * a.lds + my_block] = scale;
#pragma unroll
        for (int i = 0; i < B; ++i)
          if (i < mine) *reinterpret_cast<uint2*>(row + i * step) = q[i];
      }
    }
    return;
  }
  int count[B];  // values of the block that lie inside the row
  bool some[B];  // whether either half of the warp has any
#pragma unroll
  for (int i = 0; i < B; ++i) {
    count[i] = i < blocks ? int(min(a.cols - (col0 + i * step), 128u)) : 0;
    some[i] = __any_sync(0xffffffffu, count[i] > 0);
    if (!some[i]) continue;
    const int left = min(max(count[i] - int(8 * l), 0), 8);
    if (VEC) {
      e[i].load(x + i * step, left);
    } else {
      const T* begin = reinterpret_cast<const T*>(a.x);
      const T* end = reinterpret_cast<const T*>(a.x + (a.tokens - 1) * a.ldx) + a.cols;
      e[i].template load_granules<false>(x + i * step, begin, end);
      e[i].align(x + i * step, left);
    }
  }
  quantise();
#pragma unroll 1
  for (uint32_t j = 0; j < a.topk; ++j) {
    const uint32_t to = uint32_t(slot[j]);
    const bool on = to < a.nrows && there;
    uint8_t* row = a.rows + (on ? to * a.ldr + col0 : 0);
    if (on && scales) a.scale[to * a.lds + my_block] = scale;
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (some[i]) store_row(row + i * step, q[i], on ? count[i] : 0);
  }
}

// ---------------------------------------------------------------------------- combine
struct CombineArgs {
  const unsigned char *rows, *dout;
  unsigned char *out, *drows;
  const int32_t* slot;
  const float* weight;
  float* dweight;
  int64_t ldr, ldo;        // bytes
  uint32_t tokens, cols, vecs;  // accesses of a row
  uint32_t chunks, span;   // CTAs that share a row, and their accesses
  uint32_t nrows, topk, lanes;
};

// Elements of one access of W bytes as they lie in memory: whole words, which the compiler would
// take apart into a register an element, and their values.
template <typename T, int W>
struct Access {
  static_assert(W >= int(sizeof(T)), "whole elements");
  static constexpr int kWords = W < 4 ? 1 : W / 4, kElements = W / int(sizeof(T));
  uint32_t word[kWords];

  // Zeros, or what lies at `at` where `on`: one predicated instruction, behind which the next load
  // follows at once (as a branch the compiler draws what is done with the values into it, so that
  // one load waits for another: 158 us for 4096 x 8 rows of 7168 instead of 85).
  __device__ void load_if(bool on, const unsigned char* at) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) word[i] = 0;
    if constexpr (W == 16) {
      asm volatile("{.reg .pred p; setp.ne.u32 p, %5, 0; @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];}"
                   : "+r"(word[0]), "+r"(word[1]), "+r"(word[2]), "+r"(word[3])
                   : "l"(at), "r"(uint32_t(on)));
    } else if constexpr (W == 8) {
      asm volatile("{.reg .pred p; setp.ne.u32 p, %3, 0; @p ld.global.v2.u32 {%0, %1}, [%2];}"
                   : "+r"(word[0]), "+r"(word[1])
                   : "l"(at), "r"(uint32_t(on)));
    } else if constexpr (W == 4) {
      asm volatile("{.reg .pred p; setp.ne.u32 p, %2, 0; @p ld.global.u32 %0, [%1];}"
                   : "+r"(word[0])
                   : "l"(at), "r"(uint32_t(on)));
    } else {
      asm volatile("{.reg .pred p; setp.ne.u32 p, %2, 0; @p ld.global.u16 %0, [%1];}"
                   : "+r"(word[0])
                   : "l"(at), "r"(uint32_t(on)));
    }
  }
  __device__ void load(const unsigned char* at) {
    if constexpr (W == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(at);
      word[0] = v.x, word[1] = v.y, word[2] = v.z, word[3] = v.w;
    } else if constexpr (W == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(at);
      word[0] = v.x, word[1] = v.y;
    } else if constexpr (W == 4) {
      word[0] = *reinterpret_cast<const uint32_t*>(at);
    } else {
      word[0] = *reinterpret_cast<const uint16_t*>(at);
    }
  }
  __device__ void store(unsigned char* at) const {
    if constexpr (W == 16) *reinterpret_cast<uint4*>(at) = make_uint4(word[0], word[1], word[2], word[3]);
    else if constexpr (W == 8) *reinterpret_cast<uint2*>(at) = make_uint2(word[0], word[1]);
    else if constexpr (W == 4) *reinterpret_cast<uint32_t*>(at) = word[0];
    else *reinterpret_cast<uint16_t*>(at) = uint16_t(word[0]);
  }
  __device__ float value(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(word[i]);
    const uint32_t w = word[i / 2];
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
    else
      return __half2float(__ushort_as_half(uint16_t(i % 2 ? w >> 16 : w)));
  }
  __device__ void set(const float (&f)[kElements]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kElements; ++i) word[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kElements; i += 2) {
        const float2 v = make_float2(f[i], i + 1 < kElements ? f[i + 1] : 0.0f);
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          const __nv_bfloat162 h = __float22bfloat162_rn(v);
          word[i / 2] = reinterpret_cast<const uint32_t&>(h);
        } else {
          const __half2 h = __float22half2_rn(v);
          word[i / 2] = reinterpret_cast<const uint32_t&>(h);
        }
      }
    }
  }
};

constexpr int kTogether = 8;  // choices whose rows are on their way at a time

// out = sum of weight x row over a token's choices, in float32 in the order of the choices.  A CTA
// has `span` accesses of its tokens' rows: with whole rows its warps have the rows of 8 choices on their
// way one after another.  80 registers, so that three CTAs an SM do (83 us for 4096 x 8 rows of 7168;
// 97 us without that limit).
template <typename T, int W>
__global__ void __launch_bounds__(256, 3) combine_kernel(const __grid_constant__ CombineArgs a) {
  using A = Access<T, W>;
  constexpr int N = A::kElements;
  const uint32_t lane = threadIdx.x & (a.lanes - 1);
  const uint32_t t = blockIdx.x / a.chunks * (256 / a.lanes) + threadIdx.x / a.lanes;
  if (t >= a.tokens) return;
  const uint32_t c0 = blockIdx.x % a.chunks * a.span + lane, c1 = min(c0 - lane + a.span, a.vecs);
  const int64_t first = int64_t(t) * a.topk;
  unsigned char* out = a.out + t * a.ldo;
  const unsigned char* row[kTogether];
  float w[kTogether];
  auto places = [&](uint32_t j0) {
#pragma unroll
    for (uint32_t j = 0; j < kTogether; ++j) {
      const uint32_t s = j0 + j < a.topk ? uint32_t(a.slot[first + j0 + j]) : 0xffffffffu;
      w[j] = s < a.nrows && a.weight ? a.weight[first + j0 + j] : 1.0f;
      row[j] = s < a.nrows ? a.rows + s * a.ldr : nullptr;
    }
  };
  auto add = [&](float(&sum)[N], uint32_t c) {
    A v[kTogether];
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      v[j].load_if(row[j] != nullptr, row[j] + c * uint64_t(W));
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] = fmaf(w[j], v[j].value(i), sum[i]);
  };
  let_next_start();
  wait_for_previous();
  places(0);
  for (uint32_t c = c0; c < c1; c += a.lanes) {
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.0f;
    add(sum, c);
    if (a.topk > kTogether) {
      for (uint32_t j0 = kTogether; j0 < a.topk; j0 += kTogether) places(j0), add(sum, c);
      places(0);
    }
    A v;
    v.set(sum);
    v.store(out + c * uint64_t(W));
  }
}

// drows = weight x dout at the places of a token's choices; dweight = the products of dout with
// its rows, float32 chains of a lane joined in one order.  dout and each row are read once.  LANES: of a
// token, a warp or a CTA.  (80 registers; with 16-byte accesses and dweight 20 to 36 bytes are spilled.)
template <typename T, int W, int LANES, bool DOT>
__global__ void __launch_bounds__(256, 3) combine_grad_kernel(const __grid_constant__ CombineArgs a) {
  using A = Access<T, W>;
  constexpr int N = A::kElements;
  __shared__ float part[8][kTogether];
  const uint32_t lane = threadIdx.x % LANES, warp = threadIdx.x / 32;
  const uint32_t t = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (t >= a.tokens) return;  // (whole warps, and with a CTA a token none)
  const int64_t first = int64_t(t) * a.topk;
  const unsigned char* dout = a.dout + t * a.ldo;
  let_next_start();
  wait_for_previous();
  for (uint32_t j0 = 0; j0 < a.topk; j0 += kTogether) {
    const uint32_t together = min(uint32_t(kTogether), a.topk - j0);
    uint32_t s[kTogether];
    float w[kTogether], dot[kTogether];
#pragma unroll
    for (uint32_t j = 0; j < kTogether; ++j) {
      s[j] = j < together ? uint32_t(a.slot[first + j0 + j]) : 0xffffffffu;
      w[j] = j < together && a.weight ? a.weight[first + j0 + j] : 1.0f;
      dot[j] = 0.0f;
    }
    for (uint32_t c = lane; c < a.vecs; c += LANES) {
      A d, r[kTogether];
      d.load(dout + c * uint64_t(W));
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        if (DOT) r[j].load_if(s[j] < a.nrows, a.rows + s[j] * a.ldr + c * uint64_t(W));
      }
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        if (s[j] >= a.nrows) continue;
        if (DOT) {
#pragma unroll
          for (int i = 0; i < N; ++i) dot[j] = fmaf(d.value(i), r[j].value(i), dot[j]);
        }
        if (!a.drows) continue;
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = w[j] * d.value(i);
        A g;
        g.set(f);
        g.store(a.drows + s[j] * a.ldr + c * uint64_t(W));
      }
    }
    if constexpr (DOT) {
#pragma unroll
      for (int j = 0; j < kTogether; ++j) dot[j] = warp_sum(dot[j]);
      float* to = a.dweight + first + j0;
      if (LANES == 32) {
        if (lane == 0)
          for (uint32_t j = 0; j < kTogether; ++j)
            if (j < together) to[j] = dot[j];
      } else {
        if (threadIdx.x % 32 == 0)
          for (int j = 0; j < kTogether; ++j) part[warp][j] = dot[j];
        __syncthreads();
        if (threadIdx.x < together) {
          float sum = 0.0f;
          for (int i = 0; i < 8; ++i) sum += part[i][threadIdx.x];
          to[threadIdx.x] = sum;
        }
        __syncthreads();
      }
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

// f(std::integral_constant<int, W>()) with W the widest access, from LEAST bytes, those of an element, to 16.
template <size_t LEAST, typename F>
reshard_status_t by_width(std::initializer_list<const void*> pointers, std::initializer_list<int64_t> bytes, F&& f) {
  if (all_aligned(16, pointers, bytes)) return f(std::integral_constant<int, 16>());
  if (all_aligned(8, pointers, bytes)) return f(std::integral_constant<int, 8>());
  if constexpr (LEAST == 2)
    if (!all_aligned(4, pointers, bytes)) return f(std::integral_constant<int, 2>());
  return f(std::integral_constant<int, 4>());
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

// Launches `grid` CTAs of 256 threads, which may start before the kernel in front of them has ended.
template <auto Kernel, typename Args>
reshard_status_t start(const char* what, int64_t grid, cudaStream_t stream, const Args& a) {
  void* args[] = {const_cast<Args*>(&a)};
  return launch<Kernel, 0>(what, 0, {grid, 256, 0, 0, stream}, args);
}

// Whether rows go in shifted granules: of 16-bit elements, long enough for a warp's worth, and not
// aligned to `least` bytes.  4096 x 8 rows of 7169 bf16, in accesses of an element and shifted: to their
// places 128 and 105 us, back 154 and 119, gradients 278 and 229; of 7170, in accesses of two elements
// and shifted: 106 and 102, 103 and 120, 199 and 225 (4099 x 6 rows of 4098 to their places 43 and 40).  So
// least is 8 to their places, else 4.  (Few tokens lose by it, 32 x 8 rows of 7170 2.3 and 9.2 us.)  Rows of
// 131 columns, 8192 x 4 of them, would gain (18 and 11, 17 and 7, 25 and 13 us), of 255 not (18 and 25, 19
// and 10, 26 and 26), and few tokens would lose (128: 1.9 and 2.5, 1.8 and 2.4, 2.1 and 3.1): from 256 on.
bool goes_shifted(int64_t size, int64_t cols, int64_t least, std::initializer_list<const void*> pointers,
                  std::initializer_list<int64_t> bytes) {
  return size == 2 && cols >= 256 && !all_aligned(least, pointers, bytes);
}
// Columns from which a CTA has a token of them, else a warp.  CTA and warp, 4 choices of 1027 columns: 128
// tokens to their places 2.9 and 6.1 us, back 2.7 and 5.6, gradients 3.9 and 8.4; 8192 tokens 19 and 20, 25 and
// 20, 72 and 38.  Of 515: 128 tokens 2.7 and 3.9, 2.5 and 3.7, 3.7 and 5.3; 8192 13 and 11, 19 and 11, 50 and 18.
constexpr int64_t kLongRow = 1024;

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
  // one CTA up to kKept times 32 choices for each of its warps; a warp for each 32 choices while
  // there are few, and no more than the counts of shared memory
  int64_t warps = 8;
  while (warps < 32 && warps * 32 < n) warps *= 2;
  while ((warps + 2) * nexperts * 4 > int64_t(rs::kSortSmem)) warps /= 2;
  const int ctas = n <= warps * 32 * rs::kKept ? 1 : rs::kSortCluster;
  void* args[] = {&a};
  // clusters that share the places: a warp of each scheduler has some in all of them
  const int64_t copies = n <= ctas * warps * 32 || warps < 8 ? 1 : warps / 4;
  return rs::op::launch<rs::sort_kernel, rs::kSortSmem>(
      "reshard_expert_sort", dev,
      {copies * ctas, int(32 * warps), size_t((warps + 2) * nexperts * 4), ctas, st, true}, args);
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
  a.tokens = uint32_t(tokens);
  a.cols = uint32_t(cols);
  a.nrows = uint32_t(nrows);
  a.topk = uint32_t(topk);
  if (scale) {
    // sixteen lanes a block: as many of a CTA's sixteen on one token as it has blocks for
    a.lanes = 1;
    while (a.lanes < 16 && a.lanes < blocks) a.lanes *= 2;
    const bool vec = rs::all_aligned(16, {x}, {a.ldx}) && rs::all_aligned(8, {rows}, {a.ldr});
    // four blocks a lane where every SM has a few CTAs all the same, and five eighths of them are blocks of
    // the row (4096 tokens to 8 places: 5120 columns 39.7 us, with one block 42.3; 4096 columns 36.6 and 31.6)
    const int64_t four = rs::kDispatchBlocks * int64_t(a.lanes), fours = rs::op::cdiv(blocks, four);
    const bool many = tokens * blocks >= 64 * 1024 && blocks * 8 >= fours * four * 5;
    const int64_t chunks = many ? fours : rs::op::cdiv(blocks, int64_t(a.lanes));
    const int64_t grid = rs::op::cdiv(tokens, 16 / a.lanes) * chunks;
    a.chunks = uint32_t(chunks);
    if (const reshard_status_t s = rs::too_many(grid); s != RESHARD_OK) return s;
    return rs::op::by_dtype(dtype, [&](auto t) {
      using T = decltype(t);
      constexpr int B = rs::kDispatchBlocks;
      if (vec && many) return rs::start<rs::dispatch_fp8_kernel<T, true, B>>("reshard_expert_dispatch", grid, st, a);
      if (vec) return rs::start<rs::dispatch_fp8_kernel<T, true, 1>>("reshard_expert_dispatch", grid, st, a);
      if (many) return rs::start<rs::dispatch_fp8_kernel<T, false, B>>("reshard_expert_dispatch", grid, st, a);
      return rs::start<rs::dispatch_fp8_kernel<T, false, 1>>("reshard_expert_dispatch", grid, st, a);
    });
  }
  if (rs::goes_shifted(size, cols, 8, {x, rows}, {a.ldx, a.ldr, cols * size})) {
    const bool cta = cols >= rs::kLongRow;  // (elements are moved as they are: one type does)
    const int64_t grid = cta ? tokens : rs::op::cdiv(tokens, 8);
    return cta ? rs::start<rs::shifted::dispatch_kernel<__half, 256, rs::DispatchArgs>>("reshard_expert_dispatch", grid, st, a)
               : rs::start<rs::shifted::dispatch_kernel<__half, 32, rs::DispatchArgs>>("reshard_expert_dispatch", grid, st, a);
  }
  // (accesses know no type: two bytes serve none that is aligned to four)
  return rs::by_width<2>({x, rows}, {a.ldx, a.ldr, cols * size}, [&](auto w) {
    const int64_t vecs = cols * size / w;
    a.lanes = uint32_t(rs::lanes_of(vecs));
    const int64_t chunks = rs::op::cdiv(vecs, rs::kDispatchVecs * int64_t(a.lanes));
    const int64_t grid = rs::op::cdiv(tokens, 256 / a.lanes) * chunks;
    a.vecs = uint32_t(vecs);
    a.chunks = uint32_t(chunks);
    if (const reshard_status_t s = rs::too_many(grid); s != RESHARD_OK) return s;
    return rs::start<rs::dispatch_kernel<typename rs::Word<w>::type>>("reshard_expert_dispatch", grid, st, a);
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
  a.rows = static_cast<const unsigned char*>(rows);
  a.out = static_cast<unsigned char*>(out);
  a.slot = slot;
  a.weight = weight;
  a.ldr = ldr * size;
  a.ldo = ldo * size;
  a.tokens = uint32_t(tokens);
  a.nrows = uint32_t(nrows);
  a.topk = uint32_t(topk);
  a.cols = uint32_t(cols);
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if constexpr (sizeof(T) == 2) {
      if (rs::goes_shifted(size, cols, 4, {rows, out}, {a.ldr, a.ldo, cols * size})) {
        const bool cta = cols >= rs::kLongRow;
        const int64_t grid = cta ? tokens : rs::op::cdiv(tokens, 8);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        return cta ? rs::start<rs::shifted::combine_kernel<T, 256, rs::CombineArgs>>("reshard_expert_combine", grid, st, a)
                   : rs::start<rs::shifted::combine_kernel<T, 32, rs::CombineArgs>>("reshard_expert_combine", grid, st, a);
      }
    }
    return rs::by_width<sizeof(T)>({rows, out}, {ldr * size, ldo * size, cols * size}, [&](auto w) {
      const int64_t vecs = cols * size / w, lanes = rs::lanes_of(vecs), groups = rs::op::cdiv(tokens, 256 / lanes);
      // a CTA a whole row, or so much of it that there are some 2048 of them (8 choices of 7168 bf16, with 512,
      // 2048 and 8192: 200 tokens 3.5, 4.2 and 4.2 us, 1000 23.4, 22.9 and 23.9, 2048 42.1, 42.0 and 45.5)
      int64_t rounds = rs::op::cdiv(vecs, lanes);
      if (groups * rounds > 2048) rounds = rs::op::cdiv(groups * rounds, 2048) < rounds ? rs::op::cdiv(groups * rounds, 2048) : rounds;
      else rounds = 1;
      const int64_t chunks = rs::op::cdiv(vecs, lanes * rounds), grid = groups * chunks;
      a.vecs = uint32_t(vecs);
      a.lanes = uint32_t(lanes);
      a.span = uint32_t(lanes * rounds);
      a.chunks = uint32_t(chunks);
      if (const reshard_status_t s = rs::too_many(grid); s != RESHARD_OK) return s;
      return rs::start<rs::combine_kernel<T, w>>("reshard_expert_combine", grid, static_cast<cudaStream_t>(stream), a);
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
  a.rows = static_cast<const unsigned char*>(rows);
  a.dout = static_cast<const unsigned char*>(dout);
  a.drows = static_cast<unsigned char*>(drows);
  a.slot = slot;
  a.weight = weight;
  a.dweight = dweight;
  a.ldr = ldr * size;
  a.ldo = ldo * size;
  a.tokens = uint32_t(tokens);
  a.nrows = uint32_t(nrows);
  a.topk = uint32_t(topk);
  a.cols = uint32_t(cols);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return rs::op::by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const void* read = dweight ? rows : nullptr;
    const char* what = "reshard_expert_combine_grad";
    if constexpr (sizeof(T) == 2) {
      if (rs::goes_shifted(size, cols, 4, {dout, read, drows}, {a.ldr, a.ldo, cols * size})) {
        const bool cta = cols >= rs::kLongRow;
        const int64_t grid = cta ? tokens : rs::op::cdiv(tokens, 8);
        using rs::CombineArgs;
        using namespace rs::shifted;
        if (dweight && cta) return rs::start<combine_grad_kernel<T, 256, true, CombineArgs>>(what, grid, st, a);
        if (dweight) return rs::start<combine_grad_kernel<T, 32, true, CombineArgs>>(what, grid, st, a);
        if (cta) return rs::start<combine_grad_kernel<T, 256, false, CombineArgs>>(what, grid, st, a);
        return rs::start<combine_grad_kernel<T, 32, false, CombineArgs>>(what, grid, st, a);
      }
    }
    return rs::by_width<sizeof(T)>({dout, read, drows}, {ldr * size, ldo * size, cols * size}, [&](auto w) {
      a.vecs = uint32_t(cols * size / w);
      // a CTA a token, else a warp (4 choices: 2048 bf16 columns, 256 accesses, 128 tokens 2.9 and 7.2 us, 8192
      // tokens 60 and 55; 1024 columns 2.5 and 4.5, 47 and 29)
      const bool cta = a.vecs > 128;
      const int64_t grid = cta ? tokens : rs::op::cdiv(tokens, 8);
      if (const reshard_status_t s = rs::too_many(grid); s != RESHARD_OK) return s;
      if (dweight && cta) return rs::start<rs::combine_grad_kernel<T, w, 256, true>>(what, grid, st, a);
      if (dweight) return rs::start<rs::combine_grad_kernel<T, w, 32, true>>(what, grid, st, a);
      if (cta) return rs::start<rs::combine_grad_kernel<T, w, 256, false>>(what, grid, st, a);
      return rs::start<rs::combine_grad_kernel<T, w, 32, false>>(what, grid, st, a);
    });
  });
}
