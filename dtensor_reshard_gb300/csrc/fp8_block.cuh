// fp8_block.cuh -- a block of 128 values as sixteen lanes hold it, its scale and its e4m3
// quotients: what fp8_quantize.cu and experts.cu make 8-bit values of.
#pragma once

#include "operators.cuh"
#include "tensor_core.cuh"

namespace rs {
namespace op {

constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: a block of zeros

// x / scale, correctly rounded, two at a time: Markstein's division (IBM Journal of Research
// and Development 34, 1990) -- with the correctly rounded reciprocal y, a quotient within one
// unit in the last place becomes the correctly rounded one by one more step of
// q + (x - q * scale) * y, and the first such step brings x * y within that unit.  No
// remainder underflows unless the quotient is below 2^-12, which e4m3 rounds to 0 anyway.
//
// The quotient is carried with its sign changed: a remainder of zero is +0, which must be taken
// from, not added to, a quotient of -0 for that to stay -0.
struct Divisor {
  uint64_t s2, minus_y;
  __device__ explicit Divisor(float s) {
    const uint32_t m = __float_as_uint(s), r = __float_as_uint(-__frcp_rn(s));
    s2 = tc::pack2(m, m);
    minus_y = tc::pack2(r, r);
  }
  // Blocks for which that holds; others (tiny or infinite scales) are divided one by one.
  __device__ static bool serves(float s) { return s >= 0x1p-90f && s < INFINITY; }
  __device__ float2 divide(float2 v) const {
    const uint64_t x = tc::pack2(__float_as_uint(v.x), __float_as_uint(v.y));
    uint64_t q;  // -x / s
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(minus_y));
    q = tc::fma2(tc::fma2(s2, q, x), minus_y, q);
    q = tc::fma2(tc::fma2(s2, q, x), minus_y, q);
    const float2 f = tc::unpack2(q);
    return make_float2(-f.x, -f.y);
  }
};

__device__ __forceinline__ float largest_magnitude(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}
// 16-bit values two at a time, with the signs taken off.
template <typename T>
__device__ __forceinline__ float largest_magnitude(const T (&v)[8]) {
  alignas(4) T a[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<uint32_t*>(a)[i] = reinterpret_cast<const uint32_t*>(v)[i] & 0x7fff7fffu;
  return fmaxf(largest_of(a), 0.0f);
}

// Eight values of a row, as they lie in memory.
template <typename T>
struct Eight {
  uint4 v[sizeof(T) / 2];
  __device__ void load(const T* row) {  // starts on 16 bytes
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(row) + i);
  }
  __device__ void load(const T* row, int left) {  // `left` of them inside the matrix, else 0
    T* e = reinterpret_cast<T*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < left ? row[i] : from_float<T>(0.0f);
  }
  // The same at any alignment, by sixteen neighbouring lanes of one row at once: aligned
  // 16-byte granules, of which a lane takes the one behind its own from the next lane.
  static constexpr int kGranules = int(sizeof(T)) / 2;  // of eight values
  static constexpr int kPer = 16 / int(sizeof(T));      // values of a granule
  __device__ static const T* granule_of(const T* row) {
    return row - reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T);
  }
  // INSIDE: all granules lie inside [begin, end); else what lies outside is not read.
  template <bool INSIDE>
  __device__ static uint4 fetch(const T* from, const T* begin, const T* end) {
    if (INSIDE || (from >= begin && from + kPer <= end))
      return __ldcs(reinterpret_cast<const uint4*>(from));
    uint4 part = make_uint4(0, 0, 0, 0);
    T* e = reinterpret_cast<T*>(&part);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (from + i >= begin && from + i < end) e[i] = from[i];
    return part;
  }
  uint4 behind;
  template <bool INSIDE>
  __device__ void load_granules(const T* row, const T* begin, const T* end) {
    const T* first = granule_of(row);
#pragma unroll
    for (int i = 0; i < kGranules; ++i) v[i] = fetch<INSIDE>(first + i * kPer, begin, end);
    behind = fetch<INSIDE>(threadIdx.x % 16 == 15 ? first + kGranules * kPer : first, begin, end);
  }
  __device__ void align(const T* row, int left) {
    const uint32_t skew = uint32_t(reinterpret_cast<uintptr_t>(row) % 16);
    uint4 next;
    next.x = __shfl_down_sync(0xffffffffu, v[0].x, 1, 16);
    next.y = __shfl_down_sync(0xffffffffu, v[0].y, 1, 16);
    next.z = __shfl_down_sync(0xffffffffu, v[0].z, 1, 16);
    next.w = __shfl_down_sync(0xffffffffu, v[0].w, 1, 16);
    if (threadIdx.x % 16 == 15) next = behind;
#pragma unroll
    for (int i = 0; i < kGranules; ++i)
      v[i] = staging::funnel16(v[i], i + 1 < kGranules ? v[i + 1] : next, skew / 4,
                               0x3210u + 0x1111u * (skew % 4));
    if (left >= 8) return;
    T* e = reinterpret_cast<T*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < left ? e[i] : from_float<T>(0.0f);
  }
  __device__ float2 pair(int i) const {
    const T* e = reinterpret_cast<const T*>(v);
    return make_float2(to_float(e[2 * i]), to_float(e[2 * i + 1]));
  }
  __device__ float largest() const {  // in magnitude; a NaN loses against any number
    return largest_magnitude(reinterpret_cast<const T(&)[8]>(v));
  }
  __device__ uint2 quotients(float s) const {
    uint32_t out[4];
    if (Divisor::serves(s)) {
      const Divisor d(s);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out[i] = __nv_cvt_float2_to_fp8x2(d.divide(pair(i)), __NV_SATFINITE, __NV_E4M3);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out[i] = __nv_cvt_float2_to_fp8x2(make_float2(pair(i).x / s, pair(i).y / s), __NV_SATFINITE,
                                          __NV_E4M3);
    }
    return make_uint2(out[0] | out[1] << 16, out[2] | out[3] << 16);
  }
};
// Eight bytes a lane from sixteen neighbouring lanes to a row's `count` bytes (at most 128)
// at any alignment: each lane stores the aligned eight bytes that end in its own, and what
// is left at both ends goes out in the widest stores that are aligned.
__device__ __forceinline__ void store_row(uint8_t* row, uint2 q, int count) {
  const int lane = threadIdx.x % 16;
  const uint32_t skew = uint32_t(reinterpret_cast<uintptr_t>(row) % 8);
  uint8_t* to = row + 8 * lane;
  if (__all_sync(0xffffffffu, count == 128)) {
    const uint32_t before_x = __shfl_up_sync(0xffffffffu, q.x, 1, 16);
    const uint32_t before_y = __shfl_up_sync(0xffffffffu, q.y, 1, 16);
    const uint64_t own = q.x | uint64_t(q.y) << 32, before = before_x | uint64_t(before_y) << 32;
    if (lane > 0 || skew == 0)
      *reinterpret_cast<uint64_t*>(to - skew) = skew ? own << (8 * skew) | before >> (64 - 8 * skew) : own;
    if (skew != 0 && (lane == 0 || lane == 15)) {
      // lane 0: up to the next aligned eight bytes; lane 15: the last `skew` bytes
      const bool head = lane == 0;
      uint32_t i = head ? 0 : 8 - skew;
      auto step = [&](uint32_t n) {
        const uint64_t v = own >> (8 * i);
        if (n == 4) *reinterpret_cast<uint32_t*>(to + i) = uint32_t(v);
        if (n == 2) *reinterpret_cast<uint16_t*>(to + i) = uint16_t(v);
        if (n == 1) to[i] = uint8_t(v);
        i += n;
      };
      const uint32_t n = head ? 8 - skew : skew;
      if (head) {
        if (n & 1) step(1);
        if (n & 2) step(2);
        if (n & 4) step(4);
      } else {
        if (n & 4) step(4);
        if (n & 2) step(2);
        if (n & 1) step(1);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * lane + i < count) to[i] = uint8_t((i < 4 ? q.x : q.y) >> (8 * (i % 4)));
  }
}

__device__ __forceinline__ float scale_of(float largest) {
  return fmaxf(largest / kE4m3Max, kScaleMin);
}

}  // namespace op
}  // namespace rs
