// vocab_row.cuh -- a row of logits as logprob.cu and distill.cu take it: granules of 16 aligned
// bytes at any alignment of the row, and exponentials relative to a maximum two at a time.
#pragma once

#include <type_traits>

#include "operators.cuh"
#include "tensor_core.cuh"

namespace rs {
namespace vocab {

using namespace op;

template <typename T>
__host__ __device__ constexpr float largest_finite() {
  return sizeof(T) == 4 ? 3.402823466e38f : 3.389531390e38f;
}
template <>
__host__ __device__ constexpr float largest_finite<__half>() { return 65504.0f; }

// A logit as it counts: +inf as the type's largest finite value, so that differences of two
// logits are never NaN; NaN as -inf; -0 as +0.
template <typename T>
__device__ __forceinline__ float clean(float l) {
  return l == l ? fminf(l, largest_finite<T>()) + 0.0f : -INFINITY;
}

// Whole numbers in the order of the floats, and back.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

constexpr float kLargest = 3.402823466e38f;
// 1 / T as a factor: 1 for T <= 0 and NaN; never infinite, and never 0 (a logit of -inf has the
// exponent -inf at any temperature).
__device__ __forceinline__ float inverse_of(const float* temperature, int64_t r) {
  const float t = temperature ? temperature[r] : 1.0f;
  return t > 0.0f ? fminf(fmaxf(1.0f / t, 0x1p-126f), kLargest) : 1.0f;
}
// A gradient's factor, finite where its gradient g is, and at most `most`: 0 times it is 0.
__device__ __forceinline__ float factor_of(float x, float g, float most = kLargest) {
  return fabsf(g) < INFINITY ? fminf(fmaxf(x, -most), most) : x;
}
// The same for powers of 2.
__device__ __forceinline__ float log2_scale(float inverse) {
  return fminf(1.4426950408889634f * inverse, kLargest);
}
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint64_t both(float v) {
  return tc::pack2(__float_as_uint(v), __float_as_uint(v));
}
__device__ __forceinline__ uint64_t pair(float2 v) {
  return tc::pack2(__float_as_uint(v.x), __float_as_uint(v.y));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum2(uint64_t v) {
  const float2 f = tc::unpack2(v);
  return f.x + f.y;
}
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Exponents below this give 0 (and stay finite: 0 times one is 0).  The maximum also takes
// the place of NaN, and of -inf.
constexpr float kLeast = -200.0f;
__device__ __forceinline__ float exponent(float x, float m, float c) { return fmaxf((x - m) * c, kLeast); }
__device__ __forceinline__ uint64_t exponents(uint64_t x, uint64_t minus_m, uint64_t c) {
  const float2 z = tc::unpack2(mul2(add2(x, minus_m), c));
  return pair(make_float2(fmaxf(z.x, kLeast), fmaxf(z.y, kLeast)));
}
__device__ __forceinline__ uint64_t exp2_both(uint64_t z) {
  const float2 f = tc::unpack2(z);
  return pair(make_float2(exp2_of(f.x), exp2_of(f.y)));
}

__device__ __forceinline__ float2 pair_of(const float* e) { return make_float2(e[0], e[1]); }
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* e) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(e));
}
__device__ __forceinline__ float2 pair_of(const __half* e) {
  return __half22float2(*reinterpret_cast<const __half2*>(e));
}
__device__ __forceinline__ void set_pair(float* to, float2 x) { to[0] = x.x, to[1] = x.y; }
__device__ __forceinline__ void set_pair(__nv_bfloat16* to, float2 x) {
  *reinterpret_cast<__nv_bfloat162*>(to) = __float22bfloat162_rn(x);
}
__device__ __forceinline__ void set_pair(__half* to, float2 x) {
  *reinterpret_cast<__half2*>(to) = __float22half2_rn(x);
}

// A CTA's slice of a row: granules of 16 aligned bytes, and what is left of the row at both ends,
// fewer elements than a granule has, one a thread.
template <typename T>
struct Slice {
  static constexpr int kPer = 16 / int(sizeof(T));
  const T* row;
  int vocab;
  int head, last;  // elements before the row's first granule; the first one behind its last
  int first;       // index of the slice's first element
  int n;           // granules of the slice

  __device__ Slice(const void* logits, int64_t r, int64_t ld, int64_t vocab_, int part, int parts)
      : row(static_cast<const T*>(logits) + r * ld), vocab(int(vocab_)) {
    head = min(vocab, int((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T)));
    const int granules = (vocab - head) / kPer;
    last = head + granules * kPer;
    const int a = int(int64_t(granules) * part / parts);
    first = head + a * kPer;
    n = int(int64_t(granules) * (part + 1) / parts) - a;
  }
  __device__ const uint4* granules() const { return reinterpret_cast<const uint4*>(row + first); }
  // The element at the row's ends that is this thread's, or -1.
  __device__ int edge() const {
    const int i = int(threadIdx.x) < head ? int(threadIdx.x) : int(threadIdx.x) - head + last;
    return i < vocab ? i : -1;
  }
  __device__ float at(int i) const { return clean<T>(to_float(row[i])); }
  __device__ static uint4 nothing() {
    alignas(16) T v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = from_float<T>(-INFINITY);
    return *reinterpret_cast<const uint4*>(v);
  }
};

// A granule to a row whose elements lie at `to`; ALIKE: on 16 bytes as those it was made of.
template <bool ALIKE, typename T>
__device__ __forceinline__ void store_granule(T* to, const uint4& v) {
  if (ALIKE) {
    __stcs(reinterpret_cast<uint4*>(to), v);
    return;
  }
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int j = 0; j < Slice<T>::kPer; ++j) to[j] = e[j];
}
// The same of a whole warp whose lanes have granules next to each other: each lane stores the 16
// aligned bytes that end in its own granule, the first and the last the elements that are left at both
// ends (gradient of 2048 x 131072 bf16: 241 us, element by element 483; in float32, whose elements are
// twice as wide, 349 against 309).
template <bool ALIKE, typename T>
__device__ __forceinline__ void store_granules(T* to, const uint4& v) {
  if (ALIKE || sizeof(T) == 4) return store_granule<ALIKE>(to, v);
  constexpr int kPer = Slice<T>::kPer;
  const int lane = threadIdx.x % 32;
  const uint32_t skew = uint32_t(reinterpret_cast<uintptr_t>(to) % 16);  // bytes, alike in all lanes
  if (skew == 0) {
    __stcs(reinterpret_cast<uint4*>(to), v);
    return;
  }
  uint4 before;
  before.x = __shfl_up_sync(0xffffffffu, v.x, 1);
  before.y = __shfl_up_sync(0xffffffffu, v.y, 1);
  before.z = __shfl_up_sync(0xffffffffu, v.z, 1);
  before.w = __shfl_up_sync(0xffffffffu, v.w, 1);
  const uint32_t shift = 16 - skew;  // of the two granules' bytes, those from here on
  const uint4 out = staging::funnel16(before, v, shift / 4, 0x3210u + 0x1111u * (shift % 4));
  if (lane > 0) __stcs(reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(to) - skew), out);
  const int in_front = kPer - int(skew / sizeof(T));  // elements up to the next 16 bytes
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if ((lane == 0 && j < in_front) || (lane == 31 && j >= in_front)) to[j] = e[j];
}

// The largest value of some granules: a NaN loses against any number, or (_or_nan) wins.
template <typename T, int N>
__device__ __forceinline__ float largest_in(const uint4 (&v)[N]) {
  return largest_of(reinterpret_cast<const T(&)[N * Slice<T>::kPer]>(v));
}
// +inf as the largest finite value, in place.
template <typename T, int N>
__device__ __forceinline__ void make_finite(uint4 (&v)[N]) {
  T* e = reinterpret_cast<T*>(v);
#pragma unroll
  for (int i = 0; i < N * Slice<T>::kPer; ++i)
    if (to_float(e[i]) == INFINITY) e[i] = from_float<T>(largest_finite<T>());
}

template <typename T, int N>
__device__ __forceinline__ float largest_or_nan(const uint4 (&v)[N]) {
  if constexpr (sizeof(T) == 4) {
    const float* e = reinterpret_cast<const float*>(v);
    float m = e[0];
#pragma unroll
    for (int i = 1; i < 4 * N; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(e[i]));
    return m;
  } else {
    using P = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const P* e = reinterpret_cast<const P*>(v);
    P m = e[0];
#pragma unroll
    for (int i = 1; i < 4 * N; ++i) m = __hmax2_nan(m, e[i]);
    float f = to_float(m.x);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(f) : "f"(to_float(m.y)));
    return f;
  }
}
// NaN as -inf and +inf as the largest finite value, in place.
template <typename T, int N>
__device__ __forceinline__ void make_clean(uint4 (&v)[N]) {
  T* e = reinterpret_cast<T*>(v);
#pragma unroll
  for (int i = 0; i < N * Slice<T>::kPer; ++i) e[i] = from_float<T>(clean<T>(to_float(e[i])));
}

}  // namespace vocab
}  // namespace rs
