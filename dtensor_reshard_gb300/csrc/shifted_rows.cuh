// shifted_rows.cuh -- dispatch, combination and its gradients for rows of 16-bit elements that lie
// anyhow on 16 bytes (experts.cu): eight elements a lane out of the two aligned granules that hold
// them, and back in aligned granules of which a lane gets its predecessor's part by a shuffle.  In
// accesses of an element or two the same rows keep the load and store units busy, not the memory.
#pragma once

#include "vocab_row.cuh"

namespace rs {
namespace shifted {

using namespace op;

// The two granules in which the 16 bytes at `at` lie.
struct Granules {
  uint4 a, b;
  // Zeros unless `on`.  Predicated, so that no load waits for another's use.
  __device__ __forceinline__ void load(bool on, const unsigned char* at) {
    const uint32_t skew = uint32_t(reinterpret_cast<uintptr_t>(at) % 16);
    a = b = make_uint4(0, 0, 0, 0);
    asm volatile("{.reg .pred p; setp.ne.u32 p, %5, 0; @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];}"
                 : "+r"(a.x), "+r"(a.y), "+r"(a.z), "+r"(a.w)
                 : "l"(at - skew), "r"(uint32_t(on)));
    asm volatile("{.reg .pred p; setp.ne.u32 p, %5, 0; @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];}"
                 : "+r"(b.x), "+r"(b.y), "+r"(b.z), "+r"(b.w)
                 : "l"(at - skew + 16), "r"(uint32_t(on && skew)));
  }
  __device__ __forceinline__ uint4 at(const unsigned char* at) const {
    const uint32_t skew = uint32_t(reinterpret_cast<uintptr_t>(at) % 16);
    return staging::funnel16(a, b, skew / 4, 0x3210u + 0x1111u * (skew % 4));
  }
};
// The same element by element, for a buffer's first and last rows, whose granules may reach out of it.
__device__ __forceinline__ uint4 load_elements(bool on, const unsigned char* at) {
  alignas(16) uint16_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = on ? reinterpret_cast<const uint16_t*>(at)[i] : uint16_t(0);
  return *reinterpret_cast<const uint4*>(e);
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 two = vocab::pair_of(reinterpret_cast<const T*>(&v) + i);
    f[i] = two.x, f[i + 1] = two.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  alignas(16) T e[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) vocab::set_pair(e + i, make_float2(f[i], f[i + 1]));
  return *reinterpret_cast<const uint4*>(e);
}
// Eight elements of each lane of a warp to a row; full: of all lanes, and whether this lane has any.
template <typename T>
__device__ __forceinline__ void store(unsigned char* to, const uint4& v, bool full, bool mine) {
  if (full) vocab::store_granules<false>(reinterpret_cast<T*>(to), v);
  else if (mine) vocab::store_granule<false>(reinterpret_cast<T*>(to), v);
}

// What a warp has of its token: granules base + lane for base from `first` on in steps of LANES, and the
// row's last elements.
template <int LANES>
struct Part {
  uint32_t token, lane, first;
  __device__ Part()
      : token(blockIdx.x * (256 / LANES) + threadIdx.x / LANES),
        lane(threadIdx.x % 32),
        first(threadIdx.x % LANES / 32 * 32) {}
};

constexpr int kTogether = 4;  // choices whose rows are on their way at a time

template <typename T, int LANES, typename Args>
__global__ void __launch_bounds__(256) dispatch_kernel(const __grid_constant__ Args a) {
  const Part<LANES> p;
  if (p.token >= a.tokens) return;  // (whole warps)
  let_next_start();
  wait_for_previous();
  const unsigned char* x = a.x + p.token * a.ldx;
  const bool inside = p.token > 0 && p.token + 1 < a.tokens;
  const int32_t* slot = a.slot + int64_t(p.token) * a.topk;
  const uint32_t vecs = a.cols / 8;
  for (uint32_t base = p.first; base < vecs; base += LANES) {
    const uint32_t c = base + p.lane;
    const bool full = base + 32 <= vecs, mine = c < vecs;
    const unsigned char* at = x + c * uint64_t(16);
    uint4 v;
    if (inside) {
      Granules g;
      g.load(mine, at);
      v = g.at(at);
    } else {
      v = load_elements(mine, at);
    }
    for (uint32_t j0 = 0; j0 < a.topk; j0 += kPlaces) {
      uint32_t s[kPlaces];
      load_places(s, slot, j0, a.topk);
#pragma unroll
      for (uint32_t j = 0; j < kPlaces; ++j)
        if (s[j] < a.nrows) store<T>(a.rows + s[j] * a.ldr + c * uint64_t(16), v, full, mine);
    }
  }
  const uint32_t e = vecs * 8 + p.lane;
  if (p.first == 0 && e < a.cols)
    for (uint32_t j = 0; j < a.topk; ++j) {
      const uint32_t s = uint32_t(slot[j]);
      if (s < a.nrows) reinterpret_cast<T*>(a.rows + s * a.ldr)[e] = reinterpret_cast<const T*>(x)[e];
    }
}

template <typename T, int LANES, typename Args>
__global__ void __launch_bounds__(256, 3) combine_kernel(const __grid_constant__ Args a) {
  const Part<LANES> p;
  if (p.token >= a.tokens) return;  // (whole warps)
  let_next_start();
  wait_for_previous();
  const int64_t first = int64_t(p.token) * a.topk;
  unsigned char* out = a.out + p.token * a.ldo;
  const uint32_t vecs = a.cols / 8;
  for (uint32_t base = p.first; base < vecs; base += LANES) {
    const uint32_t c = base + p.lane;
    const bool full = base + 32 <= vecs, mine = c < vecs;
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    for (uint32_t j0 = 0; j0 < a.topk; j0 += kTogether) {
      const unsigned char* at[kTogether];
      float w[kTogether];
      bool inside = true, on[kTogether];
#pragma unroll
      for (uint32_t j = 0; j < kTogether; ++j) {
        const uint32_t s = j0 + j < a.topk ? uint32_t(a.slot[first + j0 + j]) : 0xffffffffu;
        on[j] = s < a.nrows;
        w[j] = on[j] && a.weight ? a.weight[first + j0 + j] : 1.0f;
        at[j] = a.rows + (on[j] ? s * a.ldr : 0) + c * uint64_t(16);
        inside = inside && (!on[j] || (s > 0 && s + 1 < a.nrows));
      }
      uint4 v[kTogether];
      if (inside) {
        Granules g[kTogether];
#pragma unroll
        for (int j = 0; j < kTogether; ++j) g[j].load(on[j] && mine, at[j]);
#pragma unroll
        for (int j = 0; j < kTogether; ++j) v[j] = g[j].at(at[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kTogether; ++j) v[j] = load_elements(on[j] && mine, at[j]);
      }
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        float f[8];
        unpack<T>(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[j], f[i], sum[i]);
      }
    }
    store<T>(out + c * uint64_t(16), pack<T>(sum), full, mine);
  }
  const uint32_t e = vecs * 8 + p.lane;
  if (p.first != 0 || e >= a.cols) return;
  float sum = 0.0f;
  for (uint32_t j = 0; j < a.topk; ++j) {
    const uint32_t s = uint32_t(a.slot[first + j]);
    if (s >= a.nrows) continue;
    const float w = a.weight ? a.weight[first + j] : 1.0f;
    sum = fmaf(w, to_float(reinterpret_cast<const T*>(a.rows + s * a.ldr)[e]), sum);
  }
  reinterpret_cast<T*>(out)[e] = from_float<T>(sum);
}

template <typename T, int LANES, bool DOT, typename Args>
__global__ void __launch_bounds__(256, 3) combine_grad_kernel(const __grid_constant__ Args a) {
  __shared__ float part[8][kTogether];
  const Part<LANES> p;
  if (p.token >= a.tokens) return;  // (whole warps, and with a CTA a token none)
  let_next_start();
  wait_for_previous();
  const int64_t first = int64_t(p.token) * a.topk;
  const unsigned char* dout = a.dout + p.token * a.ldo;
  const bool dout_inside = p.token > 0 && p.token + 1 < a.tokens;
  const uint32_t vecs = a.cols / 8;
  for (uint32_t j0 = 0; j0 < a.topk; j0 += kTogether) {
    float w[kTogether], dot[kTogether];
    uint32_t s[kTogether];
    bool inside = dout_inside;
#pragma unroll
    for (uint32_t j = 0; j < kTogether; ++j) {
      s[j] = j0 + j < a.topk ? uint32_t(a.slot[first + j0 + j]) : 0xffffffffu;
      w[j] = j0 + j < a.topk && a.weight ? a.weight[first + j0 + j] : 1.0f;
      dot[j] = 0.0f;
      inside = inside && (s[j] >= a.nrows || (s[j] > 0 && s[j] + 1 < a.nrows));
    }
    for (uint32_t base = p.first; base < vecs; base += LANES) {
      const uint32_t c = base + p.lane;
      const bool full = base + 32 <= vecs, mine = c < vecs;
      const unsigned char* at = dout + c * uint64_t(16);
      uint4 d, v[kTogether];
      if (inside) {
        Granules g, h[kTogether];
        g.load(mine, at);
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
          if (DOT) h[j].load(mine && s[j] < a.nrows, a.rows + (s[j] < a.nrows ? s[j] * a.ldr : 0) + c * uint64_t(16));
        d = g.at(at);
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
          if (DOT) v[j] = h[j].at(a.rows + (s[j] < a.nrows ? s[j] * a.ldr : 0) + c * uint64_t(16));
      } else {
        d = load_elements(mine, at);
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
          if (DOT)
            v[j] = load_elements(mine && s[j] < a.nrows, a.rows + (s[j] < a.nrows ? s[j] * a.ldr : 0) + c * uint64_t(16));
      }
      float f[8];
      unpack<T>(d, f);
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        if (DOT) {
          float r[8];
          unpack<T>(v[j], r);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[j] = fmaf(f[i], r[i], dot[j]);
        }
        if (!a.drows || s[j] >= a.nrows) continue;
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = w[j] * f[i];
        store<T>(a.drows + s[j] * a.ldr + c * uint64_t(16), pack<T>(g), full, mine);
      }
    }
    const uint32_t e = vecs * 8 + p.lane;
    if (p.first == 0 && e < a.cols) {
      const float d = to_float(reinterpret_cast<const T*>(dout)[e]);
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        if (s[j] >= a.nrows) continue;
        if (DOT) dot[j] = fmaf(d, to_float(reinterpret_cast<const T*>(a.rows + s[j] * a.ldr)[e]), dot[j]);
        if (a.drows) reinterpret_cast<T*>(a.drows + s[j] * a.ldr)[e] = from_float<T>(w[j] * d);
      }
    }
    if constexpr (DOT) {
      const uint32_t together = min(uint32_t(kTogether), a.topk - j0);
#pragma unroll
      for (int j = 0; j < kTogether; ++j) dot[j] = warp_sum(dot[j]);
      float* to = a.dweight + first + j0;
      if (LANES == 32) {
        if (p.lane == 0)
          for (uint32_t j = 0; j < kTogether; ++j)
            if (j < together) to[j] = dot[j];
      } else {
        if (p.lane == 0)
          for (int j = 0; j < kTogether; ++j) part[threadIdx.x / 32][j] = dot[j];
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

}  // namespace shifted
}  // namespace rs
