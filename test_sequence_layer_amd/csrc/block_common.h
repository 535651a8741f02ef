// Shared by the kernels around a layer's state: rows of bf16 or fp32 in pieces, softplus, silu.
#pragma once
#include "args_block.h"
#include "mfma_common.h"

namespace ttt {
namespace block {

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(uint16_t x) { return bf16_bits_to_f32(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = f32_to_bf16_bits(x); }

// N neighbouring elements as they lie in memory (16-byte loads and stores; 8 bytes where N of them are no more).
template <typename T, int N>
struct Piece {
  static constexpr int kWords = static_cast<int>(N * sizeof(T) / 4);
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
  // element by element: the first n of N, the others zero
  __device__ __forceinline__ void load_some(const T* p, int n) {
#pragma unroll
    for (int i = 0; i < N; ++i) set_bits(i, i < n ? p[i] : T(0));
  }
  __device__ __forceinline__ void store_some(T* p, int n) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = bits(i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ T bits(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return static_cast<T>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
  }
  __device__ __forceinline__ void set_bits(int i, T x) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x);
    else if (i & 1) w[i / 2] = (w[i / 2] & 0xffffu) | static_cast<uint32_t>(x) << 16;
    else w[i / 2] = (w[i / 2] & 0xffff0000u) | x;
  }
  __device__ __forceinline__ void set_all(const float* x) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2)
        w[i / 2] = static_cast<uint32_t>(f32_to_bf16_bits(x[i])) | static_cast<uint32_t>(f32_to_bf16_bits(x[i + 1])) << 16;
    }
  }
};

// The first n of N elements, the others zero.  Wide: all or none of them.
template <bool Wide, typename T, int N>
__device__ __forceinline__ void load(Piece<T, N>& v, const T* p, int n) {
  if constexpr (Wide) {
    if (n > 0) v.load(p);
    else v.zero();
  } else {
    v.load_some(p, n);
  }
}

// The same for loads that stay on their way over other work.  Wide: p is always good to read and ``keep`` drops what should
// not have been: with a branch around a load the compiler waits for all that is on its way, stores too, before it uses one.
template <bool Wide, typename T, int N>
__device__ __forceinline__ void load_ahead(Piece<T, N>& v, const T* p, int n) {
  if constexpr (Wide) v.load(p);
  else v.load_some(p, n);
}

template <bool Wide, typename T, int N>
__device__ __forceinline__ void keep(Piece<T, N>& v, int n) {
  if constexpr (Wide) {
#pragma unroll
    for (int i = 0; i < Piece<T, N>::kWords; ++i) v.w[i] = n > 0 ? v.w[i] : 0;
  }
}

template <bool Wide, typename T, int N>
__device__ __forceinline__ void store(const Piece<T, N>& v, T* p, int n) {
  if constexpr (Wide) {
    if (n > 0) v.store(p);
  } else {
    v.store_some(p, n);
  }
}

// N fp32 parameters of neighbouring channels, or a constant where there are none
template <int N>
__device__ __forceinline__ void params(float* x, const float* p, int n, float none) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = p && i < n ? p[i] : none;
}

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// 1 / (1 + e^-x).  v_exp_f32 and v_rcp_f32 are good to 1 ulp; x log2(e) is rounded, which shows where the result is e^x:
// |x| 2^-24 of it.  Below x = -88 e^-x is infinite and the result 0.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x)); }

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| <= 1, and its slope, the sigmoid.  log(1 + e) = 2 artanh(s) with
// s = e / (2 + e) <= 1/3, and 2 artanh(s) / s a polynomial of degree 4 in s^2 (its interpolation at Chebyshev points of
// [0, 1/9]), 4e-9 of it off.  (log of the rounded 1 + e would lose the digits of a small e, and steps of 10^-3 are the rule.)
__device__ __forceinline__ float softplus_tail(float e) {
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
  float p = 0.28174657f;
  p = fmaf(p, q, 0.27961418f);
  p = fmaf(p, q, 0.40024853f);
  p = fmaf(p, q, 0.66666317f);
  p = fmaf(p, q, 2.f);
  return s * p;
}

__device__ __forceinline__ float softplus(float x) { return softplus_tail(fast_exp(-fabsf(x))) + fmaxf(x, 0.f); }

__device__ __forceinline__ float softplus(float x, float& slope) {
  const float e = fast_exp(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.f + e);
  slope = x >= 0.f ? r : e * r;
  return softplus_tail(e) + fmaxf(x, 0.f);
}

__device__ __forceinline__ float quad_sum(float x) {
  x += mfma::dpp_mov<0xB1>(x);
  x += mfma::dpp_mov<0x4E>(x);
  return x;
}

}  // namespace block
}  // namespace ttt
