// Device pieces shared by the linear-attention kernels (forward and backward):
// matrix products on 16 x 16 blocks in bf16 or fp32, the split of fp32 values
// into bf16 parts, chunk loads, and decays.
//
// Blocks.  Every product is a sum of 16 x 16 x 16 block products.  A wave holds
// a block operand as a Frag: lane l (li = l % 16, g = l / 16) holds the four
// values of contraction indices 4g .. 4g + 3 at row (A) or column (B) li.  An
// accumulator block X (lane holds X[4g + r][li]) is therefore directly the
// A operand of X^T or the B operand of X: states and scores go back into the
// matrix cores from registers.
//   bf16: v_mfma_f32_16x16x32_bf16 takes two Frags at once (blocks p and p + 1 of
//         the contraction); products of bf16 values are exact, sums are fp32.
//   fp32: four v_mfma_f32_16x16x4_f32, the r-th on contraction indices 4g + r.
//
// Splits.  An fp32 operand (state, score, decayed value) of a bf16 product is
// the sum of NP bf16 parts, each the rounding of what the parts before it leave:
// the error is 2^-8 (half a step of bf16 relative to the value) to the power NP,
// so 2^-24 with three parts, an fp32 rounding, and 2^-16 with two, which is
// 1/256 of what rounding an output to bf16 costs.  Kernels with bf16 outputs use
// two parts where only an output depends on them; states always get three.
#pragma once

#include "args_attn.h"
#include "mfma_common.h"
#include "wave_prio.h"

namespace ttt {
namespace attn {

using mfma::bf16x4;
using mfma::bf16x8;
using mfma::float2v;
using mfma::float4v;
using mfma::u32x2;
using mfma::u32x4;

constexpr int C = kAttnChunk;

template <typename CT>
struct Ops;

template <>
struct Ops<uint16_t> {
  typedef bf16x4 Frag;
  static constexpr bool kSplit = true;
  template <int D>
  static constexpr int row_stride() { return D + 8; }
  // X[row0 + li][16 blk + 4g ..]
  template <int RS>
  __device__ static __forceinline__ Frag rows(const uint16_t* tile, int row0, int blk, int li, int g) {
    return *reinterpret_cast<const bf16x4*>(tile + (row0 + li) * RS + 16 * blk + 4 * g);
  }
  // X[row0 + 4g ..][col0 + li]
  template <int RS>
  __device__ static __forceinline__ Frag cols(const uint16_t* tile, int row0, int col0, int li, int g) {
    return mfma::read_cols<RS>(tile, row0, col0, li, g);
  }
  __device__ static __forceinline__ Frag zero() { return __builtin_bit_cast(bf16x4, u32x2{0u, 0u}); }
  __device__ static __forceinline__ float4v widen(Frag x) {
    const u32x2 w = __builtin_bit_cast(u32x2, x);
    return float4v{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                   __uint_as_float(w[1] & 0xffff0000u)};
  }
  __device__ static __forceinline__ float4v mm2(Frag a0, Frag a1, Frag b0, Frag b1, float4v c) {
    return mfma::mfma32(mfma::cat(a0, a1), mfma::cat(b0, b1), c);
  }
  // x = p[0] + p[1] (+ p[2])
  template <int NP>
  __device__ static __forceinline__ void split(float4v x, Frag p[NP]) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const mfma::bf16x2 h0 = __builtin_convertvector(float2v{x[0], x[1]}, mfma::bf16x2);
      const mfma::bf16x2 h1 = __builtin_convertvector(float2v{x[2], x[3]}, mfma::bf16x2);
      const u32x2 w = {__builtin_bit_cast(uint32_t, h0), __builtin_bit_cast(uint32_t, h1)};
      p[n] = __builtin_bit_cast(bf16x4, w);
      if (n + 1 < NP) x = x - widen(p[n]);
    }
  }
};

template <>
struct Ops<float> {
  typedef float4v Frag;
  static constexpr bool kSplit = false;
  template <int D>
  static constexpr int row_stride() { return D + 4; }
  template <int RS>
  __device__ static __forceinline__ Frag rows(const float* tile, int row0, int blk, int li, int g) {
    return *reinterpret_cast<const float4v*>(tile + (row0 + li) * RS + 16 * blk + 4 * g);
  }
  template <int RS>
  __device__ static __forceinline__ Frag cols(const float* tile, int row0, int col0, int li, int g) {
    const float* p = tile + (row0 + 4 * g) * RS + col0 + li;
    return float4v{p[0], p[RS], p[2 * RS], p[3 * RS]};
  }
  __device__ static __forceinline__ Frag zero() { return mfma::zero4v(); }
  __device__ static __forceinline__ float4v widen(Frag x) { return x; }
  __device__ static __forceinline__ float4v mm1(Frag a, Frag b, float4v c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
  }
  __device__ static __forceinline__ float4v mm2(Frag a0, Frag a1, Frag b0, Frag b1, float4v c) {
    return mm1(a1, b1, mm1(a0, b0, c));
  }
  template <int NP>
  __device__ static __forceinline__ void split(float4v x, Frag p[NP]) {
    static_assert(NP == 1, "fp32 products take fp32 operands whole");
    p[0] = x;
  }
};

// Parts of an fp32 operand: where only an output of type OT depends on it, and of state updates.
template <typename CT, typename OT>
__host__ __device__ constexpr int out_parts() { return Ops<CT>::kSplit ? (sizeof(OT) == 2 ? 2 : 3) : 1; }
template <typename CT>
__host__ __device__ constexpr int state_parts() { return Ops<CT>::kSplit ? 3 : 1; }

// c += sum over NB contraction blocks of a[b] . x[b]
template <typename CT, int NB>
__device__ __forceinline__ float4v dot(const typename Ops<CT>::Frag a[NB], const typename Ops<CT>::Frag x[NB],
                                       float4v c) {
  typedef Ops<CT> O;
#pragma unroll
  for (int b = 0; b + 1 < NB; b += 2) c = O::mm2(a[b], a[b + 1], x[b], x[b + 1], c);
  if constexpr (NB % 2 == 1) {
    if constexpr (O::kSplit) {
      c = O::mm2(a[NB - 1], O::zero(), x[NB - 1], O::zero(), c);
    } else {
      c = O::mm1(a[NB - 1], x[NB - 1], c);
    }
  }
  return c;
}

// c += a . (x[0] + ... + x[NP-1]) over one contraction block: two parts per instruction
template <typename CT, int NP>
__device__ __forceinline__ float4v dot_parts(typename Ops<CT>::Frag a, const typename Ops<CT>::Frag x[NP], float4v c) {
  typedef Ops<CT> O;
  if constexpr (NP == 1) {
    const typename O::Frag av[1] = {a};
    return dot<CT, 1>(av, x, c);
  } else {
#pragma unroll
    for (int n = 0; n < NP; n += 2) c = O::mm2(a, a, x[n], n + 1 < NP ? x[n + 1] : O::zero(), c);
    return c;
  }
}

// Eight elements of one row of a chunk, from global memory to LDS.
template <typename T>
struct Slab {
  u32x4 r[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, bool ok) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
      r[i] = u32x4{0u, 0u, 0u, 0u};
      if (ok) r[i] = mfma::ld_stream(reinterpret_cast<const u32x4*>(p) + i);
    }
  }
  __device__ __forceinline__ void put(T* p) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<u32x4*>(p)[i] = r[i];
  }
};
__device__ __forceinline__ void put_slab(const Slab<uint16_t>& s, uint16_t* p) { s.put(p); }
__device__ __forceinline__ void put_slab(const Slab<float>& s, float* p) { s.put(p); }
__device__ __forceinline__ void put_slab(const Slab<uint16_t>& s, float* p) {  // widened on the way
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w0 = s.r[0][2 * i], w1 = s.r[0][2 * i + 1];
    *reinterpret_cast<float4v*>(p + 4 * i) =
        float4v{__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u), __uint_as_float(w1 << 16),
                __uint_as_float(w1 & 0xffff0000u)};
  }
}

// lambda^n for n >= 0 (lambda^0 = 1 also where lambda = 0), and x lambda^n with
// lambda^n taken as 1 + expm1(n log lambda): for a decay close to 1 the product
// of thousands of chunks then keeps the accuracy that a rounded lambda^n loses.
__device__ __forceinline__ float powl(float g, int n) { return n == 0 ? 1.f : expf(g * static_cast<float>(n)); }
__device__ __forceinline__ float powm1(float g, int n) { return n == 0 ? 0.f : expm1f(g * static_cast<float>(n)); }
__device__ __forceinline__ float4v decayed(float4v x, float em1) {
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = fmaf(x[r], em1, x[r]);
  return x;
}

// Rows 16w .. 16w+15 of a d x d state as accumulator blocks: lane holds
// S[16w + li][16a + 4g + r]; from memory as S, or as S^T.
template <int D>
__device__ __forceinline__ void load_state(const float* p, bool transposed, int w, int li, int g, float4v s[D / 16]) {
#pragma unroll
  for (int a = 0; a < D / 16; ++a) {
    if (!transposed) {
      s[a] = *reinterpret_cast<const float4v*>(p + (16 * w + li) * D + 16 * a + 4 * g);
    } else {
      const float* c = p + (16 * a + 4 * g) * D + 16 * w + li;
      s[a] = float4v{c[0], c[D], c[2 * D], c[3 * D]};
    }
  }
}
template <int D>
__device__ __forceinline__ void store_state(float* p, int w, int li, int g, const float4v s[D / 16]) {
#pragma unroll
  for (int a = 0; a < D / 16; ++a) *reinterpret_cast<float4v*>(p + (16 * w + li) * D + 16 * a + 4 * g) = s[a];
}

// Four consecutive outputs of one token.
__device__ __forceinline__ void store4(float* p, float4v x) { *reinterpret_cast<float4v*>(p) = x; }
__device__ __forceinline__ void store4(uint16_t* p, float4v x) {
  const mfma::bf16x2 h0 = __builtin_convertvector(float2v{x[0], x[1]}, mfma::bf16x2);
  const mfma::bf16x2 h1 = __builtin_convertvector(float2v{x[2], x[3]}, mfma::bf16x2);
  *reinterpret_cast<u32x2*>(p) = u32x2{__builtin_bit_cast(uint32_t, h0), __builtin_bit_cast(uint32_t, h1)};
}

// Zeros to rows t0 .. t1 - 1 (padding behind a sequence's last token).
template <int D, typename OT>
__device__ __forceinline__ void zero_rows(OT* o, int64_t st, int t0, int t1) {
  constexpr int PR = D / 4;  // threads per row
  for (int t = t0 + static_cast<int>(threadIdx.x) / PR; t < t1; t += static_cast<int>(blockDim.x) / PR)
    store4(o + t * st + 4 * (threadIdx.x % PR), mfma::zero4v());
}

__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int T) {
  if (!lens) return T;
  const int n = lens[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

}  // namespace attn
}  // namespace ttt
