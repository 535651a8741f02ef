// Device pieces shared by the linear-attention kernels: matrix products on 16 x 16
// blocks, operands in bf16 parts, chunk loads, and decays.
//
// Blocks.  Every product is a sum of 16 x 16 x 16 block products.  A wave holds
// a block operand as a Frag: lane l (li = l % 16, g = l / 16) holds the four
// values of contraction indices 4g .. 4g + 3 at row (A) or column (B) li.  An
// accumulator block X (lane holds X[4g + r][li]) is therefore directly the
// A operand of X^T or the B operand of X: states and scores go back into the
// matrix cores from registers.  v_mfma_f32_16x16x32_bf16 takes two Frags of either
// operand at once; products of bf16 values are exact and sums are fp32.
//
// Parts.  An fp32 operand (an fp32 input, the state, a score, a decayed value) is
// the sum of bf16 parts, each the rounding of what the parts before it leave, so
// that n parts are off by at most 2^-8n: half a bf16 step, n times.  A product of
// level LV takes the part pairs (p, q) with p + q < LV: level 3 is an fp32 product
// (2^-24), level 2 is off by 2^-16, 1/256 of what rounding the output to bf16
// costs.  States and fp32 outputs are level 3, products that only a bf16 output
// depends on are level 2.  The fp32 matrix instruction (v_mfma_f32_16x16x4_f32)
// does the same at 1/16 of the bf16 rate: six part pairs take 3/8 of its time.
#pragma once

#include "args_attn.h"
#include "mfma_common.h"
#include "wave_prio.h"

namespace ttt {
namespace attn {

using mfma::bf16x4;
using mfma::float2v;
using mfma::float4v;
using mfma::u32x2;
using mfma::u32x4;

constexpr int C = kAttnChunk;
typedef bf16x4 Frag;

// parts of an input of type T, and the level of products that only an output of type T depends on
template <typename T>
__host__ __device__ constexpr int parts_of() { return sizeof(T) == 2 ? 1 : 3; }
template <typename T>
__host__ __device__ constexpr int level_of() { return sizeof(T) == 2 ? 2 : 3; }

__device__ __forceinline__ float4v widen(Frag x) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  return float4v{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                 __uint_as_float(w[1] & 0xffff0000u)};
}

// x = p[0] + ... + p[N-1]
template <int N>
__device__ __forceinline__ void split(float4v x, Frag p[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const mfma::bf16x2 h0 = __builtin_convertvector(float2v{x[0], x[1]}, mfma::bf16x2);
    const mfma::bf16x2 h1 = __builtin_convertvector(float2v{x[2], x[3]}, mfma::bf16x2);
    const u32x2 w = {__builtin_bit_cast(uint32_t, h0), __builtin_bit_cast(uint32_t, h1)};
    p[n] = __builtin_bit_cast(bf16x4, w);
    if (n + 1 < N) x = x - widen(p[n]);
  }
}

__device__ __forceinline__ Frag zero_frag() { return __builtin_bit_cast(bf16x4, u32x2{0u, 0u}); }
__device__ __forceinline__ float4v mm2(Frag a0, Frag a1, Frag b0, Frag b1, float4v c) {
  return mfma::mfma32(mfma::cat(a0, a1), mfma::cat(b0, b1), c);
}

// c += a . x over one contraction block: two part pairs per instruction
template <int NA, int NX, int LV>
__device__ __forceinline__ float4v dot1(const Frag a[NA], const Frag x[NX], float4v c) {
  Frag l[8], r[8];
  int n = 0;
#pragma unroll
  for (int p = 0; p < NA; ++p)
#pragma unroll
    for (int q = 0; q < NX; ++q)
      if (p + q < LV) {
        l[n] = a[p];
        r[n] = x[q];
        ++n;
      }
  if (n % 2) {
    l[n] = r[n] = zero_frag();
    ++n;
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    if (i < n) c = mm2(l[i], l[i + 1], r[i], r[i + 1], c);
  return c;
}

// c += a0 . x0 + a1 . x1, two contraction blocks
template <int NA, int NX, int LV>
__device__ __forceinline__ float4v dot2(const Frag a0[NA], const Frag a1[NA], const Frag x0[NX], const Frag x1[NX],
                                        float4v c) {
#pragma unroll
  for (int p = 0; p < NA; ++p)
#pragma unroll
    for (int q = 0; q < NX; ++q)
      if (p + q < LV) c = mm2(a0[p], a1[p], x0[q], x1[q], c);
  return c;
}

// One tensor's chunk in LDS: C rows of D elements, a plane for each part.
template <int D, int N>
struct Tile {
  static constexpr int RS = D + 8;  // row stride: the rows of a Frag in different banks
  static constexpr int kPlane = C * RS;
  static constexpr int kSize = N * kPlane;
  // X[row0 + li][16 blk + 4g ..]
  __device__ static __forceinline__ void rows(const uint16_t* t, int row0, int blk, int li, int g, Frag f[N]) {
#pragma unroll
    for (int p = 0; p < N; ++p)
      f[p] = *reinterpret_cast<const bf16x4*>(t + p * kPlane + (row0 + li) * RS + 16 * blk + 4 * g);
  }
  // X[row0 + 4g ..][col0 + li]
  __device__ static __forceinline__ void cols(const uint16_t* t, int row0, int col0, int li, int g, Frag f[N]) {
#pragma unroll
    for (int p = 0; p < N; ++p) f[p] = mfma::read_cols<RS>(t + p * kPlane, row0, col0, li, g);
  }
  __device__ static __forceinline__ float4v sum(const Frag f[N]) {
    float4v x = widen(f[N - 1]);
#pragma unroll
    for (int p = N - 2; p >= 0; --p) x = widen(f[p]) + x;
    return x;
  }
};

// A 16 x 16 block of A B^T: lane holds [4g + r of A's rows][li of B's rows].
template <int D, int NA, int NX, int LV>
__device__ __forceinline__ float4v rows_dot(const uint16_t* a, int ra, const uint16_t* x, int rx, int li, int g) {
  constexpr int NB = D / 16;
  float4v c = mfma::zero4v();
  if constexpr (NB == 1) {
    Frag f[NA], h[NX];
    Tile<D, NA>::rows(a, ra, 0, li, g, f);
    Tile<D, NX>::rows(x, rx, 0, li, g, h);
    c = dot1<NA, NX, LV>(f, h, c);
  } else {
#pragma unroll
    for (int k = 0; k < NB; k += 2) {
      Frag f0[NA], f1[NA], h0[NX], h1[NX];
      Tile<D, NA>::rows(a, ra, k, li, g, f0);
      Tile<D, NA>::rows(a, ra, k + 1, li, g, f1);
      Tile<D, NX>::rows(x, rx, k, li, g, h0);
      Tile<D, NX>::rows(x, rx, k + 1, li, g, h1);
      c = dot2<NA, NX, LV>(f0, f1, h0, h1, c);
    }
  }
  return c;
}

// Eight elements of one row of a chunk, from global memory to LDS.
template <typename T>
struct Slab {
  static constexpr int kWords = sizeof(T) / 2;
  u32x4 r[kWords];
  __device__ __forceinline__ void load(const T* p, bool ok) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      r[i] = u32x4{0u, 0u, 0u, 0u};
      if (ok) r[i] = reinterpret_cast<const u32x4*>(p)[i];
    }
  }
  // to the planes of a Tile<D, parts_of<T>()>
  template <int PLANE>
  __device__ __forceinline__ void put(uint16_t* t) const {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<u32x4*>(t) = r[0];
    } else {
      Frag f[2][3];
#pragma unroll
      for (int i = 0; i < 2; ++i) split<3>(__builtin_bit_cast(float4v, r[i]), f[i]);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const u32x2 lo = __builtin_bit_cast(u32x2, f[0][p]), hi = __builtin_bit_cast(u32x2, f[1][p]);
        *reinterpret_cast<u32x4*>(t + p * PLANE) = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
  }
};

// lambda^n for n >= 0 (lambda^0 = 1 also where lambda = 0)
__device__ __forceinline__ float powl(float g, int n) { return n == 0 ? 1.f : expf(g * static_cast<float>(n)); }

// x lambda^n as m x + a x.  Near 1 lambda^n is taken as 1 + expm1(n log lambda): a rounded lambda^n is off by
// up to 2^-25 the same way in every chunk, which thousands of chunks add up.  Below 1/2 it is lambda^n itself.
struct Decay {
  float m, a;
};
__device__ __forceinline__ Decay decay(float g, int n) {
  const float p = powl(g, n);
  return p > 0.5f ? Decay{1.f, n == 0 ? 0.f : expm1f(g * static_cast<float>(n))} : Decay{0.f, p};
}
__device__ __forceinline__ float4v decayed(float4v x, Decay d) {
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = fmaf(x[r], d.a, x[r] * d.m);
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
