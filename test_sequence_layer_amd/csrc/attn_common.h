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
// the sum of three bf16 parts, each the rounding of what the parts before it leave:
// half a bf16 step, three times, so that less than 2^-24 is left.  A product takes the
// part pairs (p, q) with p + q < 3, six of nine; the others are below 2^-24 of it.  With
// a bf16 operand, which is its own single part, it is three of three.  The fp32 matrix
// instruction (v_mfma_f32_16x16x4_f32) does the same at 1/16 of the bf16 rate: six part
// pairs take 3/8 of its time.  Outputs of bf16 take three parts as well: with two (2^-16
// of the sum of the terms' magnitudes) terms that cancel leave the bits that were cut
// off, and 0.25% of ordinary bf16 outputs round to the neighbouring value, with three
// 0.02%.  What that costs, us with two parts and with three: B16 H32 T8192 d64 [B, H, T, d]
// 431 and 498, [B, T, H, d] 501 and 492, d128 571 and 667, gradients at T2048 406 and 434.
// A state or a sum above bf16's largest value (3.39e38) rounds to an infinite first part,
// and an infinity leaves NaN behind its first part: both come out as NaN.
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

constexpr int kParts = 3;  // of an fp32 value
// parts of an input of type T
template <typename T>
__host__ __device__ constexpr int parts_of() { return sizeof(T) == 2 ? 1 : kParts; }

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

// The same of an fp32 input, or of one that has only decayed: its first part stays finite where x does, so that the
// type's largest and lowest values have three parts as all others, and come to nothing where their score is zero.  (0 to
// 2% of the time of fp32 calls; states and sums, which are as large only next to overflow, do without.)
__device__ __forceinline__ void split_input(float4v x, Frag p[kParts]) {
  constexpr float kMost = 3.3895313892515355e38f;  // bf16's largest
  float4v near;
#pragma unroll
  for (int i = 0; i < 4; ++i) near[i] = __builtin_amdgcn_fmed3f(x[i], -kMost, kMost);
  split<1>(near, p);
  split<kParts - 1>(x - widen(p[0]), p + 1);
}

__device__ __forceinline__ Frag zero_frag() { return __builtin_bit_cast(bf16x4, u32x2{0u, 0u}); }
__device__ __forceinline__ float4v mm2(Frag a0, Frag a1, Frag b0, Frag b1, float4v c) {
  return mfma::mfma32(mfma::cat(a0, a1), mfma::cat(b0, b1), c);
}

// c += a . x over one contraction block: two part pairs per instruction
template <int NA, int NX>
__device__ __forceinline__ float4v dot1(const Frag a[NA], const Frag x[NX], float4v c) {
  Frag l[8], r[8];
  int n = 0;
#pragma unroll
  for (int p = 0; p < NA; ++p)
#pragma unroll
    for (int q = 0; q < NX; ++q)
      if (p + q < kParts) {
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
template <int NA, int NX>
__device__ __forceinline__ float4v dot2(const Frag a0[NA], const Frag a1[NA], const Frag x0[NX], const Frag x1[NX],
                                        float4v c) {
#pragma unroll
  for (int p = 0; p < NA; ++p)
#pragma unroll
    for (int q = 0; q < NX; ++q)
      if (p + q < kParts) c = mm2(a0[p], a1[p], x0[q], x1[q], c);
  return c;
}

// One tensor's chunk in LDS: C rows of D elements, a plane for each part.  Within a row the 8-byte units are
// exchanged by an exclusive or with a function of the row, chosen so that both ways of reading a Frag touch
// all 32 banks once: by rows (16 lanes: one unit of 16 rows) and by columns (16 lanes: four units of four
// rows).  A padded row (D + 8 elements) leaves two-way conflicts in both: 43% of the LDS cycles.
template <int D>
__host__ __device__ constexpr int swizzle(int row) {
  return D >= 64 ? ((row & 3) << 2) | ((row >> 2) & 3) : D == 32 ? (((row >> 1) & 1) << 2) | ((row >> 2) & 3) : (row >> 2) & 3;
}
// Elements from row 0 to row 16.  Eight bytes over: reads of a unit in both halves then have no common
// ds_read2 form, which the compiler would take and then need two moves each to pair up units of one half.
template <int D>
__host__ __device__ constexpr int half_at() { return 16 * D + 4; }
template <int D>
__device__ __forceinline__ int unit_at(int row, int unit) {
  return row * D + (row >= 16 ? half_at<D>() - 16 * D : 0) + 4 * (unit ^ swizzle<D>(row));
}

// Where a lane finds its Frags X[li][16k + 4g ..] and X[4g ..][16k + li]; half_at further: 16 rows on.
template <int D>
struct Places {
  int row[D / 16], col[D / 16];
  __device__ __forceinline__ Places(int li, int g) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      row[k] = unit_at<D>(li, 4 * k + g);
      col[k] = unit_at<D>(4 * g + (li >> 2), 4 * k + (li & 3));
    }
  }
};

template <int D, int N>
struct Tile {
  static constexpr int kPlane = half_at<D>() + 16 * D + 4;  // (16-byte steps)
  static constexpr int kSize = N * kPlane;
  __device__ static __forceinline__ void rows(const uint16_t* t, Frag f[N]) {
#pragma unroll
    for (int p = 0; p < N; ++p) f[p] = *reinterpret_cast<const bf16x4*>(t + p * kPlane);
  }
  // ds_read_b64_tr_b16: lane l of 16 gets element r of the 8 bytes that lane 4r + l / 4 addresses, position l % 4
  __device__ static __forceinline__ void cols(const uint16_t* t, Frag f[N]) {
    typedef mfma::short4v __attribute__((address_space(3))) * ptr;
#pragma unroll
    for (int p = 0; p < N; ++p)
      f[p] = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(t + p * kPlane)));
  }
  __device__ static __forceinline__ float4v sum(const Frag f[N]) {
    float4v x = widen(f[N - 1]);
#pragma unroll
    for (int p = N - 2; p >= 0; --p) x = widen(f[p]) + x;
    return x;
  }
};

// A 16 x 16 block of A B^T: lane holds [4g + r of A's rows][li of B's rows].  a, x: the first of the 16 rows.
template <int D, int NA, int NX>
__device__ __forceinline__ float4v rows_dot(const uint16_t* a, const uint16_t* x, const Places<D>& at) {
  constexpr int NB = D / 16;
  float4v c = mfma::zero4v();
  if constexpr (NB == 1) {
    Frag f[NA], h[NX];
    Tile<D, NA>::rows(a + at.row[0], f);
    Tile<D, NX>::rows(x + at.row[0], h);
    c = dot1<NA, NX>(f, h, c);
  } else {
#pragma unroll
    for (int k = 0; k < NB; k += 2) {
      Frag f0[NA], f1[NA], h0[NX], h1[NX];
      Tile<D, NA>::rows(a + at.row[k], f0);
      Tile<D, NA>::rows(a + at.row[k + 1], f1);
      Tile<D, NX>::rows(x + at.row[k], h0);
      Tile<D, NX>::rows(x + at.row[k + 1], h1);
      c = dot2<NA, NX>(f0, f1, h0, h1, c);
    }
  }
  return c;
}

// Eight elements of one row of a chunk, from global memory to LDS.
template <typename T>
struct Slab {
  static constexpr int kWords = sizeof(T) / 2;
  u32x4 r[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) r[i] = reinterpret_cast<const u32x4*>(p)[i];
  }
  // the two units to the planes of a Tile<D, parts_of<T>()>
  template <int PLANE>
  __device__ __forceinline__ void put(uint16_t* t, int u0, int u1) const {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<u32x2*>(t + u0) = u32x2{r[0][0], r[0][1]};
      *reinterpret_cast<u32x2*>(t + u1) = u32x2{r[0][2], r[0][3]};
    } else {
      Frag f[2][kParts];
#pragma unroll
      for (int i = 0; i < 2; ++i) split_input(__builtin_bit_cast(float4v, r[i]), f[i]);
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        *reinterpret_cast<bf16x4*>(t + p * PLANE + u0) = f[0][p];
        *reinterpret_cast<bf16x4*>(t + p * PLANE + u1) = f[1][p];
      }
    }
  }
};

// lambda^n for n >= 0 (lambda^0 = 1 also where lambda = 0)
__device__ __forceinline__ float powl(float g, int n) { return n == 0 ? 1.f : expf(g * static_cast<float>(n)); }

// lambda^C, chunk after chunk.  A rounded power near 1 is off by up to 2^-25 the same way every time, which
// thousands of chunks add up: the two fp32 values around it are taken in turn, by a running sum of where it
// lies between them, so that the product of any number of chunks' factors is off by one such step at most.
struct Decays {
  float lo, step, frac, sum;
  __device__ __forceinline__ explicit Decays(float g) {
    const double p = exp(static_cast<double>(g) * C);
    lo = __double2float_rd(p);
    // the next value up (p = 0 and p = inf have none to share with)
    const float hi = lo > 0.f && lo < 3.0e38f ? __uint_as_float(__float_as_uint(lo) + 1u) : lo;
    step = hi - lo;
    frac = step > 0.f ? static_cast<float>((p - lo) / step) : 0.f;
    sum = 0.5f;
  }
  __device__ __forceinline__ float next() {
    sum += frac;
    const bool up = sum >= 1.f;
    sum -= up ? 1.f : 0.f;
    return up ? lo + step : lo;
  }
};

// lambda^n of a whole segment, n > 0, in two fp32 parts: one rounded power, taken by up to 63 segments one after the
// other, would be off the same way in each (64 segments of 512 tokens, log_decay -3e-5: the oldest tokens' share is
// off by 29 steps of 2^-24, in two parts by 1).
struct SegmentDecay {
  float hi, lo;
  __device__ __forceinline__ SegmentDecay(float g, int n) {
    const double p = exp(static_cast<double>(g) * n);
    hi = static_cast<float>(p);
    lo = hi <= 3.0e38f ? static_cast<float>(p - static_cast<double>(hi)) : 0.f;
  }
  // s lambda^n + x, rounded once
  __device__ __forceinline__ float4v carry(float4v s, float4v x) const {
    float4v r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = fmaf(s[i], hi, fmaf(s[i], lo, x[i]));
    return r;
  }
};

// Workgroup -> unit and kind of work: kinds change every 8 units.  Workgroups go round the eight XCDs, so the
// kinds of one unit run on the same XCD, at about the same time.
struct Unit {
  int64_t unit;
  int kind;
};
__device__ __forceinline__ Unit unit_of(int64_t id, int kinds, int64_t units) {
  const int64_t whole = units / 8 * 8;  // in full groups of 8
  if (id < whole * kinds) return Unit{id / (8 * kinds) * 8 + id % 8, static_cast<int>(id / 8 % kinds)};
  const int64_t r = id - whole * kinds, left = units - whole;
  return Unit{whole + r % left, static_cast<int>(r / left)};
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
// s carried over n segments: s <- e s + (the c-th state at p + c step), four loads at a time on their way.
template <int D>
__device__ __forceinline__ void carry_states(const float* p, int64_t step, int n, SegmentDecay e, bool transposed, int w, int li,
                                             int g, float4v s[D / 16]) {
  constexpr int U = D <= 64 ? 4 : 2;
  int c = 0;
  for (; c + U <= n; c += U) {
    float4v x[U][D / 16];
#pragma unroll
    for (int i = 0; i < U; ++i) load_state<D>(p + (c + i) * step, transposed, w, li, g, x[i]);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int k = 0; k < D / 16; ++k) s[k] = e.carry(s[k], x[i][k]);
  }
  for (; c < n; ++c) {
    float4v x[D / 16];
    load_state<D>(p + c * step, transposed, w, li, g, x);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) s[k] = e.carry(s[k], x[k]);
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
