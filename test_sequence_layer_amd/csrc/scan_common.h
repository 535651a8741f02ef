// The selective scan's walk over tokens: how a workgroup stages its tile and how the sums cross lanes.
//
//   h_t[c,n] = exp(dt_t[c] A[c,n]) h_{t-1}[c,n] + dt_t[c] B_t[n] u_t[c],   y_t[c] = sum_n C_t[n] h_t[c,n] + D[c] u_t[c]
//
// A workgroup holds 64 channels of one sequence, several lanes to a channel, each with NS states in registers for the whole
// walk.  Tokens go through LDS a tile at a time, where each thread has prepared some channels of one token (softplus once
// per token and channel, not once per state); B and C, which all channels of a group share, lie there as fp32, C behind B,
// NP states each, zeros from N on.
#pragma once
#include "block_common.h"

namespace ttt {
namespace scan {

using namespace block;

constexpr int CH = kScanCh;

// The channels of a workgroup and its sequence.
struct Place {
  int b, g, tile, c0, nc;  // first channel, how many of the 64 are there
  int len;                 // the sequence's tokens
};

__device__ __forceinline__ Place place(const ScanArgs& a, int64_t blk) {
  Place p;
  const int dg = a.D / a.G, tiles = (dg + CH - 1) / CH;
  p.tile = static_cast<int>(blk % tiles);
  p.g = static_cast<int>(blk / tiles % a.G);
  p.b = static_cast<int>(blk / tiles / a.G);
  p.c0 = p.g * dg + p.tile * CH;
  p.nc = min(CH, dg - p.tile * CH);
  p.len = a.lens ? max(0, min(a.lens[p.b], a.T)) : a.T;
  return p;
}

// A log2(e), finite: exp(0 A) of a token that is not there has to be 1.  -inf becomes -3e38, which keeps nothing over steps of
// 1e-36 and more.
__device__ __forceinline__ float scaled_decay(float A) {
  const float x = A * kLog2e;
  return x != x ? x : fminf(fmaxf(x, -3.0e38f), 3.0e38f);
}

// of a lane's states
template <int NS>
__device__ __forceinline__ void decays(float (&a2)[NS], const ScanArgs& a, int c, int q, bool on) {
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = q * NS + i;
    a2[i] = scaled_decay(on && n < a.N ? a.A[static_cast<int64_t>(c) * a.N + n] : 0.f);
  }
}

template <int NS>
__device__ __forceinline__ void load_states(float (&h)[NS], const float* p, int N, int q, bool on) {
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = q * NS + i;
    h[i] = p && on && n < N ? p[n] : 0.f;
  }
}

template <int NS>
__device__ __forceinline__ void store_states(const float (&h)[NS], float* p, int N, int q, bool on) {
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = q * NS + i;
    if (on && n < N) p[n] = h[i];
  }
}

// NS neighbouring floats of LDS
template <int NS>
__device__ __forceinline__ void lds_floats(float (&x)[NS], const float* p) {
  if constexpr (NS == 1) {
    x[0] = p[0];
  } else if constexpr (NS == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x; x[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
  }
}

// A thread's pieces of a tile's B and C, four states of a token each, between the load and LDS.  Piece id is B's or C's
// (id / (NQ TT)) of token id / NQ % TT, states 4 (id % NQ) on, for 256 threads.
template <typename T, int NP, int TT, bool Wide>
struct BcRows {
  static constexpr int NQ = NP / 4, kEach = (2 * TT * NQ + 255) / 256;
  typedef Piece<T, 4> Values[kEach];
  const T* p[kEach];
  int64_t row[kEach];  // elements from a token to the next
  int t[kEach], n[kEach], lds[kEach];
  __device__ __forceinline__ BcRows(const ScanArgs& a, const Place& at, int first, int tid, bool with_c) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int id = tid + 256 * k, w = id / (NQ * TT), m = id % NQ;
      t[k] = id / NQ % TT;
      n[k] = w > (with_c ? 1 : 0) ? 0 : min(4, a.N - 4 * m);  // (may be negative)
      lds[k] = w > 1 ? -1 : (w * TT + t[k]) * NP + 4 * m;
      const T* base = static_cast<const T*>(w ? a.Cm : a.Bm) + (w ? at.b * a.cs.b + at.g * a.cs.h : at.b * a.bs.b + at.g * a.bs.h);
      row[k] = w ? a.cs.t : a.bs.t;
      p[k] = base + (first + t[k]) * row[k] + (Wide && n[k] <= 0 ? 0 : 4 * m);
    }
  }
  // the tile that begins at token first, as far as end (> first); then on to the next tile (dir 1), the one before (-1) or none
  __device__ __forceinline__ void load(Values& v, int first, int end, int dir) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const T* src = p[k];
      if (Wide && first + TT > end) src -= max(0, first + t[k] - (end - 1)) * row[k];  // (the last token instead)
      load_ahead<Wide>(v[k], src, first + t[k] < end ? n[k] : 0);
      if (dir > 0) p[k] += row[k] * TT;
      else if (dir < 0) p[k] -= row[k] * TT;
    }
  }
  __device__ __forceinline__ void stage(Values& v, float* bc, int first, int end) const {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (first + TT > end || n[k] <= 0) keep<Wide>(v[k], first + t[k] < end ? n[k] : 0);
      if (256 * (k + 1) <= 2 * TT * NQ || lds[k] >= 0)
        *reinterpret_cast<float4*>(bc + lds[k]) = make_float4(v[k].get(0), v[k].get(1), v[k].get(2), v[k].get(3));
    }
  }
};

// A group of GS tokens as a lane reads it: dt and dt u of its channel (a pair every ROW floats of its tokens), B of its NS
// states.
template <int NS, int GS, int NP, int ROW>
struct Group {
  float2 d[GS];
  float B[GS][NS];
  __device__ __forceinline__ void read(const float* sd, const float* bc, int k) {
#pragma unroll
    for (int j = 0; j < GS; ++j) {
      d[j] = *reinterpret_cast<const float2*>(sd + (k + j) * ROW);
      lds_floats(B[j], bc + (k + j) * NP);
    }
  }
};

// The state before segment seg from what each earlier one adds and how far it decays.
template <int NS>
__device__ __forceinline__ void start_state(float (&h)[NS], const float (&a2)[NS], const ScanArgs& a, const Place& p, int seg,
                                            int c, int q, bool on) {
  const int64_t row = static_cast<int64_t>(p.b) * a.nseg;
  load_states(h, a.hseg + (row * a.D + c) * a.N, a.N, q, on);
  for (int s = 0; s < seg; ++s) {
    const float sum = on ? a.sseg[(row + s) * a.D + c] : 0.f;
    float x[NS];
    load_states(x, a.hseg + ((row + s + 1) * a.D + c) * a.N, a.N, q, on);
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(sum * a2[i]), h[i], x[i]);
  }
}

}  // namespace scan
}  // namespace ttt
