// The selective scan's walk over tokens: how a workgroup stages its tile and how the sums cross lanes.
//
//   h_t[c,n] = exp(dt_t[c] A[c,n]) h_{t-1}[c,n] + dt_t[c] B_t[n] u_t[c],   y_t[c] = sum_n C_t[n] h_t[c,n] + D[c] u_t[c]
//
// A workgroup of four waves holds 64 channels of one sequence; a wave 16 of them, four lanes to a channel, each with NS
// = N / 4 states in registers for the whole walk.  Tokens go through LDS 32 at a time, where each thread has prepared 8
// channels of one token (softplus once per token and channel, not once per state); B and C, which all channels of a group
// share, lie there as fp32.
#pragma once
#include "block_common.h"

namespace ttt {
namespace scan {

using namespace block;

constexpr int CH = kScanCh, TT = kScanTile;

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

// A log2(e) of a lane's states, finite: -inf keeps nothing, and exp(0 A) of a token that is not there is 1.
template <int NS>
__device__ __forceinline__ void decays(float (&a2)[NS], const ScanArgs& a, int c, int q, bool on) {
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = q * NS + i;
    const float x = on && n < a.N ? a.A[static_cast<int64_t>(c) * a.N + n] * kLog2e : 0.f;
    a2[i] = x != x ? x : fminf(fmaxf(x, -3.0e38f), 3.0e38f);
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

// B or C of a tile as a thread holds it between the load and LDS: elements tid, tid + 256, ... of [TT][4 NS].
template <typename T, int NS>
struct Rows {
  static constexpr int kN = 4 * NS, kEach = TT * kN / 256 > 0 ? TT * kN / 256 : 1;
  T v[kEach];
  __device__ __forceinline__ void load(const T* p, int64_t stride, int N, int t0, int t1, int tid) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int e = tid + 256 * k, t = t0 + e / kN, n = e % kN;
      v[k] = e < TT * kN && t < t1 && n < N ? p[t * stride + n] : T(0);
    }
  }
  __device__ __forceinline__ void stage(float* lds, int tid) const {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int e = tid + 256 * k;
      if (e < TT * kN) lds[e] = as_f32(v[k]);
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
