// Rotary positions of q and k: the pairs of each row turned by position * frequency.
//
//   (y1, y2) = scale ((x1, x2) cos t - (x2, -x1) sin t),   t = position * freqs[i]
// The gradient turns back by the same angle with the same scale.  Every value is
// read and written once and costs three flops, so the kernel is a copy: what it
// must not do is compute an angle (64-bit product, sine and cosine) per value.
// A thread owns V pairs of one (sequence, token), computes their V angles once and
// walks the heads of q and of k with them; where there are too few tokens to
// fill the chip, the heads are dealt out over blockIdx.y.
#include <type_traits>

#include "mfma_common.h"
#include "rope.h"

namespace ttt {
namespace {

using mfma::u32x2;
using mfma::u32x4;

// N consecutive elements as fp32, aligned to their own size (at most 16 bytes at a time)
template <int N, typename T>
__device__ __forceinline__ void ld(const T* p, float x[N]) {
  if constexpr (N == 1) {
    if constexpr (sizeof(T) == 4) x[0] = p[0];
    else x[0] = bf16_bits_to_f32(p[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 w = mfma::ld_stream(reinterpret_cast<const u32x4*>(p) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * i + j] = __uint_as_float(w[j]);
    }
  } else {
    static_assert(N == 8, "16 bytes of bf16");
    const u32x4 w = mfma::ld_stream(reinterpret_cast<const u32x4*>(p));
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = __uint_as_float(w[j] << 16), x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
template <int N, typename T>
__device__ __forceinline__ void st(T* p, const float x[N]) {
  if constexpr (N == 1) {
    if constexpr (sizeof(T) == 4) p[0] = x[0];
    else p[0] = f32_to_bf16_bits(x[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(x[4 * i + j]);
      mfma::st_stream(reinterpret_cast<u32x4*>(p) + i, w);
    }
  } else {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(mfma::float2v{x[2 * j], x[2 * j + 1]}, mfma::bf16x2));
    mfma::st_stream(reinterpret_cast<u32x4*>(p), w);
  }
}

// E elements a thread: 16 bytes twice (half layout), or E elements in a row (interleaved); E = 1: one
// pair, element by element, where alignment or an odd rot allows no more.
template <typename T, bool INTER, int E>
__global__ __launch_bounds__(256) void ttt_rotary(RotaryArgs a) {
  constexpr int V = E == 1 ? 1 : (INTER ? E / 2 : E);  // pairs per thread
  const int half = a.rope.rot / 2;
  const int turned = half / V;                            // threads per row with pairs
  const int rest = a.in_place ? 0 : (a.d - a.rope.rot) / E;  // and with elements to pass on
  const int per = turned + rest;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= static_cast<int64_t>(a.B) * a.T * per) return;
  const int unit = static_cast<int>(id % per);
  const int64_t bt = id / per;
  const int b = static_cast<int>(bt / a.T), t = static_cast<int>(bt % a.T);
  const int heads = a.H + a.Hkv;
  const int h0 = static_cast<int>(static_cast<int64_t>(heads) * blockIdx.y / gridDim.y);
  const int h1 = static_cast<int>(static_cast<int64_t>(heads) * (blockIdx.y + 1) / gridDim.y);
  const T* qi = static_cast<const T*>(a.q) + b * a.qs.b + t * a.qs.t;
  const T* ki = static_cast<const T*>(a.k) + b * a.ks.b + t * a.ks.t;
  T* qo = static_cast<T*>(a.qo) + b * a.qos.b + t * a.qos.t;
  T* ko = static_cast<T*>(a.ko) + b * a.kos.b + t * a.kos.t;
  auto in = [&](int h) { return h < a.H ? qi + h * a.qs.h : ki + (h - a.H) * a.ks.h; };
  auto out = [&](int h) { return h < a.H ? qo + h * a.qos.h : ko + (h - a.H) * a.kos.h; };

  if (unit >= turned) {
    const int c = a.rope.rot + (unit - turned) * E;
    for (int h = h0; h < h1; ++h) {
      float x[E];
      ld<E>(in(h) + c, x);
      st<E>(out(h) + c, x);
    }
    return;
  }
  float cs[V], sn[V];
  const int64_t pos = rope_pos(a.rope, b, t);
#pragma unroll
  for (int p = 0; p < V; ++p) {
    rope_angle(pos, a.rope.freqs[unit * V + p], cs[p], sn[p]);
    cs[p] *= a.rope.scale;
    sn[p] *= a.inverse ? -a.rope.scale : a.rope.scale;
  }
  auto turn = [&](float& x, float& y, int p) {
    const float u = fmaf(-y, sn[p], x * cs[p]);
    y = fmaf(x, sn[p], y * cs[p]);
    x = u;
  };
  constexpr int HU = 4;  // heads in flight
  constexpr int N = INTER ? 2 * V : V;
  for (int h = h0; h < h1; h += HU) {
    float x[HU][N], y[HU][INTER ? 1 : N];
#pragma unroll
    for (int u = 0; u < HU; ++u) {
      if (h + u >= h1) break;
      const T* p = in(h + u);
      if constexpr (INTER && E == 1) {
        ld<1>(p + 2 * unit, &x[u][0]);
        ld<1>(p + 2 * unit + 1, &x[u][1]);
      } else if constexpr (INTER) {
        ld<N>(p + unit * N, x[u]);
      } else {
        ld<N>(p + unit * N, x[u]);
        ld<N>(p + half + unit * N, y[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < HU; ++u) {
      if (h + u >= h1) break;
      T* p = out(h + u);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (INTER) turn(x[u][2 * v], x[u][2 * v + 1], v);
        else turn(x[u][v], y[u][v], v);
      }
      if constexpr (INTER && E == 1) {
        st<1>(p + 2 * unit, &x[u][0]);
        st<1>(p + 2 * unit + 1, &x[u][1]);
      } else if constexpr (INTER) {
        st<N>(p + unit * N, x[u]);
      } else {
        st<N>(p + unit * N, x[u]);
        st<N>(p + half + unit * N, y[u]);
      }
    }
  }
}

template <typename T, bool INTER, int E>
hipError_t go(const RotaryArgs& a, hipStream_t s) {
  constexpr int V = E == 1 ? 1 : (INTER ? E / 2 : E);
  const int64_t per = a.rope.rot / 2 / V + (a.in_place ? 0 : (a.d - a.rope.rot) / E);
  const int64_t blocks = (static_cast<int64_t>(a.B) * a.T * per + 255) / 256;
  const int heads = a.H + a.Hkv;
  int64_t y = (1024 + blocks - 1) / blocks;  // four workgroups per CU
  if (y > heads) y = heads;
  ttt_rotary<T, INTER, E><<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(y)), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t pick(const RotaryArgs& a, hipStream_t s) {
  constexpr int E = 16 / sizeof(T);
  // whole 16-byte pieces: every row and both halves of its pairs begin on one
  bool wide = a.rope.rot % (a.rope.interleaved ? E : 2 * E) == 0 && a.d % E == 0;
  for (const void* p : {a.q, a.k, static_cast<const void*>(a.qo), static_cast<const void*>(a.ko)})
    wide = wide && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  for (const Strides3& x : {a.qs, a.ks, a.qos, a.kos}) wide = wide && x.b % E == 0 && x.h % E == 0 && x.t % E == 0;
  if (a.rope.interleaved) return wide ? go<T, true, E>(a, s) : go<T, true, 1>(a, s);
  return wide ? go<T, false, E>(a, s) : go<T, false, 1>(a, s);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t s) {
  return a.dtype == 0 ? pick<float>(a, s) : pick<uint16_t>(a, s);
}

}  // namespace ttt
