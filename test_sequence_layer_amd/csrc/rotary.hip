// Rotary positions of q and k: the pairs of each row turned by position * frequency.
//
//   (y1, y2) = scale (x1 cos t - x2 sin t, x1 sin t + x2 cos t),   t = position * freqs[i]
// The gradient turns back by the same angle with the same scale.  Every value is
// read and written once and costs three flops, so the kernel is a copy: what it
// must not do is compute an angle (64-bit product, sine and cosine) per value.
// A thread owns a piece of a row at one (sequence, token), computes its angles once
// and walks the heads of q and of k with them, the next four heads' loads on their
// way while it turns four; where there are too few tokens to fill the chip, the
// heads are dealt out over blockIdx.y.  Four ways of cutting rows into pieces:
//   interleaved pairs, rows of whole 16-byte pieces: a piece, its pairs within it;
//   halves of whole pieces: a piece, its partner from the lane that has it;
//   other halves: a piece, the elements of the other half through LDS, whole rows in a workgroup;
//   rows at any address, or of more than 256 pieces: one pair, element by element.
// Measured on MI355X for B2 H32+32 T32768 d64 bf16, 1.07 GB (a copy of that size: 204 us): interleaved 214 us,
// halves 212 us (through LDS 240, eight elements of both halves a thread 243, four 241), halves of 31 pairs 214 us
// (pair by pair 638), half of the head 215 us.
#include <type_traits>

#include "mfma_common.h"
#include "rope.h"

namespace ttt {
namespace {

using mfma::u32x4;

// a 16-byte piece of T as fp32 and back
template <typename T>
__device__ __forceinline__ void unpack(u32x4 w, float x[16 / sizeof(T)]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) x[j] = __uint_as_float(w[j]);
    else x[2 * j] = __uint_as_float(w[j] << 16), x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ u32x4 pack(const float x[16 / sizeof(T)]) {
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(x[j]);
    else w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(mfma::float2v{x[2 * j], x[2 * j + 1]}, mfma::bf16x2));
  }
  return w;
}
template <typename T>
__device__ __forceinline__ u32x4 ld(const T* p) {
  return mfma::ld_stream(reinterpret_cast<const u32x4*>(p));
}
template <typename T>
__device__ __forceinline__ void st(T* p, u32x4 w) {
  mfma::st_stream(reinterpret_cast<u32x4*>(p), w);
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_bits_to_f32(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = f32_to_bf16_bits(x); }

enum { kInterleaved, kHalves, kOddHalves, kPairs };

// Threads a row takes.
template <typename T, int WAY>
__host__ __device__ __forceinline__ int row_threads(int d, int rot, bool in_place) {
  constexpr int E = 16 / sizeof(T);
  if (WAY == kInterleaved || WAY == kOddHalves) return in_place ? (rot + E - 1) / E : d / E;
  if (WAY == kHalves) return d / E;
  return rot / 2 + (in_place ? 0 : d - rot);
}

// Threads of a workgroup that have rows: of kOddHalves whole rows, whose pieces meet in its LDS (rows that went on in
// the next workgroup, and took the partners there from memory: d 96 397 us for 215, d 48 491 for 223, q alone).
template <int WAY>
__host__ __device__ __forceinline__ int busy_threads(int per) { return WAY == kOddHalves ? 256 / per * per : 256; }

// The rows of one (sequence, token) that a thread walks: heads h0 .. h1 - 1 of q, then k.
template <typename T>
struct Heads {
  const T *qi, *ki;
  T *qo, *ko;
  int64_t qih, kih, qoh, koh;
  int H, h0, h1;
  __device__ __forceinline__ Heads(const RotaryArgs& a, int b, int t) {
    qi = static_cast<const T*>(a.q) + b * a.qs.b + t * a.qs.t;
    ki = static_cast<const T*>(a.k) + b * a.ks.b + t * a.ks.t;
    qo = static_cast<T*>(a.qo) + b * a.qos.b + t * a.qos.t;
    ko = static_cast<T*>(a.ko) + b * a.kos.b + t * a.kos.t;
    qih = a.qs.h, kih = a.ks.h, qoh = a.qos.h, koh = a.kos.h;
    H = a.H;
    const int64_t heads = a.H + static_cast<int64_t>(a.Hkv);
    h0 = static_cast<int>(heads * blockIdx.y / gridDim.y);
    h1 = static_cast<int>(heads * (blockIdx.y + 1) / gridDim.y);
  }
  __device__ __forceinline__ const T* in(int h) const { return h < H ? qi + h * qih : ki + (h - H) * kih; }
  __device__ __forceinline__ T* out(int h) const { return h < H ? qo + h * qoh : ko + (h - H) * koh; }
};

template <typename T, int WAY>
__global__ __launch_bounds__(256) void ttt_rotary(RotaryArgs a) {
  constexpr int E = 16 / sizeof(T);
  constexpr int HU = 4;  // heads a step: 212 us [B, H, T, d] and 222 [B, T, H, d]; 2: 208 and 234, 8: 232 and 218
  const int rot = a.rope.rot, half = rot / 2;
  const int per = row_threads<T, WAY>(a.d, rot, a.in_place);
  const int busy = busy_threads<WAY>(per);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * busy + threadIdx.x;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  // (kOddHalves: all threads of a workgroup keep step; the ones left over walk the last row and store nothing)
  const bool live = id < rows * per && static_cast<int>(threadIdx.x) < busy;
  if (WAY != kOddHalves && !live) return;
  const int unit = static_cast<int>(id % per);
  const int64_t bt = live ? id / per : rows - 1;
  const int b = static_cast<int>(bt / a.T), t = static_cast<int>(bt % a.T);
  const Heads<T> hd(a, b, t);
  const int64_t pos = rope_pos(a.rope, b, t);
  auto angle = [&](int i, float& c, float& s) {
    rope_angle(pos, a.rope.freqs[i], c, s);
    c *= a.rope.scale;
    s *= a.inverse ? -a.rope.scale : a.rope.scale;
  };
  auto turn = [](float& x, float& y, float c, float s) {
    const float u = fmaf(-y, s, x * c);
    y = fmaf(x, s, y * c);
    x = u;
  };

  if constexpr (WAY == kInterleaved || WAY == kHalves) {
    constexpr int V = WAY == kHalves ? E : E / 2;  // angles
    typedef u32x4 W;
    const int o = unit * E, pieces = half / E;
    const bool turned = o < rot, first = o < half;
    const int partner = static_cast<int>(threadIdx.x % 64) + (!turned ? 0 : first ? pieces : -pieces);  // lane
    auto load = [&](W r[HU], int h) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < HU; ++u) r[u] = ld(hd.in(min(h + u, hd.h1 - 1)) + o);
    };
    W now[HU], next[HU];
    load(now, hd.h0);
    float cs[V], sn[V];
#pragma unroll
    for (int p = 0; p < V; ++p) {
      const int i = WAY == kHalves ? (first ? o : o - half) + p : o / 2 + p;
      cs[p] = 1.f;
      sn[p] = 0.f;
      if (turned && i < half) angle(i, cs[p], sn[p]);
      if (WAY == kHalves && first) sn[p] = -sn[p];
    }
    for (int h = hd.h0; h < hd.h1; h += HU) {
      if (h + HU < hd.h1) load(next, h + HU);
#pragma unroll
      for (int u = 0; u < HU; ++u) {
        float x[E];
        unpack<T>(now[u], x);
        if constexpr (WAY == kHalves) {
          W other;
#pragma unroll
          for (int j = 0; j < 4; ++j) other[j] = __shfl(now[u][j], partner);
          float y[E];
          unpack<T>(other, y);
#pragma unroll
          for (int i = 0; i < V; ++i) x[i] = fmaf(y[i], sn[i], x[i] * cs[i]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (o / 2 + i < half) turn(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
        }
        if (turned) now[u] = pack<T>(x);
        if (h + u < hd.h1) st(hd.out(h + u) + o, now[u]);
        now[u] = next[u];
      }
    }
  } else if constexpr (WAY == kOddHalves) {
    // Each thread's piece goes to LDS, where the threads of its row find the elements that their own are paired with.
    constexpr int kStep = 20 / sizeof(T);  // elements between pieces: 20 bytes, so that pieces begin in other banks
    __shared__ __align__(16) T buf[2][2][256 * kStep];
    const int o = unit * E;
    const int mine = static_cast<int>(threadIdx.x);
    constexpr int HL = 2;  // heads a barrier
    typedef u32x4 W;
    W now[HL], next[HL];
    auto load = [&](W* r, int h) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < HL; ++u) r[u] = ld(hd.in(min(h + u, hd.h1 - 1)) + o);
    };
    load(now, hd.h0);
    float cs[E], sn[E];
    int from[E];  // the partner in LDS
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int c = o + j;
      cs[j] = 1.f;
      sn[j] = 0.f;
      from[j] = mine * kStep + j;
      if (live && c < rot) {
        angle(c < half ? c : c - half, cs[j], sn[j]);
        if (c < half) sn[j] = -sn[j];
        const int other = c < half ? c + half : c - half;
        from[j] = (mine - unit + other / E) * kStep + other % E;
      }
    }
    int n = 0;
    for (int h = hd.h0; h < hd.h1; h += HL, n ^= 1) {
#pragma unroll
      for (int u = 0; u < HL; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t*>(buf[n][u] + mine * kStep)[j] = now[u][j];
      if (h + HL < hd.h1) load(next, h + HL);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < HL; ++u) {
        if (h + u >= hd.h1) break;
        float x[E];
        unpack<T>(now[u], x);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          if (o + j < rot) x[j] = fmaf(widen(buf[n][u][from[j]]), sn[j], x[j] * cs[j]);
        }
        if (live) st(hd.out(h + u) + o, pack<T>(x));
        now[u] = next[u];
      }
    }
  } else {
    if (unit >= half) {
      const int c = rot + unit - half;
      for (int h = hd.h0; h < hd.h1; ++h) hd.out(h)[c] = hd.in(h)[c];
      return;
    }
    const int o1 = a.rope.interleaved ? 2 * unit : unit, o2 = a.rope.interleaved ? o1 + 1 : o1 + half;
    float c, s;
    angle(unit, c, s);
    for (int h = hd.h0; h < hd.h1; ++h) {
      float x = widen(hd.in(h)[o1]), y = widen(hd.in(h)[o2]);
      turn(x, y, c, s);
      put(hd.out(h) + o1, x);
      put(hd.out(h) + o2, y);
    }
  }
}

template <typename T, int WAY>
hipError_t go(const RotaryArgs& a, hipStream_t s) {
  const int64_t per = row_threads<T, WAY>(a.d, a.rope.rot, a.in_place);
  const int64_t busy = busy_threads<WAY>(static_cast<int>(per));
  const int64_t blocks = (static_cast<int64_t>(a.B) * a.T * per + busy - 1) / busy;
  const int64_t heads = static_cast<int64_t>(a.H) + a.Hkv;
  int64_t y = (1024 + blocks - 1) / blocks;  // four workgroups per CU
  if (y > heads) y = heads;
  ttt_rotary<T, WAY><<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(y)), 256, 0, s>>>(a);
  return hipGetLastError();
}

// every row of the tensors that there are begins on a multiple of `bytes`
bool aligned_to(const RotaryArgs& a, int bytes, int size) {
  auto ok = [&](const void* p, const Strides3& x) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && x.b * size % bytes == 0 && x.h * size % bytes == 0 &&
           x.t * size % bytes == 0;
  };
  return (a.H == 0 || (ok(a.q, a.qs) && ok(a.qo, a.qos))) && (a.Hkv == 0 || (ok(a.k, a.ks) && ok(a.ko, a.kos)));
}

int pick(const RotaryArgs& a) {
  const int size = a.dtype == 0 ? 4 : 2, e = 16 / size;
  if (a.d % e != 0 || !aligned_to(a, 16, size)) return kPairs;
  if (a.rope.interleaved) return kInterleaved;
  // (whole rows in a wave)
  if (a.rope.rot % (2 * e) == 0 && 64 % (a.d / e) == 0) return kHalves;
  // (a row's pieces in a workgroup)
  return a.d / e <= 256 ? kOddHalves : kPairs;
}

template <typename T>
hipError_t launch(const RotaryArgs& a, hipStream_t s) {
  switch (pick(a)) {
    case kInterleaved: return go<T, kInterleaved>(a, s);
    case kHalves: return go<T, kHalves>(a, s);
    case kOddHalves: return go<T, kOddHalves>(a, s);
    default: return go<T, kPairs>(a, s);
  }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t s) {
  return a.dtype == 0 ? launch<float>(a, s) : launch<uint16_t>(a, s);
}

const char* rotary_name(const RotaryArgs& a) {
  switch (pick(a)) {
    case kInterleaved: return "ttt_rotary_interleaved";
    case kHalves: return "ttt_rotary_halves";
    case kOddHalves: return "ttt_rotary_odd_halves";
    default: return "ttt_rotary_pairs";
  }
}

}  // namespace ttt
