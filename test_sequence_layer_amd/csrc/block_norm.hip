// The join of two blocks: a norm behind a block, its gate, the residual scale and sum, and the norm before the next block.
//
// Pages: [TTT] = news article "大模型最强架构TTT问世！斯坦福UCSD等5年磨一剑，一夜推翻Transformer"
// (aharts.cn / itmax.cn), part 03 §9 (layer norm and residual around the layer), part 04 (backbones).
//
//   n = NORM(x) gamma_post + beta_post,   v = n silu(z)      (or, gate first, n = NORM(x silu(z)) ..., v = n)
//   s = res + alpha v,                    y = NORM(s) gamma_pre + beta_pre
// NORM divides by the root of the mean square plus eps, the layer norm after taking the mean off.  Each row is read once,
// kept in registers and written once: memory is the bound.
// 4 x 8192 rows of 2048, bf16 with an fp32 residual stream: 206 us, 4.6 TB/s (fp32 throughout 268, 4.9 TB/s).  Gradients of
// 8 x 2048 rows of 768: 76 us, two launches.  Rows over 4096 keep values in scratch in the gradients (96 bytes a lane, 350 element
// by element) and element by element in the forward (44): 8 x 2048 rows of 8192 in bf16 take 370 and 1117 us, of 8188 1112 and 3037.
#include <type_traits>

#include "block_common.h"

namespace ttt {
namespace {

using namespace block;

constexpr int NE = 8;  // elements of a row that a thread holds

__device__ __forceinline__ float wave_sum(float x) { return mfma::sum_rows(mfma::sum16(x)); }

__device__ __forceinline__ double wave_sum(double x) {
  auto step = [&](auto ctrl) {
    const uint64_t v = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_mov_dpp(static_cast<int>(v), decltype(ctrl)::value, 0xf, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_mov_dpp(static_cast<int>(v >> 32), decltype(ctrl)::value, 0xf, 0xf, true);
    x += __longlong_as_double(static_cast<uint64_t>(hi) << 32 | lo);
  };
  step(std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
  step(std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
  step(std::integral_constant<int, 0x141>{});  // row_half_mirror
  step(std::integral_constant<int, 0x140>{});  // row_mirror
  auto pair = [&](auto swap) {
    const uint64_t v = __double_as_longlong(x);
    const auto lo = swap(static_cast<uint32_t>(v)), hi = swap(static_cast<uint32_t>(v >> 32));
    x = __longlong_as_double(static_cast<uint64_t>(hi[0]) << 32 | lo[0]) + __longlong_as_double(static_cast<uint64_t>(hi[1]) << 32 | lo[1]);
  };
  pair([](uint32_t v) { return __builtin_amdgcn_permlane16_swap(v, v, false, false); });
  pair([](uint32_t v) { return __builtin_amdgcn_permlane32_swap(v, v, false, false); });
  return x;
}

// Sums over the W waves of a row's team.  Each sum has a slot of its own, eight of them in turn, so that one barrier a sum is
// enough: who writes a slot again is seven barriers further on than who still reads it could be.
template <int W>
struct Team {
  double (*slots)[W][2];  // [slot][wave][2] of this team
  int wave, next;
  static constexpr int kSlots = 8;
  template <typename F>
  __device__ __forceinline__ void sum2(F& a, F& b) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (W > 1) {
      double (*s)[2] = slots[next];
      next = next + 1 == kSlots ? 0 : next + 1;
      if ((threadIdx.x & 63) == 0) {
        s[wave][0] = a;
        s[wave][1] = b;
      }
      __syncthreads();
      a = static_cast<F>(s[0][0]);
      b = static_cast<F>(s[0][1]);
#pragma unroll
      for (int i = 1; i < W; ++i) {
        a += static_cast<F>(s[i][0]);
        b += static_cast<F>(s[i][1]);
      }
    }
  }
};

// mean (0 for the root-mean-square norm) and 1 / sqrt(var + eps) of a row of 1 / inv elements, NE of them in a thread (zeros
// behind the row's end).  The layer norm's two sums go in 64 bits, so that one pass is enough: nothing cancels in
// sum x^2 - D mean^2 that 32 bits would have kept.
template <int W>
__device__ __forceinline__ float2 stats(const float (&x)[NE], int valid, double inv, bool layer, float eps, Team<W>& team) {
  if (layer) {
    double s = 0.0, ss = 0.0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const double v = i < valid ? static_cast<double>(x[i]) : 0.0;
      s += v;
      ss = fma(v, v, ss);
    }
    team.sum2(s, ss);
    const double mean = s * inv, var = fma(ss, inv, -mean * mean);
    // (a row with an infinity has inf - inf here, and the NaN has to stay: fmax would drop it)
    return make_float2(static_cast<float>(mean), __builtin_amdgcn_rsqf(static_cast<float>(var < 0.0 ? 0.0 : var) + eps));
  }
  float s = 0.f, none = 0.f;
#pragma unroll
  for (int i = 0; i < NE; ++i) s = i < valid ? fmaf(x[i], x[i], s) : s;
  team.sum2(s, none);
  return make_float2(0.f, __builtin_amdgcn_rsqf(fmaf(s, static_cast<float>(inv), eps)));
}

// A row's sequence and token, and the one that is ``step`` rows further on (B and T are below 2^31, a step below 2^15).  In 32
// bits for the gradients, whose scalar registers run out (8 x 2048 x 768: 75.7 us, in 64 bits 78.8), in 64 for the forward
// (4 x 8192 x 2048: 207.0, in 32 bits 208.8).
template <typename I>
struct Walk {
  I b, t, T, db, dt;
  __device__ __forceinline__ Walk(int64_t line, int64_t step, int T_) : T(T_) {
    b = static_cast<I>(line / T);
    t = static_cast<I>(line - static_cast<int64_t>(b) * T);
    db = static_cast<I>(step) / T;
    dt = static_cast<I>(step) - db * T;
  }
  __device__ __forceinline__ void advance() {
    b += db;
    t += dt;
    if (t >= T) {
      t -= T;
      ++b;
    }
  }
};

// A thread's elements of a row: a piece at 8 r; element by element instead at i R + r.
template <int R, bool Wide>
struct Cols {
  int r, D;
  __device__ __forceinline__ int valid() const {  // of the thread's elements, in their order
    if constexpr (Wide) return 8 * r < D ? 8 : 0;
    else return r < D ? min(NE, (D - r + R - 1) / R) : 0;
  }
  template <typename T>
  __device__ __forceinline__ void load(float (&x)[NE], const T* p) const {
    if constexpr (Wide) {
      const int c = 8 * r;
      Piece<T, 8> v;
      if (c < D) v.load(p + c);
      else v.zero();
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = v.get(j);
    } else {
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        const int c = j * R + r;
        x[j] = c < D ? as_f32(p[c]) : 0.f;
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(const float (&x)[NE], T* p) const {
    if constexpr (Wide) {
      const int c = 8 * r;
      Piece<T, 8> v;
      v.set_all(x);
      if (c < D) v.store(p + c);
    } else {
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        const int c = j * R + r;
        if (c < D) put(p + c, x[j]);
      }
    }
  }
  __device__ __forceinline__ void param(float (&x)[NE], const float* p, float none) const {
    if (p) {
      load(x, p);
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) x[i] = none;
    }
  }
};

__device__ __forceinline__ bool dead(const NormArgs& a, int64_t b, int64_t t) {
  return a.lens && t >= max(0, min(a.lens[b], a.T));
}

template <typename T, typename RT, int R, bool Wide>
__global__ __launch_bounds__(R) void ttt_norm_fwd(NormArgs a) {
  constexpr int W = R / 64;
  __shared__ double slots[Team<W>::kSlots][W][2];
  Team<W> team{slots, static_cast<int>(threadIdx.x >> 6), 0};
  const Cols<R, Wide> cols{static_cast<int>(threadIdx.x), a.D};
  const int valid = cols.valid();
  const double inv = 1.0 / static_cast<double>(a.D);
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  Walk<int64_t> at(blockIdx.x, gridDim.x, a.T);
  for (int64_t line = blockIdx.x; line < rows; line += gridDim.x, at.advance()) {
    const int64_t b = at.b, t = at.t;
    RT* sp = a.S ? static_cast<RT*>(a.S) + b * a.ss.b + t * a.ss.t : nullptr;
    T* yp = a.Y ? static_cast<T*>(a.Y) + b * a.ys.b + t * a.ys.t : nullptr;
    float v[NE], w[NE];
    if (dead(a, b, t)) {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = 0.f;
      if (sp) cols.store(v, sp);
      if (yp) cols.store(v, yp);
      continue;
    }
    float z[NE], res[NE];
    cols.load(v, static_cast<const T*>(a.X) + b * a.xs.b + t * a.xs.t);
    if (a.Z) cols.load(z, static_cast<const T*>(a.Z) + b * a.zs.b + t * a.zs.t);
    if (a.res) cols.load(res, static_cast<const RT*>(a.res) + b * a.rs.b + t * a.rs.t);
    if (a.Z) {
#pragma unroll
      for (int i = 0; i < NE; ++i) z[i] *= sigmoid(z[i]);
      if (a.gate_first) {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] *= z[i];
      }
    }
    if (a.gamma_post) {
      const float2 st = stats<W>(v, valid, inv, a.layer, a.eps, team);
      cols.param(w, a.gamma_post, 1.f);
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = (v[i] - st.x) * st.y * w[i];
      if (a.beta_post) {
        cols.param(w, a.beta_post, 0.f);
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] += w[i];
      }
    }
    if (a.Z && !a.gate_first) {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] *= z[i];
    }
    if (a.alpha) {
      cols.param(w, a.alpha, 1.f);
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] *= w[i];
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] += res[i];
    }
    if (sp) cols.store(v, sp);
    if (yp) {
      const float2 st = stats<W>(v, valid, inv, a.layer, a.eps, team);
      cols.param(w, a.gamma_pre, 1.f);
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = (v[i] - st.x) * st.y * w[i];
      if (a.beta_pre) {
        cols.param(w, a.beta_pre, 0.f);
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] += w[i];
      }
      cols.store(v, yp);
    }
  }
}

// The gradient through unit = (x - mean) rstd, in place: h holds the gradient of unit.
template <int W>
__device__ __forceinline__ void norm_back(float (&h)[NE], const float (&unit)[NE], float rstd, int valid, float inv, bool layer,
                                          Team<W>& team) {
  float s = 0.f, m = 0.f;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    if (i >= valid) h[i] = 0.f;
    s = fmaf(h[i], unit[i], s);
    m += h[i];
  }
  team.sum2(s, m);
  const float cs = s * inv, cm = layer ? m * inv : 0.f;
#pragma unroll
  for (int i = 0; i < NE; ++i) h[i] = (h[i] - cm - unit[i] * cs) * rstd;
}

// Backward: everything of the forward again from the row, then back through it.  A thread keeps its columns' sums of the
// parameters' gradients over all rows of its workgroup; teams of fewer than 256 threads share a workgroup, which adds theirs up.
template <typename T, typename RT, int R, bool Wide>
__global__ __launch_bounds__(R < 256 ? 256 : R) void ttt_norm_bwd(NormArgs a) {
  constexpr int W = R / 64, TEAMS = R < 256 ? 256 / R : 1;
  __shared__ double slots[TEAMS][Team<W>::kSlots][W][2];
  __shared__ float sums[TEAMS > 1 ? 256 : 1][TEAMS > 1 ? 9 : 1];
  const int who = R < 256 ? __builtin_amdgcn_readfirstlane(threadIdx.x / R) : 0, r = threadIdx.x % R;
  Team<W> team{slots[who], r >> 6, 0};
  const Cols<R, Wide> cols{r, a.D};
  const int valid = cols.valid();
  const double inv = 1.0 / static_cast<double>(a.D);
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  // the columns' parameters stay in registers too, and the next row is on its way.  Teams of 1024 have no registers left for
  // either: at 8 x 2048 rows of 8192, bf16, a row ahead took 1400 us, reading each row as it comes 1114
  constexpr bool kHeld = R < 1024, kAhead = Wide && kHeld;
  float wa[NE], wp[NE], wb[NE], wn[NE];
  auto fill = [&] {
    cols.param(wa, a.alpha, 1.f);
    cols.param(wp, a.gamma_post, 1.f);
    cols.param(wb, a.beta_post, 0.f);
    cols.param(wn, a.gamma_pre, 1.f);
  };
  if constexpr (kHeld) fill();
  float acc[5][NE];
#pragma unroll
  for (int k = 0; k < 5; ++k)
#pragma unroll
    for (int i = 0; i < NE; ++i) acc[k][i] = 0.f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
  int64_t first = static_cast<int64_t>(blockIdx.x) * TEAMS;
  Walk<uint32_t> ahead(first + who, step, max(a.T, 1));  // of the next row that is read
  // the row's pieces as they lie in memory, on their way a row ahead.  Rows behind their sequence's last token and tensors that
  // are not there are not read: their loads go to this workgroup's own partial sums, which it writes at its end, and are dropped
  struct Raw {
    Piece<T, 8> x, z, dy;
    Piece<RT, 8> res, ds;
  } raw;
  float* const part = a.part + static_cast<int64_t>(blockIdx.x) * 5 * a.D;
  auto skipped = [&](int64_t line) { return line >= rows || dead(a, ahead.b, ahead.t); };
  auto fetch = [&](bool skip) {
    auto get = [&](auto& v, const auto* p, const Strides2& st) {
      typedef std::remove_const_t<std::remove_pointer_t<decltype(p)>> E;
      const E* from = p && !skip ? p + (ahead.b * st.b + ahead.t * st.t) : reinterpret_cast<const E*>(part);
      v.load(from + (8 * r < a.D ? 8 * r : 0));
    };
    get(raw.x, static_cast<const T*>(a.X), a.xs);
    get(raw.z, static_cast<const T*>(a.Z), a.zs);
    get(raw.res, static_cast<const RT*>(a.res), a.rs);
    get(raw.ds, static_cast<const RT*>(a.dS), a.ss);
    get(raw.dy, static_cast<const T*>(a.dY), a.ys);
  };
  bool next_none = skipped(first + who);
  if constexpr (kAhead) {
    if (first < rows) fetch(next_none);
  }
  for (; first < rows; first += step) {
    const int64_t b = ahead.b, t = ahead.t;
    const bool off = first + who >= rows, none = next_none;
    ahead.advance();
    next_none = skipped(first + step + who);
    // (a team without a row goes along on zeros: the others wait for it at the sums)
    float x[NE], z[NE], u1[NE], v[NE], u2[NE], g[NE];
    float gate[NE], slope[NE];
    if constexpr (kAhead) {
      auto take = [&](float (&to)[NE], auto& from, bool on) {
        const bool here = on && !none && 8 * r < a.D;
#pragma unroll
        for (int j = 0; j < 8; ++j) to[j] = here ? from.get(j) : 0.f;
      };
      take(x, raw.x, true);
      take(z, raw.z, a.Z != nullptr);
      take(u2, raw.res, a.res != nullptr);
      take(v, raw.ds, a.dS != nullptr);
      take(g, raw.dy, a.dY != nullptr);
      if (first + step < rows) fetch(next_none);
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) x[i] = z[i] = g[i] = u2[i] = v[i] = 0.f;
      if (!none) {
        cols.load(x, static_cast<const T*>(a.X) + b * a.xs.b + t * a.xs.t);
        if (a.Z) cols.load(z, static_cast<const T*>(a.Z) + b * a.zs.b + t * a.zs.t);
        if (a.res) cols.load(u2, static_cast<const RT*>(a.res) + b * a.rs.b + t * a.rs.t);
        if (a.dS) cols.load(v, static_cast<const RT*>(a.dS) + b * a.ss.b + t * a.ss.t);
        if (a.dY) cols.load(g, static_cast<const T*>(a.dY) + b * a.ys.b + t * a.ys.t);
      }
    }
    float ds[NE], n1[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) ds[i] = v[i];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      gate[i] = 1.f;
      slope[i] = 0.f;
      if (a.Z) {
        const float s = sigmoid(z[i]);
        gate[i] = z[i] * s;
        slope[i] = fmaf(gate[i], 1.f - s, s);
      }
      u1[i] = a.gate_first ? x[i] * gate[i] : x[i];
      n1[i] = u1[i];
    }
    float rstd1 = 1.f;
    if (a.gamma_post) {
      const float2 st = stats<W>(u1, valid, inv, a.layer, a.eps, team);
      rstd1 = st.y;
      if constexpr (!kHeld) fill();
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        u1[i] = i < valid ? (u1[i] - st.x) * st.y : 0.f;
        n1[i] = fmaf(u1[i], wp[i], wb[i]);
      }
    }
    if constexpr (!kHeld) cols.param(wa, a.alpha, 1.f);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      v[i] = a.gate_first ? n1[i] : n1[i] * gate[i];
      u2[i] = fmaf(wa[i], v[i], u2[i]);
    }
    if (a.dY) {
      const float2 st = stats<W>(u2, valid, inv, a.layer, a.eps, team);
      if constexpr (!kHeld) cols.param(wn, a.gamma_pre, 1.f);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        u2[i] = i < valid ? (u2[i] - st.x) * st.y : 0.f;
        if (!none) {
          acc[3][i] = fmaf(g[i], u2[i], acc[3][i]);
          acc[4][i] += g[i];
        }
        g[i] *= wn[i];
      }
      norm_back<W>(g, u2, st.y, valid, static_cast<float>(inv), a.layer, team);
#pragma unroll
      for (int i = 0; i < NE; ++i) ds[i] += g[i];
    }
    if (none) {
#pragma unroll
      for (int i = 0; i < NE; ++i) ds[i] = 0.f;
    }
    if (a.dres && !off) cols.store(ds, static_cast<RT*>(a.dres) + b * a.drs.b + t * a.drs.t);
    if constexpr (!kHeld) cols.param(wa, a.alpha, 1.f);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      if (!none) acc[0][i] = fmaf(ds[i], v[i], acc[0][i]);
      g[i] = ds[i] * wa[i];                                  // dv
      z[i] = a.gate_first ? 0.f : g[i] * n1[i] * slope[i];   // dz
      if (!a.gate_first) g[i] *= gate[i];                    // dn
    }
    if (a.gamma_post) {
      if constexpr (!kHeld) cols.param(wp, a.gamma_post, 1.f);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        if (!none) {
          acc[1][i] = fmaf(g[i], u1[i], acc[1][i]);
          acc[2][i] += g[i];
        }
        g[i] *= wp[i];
      }
      norm_back<W>(g, u1, rstd1, valid, static_cast<float>(inv), a.layer, team);
    }
    if (a.gate_first) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        z[i] = g[i] * x[i] * slope[i];
        g[i] *= gate[i];
      }
    }
    if (none) {
#pragma unroll
      for (int i = 0; i < NE; ++i) g[i] = z[i] = 0.f;
    }
    if (!off) {
      cols.store(g, static_cast<T*>(a.dX) + b * a.dxs.b + t * a.dxs.t);
      if (a.dZ) cols.store(z, static_cast<T*>(a.dZ) + b * a.dzs.b + t * a.dzs.t);
    }
  }
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    if constexpr (TEAMS > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NE; ++i) sums[threadIdx.x][i] = acc[k][i];
      __syncthreads();
      if (who == 0) {
#pragma unroll
        for (int i = 0; i < NE; ++i)
#pragma unroll
          for (int m = 1; m < TEAMS; ++m) acc[k][i] += sums[m * R + r][i];
      }
    }
    if (who == 0) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = Wide ? 8 * r + i : i * R + r;
        if (c < a.D) part[static_cast<int64_t>(k) * a.D + c] = acc[k][i];
      }
    }
  }
}

template <typename T, typename RT, int R>
hipError_t go(bool backward, const NormArgs& a, hipStream_t s) {
  if (backward) {
    constexpr int threads = R < 256 ? 256 : R;
    const unsigned grid = static_cast<unsigned>(a.blocks);
    if (a.wide) ttt_norm_bwd<T, RT, R, true><<<grid, threads, 0, s>>>(a);
    else ttt_norm_bwd<T, RT, R, false><<<grid, threads, 0, s>>>(a);
  } else {
    const int64_t rows = static_cast<int64_t>(a.B) * a.T, most = 256 * 2048 / R;  // all that run at a time
    const unsigned grid = static_cast<unsigned>(rows < most ? rows : most);
    if (a.wide) ttt_norm_fwd<T, RT, R, true><<<grid, R, 0, s>>>(a);
    else ttt_norm_fwd<T, RT, R, false><<<grid, R, 0, s>>>(a);
  }
  return hipGetLastError();
}

// Threads of a row: the fewest whose 8 elements each hold it.
template <typename T, typename RT>
hipError_t go(bool backward, const NormArgs& a, hipStream_t s) {
  if (a.D <= 512) return go<T, RT, 64>(backward, a, s);
  if (a.D <= 1024) return go<T, RT, 128>(backward, a, s);
  if (a.D <= 2048) return go<T, RT, 256>(backward, a, s);
  if (a.D <= 4096) return go<T, RT, 512>(backward, a, s);
  if (a.D <= 8192) return go<T, RT, 1024>(backward, a, s);
  return hipErrorInvalidValue;
}

hipError_t go(bool backward, const NormArgs& a, hipStream_t s) {
  const bool f = a.in_dtype == 0, rf = a.res_dtype == 0;
  if (f && rf) return go<float, float>(backward, a, s);
  if (f) return go<float, uint16_t>(backward, a, s);
  if (rf) return go<uint16_t, float>(backward, a, s);
  return go<uint16_t, uint16_t>(backward, a, s);
}

}  // namespace

int norm_max_d() { return 8192; }
int norm_teams(int D) { return D <= 512 ? 4 : D <= 1024 ? 2 : 1; }

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) { return go(false, a, s); }
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) { return go(true, a, s); }

}  // namespace ttt
