// Short causal convolution of each channel: forward, backward, single tokens.
//
// Pages: [TTT] = news article "大模型最强架构TTT问世！斯坦福UCSD等5年磨一剑，一夜推翻Transformer"
// (aharts.cn / itmax.cn), part 04 (the Mamba backbone the layer is measured in).
//
//   y_t = act(bias + sum_j w_j x_{t-K+1+j}),   K = 2, 3, 4, act the identity or silu
// 2 K flops a token and channel against 4 bytes: memory is the bound.  bf16, K = 4: 4 x 8192 tokens of 4096 channels 111 us, 4.9
// TB/s (fp32 192, 5.6); gradients of 8 x 2048 of 1536 54 us, 2.8 TB/s (fp32 77); one token of 512 x 4096 9.3 us.
#include <type_traits>

#include "block_common.h"

namespace ttt {
namespace {

using namespace block;

template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// w and bias of a piece of channels
template <int K, bool Wide, int V>
__device__ __forceinline__ void taps(float (&w)[K][V], float (&bias)[V], const ConvArgs& a, int c, int n) {
  if constexpr (Wide) {
    Piece<float, V * K> all;
    all.load(a.w + static_cast<int64_t>(c) * K);
    Piece<float, V> b;
    if (a.bias) b.load(a.bias + c);
    else b.zero();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bias[i] = b.get(i);
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][i] = all.get(i * K + j);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bias[i] = a.bias && i < n ? a.bias[c + i] : 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][i] = i < n ? a.w[static_cast<int64_t>(c + i) * K + j] : 0.f;
    }
  }
}

// The wave's number in the launch, as a scalar: what is the same for a wave is computed once.
__device__ __forceinline__ uint32_t wave_id() { return blockIdx.x * 4u + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

__device__ __forceinline__ int length(const int32_t* lens, int b, int T) { return lens ? max(0, min(lens[b], T)) : T; }

// row r of a sequence, r = -(K-1) .. -1 from the state before it
template <bool Wide, int K, typename T, int V>
__device__ __forceinline__ void row(Piece<T, V>& x, const ConvArgs& a, const T* xp, const T* st, int64_t r, int c, int n) {
  if (r >= 0) load<Wide>(x, xp + r * a.xs.t + c, n);
  else if (st) load<Wide>(x, st + (r + K - 1) * a.D + c, n);
  else x.zero();
}

// kTok tokens of a piece of channels to a thread, all of its rows on their way at once.  32 tokens read fewer rows twice but were
// slower throughout (bf16, rows of 4096: 4 x 2048 tokens 29.2 us against 28.1, 4 x 8192 tokens 115 against 108, of a wider row 123
// against 111).
constexpr int kTok = 8;

template <typename InT, typename OutT, int K, bool Wide>
__global__ __launch_bounds__(256) void ttt_conv_fwd(ConvArgs a, int blocks, int tiles) {
  constexpr int V = kVec<InT>;
  const uint32_t id = wave_id(), line = id / blocks;  // 64 pieces of channels to a wave
  const int c = static_cast<int>((id % blocks) * 64 + (threadIdx.x & 63)) * V;
  const int b = static_cast<int>(line / tiles), tile = static_cast<int>(line % tiles);
  if (b >= a.B || c >= a.D) return;
  const int n = min(V, a.D - c), len = length(a.lens, b, a.T), t0 = tile * kTok;
  const InT* xp = static_cast<const InT*>(a.X) + b * a.xs.b;
  const InT* st = a.state ? static_cast<const InT*>(a.state) + static_cast<int64_t>(b) * (K - 1) * a.D : nullptr;
  OutT* yp = static_cast<OutT*>(a.Y) + b * a.ys.b + c;

  Piece<InT, V> x[kTok + K - 1];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int64_t r = t0 - (K - 1) + i;
    if (r < len) row<Wide, K>(x[i], a, xp, st, r, c, n);
    else x[i].zero();
  }
  if (Wide && t0 + kTok <= len) {
#pragma unroll
    for (int i = 0; i < kTok; ++i) x[K - 1 + i].load(xp + (t0 + i) * a.xs.t + c);
  } else {
#pragma unroll
    for (int i = 0; i < kTok; ++i) load<Wide>(x[K - 1 + i], xp + (t0 + i) * a.xs.t + c, t0 + i < len ? n : 0);
  }
  float w[K][V], bias[V];
  taps<K, Wide>(w, bias, a, c, n);
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    if (t0 + t >= a.T) break;
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float s = bias[i];
#pragma unroll
      for (int j = 0; j < K; ++j) s = fmaf(w[j][i], x[t + j].get(i), s);
      y[i] = t0 + t < len ? s : 0.f;
      if (a.silu) y[i] *= sigmoid(y[i]);
    }
    Piece<OutT, V> out;
    out.set_all(y);
    store<Wide>(out, yp + (t0 + t) * a.ys.t, n);
  }
  if (tile == 0 && a.state_out) {
    InT* so = static_cast<InT*>(a.state_out) + static_cast<int64_t>(b) * (K - 1) * a.D + c;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      Piece<InT, V> v;
      row<Wide, K>(v, a, xp, st, static_cast<int64_t>(len) - (K - 1) + j, c, n);
      store<Wide>(v, so + static_cast<int64_t>(j) * a.D, n);
    }
  }
}

// A few tokens from the state, which goes on in place: a thread walks a piece of channels of S sequences, which share the taps
// and whose loads are on their way together.
template <typename InT, typename OutT, int K, bool Wide, int S>
__global__ __launch_bounds__(256) void ttt_conv_decode(ConvArgs a, int blocks) {
  constexpr int V = kVec<InT>;
  const uint32_t id = wave_id();
  const int64_t b0 = static_cast<int64_t>(id / blocks) * S;
  const int c = static_cast<int>((id % blocks) * 64 + (threadIdx.x & 63)) * V;
  if (b0 >= a.B || c >= a.D) return;
  const int n = min(V, a.D - c);
  Piece<InT, V> x[S][K];
  int len[S], most = 0;
#pragma unroll
  for (int r = 0; r < S; ++r) {
    len[r] = b0 + r < a.B ? length(a.lens, static_cast<int>(b0 + r), a.T) : 0;
    most = max(most, len[r]);
    const InT* st = static_cast<const InT*>(a.state_out) + (b0 + r) * (K - 1) * a.D + c;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load<Wide>(x[r][j], st + static_cast<int64_t>(j) * a.D, len[r] > 0 ? n : 0);
  }
  float w[K][V], bias[V];
  taps<K, Wide>(w, bias, a, c, n);
  for (int64_t t = 0; t < most; ++t) {
#pragma unroll
    for (int r = 0; r < S; ++r)
      load<Wide>(x[r][K - 1], static_cast<const InT*>(a.X) + (b0 + r) * a.xs.b + t * a.xs.t + c, t < len[r] ? n : 0);
#pragma unroll
    for (int r = 0; r < S; ++r) {
      if (t >= len[r]) continue;
      float y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float s = bias[i];
#pragma unroll
        for (int j = 0; j < K; ++j) s = fmaf(w[j][i], x[r][j].get(i), s);
        y[i] = a.silu ? s * sigmoid(s) : s;
      }
      Piece<OutT, V> out;
      out.set_all(y);
      store<Wide>(out, static_cast<OutT*>(a.Y) + (b0 + r) * a.ys.b + t * a.ys.t + c, n);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) x[r][j] = x[r][j + 1];
    }
  }
  Piece<OutT, V> none;
  none.zero();
#pragma unroll
  for (int r = 0; r < S; ++r) {
    if (b0 + r >= a.B) break;
    if (len[r] > 0) {
      InT* st = static_cast<InT*>(a.state_out) + (b0 + r) * (K - 1) * a.D + c;
#pragma unroll
      for (int j = 0; j < K - 1; ++j) store<Wide>(x[r][j], st + static_cast<int64_t>(j) * a.D, n);
    }
    for (int64_t t = len[r]; t < a.T; ++t) store<Wide>(none, static_cast<OutT*>(a.Y) + (b0 + r) * a.ys.b + t * a.ys.t + c, n);
  }
}

// Backward.  With g_t = dy_t act'(pre_t), pre_t the sum before the activation:
//   dx_t = sum_j w_j g_{t+K-1-j},   dw_j = sum_t g_t x_{t-K+1+j},   dbias = sum_t g_t
// A thread walks the tokens of a segment with the last K inputs and the last K g in registers; the first K - 1 rows in front
// of the segment and behind it are read (and their g computed) a second time.  Lanes of a workgroup: 32 pieces of channels
// by 8 segments, whose sums of dw and dbias are added through LDS; the rest is summed by a second launch, in a fixed order.
constexpr int kLanes = 32, kWalks = 8;

template <typename InT, typename OutT, int K, bool Wide>
__global__ __launch_bounds__(256) void ttt_conv_bwd(ConvArgs a, int cblocks) {
  constexpr int V = kVec<InT>;
  constexpr int NP = K + 1;
  __shared__ float sums[kWalks][NP][kLanes * V + 4];
  const int lane = threadIdx.x % kLanes, walk = threadIdx.x / kLanes;
  const int cb = static_cast<int>(blockIdx.x % static_cast<uint32_t>(cblocks));
  const uint32_t line = blockIdx.x / static_cast<uint32_t>(cblocks);
  const int p = static_cast<int>(line % static_cast<uint32_t>(a.nparts));
  const int64_t b = line / static_cast<uint32_t>(a.nparts);
  const int c = (cb * kLanes + lane) * V;
  const int n = min(V, a.D - c);  // (may be negative)
  const int len = length(a.lens, static_cast<int>(b), a.T);
  const int64_t seg = static_cast<int64_t>(p) * kWalks + walk;
  const int64_t t0 = seg * a.seg;
  const InT* xp = static_cast<const InT*>(a.X) + b * a.xs.b;
  const InT* st = a.state ? static_cast<const InT*>(a.state) + b * (K - 1) * a.D : nullptr;
  const OutT* gp = static_cast<const OutT*>(a.dY) + b * a.ys.b + c;
  OutT* dxp = static_cast<OutT*>(a.dX) + b * a.dxs.b + c;
  const OutT* ds = a.dstate_out ? static_cast<const OutT*>(a.dstate_out) + b * (K - 1) * a.D + c : nullptr;

  float w[K][V], bias[V], dw[NP][V];
  taps<K, Wide>(w, bias, a, n > 0 ? c : 0, n);
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j) dw[j][i] = 0.f;
  if (n > 0 && (t0 < a.T || seg == 0)) {  // (without tokens the state's gradient is still handed on)
    const int64_t t1 = min(static_cast<int64_t>(a.T), t0 + a.seg), end = min(t1, static_cast<int64_t>(len));
    Piece<InT, V> x[K];   // x_{t-K+1} .. x_t
    float g[K][V];        // g_{t-K+1} .. g_t
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int64_t r = t0 - (K - 1) + j;
      if (r < len) row<Wide, K>(x[j + 1], a, xp, st, r, c, n);
      else x[j + 1].zero();
#pragma unroll
      for (int i = 0; i < V; ++i) g[j + 1][i] = 0.f;
    }
    // token t gives g_t, and with it dx_{t-K+1}; the first segment's first K - 1 steps give the state's gradient
    for (int64_t t = t0; t < t1 + K - 1; ++t) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        x[j] = x[j + 1];
#pragma unroll
        for (int i = 0; i < V; ++i) g[j][i] = g[j + 1][i];
      }
      Piece<OutT, V> dy;
      if (t < len) {
        load<Wide>(x[K - 1], xp + t * a.xs.t + c, n);
        load<Wide>(dy, gp + t * a.ys.t, n);
      } else {
        x[K - 1].zero();
        dy.zero();
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float d = dy.get(i);
        if (a.silu) {
          float s = bias[i];
#pragma unroll
          for (int j = 0; j < K; ++j) s = fmaf(w[j][i], x[j].get(i), s);
          const float sg = sigmoid(s);
          d *= fmaf(sg, s * (1.f - sg), sg);
        }
        if (t >= len) d = 0.f;
        g[K - 1][i] = d;
        if (t < end) {
          dw[K][i] += d;
#pragma unroll
          for (int j = 0; j < K; ++j) dw[j][i] = fmaf(d, x[j].get(i), dw[j][i]);
        }
      }
      const int64_t r = t - (K - 1);  // the row whose gradient is whole now
      if (r >= t0 || (t0 == 0 && a.dstate)) {
        float dx[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float s = 0.f;
#pragma unroll
          for (int j = 0; j < K; ++j) s = fmaf(w[K - 1 - j][i], g[j][i], s);
          dx[i] = s;
        }
        // rows len-(K-1) .. len-1 are the final state too
        const int64_t last = r - (static_cast<int64_t>(len) - (K - 1));
        if (ds && last >= 0 && last < K - 1) {
          Piece<OutT, V> d;
          load<Wide>(d, ds + last * a.D, n);
#pragma unroll
          for (int i = 0; i < V; ++i) dx[i] += d.get(i);
        }
        Piece<OutT, V> out;
        if (r >= len) out.zero();
        else out.set_all(dx);
        if (r >= 0) store<Wide>(out, dxp + r * a.dxs.t, n);
        else store<Wide>(out, static_cast<OutT*>(a.dstate) + (b * (K - 1) + r + K - 1) * a.D + c, n);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) sums[walk][j][lane * V + i] = dw[j][i];
  __syncthreads();
  float* part = a.part + line * (static_cast<int64_t>(a.D) * NP);
  for (int e = threadIdx.x; e < kLanes * V * NP; e += 256) {
    const int j = e % NP, cc = e / NP, ch = cb * kLanes * V + cc;
    if (ch >= a.D) break;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWalks; ++k) s += sums[k][j][cc];
    if (j < K) part[static_cast<int64_t>(ch) * K + j] = s;
    else part[static_cast<int64_t>(a.D) * K + ch] = s;
  }
}

enum Which { FWD, BWD, DECODE };

template <typename InT, typename OutT, int K, bool Wide>
hipError_t go(Which which, const ConvArgs& a, hipStream_t s) {
  constexpr int V = kVec<InT>;
  const int pieces = (a.D + V - 1) / V, blocks = (pieces + 63) / 64;
  if (which == FWD) {
    const int tiles = a.T > 0 ? (a.T + kTok - 1) / kTok : 1;  // (without tokens the state is still handed on)
    const int64_t waves = static_cast<int64_t>(a.B) * tiles * blocks;
    ttt_conv_fwd<InT, OutT, K, Wide><<<static_cast<unsigned>((waves + 3) / 4), 256, 0, s>>>(a, blocks, tiles);
  } else if (which == DECODE) {
    // four sequences to a thread from 2^18 pieces on; one against four, rows of 4096 in bf16: 256 sequences (2^17) 5.7 and 6.1 us,
    // 512 9.5 and 8.0, 2048 27.3 and 21.6
    const bool four = static_cast<int64_t>(a.B) * pieces >= 1 << 18;
    const int64_t waves = static_cast<int64_t>(four ? (a.B + 3) / 4 : a.B) * blocks;
    const unsigned grid = static_cast<unsigned>((waves + 3) / 4);
    if (four) ttt_conv_decode<InT, OutT, K, Wide, 4><<<grid, 256, 0, s>>>(a, blocks);
    else ttt_conv_decode<InT, OutT, K, Wide, 1><<<grid, 256, 0, s>>>(a, blocks);
  } else {
    const int cblocks = (pieces + kLanes - 1) / kLanes;
    const int64_t n = static_cast<int64_t>(a.B) * a.nparts * cblocks;
    ttt_conv_bwd<InT, OutT, K, Wide><<<static_cast<unsigned>(n), 256, 0, s>>>(a, cblocks);
  }
  return hipGetLastError();
}

template <typename InT, typename OutT, int K>
hipError_t go(Which which, const ConvArgs& a, hipStream_t s) {
  return a.wide ? go<InT, OutT, K, true>(which, a, s) : go<InT, OutT, K, false>(which, a, s);
}

template <typename InT, typename OutT>
hipError_t go(Which which, const ConvArgs& a, hipStream_t s) {
  switch (a.K) {
    case 2: return go<InT, OutT, 2>(which, a, s);
    case 3: return go<InT, OutT, 3>(which, a, s);
    case 4: return go<InT, OutT, 4>(which, a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t go(Which which, const ConvArgs& a, hipStream_t s) {
  const bool inf = a.in_dtype == 0, outf = a.out_dtype == 0;
  if (inf && outf) return go<float, float>(which, a, s);
  if (inf) return go<float, uint16_t>(which, a, s);
  if (outf) return go<uint16_t, float>(which, a, s);
  return go<uint16_t, uint16_t>(which, a, s);
}

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s) { return go(FWD, a, s); }
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s) { return go(BWD, a, s); }
hipError_t launch_conv_decode(const ConvArgs& a, hipStream_t s) { return go(DECODE, a, s); }

}  // namespace ttt
