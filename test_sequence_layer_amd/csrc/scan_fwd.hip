// Selective scan, forward: prompts.
//
// Pages: [TTT] = news article "大模型最强架构TTT问世！斯坦福UCSD等5年磨一剑，一夜推翻Transformer"
// (aharts.cn / itmax.cn), part 04 (the Mamba layer that TTT is compared with).
//
// Per token, channel and state one exp, two products and two multiply-adds, against (with N = 16) half a byte: vector issue is
// the bound.  4 x 8192 tokens, 4096 channels, N = 16, bf16: 525 us, 2.0 TB/s, at a clock of 2.42 GHz (590 in the first launches
// after a pause, before the clock has risen); by its bytes 203 at the 5.3 TB/s of a large copy.  Those five instructions by
// themselves, from registers, take 356 us for as many states with one wave to a SIMD, 329 with two and 315 with eight.  They are
// 1.68e8 of the kernel's 2.54e8 vector instructions (the others: softplus, skip, gate, conversions, sums over lanes, addresses),
// which keep the vector unit busy in 93% of the cycles.
#include <utility>

#include "scan_common.h"

namespace ttt {
namespace {

using namespace scan;

constexpr int TT = kScanTile;
constexpr int LANES = 4;                      // to a channel
constexpr int WALKERS = CH * LANES;           // threads that walk
constexpr int THREADS = WALKERS + 256;        // and those that bring the tiles in and out
constexpr int GS = 4;                         // tokens whose decays and sums go together

// Sums over the four lanes of a channel (16 apart) of four tokens' values: lane row r gets token r's.
__device__ __forceinline__ float row_sums(const float (&y)[4]) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(y[0]), __float_as_uint(y[2]), false, false);
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(y[1]), __float_as_uint(y[3]), false, false);
  const float a = __uint_as_float(p[0]) + __uint_as_float(p[1]), b = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// f(0) .. f(N - 1) with constants for arguments
template <typename F, int... I>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  each(f, std::make_integer_sequence<int, N>{});
}

// States: only what the segment adds to a zero state and the sum of its dt.
// Waves 0 to 3 walk a tile while waves 4 to 7 bring the next one into LDS (softplus) and take the last one out (D u, the
// gate), one barrier a tile: a wave by itself issues a vector instruction every 5 cycles and one that needs the last one's
// result every 8 (measured; two waves to a SIMD every 4), and 64 channels to a workgroup often leave one workgroup to a CU.
// The 16 channels of a lane row share their B, so that a lane reads one state of one token, and all of the row take it from
// there by a broadcast inside the multiplication (DPP): four states of B and C for each token and lane kept LDS busy for more
// than half of the time.
template <typename InT, typename OutT, int NS, bool Wide, bool States>
__global__ __launch_bounds__(THREADS, 2) void ttt_scan_fwd(ScanArgs a) {
  constexpr int NP = LANES * NS;
  __shared__ __align__(16) float2 sdt[2][TT][CH];  // dt, dt u
  __shared__ __align__(16) float bc[2][2 * TT * NP];
  __shared__ __align__(16) float sy[States ? 1 : 2][States ? 1 : TT][CH];
  const int segs = States ? a.nseg - 1 : a.nseg;
  const int seg = static_cast<int>(blockIdx.x % segs);
  const Place p = place(a, blockIdx.x / segs);
  const int begin = seg * a.seglen, tokens = min(a.T, begin + a.seglen), end = min(p.len, tokens);
  const int64_t slot = static_cast<int64_t>(p.b) * a.nseg + seg;

  if (__builtin_amdgcn_readfirstlane(threadIdx.x) < WALKERS) {
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, cw = (tid >> 6) * 16 + (lane & 15);
    const int c = p.c0 + cw;
    const bool on = cw < p.nc;
    float a2[NS], h[NS], sum = 0.f;
    decays(a2, a, c, q, on);
    if (States || a.nseg == 1) {
      load_states(h, States || !a.h0 ? nullptr : a.h0 + (static_cast<int64_t>(p.b) * a.D + c) * a.N, a.N, q, on);
    } else {
      start_state(h, a2, a, p, seg, c, q, on);
    }
    int buf = 0;
    for (int t0 = begin; t0 < end; t0 += TT, buf ^= 1) {
      __syncthreads();
      constexpr int RB = 16 / NS;  // tokens whose B lies in a row's lanes: state lane % NS of token lane / NS
      const float* sb = bc[buf] + (lane & 15) / NS * NP + q * NS + (lane & 15) % NS;
      float Br[TT / RB];
#pragma unroll
      for (int k = 0; k < TT / RB; ++k) Br[k] = sb[k * RB * NP];
      // dt, dt u and C of a group of tokens: the next one's are on their way while this one is worked on
      float2 d[2][GS];
      float C[2][GS][NS];
      auto read = [&](int buf2, int k) {
#pragma unroll
        for (int j = 0; j < GS; ++j) {
          d[buf2][j] = sdt[buf][k + j][cw];
          if constexpr (!States) lds_floats(C[buf2][j], bc[buf] + (TT + k + j) * NP + q * NS);
        }
      };
      read(0, 0);
      each<TT / GS>([&](auto group) {
        constexpr int k = group * GS;
        if constexpr (k + GS < TT) read((group + 1) & 1, k + GS);
        float e[GS][NS], y[GS];
#pragma unroll
        for (int j = 0; j < GS; ++j)
#pragma unroll
          for (int i = 0; i < NS; ++i) e[j][i] = __builtin_amdgcn_exp2f(d[group & 1][j].x * a2[i]);
        each<GS>([&](auto j) {
          constexpr int t = k + j;
          const float2 x = d[group & 1][j];
          float s = 0.f;
          each<NS>([&](auto i) {
            constexpr int from = 0x150 + t % RB * NS + i;  // row_newbcast
            h[i] = fmaf(e[j][i], h[i], mfma::dpp_mov<from>(Br[t / RB]) * x.y);
            if constexpr (!States) s = fmaf(C[group & 1][j][i], h[i], s);
          });
          if constexpr (States) sum += x.x;
          y[j] = s;
        });
        if constexpr (!States) sy[buf][k + q][cw] = row_sums(y);
      });
    }
    __syncthreads();
    if constexpr (States) {
      store_states(h, a.hseg + ((slot + 1) * a.D + c) * a.N, a.N, q, on);
      if (on && q == 0) a.sseg[slot * a.D + c] = sum;
      if (seg == 0) {
        load_states(h, a.h0 ? a.h0 + (static_cast<int64_t>(p.b) * a.D + c) * a.N : nullptr, a.N, q, on);
        store_states(h, a.hseg + (slot * a.D + c) * a.N, a.N, q, on);
      }
    } else {
      if (seg == a.nseg - 1) store_states(h, a.h_final + (static_cast<int64_t>(p.b) * a.D + c) * a.N, a.N, q, on);
    }
    return;
  }

  // this thread's piece of a tile: token row, channels oct .. oct + 7
  const int tid = threadIdx.x - WALKERS, row = tid >> 3, oct = (tid & 7) * 8;
  const int n8 = min(8, p.nc - oct);  // (may be negative)
  const int64_t first = begin + row, oc = p.c0 + (Wide && n8 <= 0 ? 0 : oct);
  const InT* up = static_cast<const InT*>(a.u) + p.b * a.us.b + first * a.us.t + oc;
  const InT* dp = static_cast<const InT*>(a.dt) + p.b * a.dts.b + first * a.dts.t + oc;
  const InT* zp = States || !a.z ? nullptr : static_cast<const InT*>(a.z) + p.b * a.zs.b + first * a.zs.t + oc;
  OutT* yp = static_cast<OutT*>(a.y) + p.b * a.ys.b + first * a.ys.t + oc;
  BcRows<InT, NP, TT, Wide> rows(a, p, begin, tid, !States);
  typename BcRows<InT, NP, TT, Wide>::Values bc_far;
  float bias[8], skip[8];
  params<8>(bias, a.dt_bias ? a.dt_bias + p.c0 + oct : nullptr, n8, 0.f);
  if constexpr (!States) params<8>(skip, a.Dskip ? a.Dskip + p.c0 + oct : nullptr, n8, 0.f);
  // u of the tile before, this one, the next and the one behind it; the others' as far as they are wanted
  Piece<InT, 8> u_old, u_now, u_next, u_far, dt_next, dt_far, z_old, z_now;
  auto count = [&](int t0) { return t0 + row < end ? n8 : 0; };  // of this thread's 8 channels in the tile at t0
  auto fetch = [&](int t0) {
    const int n = count(t0);
    const InT *u = up, *d = dp;
    if (Wide && t0 + TT > end) {  // rows behind the end: the last one instead
      const int over = max(0, t0 + row - (end - 1));
      u -= over * a.us.t;
      d -= over * a.dts.t;
    }
    load_ahead<Wide>(u_far, u, n);
    load_ahead<Wide>(dt_far, d, n);
    up += TT * a.us.t;
    dp += TT * a.dts.t;
    rows.load(bc_far, t0, end, 1);
  };
  // (u is zero where there is no token, and so has its dt to be)
  auto stage = [&](int buf, int t0) {
    const int n = count(t0);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = dt_next.get(i) + bias[i];
    if (a.softplus) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = softplus(x[i]);
    }
    if (!Wide || t0 + TT > end || p.nc < CH) {
      keep<Wide>(u_next, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = i < n ? x[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      *reinterpret_cast<float4*>(&sdt[buf][row][oct + i]) = make_float4(x[i], x[i] * u_next.get(i), x[i + 1], x[i + 1] * u_next.get(i + 1));
  };
  auto finish = [&](int buf, int n) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(&sy[buf][row][oct + i]);
      y[i] = v.x; y[i + 1] = v.y; y[i + 2] = v.z; y[i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(skip[i], u_old.get(i), y[i]);
    if (a.z) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= z_old.get(i) * sigmoid(z_old.get(i));
    }
    Piece<OutT, 8> out;
    out.set_all(y);
    store<Wide>(out, yp, n);
    yp += TT * a.ys.t;
  };
  if (begin < end) {
    fetch(begin);
    u_next = u_far;
    dt_next = dt_far;
    rows.stage(bc_far, bc[0], begin, end);
    stage(0, begin);
    if (begin + TT < end) fetch(begin + TT);
  }
  u_now = u_next;
  z_now.zero();
  int buf = 0;
  for (int t0 = begin; t0 < end; t0 += TT, buf ^= 1) {
    __syncthreads();
    u_old = u_now;
    u_now = u_next;
    u_next = u_far;
    dt_next = dt_far;
    z_old = z_now;
    rows.stage(bc_far, bc[buf ^ 1], t0 + TT, end);
    if (t0 + 2 * TT < end) fetch(t0 + 2 * TT);
    if constexpr (!States) {
      if (a.z) {
        const InT* z = zp;
        if (Wide && t0 + TT > end) z -= max(0, t0 + row - (end - 1)) * a.zs.t;
        load_ahead<Wide>(z_now, z, count(t0));
        zp += TT * a.zs.t;
      }
    }
    stage(buf ^ 1, t0 + TT);  // (zeros behind the last tile)
    if constexpr (!States) {
      if (t0 > begin) finish(buf ^ 1, n8);
    }
  }
  __syncthreads();
  if constexpr (!States) {
    if (begin < end) {
      u_old = u_now;
      z_old = z_now;
      finish(buf ^ 1, count(begin + (end - begin - 1) / TT * TT));
    }
    // rows behind the sequence's end (those of its last tile too)
    OutT* y0 = static_cast<OutT*>(a.y) + p.b * a.ys.b + p.c0 + oct;
    Piece<OutT, 8> none;
    none.zero();
    for (int64_t t = max(begin, end) + row; t < tokens; t += TT) store<Wide>(none, y0 + t * a.ys.t, n8);
  }
}

// NS states from q NS on, in fours where N and the addresses allow it.
template <bool Wide, int NS>
__device__ __forceinline__ void token_states(float (&x)[NS], const float* p, int N, int q) {
  if constexpr (Wide && NS >= 4) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      const float4 v = q * NS + i < N ? *reinterpret_cast<const float4*>(p + q * NS + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
  } else {
    load_states(x, p, N, q, true);
  }
}

template <bool Wide, typename T, int NS>
__device__ __forceinline__ void token_row(float (&x)[NS], const T* p, int N, int q) {
  if constexpr (Wide && NS >= 4) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      Piece<T, 4> v;
      if (q * NS + i < N) v.load(p + q * NS + i);
      else v.zero();
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i + j] = v.get(j);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) x[i] = q * NS + i < N ? as_f32(p[q * NS + i]) : 0.f;
  }
}

// A few tokens, the state in place: four lanes to a channel, NS states each.  8 N bytes of state a channel against 5 N flops: a
// copy of the state with the arithmetic on the way.  512 sequences of 4096 channels, N = 16, bf16, one token: 69 us, 4.1 TB/s.
// Four sequences to a thread, which share the channel's parameters, took 90 (16 sequences 6.6 against 4.4, 1024 sequences 176
// against 142, four tokens of them 442 against 266; in fp32 1024 sequences 118 against 128, four tokens 231 against 224).
template <typename InT, typename OutT, int NS, bool Wide>
__global__ __launch_bounds__(256) void ttt_scan_decode(ScanArgs a) {
  const uint32_t blocks = (static_cast<uint32_t>(a.D) + 15) / 16;  // 16 channels to a wave
  const uint32_t id = blockIdx.x * 4u + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = threadIdx.x & 3, c = static_cast<int>(id % blocks * 16 + (threadIdx.x >> 2 & 15));
  const int64_t b = id / blocks;
  if (b >= a.B || c >= a.D) return;
  const int g = c / (a.D / a.G), len = a.lens ? max(0, min(a.lens[b], a.T)) : a.T;
  float* const state = a.h_final + (b * a.D + c) * a.N;
  float h[NS], a2[NS];
  token_states<Wide>(h, state, a.N, q);
  token_states<Wide>(a2, a.A + static_cast<int64_t>(c) * a.N, a.N, q);
#pragma unroll
  for (int i = 0; i < NS; ++i) a2[i] = scaled_decay(a2[i]);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.Dskip ? a.Dskip[c] : 0.f;
  for (int64_t t = 0; t < len; ++t) {
    float Bv[NS], Cv[NS], y = 0.f;
    const float u = as_f32(static_cast<const InT*>(a.u)[b * a.us.b + t * a.us.t + c]);
    const float dt = as_f32(static_cast<const InT*>(a.dt)[b * a.dts.b + t * a.dts.t + c]);
    const float z = a.z ? as_f32(static_cast<const InT*>(a.z)[b * a.zs.b + t * a.zs.t + c]) : 0.f;
    token_row<Wide>(Bv, static_cast<const InT*>(a.Bm) + b * a.bs.b + g * a.bs.h + t * a.bs.t, a.N, q);
    token_row<Wide>(Cv, static_cast<const InT*>(a.Cm) + b * a.cs.b + g * a.cs.h + t * a.cs.t, a.N, q);
    float step = dt + bias;
    if (a.softplus) step = softplus(step);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      h[i] = fmaf(__builtin_amdgcn_exp2f(step * a2[i]), h[i], step * u * Bv[i]);
      if (Wide || q * NS + i < a.N) y = fmaf(Cv[i], h[i], y);
    }
    y = fmaf(skip, u, quad_sum(y));
    if (a.z) y *= z * sigmoid(z);
    if (q == 0) put(static_cast<OutT*>(a.y) + b * a.ys.b + t * a.ys.t + c, y);
  }
  if (len > 0) {
    if constexpr (Wide && NS >= 4) {
#pragma unroll
      for (int i = 0; i < NS; i += 4)
        if (q * NS + i < a.N) *reinterpret_cast<float4*>(state + q * NS + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    } else {
      store_states(h, state, a.N, q, true);
    }
  }
  for (int64_t t = len + q; t < a.T; t += 4) put(static_cast<OutT*>(a.y) + b * a.ys.b + t * a.ys.t + c, 0.f);
}

enum Which { STATES, FWD, DECODE };

template <typename InT, typename OutT, int NS>
hipError_t go(Which which, const ScanArgs& a, hipStream_t s) {
  if (which == DECODE) {
    const int64_t waves = static_cast<int64_t>(a.B) * ((a.D + 15) / 16);
    const unsigned grid = static_cast<unsigned>((waves + 3) / 4);
    if (a.wide) ttt_scan_decode<InT, OutT, NS, true><<<grid, 256, 0, s>>>(a);
    else ttt_scan_decode<InT, OutT, NS, false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
  }
  const int dg = a.D / a.G, segs = which == STATES ? a.nseg - 1 : a.nseg;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.G * ((dg + CH - 1) / CH) * segs);
  if (which == STATES) {
    if (a.wide) ttt_scan_fwd<InT, float, NS, true, true><<<grid, THREADS, 0, s>>>(a);
    else ttt_scan_fwd<InT, float, NS, false, true><<<grid, THREADS, 0, s>>>(a);
  } else {
    if (a.wide) ttt_scan_fwd<InT, OutT, NS, true, false><<<grid, THREADS, 0, s>>>(a);
    else ttt_scan_fwd<InT, OutT, NS, false, false><<<grid, THREADS, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <typename InT, typename OutT>
hipError_t go(Which which, const ScanArgs& a, hipStream_t s) {
  switch (scan_states(a.N)) {
    case 1: return go<InT, OutT, 1>(which, a, s);
    case 2: return go<InT, OutT, 2>(which, a, s);
    case 4: return go<InT, OutT, 4>(which, a, s);
    case 8: return go<InT, OutT, 8>(which, a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t go(Which which, const ScanArgs& a, hipStream_t s) {
  const bool inf = a.in_dtype == 0, outf = a.out_dtype == 0;
  if (which == STATES) return inf ? go<float, float>(which, a, s) : go<uint16_t, float>(which, a, s);
  if (inf && outf) return go<float, float>(which, a, s);
  if (inf) return go<float, uint16_t>(which, a, s);
  if (outf) return go<uint16_t, float>(which, a, s);
  return go<uint16_t, uint16_t>(which, a, s);
}

}  // namespace

int scan_states(int N) {
  for (int n = 1; n <= 8; n *= 2)
    if (N >= 1 && N <= 4 * n) return n;
  return 0;
}

hipError_t launch_scan_states(const ScanArgs& a, hipStream_t s) { return go(STATES, a, s); }
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t s) { return go(FWD, a, s); }
hipError_t launch_scan_decode(const ScanArgs& a, hipStream_t s) { return go(DECODE, a, s); }

}  // namespace ttt
