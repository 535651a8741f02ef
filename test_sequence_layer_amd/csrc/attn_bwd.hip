// Linear attention with a decay per head: the backward, on the CDNA4 matrix cores.
//
// With W_t the state after token t, G_t its gradient (lambda = exp(log_decay)),
//   G_t = scale dZ_t Q_t^T + lambda G_{t+1}          (the last one plus dW_final)
//   dQ_t = scale W_t^T dZ_t,   dK_t = G_t^T V_t,   dV_t = G_t K_t,   dW0 = lambda G_0
// each of dQ, dK, dV is the forward's walk (attn_walk.h) over other tensors, dK and dV
// from the last token to the first.  One launch holds the three walks of every
// (sequence, head) or segment as workgroups of their own: three times the workgroups of
// one fused reverse walk, each with one state (dQ's walk, with the decay's gradient, two)
// instead of three, and no state kept in two layouts.  Measured on MI355X for B8 H12 T2048
// d64 in bf16, with two parts for bf16 outputs: a dQ launch and a fused dK, dV, decay walk
// with its states in two layouts 173 us, this 120 us; 410 us both at B16 H32 T2048; two
// launches, dK and dV first, 437 us.  Now, with three parts, 115 and 430 us.  Bound by issue
// slots in the latter (93% busy, 74% vector instructions: parts of states, scores and decayed
// values), with 1.48 GB moved.  At d = 128 the walks spill 18 to 128 registers: 672 us for
// B16 H16 T2048 in bf16.
//
// The walks of dK and dV read the same rows at the same time, on the same XCD (unit_of):
// the second finds them in its L2 (measured: 8.3 tensors fetched instead of 10).
#include "attn_walk.h"

namespace ttt {
namespace attn {
namespace {

// sum over the lanes of a wave, in the same order in every run
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

template <typename T>
__device__ __forceinline__ const T* at(const void* p, const Strides3& s, int b, int h, int64_t t) {
  return static_cast<const T*>(p) + b * s.b + h * s.h + t * s.t;
}

constexpr int max2(int a, int b) { return a > b ? a : b; }

template <int D, typename QT, typename ZT, typename OT>
__global__ __launch_bounds__(4 * D, 2) void ttt_attn_bwd(AttnBwdArgs a) {
  constexpr int NB = D / 16;
  constexpr int kLds = max2(WalkLds<D, true, true, ZT, QT, QT, QT>::kSize,
                            max2(WalkLds<D, true, false, QT, ZT, QT, QT>::kSize,
                                 WalkLds<D, true, false, QT, QT, ZT, QT>::kSize));
  __shared__ __align__(16) uint16_t lds[kLds];
  __shared__ float powers[15 + C + 1];
  const float* pw = powers + 15;
  __shared__ double part[NB];
  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  // kind 0: dQ, 1: dK, 2: dV.  The dQ walks, which take twice the others' time, begin first.
  const int64_t units = static_cast<int64_t>(a.B) * a.H * a.nseg, id = blockIdx.x;
  Unit pl{id, 0};
  if (id >= units) {
    pl = unit_of(id - units, 2, units);
    ++pl.kind;
  }
  const int chain = static_cast<int>(pl.unit / a.nseg), seg = static_cast<int>(pl.unit % a.nseg);
  const int b = chain / a.H, h = chain % a.H, hk = h / a.group;
  const float lg = a.log_decay[h];
  if (tid < 15 + C + 1) powers[tid] = tid < 15 ? 0.f : powl(lg, tid - 15);
  const int len = seq_len(a.lens, b, a.T);
  const int sb = seg * a.seglen, se = min(sb + a.seglen, a.T);
  const int n = max(0, min(len, se) - sb);
  const int64_t dd = static_cast<int64_t>(D) * D;
  const float* loc = a.loc + static_cast<int64_t>(chain) * a.nseg * 3 * dd;
  const int pad0 = max(len, sb);  // padding rows among this segment's

  float4v s[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) s[i] = mfma::zero4v();
  if (pl.kind == 0) {
    float4v u[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) u[i] = mfma::zero4v();
    if (seg == 0 && a.W0) load_state<D>(a.W0 + b * a.w0_bstride + h * dd, true, w, li, g4, s);
    if (n > 0 && a.carried && seg > 0) {
      load_state<D>(loc + (seg - 1) * 3 * dd, false, w, li, g4, s);
      load_state<D>(loc + (seg - 1) * 3 * dd + dd, false, w, li, g4, u);
    }
    if (n > 0 && !a.carried && seg > 0) {
      const SegmentDecay e(lg, a.seglen);
      const float sl = static_cast<float>(a.seglen);
      for (int c = 0; c < seg; ++c) {
        float4v x[NB], y[NB];
        load_state<D>(loc + c * 3 * dd, false, w, li, g4, x);
        load_state<D>(loc + c * 3 * dd + dd, false, w, li, g4, y);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          u[i] = e.carry(u[i] + s[i] * sl, y[i]);
          s[i] = e.carry(s[i], x[i]);
        }
      }
    }
    __syncthreads();
    ZT* dq = static_cast<ZT*>(a.dQ) + b * a.dqs.b + h * a.dqs.h;
    Walk<ZT, QT, QT, QT, ZT> k;
    k.x = at<ZT>(a.dZ, a.zs, b, h, sb);
    k.y = at<QT>(a.V, a.vs, b, hk, sb);
    k.v = at<QT>(a.K, a.ks, b, hk, sb);
    k.q = at<QT>(a.Q, a.qs, b, h, sb);
    k.o = dq + sb * a.dqs.t;
    k.xt = a.zs.t;
    k.yt = a.vs.t;
    k.vt = a.ks.t;
    k.qt = a.qs.t;
    k.ot = a.dqs.t;
    k.n = n;
    k.lg = lg;
    k.sp = k.si = a.scale;
    k.su = 1.f;
    double dg = 0.0;
    walk<D, true, true>(k, false, lds, pw, s, u, dg);
    if (pad0 < se) zero_rows<D>(dq, a.dqs.t, pad0, se);
    if (a.dWf && seg == (len > 0 ? (len - 1) / a.seglen : 0)) {  // the last state depends on the decay too
      float4v x[NB];
      load_state<D>(a.dWf + chain * dd, true, w, li, g4, x);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) dg += static_cast<double>(x[i][r]) * static_cast<double>(u[i][r]);
    }
    dg = wave_sum(dg);
    if (lane == 0) part[w] = dg;
    __syncthreads();
    if (tid == 0) {
      double sum = 0.0;
      for (int i = 0; i < NB; ++i) sum += part[i];
      if (a.nseg == 1) a.dg[chain] = static_cast<float>(sum);
      else a.dgpart[static_cast<int64_t>(chain) * a.nseg + seg] = sum;
    }
    return;
  }

  // dK, dV: token i of the walk is token len - 1 - i
  bool fresh = false;
  if (seg == 0 && a.dWf) {
    load_state<D>(a.dWf + chain * dd, pl.kind == 1, w, li, g4, s);
    fresh = true;
  }
  if (n > 0 && a.carried && seg > 0) load_state<D>(loc + (seg - 1) * 3 * dd + 2 * dd, pl.kind == 2, w, li, g4, s);
  if (n > 0 && !a.carried && seg > 0)
    carry_states<D>(loc + 2 * dd, 3 * dd, seg, SegmentDecay(lg, a.seglen), pl.kind == 2, w, li, g4, s);
  __syncthreads();
  const int64_t t0 = len - 1 - sb;  // (only for a walk of at least one token)
  const int ho = a.parts ? h : hk;
  double none = 0.0;
  OT* out = pl.kind == 1 ? static_cast<OT*>(a.dK) + b * a.dks.b + ho * a.dks.h
                         : static_cast<OT*>(a.dV) + b * a.dvs.b + ho * a.dvs.h;
  const int64_t ot = pl.kind == 1 ? a.dks.t : a.dvs.t;
  if (pl.kind == 1) {
    Walk<QT, ZT, QT, QT, OT> k;
    k.x = at<QT>(a.V, a.vs, b, hk, t0);
    k.y = at<ZT>(a.dZ, a.zs, b, h, t0);
    k.v = at<QT>(a.Q, a.qs, b, h, t0);
    k.q = nullptr;
    k.o = out + t0 * ot;
    k.xt = -a.vs.t;
    k.yt = -a.zs.t;
    k.vt = -a.qs.t;
    k.qt = 0;
    k.ot = -ot;
    k.n = n;
    k.lg = lg;
    k.sp = k.su = a.scale;
    k.si = 1.f;
    walk<D, true, false>(k, fresh, lds, pw, s, s, none);
  } else {
    Walk<QT, QT, ZT, QT, OT> k;
    k.x = at<QT>(a.K, a.ks, b, hk, t0);
    k.y = at<QT>(a.Q, a.qs, b, h, t0);
    k.v = at<ZT>(a.dZ, a.zs, b, h, t0);
    k.q = nullptr;
    k.o = out + t0 * ot;
    k.xt = -a.ks.t;
    k.yt = -a.qs.t;
    k.vt = -a.zs.t;
    k.qt = 0;
    k.ot = -ot;
    k.n = n;
    k.lg = lg;
    k.sp = k.su = a.scale;
    k.si = 1.f;
    walk<D, true, false>(k, fresh, lds, pw, s, s, none);
  }
  if (pad0 < se) zero_rows<D>(out, ot, pad0, se);
  if (pl.kind == 2 && seg == (len > 0 ? (len - 1) / a.seglen : 0)) {
    const float e1 = len > 0 ? pw[1] : 1.f;  // from the first token's state to the one before it
#pragma unroll
    for (int i = 0; i < NB; ++i) s[i] = s[i] * e1;
    store_state<D>(a.dW0 + chain * dd, w, li, g4, s);
  }
}

// The states of segments 0 .. nseg-2 at their ends, the first from the start state, the
// others from zero: W^T with its derivative, and G^T.
template <int D, typename QT, typename ZT>
__global__ __launch_bounds__(4 * D) void ttt_attn_bwd_states(AttnBwdArgs a) {
  constexpr int NB = D / 16;
  constexpr int kLds =
      max2(WalkLds<D, false, true, QT, QT, QT, QT>::kSize, WalkLds<D, false, false, QT, ZT, QT, QT>::kSize);
  __shared__ __align__(16) uint16_t lds[kLds];
  __shared__ float powers[15 + C + 1];
  const float* pw = powers + 15;
  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  const Unit pl = unit_of(blockIdx.x, 2, static_cast<int64_t>(a.B) * a.H * (a.nseg - 1));
  const int chain = static_cast<int>(pl.unit / (a.nseg - 1)), seg = static_cast<int>(pl.unit % (a.nseg - 1));
  const int b = chain / a.H, h = chain % a.H, hk = h / a.group;
  const float lg = a.log_decay[h];
  if (tid < 15 + C + 1) powers[tid] = tid < 15 ? 0.f : powl(lg, tid - 15);
  const int len = seq_len(a.lens, b, a.T);
  const int sb = seg * a.seglen;
  if (len <= sb + a.seglen) return;  // no segment behind this one has a token
  const int64_t dd = static_cast<int64_t>(D) * D;
  float* loc = a.loc + (static_cast<int64_t>(chain) * a.nseg + seg) * 3 * dd;
  float4v s[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) s[i] = mfma::zero4v();
  double none = 0.0;
  if (pl.kind == 0) {
    float4v u[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) u[i] = mfma::zero4v();
    if (seg == 0 && a.W0) load_state<D>(a.W0 + b * a.w0_bstride + h * dd, true, w, li, g4, s);
    __syncthreads();
    Walk<QT, QT, QT, QT, QT> k;
    k.x = k.q = nullptr;
    k.o = nullptr;
    k.xt = k.qt = k.ot = 0;
    k.y = at<QT>(a.V, a.vs, b, hk, sb);
    k.v = at<QT>(a.K, a.ks, b, hk, sb);
    k.yt = a.vs.t;
    k.vt = a.ks.t;
    k.n = a.seglen;
    k.lg = lg;
    k.sp = k.si = k.su = 1.f;
    walk<D, false, true>(k, false, lds, pw, s, u, none);
    store_state<D>(loc, w, li, g4, s);
    store_state<D>(loc + dd, w, li, g4, u);
    return;
  }
  bool fresh = false;
  if (seg == 0 && a.dWf) {
    load_state<D>(a.dWf + chain * dd, true, w, li, g4, s);
    fresh = true;
  }
  __syncthreads();
  const int64_t t0 = len - 1 - sb;
  Walk<QT, ZT, QT, QT, QT> k;
  k.x = k.q = nullptr;
  k.o = nullptr;
  k.xt = k.qt = k.ot = 0;
  k.y = at<ZT>(a.dZ, a.zs, b, h, t0);
  k.v = at<QT>(a.Q, a.qs, b, h, t0);
  k.yt = -a.zs.t;
  k.vt = -a.qs.t;
  k.n = a.seglen;
  k.lg = lg;
  k.sp = k.si = 1.f;
  k.su = a.scale;
  walk<D, false, false>(k, fresh, lds, pw, s, s, none);
  store_state<D>(loc + 2 * dd, w, li, g4, s);
}

// Four elements a thread: the parts of a shared head's query heads, in order; then the
// decay's gradient of a (sequence, head): its segments' sums, in order.
template <typename OT>
__global__ __launch_bounds__(256) void ttt_attn_sum(AttnSumArgs a) {
  const int per = a.d / 4;
  const int64_t half = a.dk_parts ? static_cast<int64_t>(a.B) * a.Hkv * a.T * per : 0;
  int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id < 2 * half) {
    const bool second = id >= half;
    if (second) id -= half;
    const int c = 4 * static_cast<int>(id % per);
    const int64_t row = id / per;
    const int t = static_cast<int>(row % a.T);
    const int hk = static_cast<int>(row / a.T % a.Hkv), b = static_cast<int>(row / a.T / a.Hkv);
    const int64_t head = static_cast<int64_t>(a.T) * a.d;
    const float* p = (second ? a.dv_parts : a.dk_parts) + (static_cast<int64_t>(b) * a.Hkv + hk) * a.group * head +
                     static_cast<int64_t>(t) * a.d + c;
    float4v s = *reinterpret_cast<const float4v*>(p);
    for (int i = 1; i < a.group; ++i) s = s + *reinterpret_cast<const float4v*>(p + i * head);
    const Strides3 os = second ? a.dvs : a.dks;
    store4(static_cast<OT*>(second ? a.dV : a.dK) + b * os.b + hk * os.h + t * os.t + c, s);
    return;
  }
  id -= 2 * half;
  if (!a.dgpart || id >= static_cast<int64_t>(a.B) * a.Hkv * a.group) return;
  double sum = 0.0;
  for (int i = 0; i < a.nseg; ++i) sum += a.dgpart[id * a.nseg + i];
  a.dg[id] = static_cast<float>(sum);
}

template <int D>
hipError_t go(const AttnBwdArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H * a.nseg * 3), block(4 * D);
  const bool qf = a.in_dtype == 0, zf = a.out_dtype == 0;
  if (qf && zf) ttt_attn_bwd<D, float, float, float><<<grid, block, 0, s>>>(a);
  else if (zf) ttt_attn_bwd<D, uint16_t, float, float><<<grid, block, 0, s>>>(a);
  else if (qf && a.parts) ttt_attn_bwd<D, float, uint16_t, float><<<grid, block, 0, s>>>(a);
  else if (qf) ttt_attn_bwd<D, float, uint16_t, uint16_t><<<grid, block, 0, s>>>(a);
  else if (a.parts) ttt_attn_bwd<D, uint16_t, uint16_t, float><<<grid, block, 0, s>>>(a);
  else ttt_attn_bwd<D, uint16_t, uint16_t, uint16_t><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t go_states(const AttnBwdArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H * (a.nseg - 1) * 2), block(4 * D);
  const bool qf = a.in_dtype == 0, zf = a.out_dtype == 0;
  if (qf && zf) ttt_attn_bwd_states<D, float, float><<<grid, block, 0, s>>>(a);
  else if (qf) ttt_attn_bwd_states<D, float, uint16_t><<<grid, block, 0, s>>>(a);
  else if (zf) ttt_attn_bwd_states<D, uint16_t, float><<<grid, block, 0, s>>>(a);
  else ttt_attn_bwd_states<D, uint16_t, uint16_t><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_bwd(const AttnBwdArgs& a, hipStream_t s) {
  switch (a.d) {
    case 16: return attn::go<16>(a, s);
    case 32: return attn::go<32>(a, s);
    case 64: return attn::go<64>(a, s);
    case 128: return attn::go<128>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_attn_bwd_states(const AttnBwdArgs& a, hipStream_t s) {
  switch (a.d) {
    case 16: return attn::go_states<16>(a, s);
    case 32: return attn::go_states<32>(a, s);
    case 64: return attn::go_states<64>(a, s);
    case 128: return attn::go_states<128>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_attn_sum(const AttnSumArgs& a, hipStream_t s) {
  int64_t n = a.dk_parts ? 2 * static_cast<int64_t>(a.B) * a.Hkv * a.T * (a.d / 4) : 0;
  if (a.dgpart) n += static_cast<int64_t>(a.B) * a.Hkv * a.group;
  if (n == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>((n + 255) / 256));
  if (a.out_dtype == 0) attn::ttt_attn_sum<float><<<grid, 256, 0, s>>>(a);
  else attn::ttt_attn_sum<uint16_t><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ttt
