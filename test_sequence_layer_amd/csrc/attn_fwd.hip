// Linear attention with a decay per head, forward, on the CDNA4 matrix cores.
//
// Pages: [TTT] = news article "大模型最强架构TTT问世！斯坦福UCSD等5年磨一剑，一夜推翻Transformer"
// (aharts.cn / itmax.cn), part 03 §8: TTT with a linear f and batch gradient
// descent is linear attention; the state here is laid out as TTT-Linear's.
//
// One workgroup walks a (sequence, head) (attn_walk.h), or one segment of it where
// there are too few to fill the chip: then a first launch walks the segments for
// their end states alone, and each workgroup of the second carries the states of
// the segments before its own over to its first token.
#include "attn_walk.h"

namespace ttt {
namespace attn {
namespace {

// the segment's first token
template <typename T>
__device__ __forceinline__ const T* at(const void* p, const Strides3& s, int b, int h, int64_t t) {
  return static_cast<const T*>(p) + b * s.b + h * s.h + t * s.t;
}

template <int D, typename IT, typename OT>
__global__ __launch_bounds__(4 * D, 2) void ttt_attn_fwd(AttnArgs a) {
  constexpr int NB = D / 16;
  __shared__ __align__(16) uint16_t lds[WalkLds<D, true, false, IT, IT, IT, IT>::kSize];
  __shared__ float powers[15 + C + 1];
  const float* pw = powers + 15;
  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  const int chain = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const int b = chain / a.H, h = chain % a.H, hk = h / a.group;
  const float lg = a.log_decay[h];
  if (tid < 15 + C + 1) powers[tid] = tid < 15 ? 0.f : powl(lg, tid - 15);
  const int len = seq_len(a.lens, b, a.T);
  const int sb = seg * a.seglen, se = min(sb + a.seglen, a.T);  // this segment's rows
  const int n = max(0, min(len, se) - sb);                      // and tokens

  float4v s[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) s[i] = mfma::zero4v();
  if (a.nseg == 1) {
    if (a.W0) load_state<D>(a.W0 + b * a.w0_bstride + static_cast<int64_t>(h) * D * D, false, w, li, g4, s);
  } else {
    const float* loc = a.loc + static_cast<int64_t>(chain) * a.nseg * D * D;
    if (seg == 0) load_state<D>(loc + static_cast<int64_t>(a.nseg - 1) * D * D, false, w, li, g4, s);
    if (n > 0 && a.carried && seg > 0) load_state<D>(loc + static_cast<int64_t>(seg - 1) * D * D, false, w, li, g4, s);
    if (n > 0 && !a.carried && seg > 0)
      carry_states<D>(loc, static_cast<int64_t>(D) * D, seg, SegmentDecay(lg, a.seglen), false, w, li, g4, s);
  }
  __syncthreads();

  OT* z = static_cast<OT*>(a.Z) + b * a.zs.b + h * a.zs.h;
  Walk<IT, IT, IT, IT, OT> walk_args;
  walk_args.x = at<IT>(a.Q, a.qs, b, h, sb);
  walk_args.y = at<IT>(a.K, a.ks, b, hk, sb);
  walk_args.v = at<IT>(a.V, a.vs, b, hk, sb);
  walk_args.q = nullptr;
  walk_args.o = z + sb * a.zs.t;
  walk_args.xt = a.qs.t;
  walk_args.yt = a.ks.t;
  walk_args.vt = a.vs.t;
  walk_args.qt = 0;
  walk_args.ot = a.zs.t;
  walk_args.n = n;
  walk_args.lg = lg;
  walk_args.sp = walk_args.si = a.scale;
  walk_args.su = 1.f;
  double none = 0.0;
  walk<D, true, false>(walk_args, false, lds, pw, s, s, none);

  if (sb + n < se) zero_rows<D>(z, a.zs.t, sb + n, se);
  if (seg == (len > 0 ? (len - 1) / a.seglen : 0))
    store_state<D>(a.W_final + static_cast<int64_t>(chain) * D * D, w, li, g4, s);
}

// The states of segments 0 .. nseg-2 at their ends: the first from W0, the others
// from zero.  The second launch's first segment finds W0 in the last slot, since its
// last one may write W_final over W0 before it starts.
template <int D, typename IT>
__global__ __launch_bounds__(4 * D) void ttt_attn_states(AttnArgs a) {
  constexpr int NB = D / 16;
  __shared__ __align__(16) uint16_t lds[WalkLds<D, false, false, IT, IT, IT, IT>::kSize];
  __shared__ float powers[15 + C + 1];
  const float* pw = powers + 15;
  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  const int chain = blockIdx.x / (a.nseg - 1), seg = blockIdx.x % (a.nseg - 1);
  const int b = chain / a.H, h = chain % a.H, hk = h / a.group;
  const float lg = a.log_decay[h];
  if (tid < 15 + C + 1) powers[tid] = tid < 15 ? 0.f : powl(lg, tid - 15);
  const int len = seq_len(a.lens, b, a.T);
  const int sb = seg * a.seglen;
  float4v s[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) s[i] = mfma::zero4v();
  float* loc = a.loc + static_cast<int64_t>(chain) * a.nseg * D * D;
  if (seg == 0) {
    if (a.W0) load_state<D>(a.W0 + b * a.w0_bstride + static_cast<int64_t>(h) * D * D, false, w, li, g4, s);
    store_state<D>(loc + static_cast<int64_t>(a.nseg - 1) * D * D, w, li, g4, s);
  }
  if (len <= sb + a.seglen) return;  // no segment behind this one has a token
  __syncthreads();
  Walk<IT, IT, IT, IT, IT> walk_args;
  walk_args.x = walk_args.q = nullptr;
  walk_args.o = nullptr;
  walk_args.xt = walk_args.qt = walk_args.ot = 0;
  walk_args.y = at<IT>(a.K, a.ks, b, hk, sb);
  walk_args.v = at<IT>(a.V, a.vs, b, hk, sb);
  walk_args.yt = a.ks.t;
  walk_args.vt = a.vs.t;
  walk_args.n = a.seglen;
  walk_args.lg = lg;
  walk_args.sp = walk_args.si = walk_args.su = 1.f;
  double none = 0.0;
  walk<D, false, false>(walk_args, false, lds, pw, s, s, none);
  store_state<D>(loc + static_cast<int64_t>(seg) * D * D, w, li, g4, s);
}

// Four elements of one chain's states a thread, from segment to segment.
__global__ __launch_bounds__(256) void ttt_attn_carry(AttnCarryArgs a) {
  constexpr int U = 8;  // segments on their way
  const int quads = a.d * a.d / 4;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= a.chains * quads * (a.backward ? 2 : 1)) return;
  const bool grad = id >= a.chains * quads;  // of G^T
  const int64_t at = grad ? id - a.chains * quads : id, chain = at / quads;
  const int64_t dd = static_cast<int64_t>(a.d) * a.d, step = a.backward ? 3 * dd : dd;
  float* p = a.loc + chain * a.nseg * step + 4 * (at % quads) + (grad ? 2 * dd : 0);
  const SegmentDecay e(a.log_decay[chain % a.H], a.seglen);
  const float len = static_cast<float>(a.seglen);
  float4v s = mfma::zero4v(), u = s;
  const bool with_u = a.backward && !grad;
  for (int c = 0; c < a.nseg - 1; c += U) {
    float4v x[U], y[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t k = min(c + i, a.nseg - 2) * step;
      x[i] = *reinterpret_cast<const float4v*>(p + k);
      y[i] = with_u ? *reinterpret_cast<const float4v*>(p + k + dd) : x[i];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (c + i >= a.nseg - 1) break;
      const int64_t k = (c + i) * step;
      u = e.carry(u + s * len, y[i]);
      s = e.carry(s, x[i]);
      *reinterpret_cast<float4v*>(p + k) = s;
      if (with_u) *reinterpret_cast<float4v*>(p + k + dd) = u;
    }
  }
}

template <int D>
hipError_t go(const AttnArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H * a.nseg), block(4 * D);
  const bool in = a.in_dtype == 0, out = a.out_dtype == 0;
  if (in && out) ttt_attn_fwd<D, float, float><<<grid, block, 0, s>>>(a);
  else if (in) ttt_attn_fwd<D, float, uint16_t><<<grid, block, 0, s>>>(a);
  else if (out) ttt_attn_fwd<D, uint16_t, float><<<grid, block, 0, s>>>(a);
  else ttt_attn_fwd<D, uint16_t, uint16_t><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t go_states(const AttnArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H * (a.nseg - 1)), block(4 * D);
  if (a.in_dtype == 0) ttt_attn_states<D, float><<<grid, block, 0, s>>>(a);
  else ttt_attn_states<D, uint16_t><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace
}  // namespace attn

bool attn_supported(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Segments per sequence.  One workgroup walks a chain 32 tokens at a time, so a few chains leave most of the 256
// CUs idle for long; segments fill them, at the price of a first pass over K and V (Q and dZ too in the
// backward), of carrying the states and of a launch.  us at T2048 in bf16, [B, H, T, d]:
//   forward, 8 waves a CU (32768 / d workgroups at most): 96 chains d64 43 (half as many: 65, twice: 56, one
//     segment a chain: 80), 200 chains d128 153 (twice: 200), d32 37 (half: 59, twice: 45), d16 24 (half: 26, a
//     quarter: 50, twice: 29)
//   backward, three walks a segment.  d128, 240 segments: 96 chains 312 (320: 355, 160: 319).  d64, 320: 96 chains 123
//     (160: 134, 640: 140).  d32, 384: 200 chains 101 (640: 112, 200: 101), 96 chains 68 (640: 63, 320: 71).  d16, 640:
//     300 chains 79 (320: 94, 960: 88), 400 chains 102 (960: 117).
// Shortest segment.  wide (fp32 inputs or d = 128): 3 chunks of 32 tokens, from 6 chunks on (12 chains T1009 d128 fp32:
// 40, 4 chunks 45, 6 chunks 55; T200 31 for 33 in one, gradients 70 for 91).  Otherwise 4 chunks, from 12 on
// (T330: in one 17.3, in two 17.5, T512: 16.4 for 23.1 in one; T200 would cost 16 for 12, gradients 26 for 19).  At most
// 64 segments (B1 H1 T32768: 63, 109 with 256).
int attn_segments(int64_t chains, int T, int d, bool wide, bool backward) {
  if (chains <= 0 || T <= 0) return 1;
  const int all = !backward ? 32768 / d : d == 128 ? 240 : d == 64 ? 320 : d == 32 ? 384 : 640;
  const int chunks = (T + kAttnChunk - 1) / kAttnChunk;
  if (chunks < (wide ? 6 : 12)) return 1;
  int64_t most = wide ? (chunks + 2) / 3 : chunks / 4;
  if (most > 64) most = 64;
  const int64_t n = all / chains;
  return n < 1 ? 1 : static_cast<int>(n < most ? n : most);
}

hipError_t launch_attn_states(const AttnArgs& a, hipStream_t s) {
  switch (a.d) {
    case 16: return attn::go_states<16>(a, s);
    case 32: return attn::go_states<32>(a, s);
    case 64: return attn::go_states<64>(a, s);
    case 128: return attn::go_states<128>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_attn_carry(const AttnCarryArgs& a, hipStream_t s) {
  const int64_t n = a.chains * (a.d * a.d / 4) * (a.backward ? 2 : 1);
  attn::ttt_attn_carry<<<dim3(static_cast<unsigned>((n + 255) / 256)), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s) {
  switch (a.d) {
    case 16: return attn::go<16>(a, s);
    case 32: return attn::go<32>(a, s);
    case 64: return attn::go<64>(a, s);
    case 128: return attn::go<128>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ttt
