// Linear attention with a decay per head, forward (and dQ of its backward) on
// the CDNA4 matrix cores.
//
// Pages: [TTT] = news article "大模型最强架构TTT问世！斯坦福UCSD等5年磨一剑，一夜推翻Transformer"
// (aharts.cn / itmax.cn), part 03 §8: TTT with a linear f and batch gradient
// descent is linear attention; the state here is laid out as TTT-Linear's.
//
// With lambda = exp(log_decay) the recurrence S_t = lambda S_{t-1} + v_t y_t^T,
// o_t = scale S_t x_t over a chunk of C = 32 tokens (0-based i, j in the chunk) is
//   O = ((X Y^T) o D) V + diag(lambda^{i+1}) X S^T,   D_ij = lambda^{i-j} (i >= j)
//   S <- lambda^C S + (diag(lambda^{C-1-j}) V)^T Y
// Every power of lambda has an exponent >= 0, so no decay overflows.
//
// One workgroup of d / 16 waves walks a (sequence, head), or one segment of it.
// Wave w owns rows 16w .. 16w+15 of S (as accumulator blocks, for the whole
// walk) and the same 16 output columns, so waves share only the input tiles;
// each computes the three causal 16 x 16 blocks of X Y^T itself, transposed, so
// that they come out in the layout the next product reads (no LDS round trip).
// A chunk's rows are loaded PF chunks ahead into registers (16 bytes a thread
// and tensor for bf16), stored to the other half of a double LDS buffer, and
// one barrier a chunk separates its readers from the next writer.
#include <type_traits>

#include "attn_common.h"

namespace ttt {
namespace attn {
namespace {

constexpr int PF = 2;  // chunks in flight in registers

template <int D, typename XT, typename YT>
struct FwdTypes {
  typedef std::conditional_t<std::is_same<XT, float>::value || std::is_same<YT, float>::value, float, uint16_t> CT;
};

template <int D, typename XT, typename YT, typename OT>
__global__ __launch_bounds__(4 * D) void ttt_attn_fwd(AttnArgs a) {
  typedef typename FwdTypes<D, XT, YT>::CT CT;
  typedef Ops<CT> O;
  typedef typename O::Frag Frag;
  constexpr int NB = D / 16, RS = O::template row_stride<D>();
  constexpr int NP = out_parts<CT, OT>(), NS = state_parts<CT>();
  __shared__ __align__(16) CT xt[2][C * RS], yt[2][C * RS], vt[2][C * RS];

  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  const int chain = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const int b = chain / a.H, h = chain % a.H, hk = h / a.group;
  const float lg = a.log_decay[h];
  const int len = seq_len(a.lens, b, a.T);
  const int sb = seg * a.seglen, se = min(sb + a.seglen, a.T);  // this segment's rows
  const int te = max(sb, min(len, se));                         // end of its tokens
  const int nch = (te - sb + C - 1) / C;
  OT* out = static_cast<OT*>(a.O) + b * a.os.b + h * a.os.h;

  // state at the segment's first token
  float4v s[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) s[i] = mfma::zero4v();
  if (a.nseg == 1) {
    if (a.S0) load_state<D>(a.S0 + b * a.s0_bstride + static_cast<int64_t>(h) * D * D, a.transposed, w, li, g4, s);
  } else {
    const float* loc = a.loc + static_cast<int64_t>(chain) * a.nseg * D * D;
    const float em = powm1(lg, a.seglen);
    if (seg == 0) load_state<D>(loc + static_cast<int64_t>(a.nseg - 1) * D * D, a.transposed, w, li, g4, s);
    for (int c = 0; c < seg && nch > 0; ++c) {
      float4v x[NB];
      load_state<D>(loc + static_cast<int64_t>(c) * D * D, a.transposed, w, li, g4, x);
#pragma unroll
      for (int i = 0; i < NB; ++i) s[i] = decayed(s[i], em) + x[i];
    }
  }

  // this thread's eight elements of a chunk
  const int row = tid / (D / 8), col = 8 * (tid % (D / 8));
  const XT* xp = static_cast<const XT*>(a.X) + b * a.xs.b + h * a.xs.h + (sb + row) * a.xs.t + col;
  const YT* yp = static_cast<const YT*>(a.Y) + b * a.ys.b + hk * a.ys.h + (sb + row) * a.ys.t + col;
  const YT* vp = static_cast<const YT*>(a.V) + b * a.vs.b + hk * a.vs.h + (sb + row) * a.vs.t + col;
  Slab<XT> rx[PF];
  Slab<YT> ry[PF], rv[PF];
  auto fetch = [&](auto U, int n) {
    constexpr int u = decltype(U)::value;
    const bool ok = sb + n * C + row < te;
    const int64_t t = static_cast<int64_t>(n) * C;
    rx[u].load(xp + t * a.xs.t, ok);
    ry[u].load(yp + t * a.ys.t, ok);
    rv[u].load(vp + t * a.vs.t, ok);
  };
  auto stage = [&](auto U, int buf) {
    constexpr int u = decltype(U)::value;
    put_slab(rx[u], &xt[buf][row * RS + col]);
    put_slab(ry[u], &yt[buf][row * RS + col]);
    put_slab(rv[u], &vt[buf][row * RS + col]);
  };

  // decays: D of a diagonal and of the block below it (lane: j = 4g + r, i = li),
  // lambda^{i+1} of the two row blocks, lambda^{C-1-j} of the two value blocks
  float4v dd, dl, vf[2];
  float inter[2];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int j = 4 * g4 + r;
    dd[r] = li >= j ? powl(lg, li - j) : 0.f;
    dl[r] = powl(lg, 16 + li - j);
    vf[0][r] = powl(lg, C - 1 - j);
    vf[1][r] = powl(lg, C - 17 - j);
  }
  inter[0] = powl(lg, li + 1);
  inter[1] = powl(lg, li + 17);
  float em = powm1(lg, C);

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  auto chunk = [&](int buf, int n) {
    const CT *X = xt[buf], *Y = yt[buf], *V = vt[buf];
    const int t0 = sb + n * C;
    const int L = te - t0;
    if (L < C) {  // the last, ragged chunk: its state ends after L tokens
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 4 * g4 + r;
        vf[0][r] = j < L ? powl(lg, L - 1 - j) : 0.f;
        vf[1][r] = j + 16 < L ? powl(lg, L - 17 - j) : 0.f;
      }
      em = powm1(lg, L);
    }
    Frag xf[2][NB], yf[2][NB];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        xf[i][k] = O::template rows<RS>(X, 16 * i, k, li, g4);
        yf[i][k] = O::template rows<RS>(Y, 16 * i, k, li, g4);
      }
    const Frag v0 = O::template cols<RS>(V, 0, 16 * w, li, g4), v1 = O::template cols<RS>(V, 16, 16 * w, li, g4);
    // scores, transposed: block (j, i), lane holds [j = 4g + r][i = li]
    Frag p00[NP], p01[NP], p11[NP];
    float4v z0 = mfma::zero4v(), z1 = mfma::zero4v();
    {
      float4v s00 = dot<CT, NB>(yf[0], xf[0], mfma::zero4v());
      float4v s01 = dot<CT, NB>(yf[0], xf[1], mfma::zero4v());
      float4v s11 = dot<CT, NB>(yf[1], xf[1], mfma::zero4v());
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool seen = li >= 4 * g4 + r;
        s00[r] = seen ? s00[r] * dd[r] : 0.f;
        s01[r] = s01[r] * dl[r];
        s11[r] = seen ? s11[r] * dd[r] : 0.f;
      }
      O::template split<NP>(s00, p00);
      O::template split<NP>(s01, p01);
      O::template split<NP>(s11, p11);
    }
    // O^T = S X^T, decayed, plus V^T P^T
    {
      Frag sp[NB][NP];
#pragma unroll
      for (int k = 0; k < NB; ++k) O::template split<NP>(s[k], sp[k]);
#pragma unroll
      for (int n2 = 0; n2 < NP; ++n2) {
        Frag q[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) q[k] = sp[k][n2];
        z0 = dot<CT, NB>(q, xf[0], z0);
        z1 = dot<CT, NB>(q, xf[1], z1);
      }
    }
    z0 = z0 * inter[0];
    z1 = z1 * inter[1];
    z0 = dot_parts<CT, NP>(v0, p00, z0);
#pragma unroll
    for (int n2 = 0; n2 < NP; ++n2) z1 = O::mm2(v0, v1, p01[n2], p11[n2], z1);
    // S += (decayed V)^T Y
    Frag q0[NS], q1[NS];
    O::template split<NS>(O::widen(v0) * vf[0], q0);
    O::template split<NS>(O::widen(v1) * vf[1], q1);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const Frag y0 = O::template cols<RS>(Y, 0, 16 * k, li, g4), y1 = O::template cols<RS>(Y, 16, 16 * k, li, g4);
      float4v x = decayed(s[k], em);
#pragma unroll
      for (int n2 = 0; n2 < NS; ++n2) x = O::mm2(y0, y1, q0[n2], q1[n2], x);
      s[k] = x;
    }
    OT* o = out + 16 * w + 4 * g4;
    if (li < L) store4(o + (t0 + li) * a.os.t, z0 * a.scale);
    if (16 + li < L) store4(o + (t0 + 16 + li) * a.os.t, z1 * a.scale);
  };

  if (nch > 0) {
    fetch(I0{}, 0);
    fetch(I1{}, 1);
    stage(I0{}, 0);
    fetch(I0{}, 2);
    __syncthreads();
    for (int n = 0; n < nch; n += 2) {
      stage(I1{}, 1);
      fetch(I1{}, n + 3);
      chunk(0, n);
      __syncthreads();
      if (n + 1 >= nch) break;
      stage(I0{}, 0);
      fetch(I0{}, n + 4);
      chunk(1, n + 1);
      __syncthreads();
    }
  }

  if (te < se) zero_rows<D>(out, a.os.t, te, se);
  if (a.S_final && seg == (len > 0 ? (len - 1) / a.seglen : 0))
    store_state<D>(a.S_final + static_cast<int64_t>(chain) * D * D, w, li, g4, s);
}

// The states of segments 0 .. nseg-2 at their ends: the first from S0, the others
// from zero (the walk's update alone).  The walk's own first segment finds S0 in
// the last slot, since its last one may write S_final over S0 before it starts.
template <int D, typename YT>
__global__ __launch_bounds__(4 * D) void ttt_attn_states(AttnArgs a) {
  typedef YT CT;
  typedef Ops<CT> O;
  typedef typename O::Frag Frag;
  constexpr int NB = D / 16, RS = O::template row_stride<D>(), NS = state_parts<CT>();
  __shared__ __align__(16) CT yt[2][C * RS], vt[2][C * RS];
  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  const int chain = blockIdx.x / (a.nseg - 1), seg = blockIdx.x % (a.nseg - 1);
  const int b = chain / a.H, h = chain % a.H, hk = h / a.group;
  const float lg = a.log_decay[h];
  const int len = seq_len(a.lens, b, a.T);
  const int sb = seg * a.seglen, te = sb + a.seglen;
  float4v s[NB], vf[2];
#pragma unroll
  for (int i = 0; i < NB; ++i) s[i] = mfma::zero4v();
  if (seg == 0) {
    if (a.S0) load_state<D>(a.S0 + b * a.s0_bstride + static_cast<int64_t>(h) * D * D, false, w, li, g4, s);
    store_state<D>(a.loc + (static_cast<int64_t>(chain) * a.nseg + a.nseg - 1) * D * D, w, li, g4, s);
  }
  if (len <= te) return;  // no segment behind this one has a token
  const int nch = a.seglen / C;
  const int row = tid / (D / 8), col = 8 * (tid % (D / 8));
  const YT* yp = static_cast<const YT*>(a.Y) + b * a.ys.b + hk * a.ys.h + (sb + row) * a.ys.t + col;
  const YT* vp = static_cast<const YT*>(a.V) + b * a.vs.b + hk * a.vs.h + (sb + row) * a.vs.t + col;
  Slab<YT> ry[PF], rv[PF];
  auto fetch = [&](auto U, int n) {
    constexpr int u = decltype(U)::value;
    const int64_t t = static_cast<int64_t>(n) * C;
    ry[u].load(yp + t * a.ys.t, n < nch);
    rv[u].load(vp + t * a.vs.t, n < nch);
  };
  auto stage = [&](auto U, int buf) {
    constexpr int u = decltype(U)::value;
    put_slab(ry[u], &yt[buf][row * RS + col]);
    put_slab(rv[u], &vt[buf][row * RS + col]);
  };
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    vf[0][r] = powl(lg, C - 1 - 4 * g4 - r);
    vf[1][r] = powl(lg, C - 17 - 4 * g4 - r);
  }
  const float em = powm1(lg, C);
  auto chunk = [&](int buf) {
    const CT *Y = yt[buf], *V = vt[buf];
    Frag q0[NS], q1[NS];
    O::template split<NS>(O::widen(O::template cols<RS>(V, 0, 16 * w, li, g4)) * vf[0], q0);
    O::template split<NS>(O::widen(O::template cols<RS>(V, 16, 16 * w, li, g4)) * vf[1], q1);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const Frag y0 = O::template cols<RS>(Y, 0, 16 * k, li, g4), y1 = O::template cols<RS>(Y, 16, 16 * k, li, g4);
      float4v x = decayed(s[k], em);
#pragma unroll
      for (int n2 = 0; n2 < NS; ++n2) x = O::mm2(y0, y1, q0[n2], q1[n2], x);
      s[k] = x;
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  fetch(I0{}, 0);
  fetch(I1{}, 1);
  stage(I0{}, 0);
  fetch(I0{}, 2);
  __syncthreads();
  for (int n = 0; n < nch; n += 2) {
    stage(I1{}, 1);
    fetch(I1{}, n + 3);
    chunk(0);
    __syncthreads();
    if (n + 1 >= nch) break;
    stage(I0{}, 0);
    fetch(I0{}, n + 4);
    chunk(1);
    __syncthreads();
  }
  store_state<D>(a.loc + (static_cast<int64_t>(chain) * a.nseg + seg) * D * D, w, li, g4, s);
}

template <int D>
hipError_t go(const AttnArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H * a.nseg), block(4 * D);
  const bool xf = a.x_dtype == 0, yf = a.in_dtype == 0, of = a.out_dtype == 0;
  if (!xf && !yf && !of) ttt_attn_fwd<D, uint16_t, uint16_t, uint16_t><<<grid, block, 0, s>>>(a);
  else if (!xf && !yf) ttt_attn_fwd<D, uint16_t, uint16_t, float><<<grid, block, 0, s>>>(a);
  else if (xf && yf && of) ttt_attn_fwd<D, float, float, float><<<grid, block, 0, s>>>(a);
  else if (xf && yf) ttt_attn_fwd<D, float, float, uint16_t><<<grid, block, 0, s>>>(a);
  else if (xf && of) ttt_attn_fwd<D, float, uint16_t, float><<<grid, block, 0, s>>>(a);
  else if (!xf && !of) ttt_attn_fwd<D, uint16_t, float, uint16_t><<<grid, block, 0, s>>>(a);
  else return hipErrorInvalidValue;
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

// Segments per sequence: as many as it takes for about three workgroups per CU
// (256 CUs), none shorter than 128 tokens.
int attn_segments(int64_t chains, int T, int d) {
  (void)d;
  if (chains <= 0 || T <= 0) return 1;
  int64_t n = (768 + chains - 1) / chains;
  const int64_t most = T / 128;
  if (chains >= 384) n = 1;
  if (n > most) n = most;
  return n < 1 ? 1 : static_cast<int>(n);
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
