// Linear attention with a decay per head: the part of the backward that runs from
// the last token to the first (dK, dV, the decay's and the initial state's
// gradient) on the CDNA4 matrix cores.  dQ is the forward walk with dZ, V, K in
// the places of Q, K, V and W^T for the state.
//
// With G_t the gradient of the state after token t (lambda = exp(log_decay)),
//   G_t = scale dZ_t Q_t^T + lambda G_{t+1},   dV_t = G_t K_t,   dK_t = G_t^T V_t
// and over a chunk of L <= 32 tokens, G the gradient of the state at its end:
//   dV = diag(lambda^{L-1-j}) K G^T + scale ((Q K^T) o D)^T dZ,   D_ij = lambda^{i-j} (i >= j)
//   dK = diag(lambda^{L-1-j}) V G   + scale ((dZ V^T) o D)^T Q
//   G <- lambda^L G + scale (diag(lambda^{i+1}) dZ)^T Q
// The decay's gradient counts every pair j <= i by its distance:
//   dg = sum_{j <= i} (i - j) lambda^{i-j} scale (Q_i.K_j)(dZ_i.V_j)   + initial and final state
// Pairs within a chunk come from the two score blocks at hand.  For pairs across
// its end a second state carries the distances, H = dG/dlog_decay:
//   H <- lambda^L (H + L G) + scale (diag((i+1) lambda^{i+1}) dZ)^T Q
//   dg += sum_j lambda^{L-1-j} V_j . ((H + (L-1-j) G) K_j)
// so that every term is added once, with its own sign and weight; the shorter
// form sum_t t (dQ_t.Q_t - dK_t.K_t) subtracts sums T / distance times larger.
//
// One workgroup of d / 16 waves walks a (sequence, head), or a segment of it, as
// in the forward.  Wave w owns rows 16w .. of G and H (for dV and dg) and columns
// 16w .. of G (for dK), all as accumulator blocks: G is kept and updated twice
// rather than transposed through LDS in every chunk.
#include <type_traits>

#include "attn_common.h"

namespace ttt {
namespace attn {
namespace {

// sum over the lanes of a wave, the same in every run
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

template <int D, typename QT, typename ZT, typename OT>
__global__ __launch_bounds__(4 * D) void ttt_attn_bwd(AttnBwdArgs a) {
  typedef std::conditional_t<std::is_same<QT, float>::value || std::is_same<ZT, float>::value, float, uint16_t> CT;
  typedef Ops<CT> O;
  typedef typename O::Frag Frag;
  constexpr int NB = D / 16, RS = O::template row_stride<D>();
  constexpr int NP = out_parts<CT, ZT>(), NS = state_parts<CT>();
  constexpr int PF = sizeof(CT) == 2 ? 2 : 1;  // chunks in flight in registers
  __shared__ __align__(16) CT qt[2][C * RS], kt[2][C * RS], vt[2][C * RS], zt[2][C * RS];
  __shared__ double part[NB];

  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  const int chain = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const int b = chain / a.H, h = chain % a.H, hk = h / a.group;
  const float lg = a.log_decay[h];
  const int len = seq_len(a.lens, b, a.T);
  const int sb = seg * a.seglen, se = min(sb + a.seglen, a.T);
  const int te = max(sb, min(len, se));
  const int nch = (te - sb + C - 1) / C;
  const int ho = a.parts ? h : hk;
  OT* dk = static_cast<OT*>(a.dK) + b * a.dks.b + ho * a.dks.h;
  OT* dv = static_cast<OT*>(a.dV) + b * a.dvs.b + ho * a.dvs.h;

  // gradient of the state at the segment's end: rows of G and H, columns of G
  float4v gr[NB], hr[NB], gc[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) gr[i] = hr[i] = gc[i] = mfma::zero4v();
  if (a.dWf) {
    const float* p = a.dWf + static_cast<int64_t>(chain) * D * D;
    load_state<D>(p, false, w, li, g4, gr);
    load_state<D>(p, true, w, li, g4, gc);
  }
  for (int c = len > 0 ? (len - 1) / a.seglen : 0; c > seg; --c) {
    const int L = min(len - c * a.seglen, a.seglen);
    const float em = powm1(lg, L);
    const float* p = a.gloc + (static_cast<int64_t>(chain) * a.nseg + c) * 2 * D * D;
    float4v x[NB], y[NB];
    load_state<D>(p, true, w, li, g4, x);
#pragma unroll
    for (int i = 0; i < NB; ++i) gc[i] = decayed(gc[i], em) + x[i];
    load_state<D>(p, false, w, li, g4, x);
    load_state<D>(p + D * D, false, w, li, g4, y);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      hr[i] = decayed(hr[i] + gr[i] * static_cast<float>(L), em) + y[i];
      gr[i] = decayed(gr[i], em) + x[i];
    }
  }

  const int row = tid / (D / 8), col = 8 * (tid % (D / 8));
  const QT* qp = static_cast<const QT*>(a.Q) + b * a.qs.b + h * a.qs.h + (sb + row) * a.qs.t + col;
  const QT* kp = static_cast<const QT*>(a.K) + b * a.ks.b + hk * a.ks.h + (sb + row) * a.ks.t + col;
  const QT* vp = static_cast<const QT*>(a.V) + b * a.vs.b + hk * a.vs.h + (sb + row) * a.vs.t + col;
  const ZT* zp = static_cast<const ZT*>(a.dZ) + b * a.zs.b + h * a.zs.h + (sb + row) * a.zs.t + col;
  Slab<QT> rq[PF], rk[PF], rv[PF];
  Slab<ZT> rz[PF];
  auto fetch = [&](auto U, int n) {  // chunk n, none for n < 0
    constexpr int u = decltype(U)::value % PF;
    const bool ok = n >= 0 && sb + n * C + row < te;
    const int64_t t = static_cast<int64_t>(n) * C;
    rq[u].load(qp + t * a.qs.t, ok);
    rk[u].load(kp + t * a.ks.t, ok);
    rv[u].load(vp + t * a.vs.t, ok);
    rz[u].load(zp + t * a.zs.t, ok);
  };
  auto stage = [&](auto U, int buf) {
    constexpr int u = decltype(U)::value % PF;
    put_slab(rq[u], &qt[buf][row * RS + col]);
    put_slab(rk[u], &kt[buf][row * RS + col]);
    put_slab(rv[u], &vt[buf][row * RS + col]);
    put_slab(rz[u], &zt[buf][row * RS + col]);
  };

  // scale lambda^{i-j} of a diagonal block and the block below it (lane: i = 4g + r,
  // j = li), and the update's scale lambda^{i+1}
  float4v dd, dl, up[2];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = 4 * g4 + r;
    dd[r] = i >= li ? a.scale * powl(lg, i - li) : 0.f;
    dl[r] = a.scale * powl(lg, 16 + i - li);
    up[0][r] = a.scale * powl(lg, i + 1);
    up[1][r] = a.scale * powl(lg, i + 17);
  }
  double dg = 0.0;

  auto chunk = [&](int buf, int n) {
    const CT *Q = qt[buf], *K = kt[buf], *V = vt[buf], *Z = zt[buf];
    const int t0 = sb + n * C;
    const int L = min(C, te - t0);
    const int left[2] = {L - 1 - li, L - 17 - li};  // tokens of this chunk behind j
    float dgc = 0.f;
    // score blocks (i, j): lane holds [i = 4g + r][j = li]
    Frag pk[3][NP], pv[3][NP];  // (0,0), (1,0), (1,1) of scale (Q K^T) o D and scale (dZ V^T) o D
    {
      Frag x[2][NB], y[2][NB];
      float4v sk[3], sv[3];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          x[i][k] = O::template rows<RS>(Q, 16 * i, k, li, g4);
          y[i][k] = O::template rows<RS>(K, 16 * i, k, li, g4);
        }
      sk[0] = dot<CT, NB>(x[0], y[0], mfma::zero4v());
      sk[1] = dot<CT, NB>(x[1], y[0], mfma::zero4v());
      sk[2] = dot<CT, NB>(x[1], y[1], mfma::zero4v());
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          x[i][k] = O::template rows<RS>(Z, 16 * i, k, li, g4);
          y[i][k] = O::template rows<RS>(V, 16 * i, k, li, g4);
        }
      sv[0] = dot<CT, NB>(x[0], y[0], mfma::zero4v());
      sv[1] = dot<CT, NB>(x[1], y[0], mfma::zero4v());
      sv[2] = dot<CT, NB>(x[1], y[1], mfma::zero4v());
      if (w == 0) {  // pairs within the chunk, counted by one wave
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float dist = static_cast<float>(4 * g4 + r - li);
          dgc += dist > 0.f ? dist * dd[r] * (sk[0][r] * sv[0][r] + sk[2][r] * sv[2][r]) : 0.f;
          dgc += (16.f + dist) * dl[r] * (sk[1][r] * sv[1][r]);
        }
      }
#pragma unroll
      for (int t = 0; t < 3; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool seen = t == 1 || 4 * g4 + r >= li;
          const float f = t == 1 ? dl[r] : dd[r];
          sk[t][r] = seen ? sk[t][r] * f : 0.f;
          sv[t][r] = seen ? sv[t][r] * f : 0.f;
        }
        O::template split<NP>(sk[t], pk[t]);
        O::template split<NP>(sv[t], pv[t]);
      }
    }
    const Frag z0 = O::template cols<RS>(Z, 0, 16 * w, li, g4), z1 = O::template cols<RS>(Z, 16, 16 * w, li, g4);
    const Frag q0 = O::template cols<RS>(Q, 0, 16 * w, li, g4), q1 = O::template cols<RS>(Q, 16, 16 * w, li, g4);
    float far[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) far[j] = left[j] >= 0 ? powl(lg, left[j]) : 0.f;

    // dV^T = G K^T, decayed, plus dZ^T (Q K^T o D); dg's pairs across the chunk's end
    {
      Frag sp[NB][NP];
      float4v o[2], hk2[2];
      o[0] = o[1] = hk2[0] = hk2[1] = mfma::zero4v();
      Frag y[2][NB];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < NB; ++k) y[j][k] = O::template rows<RS>(K, 16 * j, k, li, g4);
#pragma unroll
      for (int k = 0; k < NB; ++k) O::template split<NP>(gr[k], sp[k]);
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        Frag s[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) s[k] = sp[k][m];
#pragma unroll
        for (int j = 0; j < 2; ++j) o[j] = dot<CT, NB>(s, y[j], o[j]);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) O::template split<NP>(hr[k], sp[k]);
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        Frag s[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) s[k] = sp[k][m];
#pragma unroll
        for (int j = 0; j < 2; ++j) hk2[j] = dot<CT, NB>(s, y[j], hk2[j]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4v vv = O::widen(O::template rows<RS>(V, 16 * j, w, li, g4));
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) t = fmaf(vv[r], fmaf(static_cast<float>(left[j]), o[j][r], hk2[j][r]), t);
        dgc += left[j] >= 0 ? far[j] * t : 0.f;
        o[j] = o[j] * far[j];
      }
#pragma unroll
      for (int m = 0; m < NP; ++m) o[0] = O::mm2(z0, z1, pk[0][m], pk[1][m], o[0]);
      o[1] = dot_parts<CT, NP>(z1, pk[2], o[1]);
      OT* p = dv + 16 * w + 4 * g4;
      if (left[0] >= 0) store4(p + (t0 + li) * a.dvs.t, o[0]);
      if (left[1] >= 0) store4(p + (t0 + 16 + li) * a.dvs.t, o[1]);
    }
    // dK^T = G^T V^T, decayed, plus Q^T (dZ V^T o D)
    {
      Frag sp[NB][NP];
      float4v o[2];
      o[0] = o[1] = mfma::zero4v();
      Frag y[2][NB];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < NB; ++k) y[j][k] = O::template rows<RS>(V, 16 * j, k, li, g4);
#pragma unroll
      for (int k = 0; k < NB; ++k) O::template split<NP>(gc[k], sp[k]);
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        Frag s[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) s[k] = sp[k][m];
#pragma unroll
        for (int j = 0; j < 2; ++j) o[j] = dot<CT, NB>(s, y[j], o[j]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) o[j] = o[j] * far[j];
#pragma unroll
      for (int m = 0; m < NP; ++m) o[0] = O::mm2(q0, q1, pv[0][m], pv[1][m], o[0]);
      o[1] = dot_parts<CT, NP>(q1, pv[2], o[1]);
      OT* p = dk + 16 * w + 4 * g4;
      if (left[0] >= 0) store4(p + (t0 + li) * a.dks.t, o[0]);
      if (left[1] >= 0) store4(p + (t0 + 16 + li) * a.dks.t, o[1]);
    }
    // the states at the chunk's first token
    {
      const float em = powm1(lg, L);
      Frag u0[NS], u1[NS], d0[NS], d1[NS], c0[NS], c1[NS];
      const float4v zu0 = O::widen(z0) * up[0], zu1 = O::widen(z1) * up[1];
      float4v zd0, zd1;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        zd0[r] = zu0[r] * static_cast<float>(4 * g4 + r + 1);
        zd1[r] = zu1[r] * static_cast<float>(4 * g4 + r + 17);
      }
      O::template split<NS>(zu0, u0);
      O::template split<NS>(zu1, u1);
      O::template split<NS>(zd0, d0);
      O::template split<NS>(zd1, d1);
      O::template split<NS>(O::widen(q0) * up[0], c0);
      O::template split<NS>(O::widen(q1) * up[1], c1);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const Frag y0 = O::template cols<RS>(Q, 0, 16 * k, li, g4), y1 = O::template cols<RS>(Q, 16, 16 * k, li, g4);
        float4v x = decayed(hr[k] + gr[k] * static_cast<float>(L), em);
        float4v y = decayed(gr[k], em);
#pragma unroll
        for (int m = 0; m < NS; ++m) {
          x = O::mm2(y0, y1, d0[m], d1[m], x);
          y = O::mm2(y0, y1, u0[m], u1[m], y);
        }
        hr[k] = x;
        gr[k] = y;
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const Frag y0 = O::template cols<RS>(Z, 0, 16 * k, li, g4), y1 = O::template cols<RS>(Z, 16, 16 * k, li, g4);
        float4v x = decayed(gc[k], em);
#pragma unroll
        for (int m = 0; m < NS; ++m) x = O::mm2(y0, y1, c0[m], c1[m], x);
        gc[k] = x;
      }
    }
    dg += static_cast<double>(dgc);
  };

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  if (nch > 0) {
    const int last = nch - 1;
    if constexpr (PF == 2) {
      fetch(I0{}, last);
      fetch(I1{}, last - 1);
      stage(I0{}, 0);
      fetch(I0{}, last - 2);
    } else {
      fetch(I0{}, last);
      stage(I0{}, 0);
      fetch(I0{}, last - 1);
    }
    __syncthreads();
    for (int n = last; n >= 0; n -= 2) {
      stage(I1{}, 1);
      fetch(I1{}, n - 1 - PF);
      chunk(0, n);
      __syncthreads();
      if (n - 1 < 0) break;
      stage(I0{}, 0);
      fetch(I0{}, n - 2 - PF);
      chunk(1, n - 1);
      __syncthreads();
    }
  }

  if (te < se) {
    zero_rows<D>(dk, a.dks.t, te, se);
    zero_rows<D>(dv, a.dvs.t, te, se);
  }
  if (seg == 0) {
    store_state<D>(a.dW0 + static_cast<int64_t>(chain) * D * D, w, li, g4, gr);
    if (a.W0) {
      float4v x[NB];
      load_state<D>(a.W0 + b * a.w0_bstride + static_cast<int64_t>(h) * D * D, false, w, li, g4, x);
#pragma unroll
      for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) dg += static_cast<double>(x[k][r]) * static_cast<double>(hr[k][r]);
    }
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
}

// G and H that segments 1 .. nseg-1 add from zero, at their first tokens.
template <int D, typename QT, typename ZT>
__global__ __launch_bounds__(4 * D) void ttt_attn_bwd_states(AttnBwdArgs a) {
  typedef std::conditional_t<std::is_same<QT, float>::value || std::is_same<ZT, float>::value, float, uint16_t> CT;
  typedef Ops<CT> O;
  typedef typename O::Frag Frag;
  constexpr int NB = D / 16, RS = O::template row_stride<D>(), NS = state_parts<CT>();
  __shared__ __align__(16) CT qt[2][C * RS], zt[2][C * RS];
  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  const int chain = blockIdx.x / (a.nseg - 1), seg = 1 + blockIdx.x % (a.nseg - 1);
  const int b = chain / a.H, h = chain % a.H;
  const float lg = a.log_decay[h];
  const int len = seq_len(a.lens, b, a.T);
  const int sb = seg * a.seglen, te = min(sb + a.seglen, len);
  if (te <= sb) return;  // nobody reads it
  const int nch = (te - sb + C - 1) / C;
  const int row = tid / (D / 8), col = 8 * (tid % (D / 8));
  const QT* qp = static_cast<const QT*>(a.Q) + b * a.qs.b + h * a.qs.h + (sb + row) * a.qs.t + col;
  const ZT* zp = static_cast<const ZT*>(a.dZ) + b * a.zs.b + h * a.zs.h + (sb + row) * a.zs.t + col;
  Slab<QT> rq[2];
  Slab<ZT> rz[2];
  auto fetch = [&](auto U, int n) {
    constexpr int u = decltype(U)::value;
    const bool ok = n >= 0 && sb + n * C + row < te;
    const int64_t t = static_cast<int64_t>(n) * C;
    rq[u].load(qp + t * a.qs.t, ok);
    rz[u].load(zp + t * a.zs.t, ok);
  };
  auto stage = [&](auto U, int buf) {
    constexpr int u = decltype(U)::value;
    put_slab(rq[u], &qt[buf][row * RS + col]);
    put_slab(rz[u], &zt[buf][row * RS + col]);
  };
  float4v up[2], gr[NB], hr[NB];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    up[0][r] = a.scale * powl(lg, 4 * g4 + r + 1);
    up[1][r] = a.scale * powl(lg, 4 * g4 + r + 17);
  }
#pragma unroll
  for (int k = 0; k < NB; ++k) gr[k] = hr[k] = mfma::zero4v();
  auto chunk = [&](int buf, int n) {
    const CT *Q = qt[buf], *Z = zt[buf];
    const int L = min(C, te - sb - n * C);
    const float em = powm1(lg, L);
    const float4v zu0 = O::widen(O::template cols<RS>(Z, 0, 16 * w, li, g4)) * up[0];
    const float4v zu1 = O::widen(O::template cols<RS>(Z, 16, 16 * w, li, g4)) * up[1];
    float4v zd0, zd1;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      zd0[r] = zu0[r] * static_cast<float>(4 * g4 + r + 1);
      zd1[r] = zu1[r] * static_cast<float>(4 * g4 + r + 17);
    }
    Frag u0[NS], u1[NS], d0[NS], d1[NS];
    O::template split<NS>(zu0, u0);
    O::template split<NS>(zu1, u1);
    O::template split<NS>(zd0, d0);
    O::template split<NS>(zd1, d1);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const Frag y0 = O::template cols<RS>(Q, 0, 16 * k, li, g4), y1 = O::template cols<RS>(Q, 16, 16 * k, li, g4);
      float4v x = decayed(hr[k] + gr[k] * static_cast<float>(L), em);
      float4v y = decayed(gr[k], em);
#pragma unroll
      for (int m = 0; m < NS; ++m) {
        x = O::mm2(y0, y1, d0[m], d1[m], x);
        y = O::mm2(y0, y1, u0[m], u1[m], y);
      }
      hr[k] = x;
      gr[k] = y;
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  const int last = nch - 1;
  fetch(I0{}, last);
  fetch(I1{}, last - 1);
  stage(I0{}, 0);
  fetch(I0{}, last - 2);
  __syncthreads();
  for (int n = last; n >= 0; n -= 2) {
    stage(I1{}, 1);
    fetch(I1{}, n - 3);
    chunk(0, n);
    __syncthreads();
    if (n - 1 < 0) break;
    stage(I0{}, 0);
    fetch(I0{}, n - 4);
    chunk(1, n - 1);
    __syncthreads();
  }
  float* p = a.gloc + (static_cast<int64_t>(chain) * a.nseg + seg) * 2 * D * D;
  store_state<D>(p, w, li, g4, gr);
  store_state<D>(p + D * D, w, li, g4, hr);
}

// The decay's gradient of a (sequence, head): its segments' sums, in order.
__global__ __launch_bounds__(256) void ttt_attn_bwd_dg(const double* part, float* dg, int64_t chains, int nseg) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= chains) return;
  double sum = 0.0;
  for (int i = 0; i < nseg; ++i) sum += part[c * nseg + i];
  dg[c] = static_cast<float>(sum);
}

// Four elements a thread: the parts of a shared head's query heads, in order.
template <typename OT>
__global__ __launch_bounds__(256) void ttt_attn_sum(AttnSumArgs a) {
  const int per = a.d / 4;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= static_cast<int64_t>(a.B) * a.Hkv * a.T * per) return;
  const int c = 4 * static_cast<int>(id % per);
  const int64_t row = id / per;
  const int t = static_cast<int>(row % a.T);
  const int hk = static_cast<int>(row / a.T % a.Hkv), b = static_cast<int>(row / a.T / a.Hkv);
  const int64_t head = static_cast<int64_t>(a.T) * a.d;
  const float* p = a.parts + (static_cast<int64_t>(b) * a.Hkv + hk) * a.group * head + static_cast<int64_t>(t) * a.d + c;
  float4v s = *reinterpret_cast<const float4v*>(p);
  for (int i = 1; i < a.group; ++i) s = s + *reinterpret_cast<const float4v*>(p + i * head);
  store4(static_cast<OT*>(a.out) + b * a.os.b + hk * a.os.h + t * a.os.t + c, s);
}

template <int D>
hipError_t go(const AttnBwdArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H * a.nseg), block(4 * D);
  const bool qf = a.in_dtype == 0, zf = a.out_dtype == 0;
  if (qf && zf) ttt_attn_bwd<D, float, float, float><<<grid, block, 0, s>>>(a);
  else if (!qf && zf) ttt_attn_bwd<D, uint16_t, float, float><<<grid, block, 0, s>>>(a);
  else if (qf && a.parts) ttt_attn_bwd<D, float, uint16_t, float><<<grid, block, 0, s>>>(a);
  else if (qf) ttt_attn_bwd<D, float, uint16_t, uint16_t><<<grid, block, 0, s>>>(a);
  else if (a.parts) ttt_attn_bwd<D, uint16_t, uint16_t, float><<<grid, block, 0, s>>>(a);
  else ttt_attn_bwd<D, uint16_t, uint16_t, uint16_t><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

template <int D>
hipError_t go_states(const AttnBwdArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H * (a.nseg - 1)), block(4 * D);
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

hipError_t launch_attn_bwd_dg(const AttnBwdArgs& a, hipStream_t s) {
  const int64_t chains = static_cast<int64_t>(a.B) * a.H;
  attn::ttt_attn_bwd_dg<<<dim3(static_cast<unsigned>((chains + 255) / 256)), 256, 0, s>>>(a.dgpart, a.dg, chains, a.nseg);
  return hipGetLastError();
}

hipError_t launch_attn_sum(const AttnSumArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.B) * a.Hkv * a.T * (a.d / 4);
  const dim3 grid(static_cast<unsigned>((n + 255) / 256));
  if (a.out_dtype == 0) attn::ttt_attn_sum<float><<<grid, 256, 0, s>>>(a);
  else attn::ttt_attn_sum<uint16_t><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ttt
