// The walk over the tokens of one (sequence, head), or of a segment of it, that
// every linear-attention pass is:
//   S_i = lambda S_{i-1} + V_i Y_i^T,   O_i = sp (own and earlier tokens) + si (start state)
// in chunks of C = 32 tokens (0-based i, j in the chunk, S the state before it)
//   O = sp ((X Y^T) o D) V + si diag(lambda^{i+1}) X S^T,   D_ij = lambda^{i-j} (i >= j)
//   S <- lambda^C S + su (diag(lambda^{C-1-j}) V)^T Y
// Every power of lambda has an exponent >= 0, so no decay overflows.
//   Z  : X, Y, V = Q, K, V        S = W
//   dQ : X, Y, V = dZ, V, K       S = W^T
//   dK : X, Y, V = V, dZ, Q       S = G^T, from the last token to the first
//   dV : X, Y, V = K, Q, dZ       S = G, from the last token to the first
// with G the gradient of the state.  A reversed walk has negative token strides.  Its
// start state, the last state's gradient, is not decayed before its first token:
// `fresh` says so, and the first chunk takes lambda^i and lambda^{C-1} for it.
//
// One workgroup of d / 16 waves.  Wave w owns rows 16w .. 16w+15 of S (as
// accumulator blocks, for the whole walk) and the same 16 output columns, so waves
// share only the input tiles; each computes the three causal 16 x 16 blocks of
// X Y^T itself, transposed, so that they come out in the layout the next product
// reads, with no LDS round trip and no second barrier.  A chunk's rows are loaded
// ahead into registers (16 bytes a thread and tensor for bf16) and stored to LDS.
//
// The decay's gradient (with dQ): a second state U = dS/dlog_decay counts each pair
// j <= i by its distance,
//   U <- lambda^C (U + C S) + (diag((C-1-j) lambda^{C-1-j}) V)^T Y
//   dg += sum_{i >= j in the chunk} (i - j) lambda^{i-j} scale (Q_i.K_j)(dZ_i.V_j)
//       + sum_i lambda^{i+1} scale Q_i . ((U + (i+1) S) dZ_i)
// so that every term is added once, with its own weight; the shorter form
// sum_t t (dQ_t.Q_t - dK_t.K_t) subtracts sums T / distance times larger.
#pragma once

#include <type_traits>

#include "attn_common.h"

namespace ttt {
namespace attn {

template <typename XT, typename YT, typename VT, typename QT, typename OT>
struct Walk {
  // first token of the segment, elements to the next
  const XT* x;
  const YT* y;
  const VT* v;
  const QT* q;  // with the decay's gradient
  OT* o;
  int64_t xt, yt, vt, qt, ot;
  int n;             // tokens
  float lg;          // log(lambda)
  float sp, si, su;  // factors of scores, start state and update
};

// LDS of a walk: tiles of X (with outputs), Y, V and Q (with the decay's gradient), once or twice
template <int D, bool OUT, bool DG, typename XT, typename YT, typename VT, typename QT>
struct WalkLds {
  static constexpr int kX = OUT ? Tile<D, parts_of<XT>()>::kSize : 0;
  static constexpr int kY = Tile<D, parts_of<YT>()>::kSize;
  static constexpr int kV = Tile<D, parts_of<VT>()>::kSize;
  static constexpr int kQ = DG && OUT ? Tile<D, parts_of<QT>()>::kSize : 0;
  static constexpr int kChunk = kX + kY + kV + kQ;
  // bf16: two halves, so that one barrier a chunk separates readers and writers.  fp32 tiles are three
  // planes: one half and two barriers leave room for two workgroups a CU, two halves for one.
  static constexpr int kHalves = sizeof(XT) + sizeof(YT) + sizeof(VT) == 6 ? 2 : 1;
  static constexpr int kSize = kHalves * kChunk;
};

// s: the state before the first token, on return after the last; u likewise dS/dlog_decay.  pw: lambda^0 ..
// lambda^C in LDS.  dg: this lane's share of the decay's gradient.
template <int D, bool OUT, bool DG, typename XT, typename YT, typename VT, typename QT, typename OT>
__device__ __forceinline__ void walk(const Walk<XT, YT, VT, QT, OT>& a, bool fresh, uint16_t* lds, const float* pw,
                                     float4v s[D / 16], float4v u[D / 16], double& dg) {
  typedef WalkLds<D, OUT, DG, XT, YT, VT, QT> Lds;
  constexpr int NB = D / 16, NX = parts_of<XT>(), NY = parts_of<YT>(), NV = parts_of<VT>(), NQ = parts_of<QT>();
  typedef Tile<D, NX> TX;
  typedef Tile<D, NY> TY;
  typedef Tile<D, NV> TV;
  typedef Tile<D, NQ> TQ;
  constexpr int RS = TX::RS, kPlane = TX::kPlane;
  constexpr int LO = DG ? 3 : level_of<OT>(), NP = LO;  // level of outputs, parts of scores and of the state for them
  constexpr bool two = Lds::kHalves == 2;

  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  const int nfull = a.n / C, nch = (a.n + C - 1) / C;
  if (nch == 0) return;

  const int row = tid / (D / 8), col = 8 * (tid % (D / 8));
  const XT* xp = a.x + row * a.xt + col;
  const YT* yp = a.y + row * a.yt + col;
  const VT* vp = a.v + row * a.vt + col;
  const QT* qp = a.q + row * a.qt + col;
  struct Ring {
    Slab<XT> x;
    Slab<YT> y;
    Slab<VT> v;
    Slab<QT> q;
  };
  auto fetch = [&](Ring& r, int n) __attribute__((always_inline)) {
    const bool ok = n * C + row < a.n;
    const int64_t t = static_cast<int64_t>(n) * C;
    if constexpr (OUT) r.x.load(xp + t * a.xt, ok);
    r.y.load(yp + t * a.yt, ok);
    r.v.load(vp + t * a.vt, ok);
    if constexpr (OUT && DG) r.q.load(qp + t * a.qt, ok);
  };
  auto stage = [&](const Ring& r, int half) __attribute__((always_inline)) {
    uint16_t* t = lds + half * Lds::kChunk + row * RS + col;
    if constexpr (OUT) r.x.template put<kPlane>(t);
    r.y.template put<kPlane>(t + Lds::kX);
    r.v.template put<kPlane>(t + Lds::kX + Lds::kY);
    if constexpr (OUT && DG) r.q.template put<kPlane>(t + Lds::kX + Lds::kY + Lds::kV);
  };

  // decays: sp D of a diagonal block and of the block below it (lane: j = 4g + r, i = li), si lambda^{i+1}
  // of the two row blocks, su lambda^{C-1-j} of the two value blocks
  float4v dd, dl, vf[2];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int j = 4 * g4 + r;
    dd[r] = li >= j ? a.sp * pw[li >= j ? li - j : 0] : 0.f;
    dl[r] = a.sp * pw[16 + li - j];
    vf[0][r] = a.su * pw[C - 1 - j];
    vf[1][r] = a.su * pw[C - 17 - j];
  }
  const Decay em = decay(a.lg, C);

  const float near0 = a.si * pw[li + 1], near1 = a.si * pw[li + 17];
  // of the first chunk: the start state may have one decay less to go
  int un = fresh ? 1 : 0;
  float far0 = a.si * pw[li + 1 - un], far1 = a.si * pw[li + 17 - un];
  Decay e = decay(a.lg, C - un);

  auto chunk = [&](auto FULL, int half, int n) __attribute__((always_inline)) {
    constexpr bool full = decltype(FULL)::value;
    const uint16_t* X = lds + half * Lds::kChunk;
    const uint16_t *Y = X + Lds::kX, *V = Y + Lds::kY, *Q = V + Lds::kV;
    const int L = full ? C : a.n - n * C;
    float4v f0 = vf[0], f1 = vf[1];
    if constexpr (!full) {  // the last, ragged chunk
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 4 * g4 + r;
        f0[r] = j < L ? a.su * pw[j < L ? L - 1 - j : 0] : 0.f;
        f1[r] = j + 16 < L ? a.su * pw[j + 16 < L ? L - 17 - j : 0] : 0.f;
      }
      e = decay(a.lg, L - un);
    }

    Frag v0[NV], v1[NV];
    TV::cols(V, 0, 16 * w, li, g4, v0);
    TV::cols(V, 16, 16 * w, li, g4, v1);
    if constexpr (OUT) {
      // scores, transposed: block (j, i), lane holds [j = 4g + r][i = li]
      float4v s00 = rows_dot<D, NY, NX, LO>(Y, 0, X, 0, li, g4);
      float4v s01 = rows_dot<D, NY, NX, LO>(Y, 0, X, 16, li, g4);
      float4v s11 = rows_dot<D, NY, NX, LO>(Y, 16, X, 16, li, g4);
      float dgc = 0.f;
      if constexpr (DG) {  // pairs within the chunk: block t of Q K^T on wave t % NB
        auto within = [&](float4v z, int rj, int ri, float4v f) __attribute__((always_inline)) {
          const float4v k = rows_dot<D, NV, NQ, 3>(V, rj, Q, ri, li, g4);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int dist = ri + li - rj - 4 * g4 - r;
            dgc += dist > 0 ? static_cast<float>(dist) * f[r] * (k[r] * z[r]) : 0.f;
          }
        };
        if constexpr (NB >= 4) {
          if (w < 3) {
            float4v z, f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              z[r] = w == 0 ? s00[r] : (w == 1 ? s01[r] : s11[r]);
              f[r] = w == 1 ? dl[r] : dd[r];
            }
            within(z, w == 2 ? 16 : 0, w == 0 ? 0 : 16, f);
          }
        } else {
          if (w == 0) within(s00, 0, 0, dd);
          if (w == NB - 1) within(s01, 0, 16, dl);
          if (w == 0) within(s11, 16, 16, dd);
        }
      }
      Frag p00[NP], p01[NP], p11[NP];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool seen = li >= 4 * g4 + r;
        s00[r] = seen ? s00[r] * dd[r] : 0.f;
        s01[r] = s01[r] * dl[r];
        s11[r] = seen ? s11[r] * dd[r] : 0.f;
      }
      split<NP>(s00, p00);
      split<NP>(s01, p01);
      split<NP>(s11, p11);
      if constexpr (D == 128) asm volatile("" ::: "memory");  // read X again rather than keep 64 or more registers
      // O^T = S X^T, decayed, plus V^T P^T
      float4v z0 = mfma::zero4v(), z1 = mfma::zero4v(), y0 = mfma::zero4v(), y1 = mfma::zero4v();
      auto times_state = [&](const float4v* st, float4v& o0, float4v& o1) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < NB; k += 2) {
          Frag a0[NP], a1[NP], x0[NX], x1[NX];
          split<NP>(st[k], a0);
          TX::rows(X, 0, k, li, g4, x0);
          if constexpr (NB == 1) {
            o0 = dot1<NP, NX, LO>(a0, x0, o0);
            TX::rows(X, 16, k, li, g4, x0);
            o1 = dot1<NP, NX, LO>(a0, x0, o1);
          } else {
            split<NP>(st[k + 1], a1);
            TX::rows(X, 0, k + 1, li, g4, x1);
            o0 = dot2<NP, NX, LO>(a0, a1, x0, x1, o0);
            TX::rows(X, 16, k, li, g4, x0);
            TX::rows(X, 16, k + 1, li, g4, x1);
            o1 = dot2<NP, NX, LO>(a0, a1, x0, x1, o1);
          }
        }
      };
      times_state(s, z0, z1);
      if constexpr (DG) {
        times_state(u, y0, y1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          Frag qf[NQ];
          TQ::rows(Q, 16 * i, w, li, g4, qf);
          const float4v qv = TQ::sum(qf);
          const float4v &z = i ? z1 : z0, &y = i ? y1 : y0;
          float t = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) t = fmaf(qv[r], fmaf(static_cast<float>(16 * i + li + 1), z[r], y[r]), t);
          dgc = fmaf(i ? far1 : far0, t, dgc);
        }
        dg += static_cast<double>(dgc);
      }
      z0 = z0 * far0;
      z1 = z1 * far1;
      z0 = dot1<NV, NP, LO>(v0, p00, z0);
      z1 = dot2<NV, NP, LO>(v0, v1, p01, p11, z1);
      OT* o = a.o + static_cast<int64_t>(n * C) * a.ot + 16 * w + 4 * g4;
      if (full || li < L) store4(o + li * a.ot, z0);
      if (full || 16 + li < L) store4(o + (16 + li) * a.ot, z1);
    }
    // S = lambda^L S + (decayed V)^T Y
    {
      Frag q0[3], q1[3], d0[3], d1[3];
      const float4v x0 = TV::sum(v0) * f0, x1 = TV::sum(v1) * f1;
      split<3>(x0, q0);
      split<3>(x1, q1);
      if constexpr (DG) {
        float4v m0, m1;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int left = L - 1 - 4 * g4 - r;
          m0[r] = x0[r] * static_cast<float>(left);
          m1[r] = x1[r] * static_cast<float>(left - 16);
        }
        split<3>(m0, d0);
        split<3>(m1, d1);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        Frag y0[NY], y1[NY];
        TY::cols(Y, 0, 16 * k, li, g4, y0);
        TY::cols(Y, 16, 16 * k, li, g4, y1);
        if constexpr (DG)
          u[k] = dot2<NY, 3, 3>(y0, y1, d0, d1, decayed(u[k] + s[k] * static_cast<float>(L), e));
        s[k] = dot2<NY, 3, 3>(y0, y1, q0, q1, decayed(s[k], e));
      }
    }
    far0 = near0;
    far1 = near1;
    e = em;
    un = 0;
  };

  using T = std::true_type;
  using F = std::false_type;
  if constexpr (two) {
    // chunk n + 2 goes to the registers that chunk n left for LDS half n % 2
    Ring r0, r1;
    fetch(r0, 0);
    fetch(r1, 1);
    stage(r0, 0);
    fetch(r0, 2);
    __syncthreads();
    for (int n = 0; n < nfull; n += 2) {
      stage(r1, 1);
      fetch(r1, n + 3);
      chunk(T{}, 0, n);
      __syncthreads();
      if (n + 1 >= nfull) break;
      stage(r0, 0);
      fetch(r0, n + 4);
      chunk(T{}, 1, n + 1);
      __syncthreads();
    }
    if (nfull < nch) chunk(F{}, nfull % 2, nfull);
  } else {
    Ring r;
    fetch(r, 0);
    for (int n = 0; n < nch; ++n) {
      stage(r, 0);
      fetch(r, n + 1);
      __syncthreads();
      if (n < nfull) chunk(T{}, 0, n);
      else chunk(F{}, 0, n);
      if (n + 1 < nch) __syncthreads();
    }
  }
}

}  // namespace attn
}  // namespace ttt
