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
// accumulator blocks, for the whole walk) and the same 16 output columns.  The three
// causal 16 x 16 blocks of X Y^T come out of the matrix cores, transposed, in the
// layout that the product with V reads: one wave computes, decays and splits a block and
// leaves it in LDS for the others (computed by every wave they were a fifth of all
// instructions, and issue slots are what this kernel runs out of: 90% busy in the
// forward, 93% in the backward at B16 H32 d64 bf16).
//
// Chunks on their way.  bf16: two chunks in registers (16 bytes a thread and tensor)
// and two LDS buffers, so a chunk is loaded three chunks before it is used and stored
// one before; two barriers a chunk, behind the scores and behind the chunk.  Otherwise
// (three planes a tensor, or the four tiles of the decay's gradient at d = 128) one of
// each, and a third barrier behind the stores.  The barrier behind the scores
// comes after the products with the start state, which do not need them (d128 bf16: B16 H16
// T8192 664 us, 708 with it before, gradients at T2048 665 and 685; fp32 inputs -1 to -3%),
// but before them for bf16 at d = 64, where the other workgroups of the CU fill the wait
// ([B, T, H, d], B16 H32 T8192: 494 us, 512 with it after, gradients at T2048 431 and 447;
// [B, H, T, d] the same either way).  At d = 64 a wave also issues a chunk's products
// before the other waves' loads and scores ([B, H, T, d]: 490 us, 509 without, gradients
// 433 and 449; at d = 128 it costs 1 to 3%, below 64 it changes 1 to 3% either way).
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

// LDS of a walk: tiles of X (with outputs), Y, V and Q (with the decay's gradient), and score blocks
template <int D, bool OUT, bool DG, typename XT, typename YT, typename VT, typename QT>
struct WalkLds {
  static constexpr int kX = OUT ? Tile<D, parts_of<XT>()>::kSize : 0;
  static constexpr int kY = Tile<D, parts_of<YT>()>::kSize;
  static constexpr int kV = Tile<D, parts_of<VT>()>::kSize;
  static constexpr int kQ = DG && OUT ? Tile<D, parts_of<QT>()>::kSize : 0;
  static constexpr int kChunk = kX + kY + kV + kQ;
  static constexpr bool kRing = sizeof(XT) + sizeof(YT) + sizeof(VT) == 6 && !(DG && OUT && D == 128);
  static constexpr int kBufs = kRing ? 2 : 1;
  static constexpr bool kScoresFirst = kRing && D == 64;  // where the barrier behind the scores stands
  static constexpr int kScores = OUT ? 3 * kParts * 64 * 4 : 0;  // a chunk's score blocks
  static constexpr int kSize = kBufs * kChunk + kScores;
};

// s: the state before the first token, on return after the last; u likewise dS/dlog_decay.  pw: lambda^0 ..
// lambda^C in LDS, 15 zeros before them.  dg: this lane's share of the decay's gradient.
template <int D, bool OUT, bool DG, typename XT, typename YT, typename VT, typename QT, typename OT>
__device__ __forceinline__ void walk(const Walk<XT, YT, VT, QT, OT>& a, bool fresh, uint16_t* lds, const float* pw,
                                     float4v s[D / 16], float4v u[D / 16], double& dg) {
  typedef WalkLds<D, OUT, DG, XT, YT, VT, QT> Lds;
  constexpr int NB = D / 16, NX = parts_of<XT>(), NY = parts_of<YT>(), NV = parts_of<VT>(), NQ = parts_of<QT>();
  typedef Tile<D, NX> TX;
  typedef Tile<D, NY> TY;
  typedef Tile<D, NV> TV;
  typedef Tile<D, NQ> TQ;
  constexpr int kPlane = TX::kPlane, kHalf = half_at<D>();
  constexpr int NP = kParts;  // of scores and of the state

  const int tid = threadIdx.x, w = tid / 64, lane = tid % 64, li = lane % 16, g4 = lane / 16;
  const int nfull = a.n / C, nch = (a.n + C - 1) / C;
  if (nch == 0) return;
  const Places<D> at(li, g4);
  const int own_col = unit_at<D>(4 * g4 + (li >> 2), 4 * w + (li & 3)), own_row = unit_at<D>(li, 4 * w + g4);
  uint16_t* const scores = lds + Lds::kBufs * Lds::kChunk + 4 * lane;

  const int row = tid / (D / 8), col = 8 * (tid % (D / 8));
  const int u0 = unit_at<D>(row, col / 4), u1 = unit_at<D>(row, col / 4 + 1);
  const XT* xp = a.x + row * a.xt + col;
  const YT* yp = a.y + row * a.yt + col;
  const VT* vp = a.v + row * a.vt + col;
  const QT* qp = a.q + row * a.qt + col;
  OT* op = a.o + li * a.ot + 16 * w + 4 * g4;
  struct Ring {
    Slab<XT> x;
    Slab<YT> y;
    Slab<VT> v;
    Slab<QT> q;
  };
  // Chunk n.  Rows behind the last token hold the last token: the update takes them times zero, and of the
  // outputs and of the decay's gradient they reach only those of rows behind the last token.
  auto fetch = [&](Ring& r, int n) __attribute__((always_inline)) {
    if (n >= nch) return;
    int64_t t = static_cast<int64_t>(n) * C;
    if (n >= nfull) t = min(n * C + row, a.n - 1) - row;
    if constexpr (OUT) r.x.load(xp + t * a.xt);
    r.y.load(yp + t * a.yt);
    r.v.load(vp + t * a.vt);
    if constexpr (OUT && DG) r.q.load(qp + t * a.qt);
  };
  auto stage = [&](const Ring& r, int buf) __attribute__((always_inline)) {
    uint16_t* t = lds + buf * Lds::kChunk;
    if constexpr (OUT) r.x.template put<kPlane>(t, u0, u1);
    r.y.template put<kPlane>(t + Lds::kX, u0, u1);
    r.v.template put<kPlane>(t + Lds::kX + Lds::kY, u0, u1);
    if constexpr (OUT && DG) r.q.template put<kPlane>(t + Lds::kX + Lds::kY + Lds::kV, u0, u1);
  };

  // decays: su lambda^{C-1-j} of the two value blocks, si lambda^{i+1} of the two row blocks
  float4v vf[2];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    vf[0][r] = a.su * pw[C - 1 - 4 * g4 - r];
    vf[1][r] = a.su * pw[C - 17 - 4 * g4 - r];
  }
  Decays chunk_decay(a.lg);
  const float near0 = a.si * pw[li + 1], near1 = a.si * pw[li + 17];
  // of the first chunk: the start state may have one decay less to go
  int un = fresh ? 1 : 0;
  float far0 = a.si * pw[li + 1 - un], far1 = a.si * pw[li + 17 - un];

  // Score block t (0: rows i and j 0..15, 1: i 16..31 and j 0..15, 2: both 16..31) of a chunk, transposed:
  // lane holds [j = 4g + r][i = li].  Its wave goes round with the chunks.
  auto score = [&](int buf, int n) __attribute__((always_inline)) {
    const uint16_t* X = lds + buf * Lds::kChunk;
    const uint16_t *Y = X + Lds::kX, *V = Y + Lds::kY, *Q = V + Lds::kV;
    float dgc = 0.f;
    auto block = [&](int t) __attribute__((always_inline)) {
      const int rj = t == 2 ? kHalf : 0, ri = t == 0 ? 0 : kHalf;
      float4v c = rows_dot<D, NY, NX>(Y + rj, X + ri, at);
      float4v f;  // sp lambda^{i-j}, or what stands before lambda^0 in the table
      const float* pt = pw + (t == 1 ? 16 : 0) + li - 4 * g4;
#pragma unroll
      for (int r = 0; r < 4; ++r) f[r] = a.sp * pt[-r];
      if constexpr (DG) {  // pairs within the chunk
        const float4v k = rows_dot<D, NV, NQ>(V + rj, Q + ri, at);
        const bool live = n * C + (t == 0 ? 0 : 16) + li < a.n;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int dist = (t == 1 ? 16 : 0) + li - 4 * g4 - r;
          dgc += dist > 0 && live ? static_cast<float>(dist) * f[r] * (k[r] * c[r]) : 0.f;
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) c[r] = t == 1 || li >= 4 * g4 + r ? c[r] * f[r] : 0.f;
      Frag p[NP];
      split<NP>(c, p);
      // parts of block 0, then blocks 1 and 2 part by part
      uint16_t* to = scores + (t == 0 ? 0 : 256 * (NP + t - 1));
#pragma unroll
      for (int m = 0; m < NP; ++m) *reinterpret_cast<bf16x4*>(to + (t == 0 ? 256 : 512) * m) = p[m];
    };
    if constexpr (NB >= 4) {
      const int t = (w - n) & (NB - 1);
      if (t < 3) block(t);
    } else {
#pragma unroll
      for (int t = 0; t < 3; ++t)
        if ((t + n) % NB == w) block(t);
    }
    if constexpr (DG) dg += static_cast<double>(dgc);
  };

  // Outputs and update of chunk n in LDS buffer buf, its scores in their half.  FULL: C tokens.
  auto chunk = [&](auto FULL, int buf, int n) __attribute__((always_inline)) {
    constexpr bool full = decltype(FULL)::value;
    const uint16_t* X = lds + buf * Lds::kChunk;
    const uint16_t *Y = X + Lds::kX, *V = Y + Lds::kY, *Q = V + Lds::kV;
    const int L = full ? C : a.n - n * C;
    float4v f0 = vf[0], f1 = vf[1];
    float e = chunk_decay.next();
    if (!full || un) e = powl(a.lg, L - un);
    if constexpr (!full) {  // the last, ragged chunk
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 4 * g4 + r;
        f0[r] = j < L ? a.su * pw[j < L ? L - 1 - j : 0] : 0.f;
        f1[r] = j + 16 < L ? a.su * pw[j + 16 < L ? L - 17 - j : 0] : 0.f;
      }
    }
    if constexpr (D == 64) prio_mfma();
    Frag v0[NV], v1[NV];
    TV::cols(V + own_col, v0);
    TV::cols(V + kHalf + own_col, v1);
    if constexpr (OUT) {
      // O^T = S X^T, decayed, plus V^T P^T
      float4v z0 = mfma::zero4v(), z1 = mfma::zero4v(), y0 = mfma::zero4v(), y1 = mfma::zero4v();
      auto times_state = [&](const float4v* st, float4v& o0, float4v& o1) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < NB; k += 2) {
          Frag a0[NP], a1[NP], x0[NX], x1[NX];
          split<NP>(st[k], a0);
          TX::rows(X + at.row[k], x0);
          if constexpr (NB == 1) {
            o0 = dot1<NP, NX>(a0, x0, o0);
            TX::rows(X + kHalf + at.row[k], x0);
            o1 = dot1<NP, NX>(a0, x0, o1);
          } else {
            split<NP>(st[k + 1], a1);
            TX::rows(X + at.row[k + 1], x1);
            o0 = dot2<NP, NX>(a0, a1, x0, x1, o0);
            TX::rows(X + kHalf + at.row[k], x0);
            TX::rows(X + kHalf + at.row[k + 1], x1);
            o1 = dot2<NP, NX>(a0, a1, x0, x1, o1);
          }
        }
      };
      times_state(s, z0, z1);
      if constexpr (DG) {
        times_state(u, y0, y1);
        float dgc = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          Frag qf[NQ];
          TQ::rows(Q + i * kHalf + own_row, qf);
          const float4v qv = TQ::sum(qf);
          const float4v &z = i ? z1 : z0, &y = i ? y1 : y0;
          float t = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) t = fmaf(qv[r], fmaf(static_cast<float>(16 * i + li + 1), z[r], y[r]), t);
          if (full || 16 * i + li < L) dgc = fmaf(i ? far1 : far0, t, dgc);
        }
        dg += static_cast<double>(dgc);
      }
      z0 = z0 * far0;
      z1 = z1 * far1;
      if constexpr (!Lds::kScoresFirst) __syncthreads();
      Frag p0[NP], p1[NP];
      const uint16_t* P = scores;
#pragma unroll
      for (int m = 0; m < NP; ++m) p0[m] = *reinterpret_cast<const bf16x4*>(P + 256 * m);
      z0 = dot1<NV, NP>(v0, p0, z0);
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        p0[m] = *reinterpret_cast<const bf16x4*>(P + 256 * (NP + 2 * m));
        p1[m] = *reinterpret_cast<const bf16x4*>(P + 256 * (NP + 2 * m + 1));
      }
      z1 = dot2<NV, NP>(v0, v1, p0, p1, z1);
      if (full || li < L) store4(op, z0);
      if (full || 16 + li < L) store4(op + 16 * a.ot, z1);
      op += C * a.ot;
    }
    // S = lambda^L S + (decayed V)^T Y
    {
      Frag q0[NP], q1[NP], d0[NP], d1[NP];
      const float4v x0 = TV::sum(v0) * f0, x1 = TV::sum(v1) * f1;
      if constexpr (NV == 1) {
        split<NP>(x0, q0);
        split<NP>(x1, q1);
      } else {
        split_input(x0, q0);
        split_input(x1, q1);
      }
      if constexpr (DG) {
        float4v m0, m1;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int left = L - 1 - 4 * g4 - r;
          m0[r] = x0[r] * static_cast<float>(left);
          m1[r] = x1[r] * static_cast<float>(left - 16);
        }
        split<NP>(m0, d0);
        split<NP>(m1, d1);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        Frag y0[NY], y1[NY];
        TY::cols(Y + at.col[k], y0);
        TY::cols(Y + kHalf + at.col[k], y1);
        if constexpr (DG) u[k] = dot2<NY, NP>(y0, y1, d0, d1, (u[k] + s[k] * static_cast<float>(L)) * e);
        s[k] = dot2<NY, NP>(y0, y1, q0, q1, s[k] * e);
      }
    }
    if constexpr (D == 64) prio_valu();
    far0 = near0;
    far1 = near1;
    un = 0;
  };

  using T = std::true_type;
  using F = std::false_type;
  if constexpr (Lds::kRing) {
    Ring r0, r1;
    fetch(r0, 0);
    fetch(r1, 1);
    stage(r0, 0);
    fetch(r0, 2);
    __syncthreads();
    auto step = [&](Ring& r, int buf, int n) __attribute__((always_inline)) {
      if constexpr (OUT) {
        score(buf, n);
        if constexpr (Lds::kScoresFirst) __syncthreads();
      }
      stage(r, 1 - buf);
      fetch(r, n + 3);
      chunk(T{}, buf, n);
      __syncthreads();
    };
    for (int n = 0; n < nfull; n += 2) {
      step(r1, 0, n);
      if (n + 1 >= nfull) break;
      step(r0, 1, n + 1);
    }
    if (nfull < nch) {
      if constexpr (OUT) {
        score(nfull % 2, nfull);
        if constexpr (Lds::kScoresFirst) __syncthreads();
      }
      chunk(F{}, nfull % 2, nfull);
    }
  } else {
    Ring r;
    fetch(r, 0);
    for (int n = 0; n < nch; ++n) {
      stage(r, 0);
      fetch(r, n + 1);
      __syncthreads();
      if constexpr (OUT) score(0, n);
      if (n < nfull) chunk(T{}, 0, n);
      else chunk(F{}, 0, n);
      if (n + 1 < nch) __syncthreads();
    }
  }
}

}  // namespace attn
}  // namespace ttt
