// Selective scan, backward.
//
// Pages: [TTT] = news article "大模型最强架构TTT问世！斯坦福UCSD等5年磨一剑，一夜推翻Transformer"
// (aharts.cn / itmax.cn), part 03 §4 (the layer is trained end to end).
//
// With a_t = exp(dt_t A), x_t = dt_t u_t and dy_t the gradient of the sum before the gate, from the last token to the first
//   g_t = C_t dy_t + a_{t+1} g_{t+1}                                   (the gradient of h_t)
//   dC_t = sum_c dy_t h_t,      dB_t = sum_c x_t g_t,                  (over the channels of the group)
//   du_t = dt_t sum_n g_t B_t + D dy_t,   dA = sum_t dt_t g_t a_t h_{t-1},
//   ddt_t = sum_n g_t a_t h_{t-1} A + u_t sum_n g_t B_t
// The walk goes forward first and writes the state before each chunk of CL tokens, then backward chunk by chunk: the chunk's
// a_t and a_t h_{t-1} are computed again into registers and used from the last token on.
#include "scan_common.h"

namespace ttt {
namespace {

using namespace scan;

template <int NS>
constexpr int kChunk = NS <= 4 ? 16 : 8;

// Sums over the 16 channels of a wave (lanes l / 4) of 2 NS values a lane; what comes back in x[0 .. max(1, NS / 2)) is
// value (l / 32) NS + (l / 16 % 2) (NS / 2) + j of the states of l % 4.
template <int NS>
__device__ __forceinline__ void channel_sums(float (&x)[2 * NS]) {
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[j]), __float_as_uint(x[j + NS]), false, false);
    x[j] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (NS == 1) {
    x[0] = mfma::sum_row_pairs(x[0]);
  } else {
#pragma unroll
    for (int j = 0; j < NS / 2; ++j) {
      const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[j]), __float_as_uint(x[j + NS / 2]), false, false);
      x[j] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
  }
#pragma unroll
  for (int j = 0; j < (NS > 1 ? NS / 2 : 1); ++j) {
    x[j] += mfma::dpp_mov<0x128>(x[j]);  // row_ror:8
    x[j] += mfma::dpp_mov<0x124>(x[j]);  // row_ror:4
  }
}

// What a segment adds to a zero state (hseg), its sum of dt (sseg) and what its own dy add to the gradient of the state
// before it (gseg): g = sum_t a_1 .. a_t C_t dy_t.
template <typename InT, typename OutT, int NS, bool Wide>
__global__ __launch_bounds__(256) void ttt_scan_bwd_states(ScanArgs a) {
  constexpr int NP = 4 * NS;
  __shared__ __align__(16) float4 tile[TT][CH];  // dt, dt u, dy
  __shared__ __align__(16) float sB[TT * NP], sC[TT * NP];
  const int tid = threadIdx.x, lane = tid & 63, q = lane & 3, cw = (tid >> 6) * 16 + (lane >> 2);
  const int seg = static_cast<int>(blockIdx.x % a.nseg);
  const Place p = place(a, blockIdx.x / a.nseg);
  const int c = p.c0 + cw;
  const bool on = cw < p.nc;
  const int begin = seg * a.seglen, end = min(p.len, min(a.T, begin + a.seglen));
  float a2[NS], h[NS], g[NS], prod[NS], sum = 0.f;
  decays(a2, a, c, q, on);
#pragma unroll
  for (int i = 0; i < NS; ++i) h[i] = g[i] = 0.f, prod[i] = 1.f;
  const int row = tid >> 3, oct = (tid & 7) * 8, n8 = min(8, p.nc - oct);
  const InT* up = static_cast<const InT*>(a.u) + p.b * a.us.b + p.c0 + oct;
  const InT* dp = static_cast<const InT*>(a.dt) + p.b * a.dts.b + p.c0 + oct;
  const InT* zp = a.z ? static_cast<const InT*>(a.z) + p.b * a.zs.b + p.c0 + oct : nullptr;
  const OutT* gp = static_cast<const OutT*>(a.dy) + p.b * a.ys.b + p.c0 + oct;
  const InT* bp = static_cast<const InT*>(a.Bm) + p.b * a.bs.b + p.g * a.bs.h;
  const InT* cp = static_cast<const InT*>(a.Cm) + p.b * a.cs.b + p.g * a.cs.h;
  float bias[8];
  params<8>(bias, a.dt_bias ? a.dt_bias + p.c0 + oct : nullptr, n8, 0.f);
  for (int t0 = begin; t0 < end; t0 += TT) {
    const int64_t t = t0 + row;
    const int n = t < end ? n8 : 0;
    Piece<InT, 8> u, dt, z;
    Piece<OutT, 8> dy;
    Rows<InT, NS> rb, rc;
    load<Wide>(u, up + t * a.us.t, n);
    load<Wide>(dt, dp + t * a.dts.t, n);
    load<Wide>(dy, gp + t * a.ys.t, n);
    if (zp) load<Wide>(z, zp + t * a.zs.t, n);
    rb.load(bp, a.bs.t, a.N, t0, end, tid);
    rc.load(cp, a.cs.t, a.N, t0, end, tid);
    if (t0 > begin) __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = dt.get(i) + bias[i], d = dy.get(i), slope;
      if (a.softplus) s = softplus(s, slope);
      if (i >= n) s = 0.f;
      if (zp) d *= z.get(i) * sigmoid(z.get(i));
      tile[row][oct + i] = make_float4(s, s * u.get(i), d, 0.f);
    }
    rb.stage(sB, tid);
    rc.stage(sC, tid);
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < TT; ++k) {
      const float4 d = tile[k][cw];
      float Bv[NS], Cv[NS];
      lds_floats(Bv, sB + k * NP + q * NS);
      lds_floats(Cv, sC + k * NP + q * NS);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float e = __builtin_amdgcn_exp2f(d.x * a2[i]);
        h[i] = fmaf(e, h[i], d.y * Bv[i]);
        prod[i] *= e;
        g[i] = fmaf(prod[i], Cv[i] * d.z, g[i]);
      }
      sum += d.x;
    }
  }
  const int64_t slot = static_cast<int64_t>(p.b) * a.nseg + seg;
  if (seg + 1 < a.nseg) store_states(h, a.hseg + ((slot + 1) * a.D + c) * a.N, a.N, q, on);
  store_states(g, a.gseg + (slot * a.D + c) * a.N, a.N, q, on);
  if (on && q == 0) a.sseg[slot * a.D + c] = sum;
  if (seg == 0) {
    load_states(h, a.h0 ? a.h0 + (static_cast<int64_t>(p.b) * a.D + c) * a.N : nullptr, a.N, q, on);
    store_states(h, a.hseg + (slot * a.D + c) * a.N, a.N, q, on);
  }
}

template <typename InT, typename OutT, int NS, bool Wide>
__global__ __launch_bounds__(256) void ttt_scan_bwd(ScanArgs a) {
  constexpr int NP = 4 * NS, CL = kChunk<NS>;
  __shared__ __align__(16) float4 tile[TT][CH];  // dt, dt u, dy; then sum g B, sum g a h A log2(e), y
  __shared__ __align__(16) float sB[TT * NP], sC[TT * NP];
  __shared__ __align__(16) float sbc[4][TT][2][NP];  // each wave's sums over its channels
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, q = lane & 3, cw = wave * 16 + (lane >> 2);
  const int seg = static_cast<int>(blockIdx.x % a.nseg);
  const Place p = place(a, blockIdx.x / a.nseg);
  const int c = p.c0 + cw;
  const bool on = cw < p.nc;
  const int begin = seg * a.seglen, tokens = min(a.T, begin + a.seglen), end = min(p.len, tokens);
  const int64_t slot = static_cast<int64_t>(p.b) * a.nseg + seg;

  float a2[NS], h[NS];
  decays(a2, a, c, q, on);
  if (a.nseg == 1) load_states(h, a.h0 ? a.h0 + (static_cast<int64_t>(p.b) * a.D + c) * a.N : nullptr, a.N, q, on);
  else start_state(h, a2, a, p, seg, c, q, on);

  const int row = tid >> 3, oct = (tid & 7) * 8, n8 = min(8, p.nc - oct);
  const InT* up = static_cast<const InT*>(a.u) + p.b * a.us.b + p.c0 + oct;
  const InT* dp = static_cast<const InT*>(a.dt) + p.b * a.dts.b + p.c0 + oct;
  const InT* zp = a.z ? static_cast<const InT*>(a.z) + p.b * a.zs.b + p.c0 + oct : nullptr;
  const OutT* gp = static_cast<const OutT*>(a.dy) + p.b * a.ys.b + p.c0 + oct;
  const InT* bp = static_cast<const InT*>(a.Bm) + p.b * a.bs.b + p.g * a.bs.h;
  const InT* cp = static_cast<const InT*>(a.Cm) + p.b * a.cs.b + p.g * a.cs.h;
  float bias[8];
  params<8>(bias, a.dt_bias ? a.dt_bias + p.c0 + oct : nullptr, n8, 0.f);
  float* ck = a.ckpt + (static_cast<int64_t>(p.b) * a.chunks * a.D + c) * a.N;  // chunk j at j * D * N
  const int64_t ckstep = static_cast<int64_t>(a.D) * a.N;

  // forward: the state before each chunk
  for (int t0 = begin; t0 < end; t0 += TT) {
    const int64_t t = t0 + row;
    const int n = t < end ? n8 : 0;
    Piece<InT, 8> u, dt;
    Rows<InT, NS> rb;
    load<Wide>(u, up + t * a.us.t, n);
    load<Wide>(dt, dp + t * a.dts.t, n);
    rb.load(bp, a.bs.t, a.N, t0, end, tid);
    if (t0 > begin) __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = dt.get(i) + bias[i], slope;
      if (a.softplus) s = softplus(s, slope);
      if (i >= n) s = 0.f;
      *reinterpret_cast<float2*>(&tile[row][oct + i]) = make_float2(s, s * u.get(i));
    }
    rb.stage(sB, tid);
    __syncthreads();
    for (int k0 = 0; k0 < TT; k0 += CL) {
      if (t0 + k0 < end) store_states(h, ck + (t0 + k0) / CL * ckstep, a.N, q, on);
#pragma unroll
      for (int k = k0; k < k0 + CL; ++k) {
        const float2 d = *reinterpret_cast<const float2*>(&tile[k][cw]);
        float Bv[NS];
        lds_floats(Bv, sB + k * NP + q * NS);
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(d.x * a2[i]), h[i], d.y * Bv[i]);
      }
    }
  }

  // the gradient of the state behind the segment
  float g[NS], dA[NS];
  load_states(g, a.dh_final ? a.dh_final + (static_cast<int64_t>(p.b) * a.D + c) * a.N : nullptr, a.N, q, on);
  for (int s = a.nseg - 1; s > seg; --s) {
    const int64_t at = static_cast<int64_t>(p.b) * a.nseg + s;
    const float sum = on ? a.sseg[at * a.D + c] : 0.f;
    float x[NS];
    load_states(x, a.gseg + (at * a.D + c) * a.N, a.N, q, on);
#pragma unroll
    for (int i = 0; i < NS; ++i) g[i] = fmaf(__builtin_amdgcn_exp2f(sum * a2[i]), g[i], x[i]);
  }
#pragma unroll
  for (int i = 0; i < NS; ++i) dA[i] = 0.f;

  OutT* dup = static_cast<OutT*>(a.du) + p.b * a.dus.b + p.c0 + oct;
  OutT* ddp = static_cast<OutT*>(a.ddt) + p.b * a.ddts.b + p.c0 + oct;
  OutT* dzp = zp ? static_cast<OutT*>(a.dz) + p.b * a.dzs.b + p.c0 + oct : nullptr;
  float skip[8], dD[8], db[8];
  params<8>(skip, a.Dskip ? a.Dskip + p.c0 + oct : nullptr, n8, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) dD[i] = db[i] = 0.f;
  float* part = a.bcpart + (static_cast<int64_t>(p.b) * a.G + p.g) * ((a.D / a.G + CH - 1) / CH) * a.T * 2 * a.N +
                static_cast<int64_t>(p.tile) * a.T * 2 * a.N;

  const int last = begin + (max(end - begin, 1) - 1) / TT * TT;
  for (int t0 = last; t0 >= begin && end > begin; t0 -= TT) {
    const int64_t t = t0 + row;
    const int n = t < end ? n8 : 0;
    Piece<InT, 8> u, dtr, z;
    Piece<OutT, 8> dyr;
    Rows<InT, NS> rb, rc;
    load<Wide>(u, up + t * a.us.t, n);
    load<Wide>(dtr, dp + t * a.dts.t, n);
    load<Wide>(dyr, gp + t * a.ys.t, n);
    if (zp) load<Wide>(z, zp + t * a.zs.t, n);
    rb.load(bp, a.bs.t, a.N, t0, end, tid);
    rc.load(cp, a.cs.t, a.N, t0, end, tid);
    __syncthreads();  // the tile before (or the forward walk's last) is done with
    float dt[8], slope[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float d = dyr.get(i);
      dt[i] = dtr.get(i) + bias[i];
      slope[i] = 1.f;
      if (a.softplus) dt[i] = softplus(dt[i], slope[i]);
      if (i >= n) dt[i] = 0.f;
      if (zp) d *= z.get(i) * sigmoid(z.get(i));
      tile[row][oct + i] = make_float4(dt[i], dt[i] * u.get(i), d, 0.f);
    }
    rb.stage(sB, tid);
    rc.stage(sC, tid);
    __syncthreads();
#pragma unroll 1
    for (int k0 = TT - CL; k0 >= 0; k0 -= CL) {
      if (t0 + k0 >= end) {  // nothing here: zeros for the sums
        for (int k = k0; k < k0 + CL; ++k) {
          reinterpret_cast<float*>(&tile[k][cw])[q] = 0.f;
          if ((lane & 12) == 0) {
#pragma unroll
            for (int j = 0; j < (NS > 1 ? NS / 2 : 1); ++j)
              sbc[wave][k][lane >> 5][NS > 1 ? q * NS + (lane >> 4 & 1) * (NS / 2) + j : q] = 0.f;
          }
        }
        continue;
      }
      float ah[CL][NS], e[CL][NS];
      load_states(h, ck + (t0 + k0) / CL * ckstep, a.N, q, on);
#pragma unroll
      for (int k = 0; k < CL; ++k) {
        const float2 d = *reinterpret_cast<const float2*>(&tile[k0 + k][cw]);
        float Bv[NS];
        lds_floats(Bv, sB + (k0 + k) * NP + q * NS);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          e[k][i] = __builtin_amdgcn_exp2f(d.x * a2[i]);
          ah[k][i] = e[k][i] * h[i];
          h[i] = fmaf(d.y, Bv[i], ah[k][i]);
        }
      }
#pragma unroll
      for (int k = CL - 1; k >= 0; --k) {
        const float4 d = tile[k0 + k][cw];
        float Bv[NS], Cv[NS], bc[2 * NS], sb = 0.f, sa = 0.f, y = 0.f;
        lds_floats(Bv, sB + (k0 + k) * NP + q * NS);
        lds_floats(Cv, sC + (k0 + k) * NP + q * NS);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          g[i] = fmaf(Cv[i], d.z, g[i]);
          const float ht = fmaf(d.y, Bv[i], ah[k][i]);
          bc[i] = d.y * g[i];
          bc[NS + i] = d.z * ht;
          sb = fmaf(g[i], Bv[i], sb);
          const float gh = g[i] * ah[k][i];
          sa = fmaf(gh, a2[i], sa);
          dA[i] = fmaf(gh, d.x, dA[i]);
          y = fmaf(Cv[i], ht, y);
          g[i] *= e[k][i];
        }
        channel_sums<NS>(bc);
        sb = quad_sum(sb);
        sa = quad_sum(sa);
        y = quad_sum(y);
        if (q < 3) reinterpret_cast<float*>(&tile[k0 + k][cw])[q] = q == 0 ? sb : q == 1 ? sa : y;
        if ((lane & 12) == 0) {
#pragma unroll
          for (int j = 0; j < (NS > 1 ? NS / 2 : 1); ++j)
            sbc[wave][k0 + k][lane >> 5][NS > 1 ? q * NS + (lane >> 4 & 1) * (NS / 2) + j : q] = bc[j];
        }
      }
    }
    __syncthreads();
    if (t < end && n8 > 0) {
      float o[3][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 v = tile[row][oct + i];
        const float uu = u.get(i);
        float d = dyr.get(i);
        o[2][i] = 0.f;
        if (zp) {
          const float x = z.get(i), s = sigmoid(x), gate = x * s;
          o[2][i] = d * fmaf(skip[i], uu, v.z) * fmaf(gate, 1.f - s, s);
          d *= gate;
        }
        o[0][i] = fmaf(dt[i], v.x, skip[i] * d);
        o[1][i] = fmaf(uu, v.x, v.y * (1.f / kLog2e)) * slope[i];
        dD[i] = fmaf(d, uu, dD[i]);
        db[i] += o[1][i];
      }
      Piece<OutT, 8> out;
      out.set_all(o[0]);
      store<Wide>(out, dup + t * a.dus.t, n8);
      out.set_all(o[1]);
      store<Wide>(out, ddp + t * a.ddts.t, n8);
      if (zp) {
        out.set_all(o[2]);
        store<Wide>(out, dzp + t * a.dzs.t, n8);
      }
    }
    for (int x = tid; x < TT * 2 * NP; x += 256) {
      const int k = x / (2 * NP), w = x / NP % 2, m = x % NP;
      if (t0 + k < end && m < a.N)
        part[(static_cast<int64_t>(t0 + k) * 2 + w) * a.N + m] =
            (sbc[0][k][w][m] + sbc[1][k][w][m]) + (sbc[2][k][w][m] + sbc[3][k][w][m]);
    }
  }
  Piece<OutT, 8> none;
  none.zero();
  for (int64_t t = max(begin, end) + row; t < tokens; t += TT) {
    store<Wide>(none, dup + t * a.dus.t, n8);
    store<Wide>(none, ddp + t * a.ddts.t, n8);
    if (zp) store<Wide>(none, dzp + t * a.dzs.t, n8);
  }
  if (seg == 0 && a.dh0) store_states(g, a.dh0 + (static_cast<int64_t>(p.b) * a.D + c) * a.N, a.N, q, on);
  float* sums = a.part + slot * (static_cast<int64_t>(a.D) * (a.N + 2));
  store_states(dA, sums + static_cast<int64_t>(c) * a.N, a.N, q, on);
  // dD and ddt_bias: over the 32 token rows
  __syncthreads();
  float2* rows = reinterpret_cast<float2*>(&tile[0][0]);
#pragma unroll
  for (int i = 0; i < 8; ++i) rows[row * CH + oct + i] = make_float2(dD[i], db[i]);
  __syncthreads();
  if (tid < p.nc) {
    float2 s = rows[tid];
    for (int r = 1; r < TT; ++r) {
      const float2 x = rows[r * CH + tid];
      s.x += x.x;
      s.y += x.y;
    }
    sums += static_cast<int64_t>(a.D) * a.N + p.c0 + tid;
    sums[0] = s.x;
    sums[a.D] = s.y;
  }
}

// dB and dC: the sum over the tiles of channels, in their order.
template <typename OutT>
__global__ __launch_bounds__(256) void ttt_scan_bc_sum(ScanBcSumArgs a) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, each = static_cast<int64_t>(a.T) * 2 * a.N;
  const int64_t bg = id / each;
  const int64_t e = id - bg * each;
  const int b = static_cast<int>(bg / a.G), g = static_cast<int>(bg % a.G);
  if (b >= a.B) return;
  const int64_t t = e / (2 * a.N);
  const int w = static_cast<int>(e / a.N % 2), n = static_cast<int>(e % a.N);
  const int len = a.lens ? max(0, min(a.lens[b], a.T)) : a.T;
  float s = 0.f;
  if (t < len) {
    const float* p = a.part + bg * a.tiles * each + e;
    for (int k = 0; k < a.tiles; ++k) s += p[k * each];
  }
  OutT* o = w ? static_cast<OutT*>(a.dC) + b * a.dcs.b + g * a.dcs.h + t * a.dcs.t
              : static_cast<OutT*>(a.dB) + b * a.dbs.b + g * a.dbs.h + t * a.dbs.t;
  put(o + n, s);
}

template <typename InT, typename OutT, int NS>
hipError_t go(bool states, const ScanArgs& a, hipStream_t s) {
  const int dg = a.D / a.G;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.G * ((dg + CH - 1) / CH) * a.nseg);
  if (states) {
    if (a.wide) ttt_scan_bwd_states<InT, OutT, NS, true><<<grid, 256, 0, s>>>(a);
    else ttt_scan_bwd_states<InT, OutT, NS, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (a.wide) ttt_scan_bwd<InT, OutT, NS, true><<<grid, 256, 0, s>>>(a);
    else ttt_scan_bwd<InT, OutT, NS, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <typename InT, typename OutT>
hipError_t go(bool states, const ScanArgs& a, hipStream_t s) {
  switch (scan_states(a.N)) {
    case 1: return go<InT, OutT, 1>(states, a, s);
    case 2: return go<InT, OutT, 2>(states, a, s);
    case 4: return go<InT, OutT, 4>(states, a, s);
    case 8: return go<InT, OutT, 8>(states, a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t go(bool states, const ScanArgs& a, hipStream_t s) {
  const bool inf = a.in_dtype == 0, outf = a.out_dtype == 0;
  if (inf && outf) return go<float, float>(states, a, s);
  if (inf) return go<float, uint16_t>(states, a, s);
  if (outf) return go<uint16_t, float>(states, a, s);
  return go<uint16_t, uint16_t>(states, a, s);
}

}  // namespace

int scan_chunk(int N) { return scan_states(N) <= 4 ? kChunk<4> : kChunk<8>; }

hipError_t launch_scan_bwd_states(const ScanArgs& a, hipStream_t s) { return go(true, a, s); }
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s) { return go(false, a, s); }

hipError_t launch_scan_bc_sum(const ScanBcSumArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.B) * a.G * a.T * 2 * a.N;
  if (n == 0) return hipSuccess;
  const unsigned grid = static_cast<unsigned>((n + 255) / 256);
  if (a.out_dtype == 0) ttt_scan_bc_sum<float><<<grid, 256, 0, s>>>(a);
  else ttt_scan_bc_sum<uint16_t><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ttt
