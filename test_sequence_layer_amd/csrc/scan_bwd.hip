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
// 8 x 2048 tokens, 1536 channels, N = 16, bf16: 657 us (67 by its bytes at 5.3 TB/s); by the trace, at the settled clock, the start
// states of 4 segments take 131, the walk 506 and the sums 16 and 5.  The walk keeps the vector unit busy in 74% of the cycles:
// 219 registers leave one walking wave to a SIMD, which waits for its own results in the rest.  Rows that do not go in pieces
// (1532 channels) take 1052.  For N > 16 60 to 68 bytes a lane are in scratch: 1404 us with N = 32, 340 with N = 4.
#include <limits.h>

#include "scan_common.h"

namespace ttt {
namespace {

using namespace scan;

constexpr int TT = 16;  // tokens staged at a time: 4 channels of one to a thread, which leaves registers for the chunk
constexpr int GS = 4;

// Tokens to a chunk, as long as its a_t and a_t h_{t-1} fit into registers (8 x 2048 tokens, 1536 channels, bf16, us):
//   N = 16: 16 tokens 657, 8 tokens 683;  N = 4: 340 and 346;  N = 32: 16 tokens 3134, 8 tokens 1401, 4 tokens 1450
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

// This thread's piece of the tiles: token row, channels quad .. quad + 3, and where they are.
template <typename InT, typename OutT>
struct Lines {
  int row, quad, n4;  // n4 may be negative
  const InT *u, *dt, *z;
  const OutT* dy;
  __device__ __forceinline__ Lines(const ScanArgs& a, const Place& p, int first, int tid) {
    row = tid >> 4;
    quad = (tid & 15) * 4;
    n4 = min(4, p.nc - quad);
    const int64_t t = first + row, c = p.c0 + (n4 > 0 ? quad : 0);
    u = static_cast<const InT*>(a.u) + p.b * a.us.b + t * a.us.t + c;
    dt = static_cast<const InT*>(a.dt) + p.b * a.dts.b + t * a.dts.t + c;
    z = a.z ? static_cast<const InT*>(a.z) + p.b * a.zs.b + t * a.zs.t + c : nullptr;
    dy = static_cast<const OutT*>(a.dy) + p.b * a.ys.b + t * a.ys.t + c;
  }
  __device__ __forceinline__ void step(const ScanArgs& a) {
    u += TT * a.us.t;
    dt += TT * a.dts.t;
    if (a.z) z += TT * a.zs.t;
    dy += TT * a.ys.t;
  }
};

template <int N>
__device__ __forceinline__ void zero_from(float (&x)[N], int n) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = i < n ? x[i] : 0.f;
}

// What a segment adds to a zero state (hseg), its sum of dt (sseg) and what its own dy add to the gradient of the state
// before it (gseg): g = sum_t a_1 .. a_t C_t dy_t.
template <typename InT, typename OutT, int NS, bool Wide>
__global__ __launch_bounds__(256, 2) void ttt_scan_bwd_states(ScanArgs a) {
  constexpr int NP = 4 * NS;
  __shared__ __align__(16) float4 tile[TT][CH];  // dt, dt u, dy
  __shared__ __align__(16) float bc[2 * TT * NP];
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
  Lines<InT, OutT> at(a, p, begin, tid);
  BcRows<InT, NP, TT, Wide> rows(a, p, begin, tid, true);
  float bias[4];
  params<4>(bias, a.dt_bias ? a.dt_bias + p.c0 + at.quad : nullptr, at.n4, 0.f);
  for (int t0 = begin; t0 < end; t0 += TT) {
    const int n = t0 + at.row < end ? at.n4 : 0;
    Piece<InT, 4> u, dt, z;
    Piece<OutT, 4> dy;
    load<Wide>(u, at.u, n);
    load<Wide>(dt, at.dt, n);
    load<Wide>(dy, at.dy, n);
    if (a.z) load<Wide>(z, at.z, n);
    typename BcRows<InT, NP, TT, Wide>::Values v;
    rows.load(v, t0, end, 1);
    at.step(a);
    if (t0 > begin) __syncthreads();
    float s[4], d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = dt.get(i) + bias[i], d[i] = dy.get(i);
    if (a.softplus) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = softplus(s[i]);
    }
    zero_from(s, n);
    if (a.z) {
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] *= z.get(i) * sigmoid(z.get(i));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) tile[at.row][at.quad + i] = make_float4(s[i], s[i] * u.get(i), d[i], 0.f);
    rows.stage(v, bc, t0, end);
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < TT; ++k) {
      const float4 x = tile[k][cw];
      float Bv[NS], Cv[NS];
      lds_floats(Bv, bc + k * NP + q * NS);
      lds_floats(Cv, bc + (TT + k) * NP + q * NS);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float e = __builtin_amdgcn_exp2f(x.x * a2[i]);
        h[i] = fmaf(e, h[i], x.y * Bv[i]);
        prod[i] *= e;
        g[i] = fmaf(prod[i], Cv[i] * x.z, g[i]);
      }
      sum += x.x;
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

// Waves 0 to 3 walk, 16 channels each; waves 4 to 7 bring the tiles into LDS one step ahead of them and take them out one
// step behind (see the forward): first the forward walk's tiles, then the same backward.  Step s works on buffer s % 2.
template <typename InT, typename OutT, int NS, bool Wide>
__global__ __launch_bounds__(512, 1) void ttt_scan_bwd(ScanArgs a) {
  constexpr int NP = 4 * NS, CL = kChunk<NS>, NV = NS > 1 ? NS / 2 : 1;
  __shared__ __align__(16) float4 tile[2][TT][CH];  // dt, dt u, dy; then sum g B, sum g a h A log2(e), y
  __shared__ __align__(16) float bc[2][2 * TT * NP];
  __shared__ __align__(16) float sbc[2][4][TT][2][NP];  // each wave's sums over its channels
  const int seg = static_cast<int>(blockIdx.x % a.nseg);
  const Place p = place(a, blockIdx.x / a.nseg);
  const int begin = seg * a.seglen, tokens = min(a.T, begin + a.seglen), end = min(p.len, tokens);
  const int64_t slot = static_cast<int64_t>(p.b) * a.nseg + seg;
  const int tiles = begin < end ? (end - begin + 2 * TT - 1) / (2 * TT) * 2 : 0;  // (an even number: two steps at a time)
  float* sums = a.part + slot * (static_cast<int64_t>(a.D) * (a.N + 2));

  if (__builtin_amdgcn_readfirstlane(threadIdx.x) < 256) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, q = lane & 3, cw = wave * 16 + (lane >> 2);
    const int c = p.c0 + cw;
    const bool on = cw < p.nc;
    float a2[NS], h[NS];
    decays(a2, a, c, q, on);
    if (a.nseg == 1) load_states(h, a.h0 ? a.h0 + (static_cast<int64_t>(p.b) * a.D + c) * a.N : nullptr, a.N, q, on);
    else start_state(h, a2, a, p, seg, c, q, on);
    const int64_t ckstep = static_cast<int64_t>(a.D) * a.N;
    // the chunk's state; always by the same thread, so that it is there when it is read again
    float* ck = a.ckpt + (static_cast<int64_t>(p.b) * a.chunks + begin / CL) * ckstep + static_cast<int64_t>(c) * a.N;
    int buf = 0;
    // forward: the state before each chunk
    for (int k = 0; k < tiles; ++k, buf ^= 1) {
      __syncthreads();
      const float* sd = &tile[buf][0][cw].x;
      const float* sb = bc[buf] + q * NS;
#pragma unroll
      for (int k0 = 0; k0 < TT; k0 += CL) {
        store_states(h, ck, a.N, q, on && begin + k * TT + k0 < end);
        ck += ckstep;
        if (k0 + CL >= TT && k == tiles - 1) break;  // (nobody asks for the state behind the last chunk)
#pragma unroll
        for (int j0 = k0; j0 < k0 + CL; j0 += GS) {
          Group<NS, GS, NP, 4 * CH> g;
          g.read(sd, sb, j0);
          float e[GS][NS];
#pragma unroll
          for (int j = 0; j < GS; ++j)
#pragma unroll
            for (int i = 0; i < NS; ++i) e[j][i] = __builtin_amdgcn_exp2f(g.d[j].x * a2[i]);
#pragma unroll
          for (int j = 0; j < GS; ++j)
#pragma unroll
            for (int i = 0; i < NS; ++i) h[i] = fmaf(e[j][i], h[i], g.d[j].y * g.B[j][i]);
        }
      }
    }
    // the gradient of the state behind the segment
    float g[NS], dA[NS];
    load_states(g, a.dh_final ? a.dh_final + (static_cast<int64_t>(p.b) * a.D + c) * a.N : nullptr, a.N, q, on);
    for (int s = a.nseg - 1; s > seg; --s) {
      const int64_t o = static_cast<int64_t>(p.b) * a.nseg + s;
      const float sum = on ? a.sseg[o * a.D + c] : 0.f;
      float x[NS];
      load_states(x, a.gseg + (o * a.D + c) * a.N, a.N, q, on);
#pragma unroll
      for (int i = 0; i < NS; ++i) g[i] = fmaf(__builtin_amdgcn_exp2f(sum * a2[i]), g[i], x[i]);
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) dA[i] = 0.f;

    float next[NS];  // the state before the chunk that comes next
    load_states(next, ck - ckstep, a.N, q, on && tiles > 0 && begin + tiles * TT - CL < end);
    for (int k = tiles - 1; k >= 0; --k, buf ^= 1) {
      __syncthreads();
      const float4* td = &tile[buf][0][cw];
      const float* sb = bc[buf] + q * NS;
      float* res = reinterpret_cast<float*>(&tile[buf][0][cw]) + q;
      float* out = &sbc[buf][wave][0][lane >> 5][NS > 1 ? q * NS + (lane >> 4 & 1) * (NS / 2) : q];
#pragma unroll 1
      for (int k0 = TT - CL; k0 >= 0; k0 -= CL) {
        float ah[CL][NS], e[CL][NS];
        ck -= ckstep;
#pragma unroll
        for (int i = 0; i < NS; ++i) h[i] = next[i];
        const int before = begin + k * TT + k0 - CL;
        load_states(next, ck - ckstep, a.N, q, on && before >= begin && before < end);
        {
          Group<NS, GS, NP, 4 * CH> in[2];
          in[0].read(&td->x, sb, k0);
#pragma unroll
          for (int m = 0; m < CL; m += GS) {
            if (m + GS < CL) in[(m / GS + 1) & 1].read(&td->x, sb, k0 + m + GS);
            __builtin_amdgcn_sched_barrier(0);  // (the reads stay ahead)
            const auto& now = in[m / GS & 1];
#pragma unroll
            for (int j = 0; j < GS; ++j)
#pragma unroll
              for (int i = 0; i < NS; ++i) e[m + j][i] = __builtin_amdgcn_exp2f(now.d[j].x * a2[i]);
#pragma unroll
            for (int j = 0; j < GS; ++j)
#pragma unroll
              for (int i = 0; i < NS; ++i) {
                ah[m + j][i] = e[m + j][i] * h[i];
                h[i] = fmaf(now.d[j].y, now.B[j][i], ah[m + j][i]);
              }
          }
        }
        // two tokens at a time, the next two's reads ahead of this two's writes (which the compiler cannot tell apart)
        float4 x[2][2];
        float Bv[2][2][NS], Cv[2][2][NS];
        auto read = [&](int to, int j) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            x[to][r] = td[(k0 + j - r) * CH];
            lds_floats(Bv[to][r], sb + (k0 + j - r) * NP);
            lds_floats(Cv[to][r], sb + (TT + k0 + j - r) * NP);
          }
        };
        read(CL / 2 & 1, CL - 1);
#pragma unroll
        for (int m = CL / 2; m > 0; --m) {
          if (m > 1) read(m - 1 & 1, 2 * m - 3);
          __builtin_amdgcn_sched_barrier(0);
          float v[2][2 * NS], s[2], sa[2], y[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j = 2 * m - 1 - r;
            const float4 xt = x[m & 1][r];
            const float(&Bt)[NS] = Bv[m & 1][r], (&Ct)[NS] = Cv[m & 1][r];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              g[i] = fmaf(Ct[i], xt.z, g[i]);
              const float ht = fmaf(xt.y, Bt[i], ah[j][i]);
              v[r][i] = xt.y * g[i];
              v[r][NS + i] = xt.z * ht;
              const float gh = g[i] * ah[j][i];
              s[r] = i ? fmaf(g[i], Bt[i], s[r]) : g[i] * Bt[i];
              sa[r] = i ? fmaf(gh, a2[i], sa[r]) : gh * a2[i];
              y[r] = i ? fmaf(Ct[i], ht, y[r]) : Ct[i] * ht;
              dA[i] = fmaf(gh, xt.x, dA[i]);
              g[i] *= e[j][i];
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            channel_sums<NS>(v[r]);
            s[r] = quad_sum(s[r]);
            sa[r] = quad_sum(sa[r]);
            y[r] = quad_sum(y[r]);
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j = 2 * m - 1 - r;
            // (lanes that hold the same value write it to the same place: no branch in the walk)
            res[(k0 + j) * 4 * CH] = q == 0 ? s[r] : q == 1 ? sa[r] : y[r];
            float* to = out + (k0 + j) * 2 * NP;
            if constexpr (NV == 4) *reinterpret_cast<float4*>(to) = make_float4(v[r][0], v[r][1], v[r][2], v[r][3]);
            else if constexpr (NV == 2) *reinterpret_cast<float2*>(to) = make_float2(v[r][0], v[r][1]);
            else to[0] = v[r][0];
          }
        }
      }
    }
    __syncthreads();
    if (seg == 0 && a.dh0) store_states(g, a.dh0 + (static_cast<int64_t>(p.b) * a.D + c) * a.N, a.N, q, on);
    store_states(dA, sums + static_cast<int64_t>(c) * a.N, a.N, q, on);
    __syncthreads();
    return;
  }

  const int tid = threadIdx.x - 256;
  Lines<InT, OutT> at(a, p, begin, tid);
  BcRows<InT, NP, TT, Wide> rows(a, p, begin, tid, true);
  const int last = begin + max(tiles - 1, 0) * TT;
  const int64_t oc = p.c0 + at.quad;
  float bias[4], skip[4], dD[4], db[4];
  params<4>(bias, a.dt_bias ? a.dt_bias + oc : nullptr, at.n4, 0.f);
  params<4>(skip, a.Dskip ? a.Dskip + oc : nullptr, at.n4, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) dD[i] = db[i] = 0.f;
  OutT* dup = static_cast<OutT*>(a.du) + p.b * a.dus.b + (last + at.row) * a.dus.t + oc;
  OutT* ddp = static_cast<OutT*>(a.ddt) + p.b * a.ddts.b + (last + at.row) * a.ddts.t + oc;
  OutT* dzp = a.z ? static_cast<OutT*>(a.dz) + p.b * a.dzs.b + (last + at.row) * a.dzs.t + oc : nullptr;
  // its sums over the four waves: element tid + 256 k of a tile's [TT][2][NP]
  constexpr int kSums = (TT * 2 * NP + 255) / 256;
  float* part[kSums];
  int sum_t[kSums];  // the token in the tile; beyond any where there is no such element
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    const int x = tid + 256 * k, t = x / (2 * NP), w = x / NP % 2, m = x % NP;
    sum_t[k] = x < TT * 2 * NP && m < a.N ? t : INT_MAX / 2;
    part[k] = a.bcpart + ((static_cast<int64_t>(p.b) * a.G + p.g) * ((a.D / a.G + CH - 1) / CH) + p.tile) * a.T * 2 * a.N +
              (static_cast<int64_t>(last + t) * 2 + w) * a.N + m;
  }

  // a tile's inputs of this thread as they come, two steps before they go into LDS (a step of the forward walk is shorter
  // than a load)
  struct Raw {
    Piece<InT, 4> u, dt, z;
    Piece<OutT, 4> dy;
    typename BcRows<InT, NP, TT, Wide>::Values bc;
  };
  Raw far[2];
  // what the way out wants of them
  struct Held {
    Piece<InT, 4> u, z;
    Piece<OutT, 4> dy;
    float dt[4], slope[4];
  };
  Held old, now, next;  // of the tile behind the walk, in the walk, before it
  const int steps = 2 * tiles;
  auto token = [&](int s) { return begin + (s < tiles ? s : steps - 1 - s) * TT; };
  // Without a branch around the loads (see load_ahead): behind the last step the last one's again, and for the forward walk
  // the last tile's dy and z, which are wanted first (z: or u), and are at hand from then on.
  const OutT* gp = at.dy + (last - begin) * a.ys.t;
  const int64_t zstride = a.z ? a.zs.t : a.us.t;
  const InT* zp = (a.z ? at.z : at.u) + (last - begin) * zstride;
  auto fetch = [&](Raw& r, int step) {
    const int s = min(step, steps - 1), t0 = token(s), n = t0 + at.row < end ? at.n4 : 0;
    const InT *u = at.u, *dt = at.dt, *z = zp;
    const OutT* dy = gp;
    if (Wide && t0 + TT > end) {  // rows behind the end: the last one instead
      const int over = max(0, t0 + at.row - (end - 1));
      u -= over * a.us.t;
      dt -= over * a.dts.t;
    }
    if (Wide && (s < tiles || t0 + TT > end)) {
      const int over = max(0, (s < tiles ? last : t0) + at.row - (end - 1));
      z -= over * zstride;
      dy -= over * a.ys.t;
    }
    load_ahead<Wide>(r.u, u, n);
    load_ahead<Wide>(r.dt, dt, n);
    load_ahead<Wide>(r.dy, dy, s < tiles ? 0 : n);
    load_ahead<Wide>(r.z, z, s < tiles ? 0 : n);
    const int dir = step + 1 < tiles ? 1 : step + 1 == tiles || step + 1 >= steps ? 0 : -1;
    rows.load(r.bc, t0, end, dir);
    if (dir > 0) {
      at.u += TT * a.us.t;
      at.dt += TT * a.dts.t;
    } else if (dir < 0) {
      at.u -= TT * a.us.t;
      at.dt -= TT * a.dts.t;
      zp -= TT * zstride;
      gp -= TT * a.ys.t;
    }
  };
  auto stage = [&](Raw& r, int s) {
    const int t0 = token(s), n = t0 + at.row < end ? at.n4 : 0;
    if (t0 + TT > end || p.nc < CH) {
      keep<Wide>(r.u, n);
      keep<Wide>(r.dy, n);
      keep<Wide>(r.z, n);
    }
    next.u = r.u;
    next.z = r.z;
    next.dy = r.dy;
    float4* to = &tile[s & 1][at.row][at.quad];
#pragma unroll
    for (int i = 0; i < 4; ++i) next.dt[i] = r.dt.get(i) + bias[i], next.slope[i] = 1.f;
    if (s < tiles) {
      if (a.softplus) {
#pragma unroll
        for (int i = 0; i < 4; ++i) next.dt[i] = softplus(next.dt[i]);
      }
      zero_from(next.dt, n);
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(to + i) = make_float2(next.dt[i], next.dt[i] * next.u.get(i));
    } else {
      float d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = next.dy.get(i);
      if (a.softplus) {
#pragma unroll
        for (int i = 0; i < 4; ++i) next.dt[i] = softplus(next.dt[i], next.slope[i]);
      }
      zero_from(next.dt, n);
      if (a.z) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] *= next.z.get(i) * sigmoid(next.z.get(i));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = make_float4(next.dt[i], next.dt[i] * next.u.get(i), d[i], 0.f);
    }
    rows.stage(r.bc, bc[s & 1], t0, end);
  };
  auto finish = [&](int s) {
    const int t0 = token(s), n = t0 + at.row < end ? at.n4 : 0;
    float o[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = tile[s & 1][at.row][at.quad + i];
      const float uu = old.u.get(i);
      float dd = old.dy.get(i);
      o[2][i] = 0.f;
      if (a.z) {
        const float x = old.z.get(i), sg = sigmoid(x), gate = x * sg;
        o[2][i] = dd * fmaf(skip[i], uu, v.z) * fmaf(gate, 1.f - sg, sg);
        dd *= gate;
      }
      o[0][i] = fmaf(old.dt[i], v.x, skip[i] * dd);
      o[1][i] = fmaf(uu, v.x, v.y * (1.f / kLog2e)) * old.slope[i];
      dD[i] = fmaf(dd, uu, dD[i]);
      db[i] += i < n ? o[1][i] : 0.f;
    }
    Piece<OutT, 4> out[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) out[k].set_all(o[k]);
    if (n > 0) {
      store<Wide>(out[0], dup, n);
      store<Wide>(out[1], ddp, n);
      if (a.z) store<Wide>(out[2], dzp, n);
    }
    dup -= TT * a.dus.t;
    ddp -= TT * a.ddts.t;
    dzp -= TT * a.dzs.t;
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      constexpr int W = TT * 2 * NP;
      const float* v = &sbc[s & 1][0][0][0][0] + (W < 256 ? tid % W : tid + 256 * k);
      const float sum = (v[0] + v[W]) + (v[2 * W] + v[3 * W]);
      if (t0 + sum_t[k] < end) *part[k] = sum;
      part[k] -= TT * 2 * a.N;
    }
  };
  if (steps) {
    fetch(far[0], 0);
    fetch(far[1], 1);
    stage(far[0], 0);
    fetch(far[0], 2);
  }
  auto step = [&](Raw& r, int s) {
    __syncthreads();
    old = now;
    now = next;
    if (s > tiles) finish(s - 1);
    if (s + 1 < steps) stage(r, s + 1);
    fetch(r, s + 3);
  };
  for (int s = 0; s < steps; s += 2) {
    step(far[1], s);
    step(far[0], s + 1);
  }
  __syncthreads();
  if (steps) {
    old = now;
    finish(steps - 1);
  }
  Piece<OutT, 4> none;
  none.zero();
  for (int64_t t = max(begin, end) + at.row; t < tokens; t += TT) {
    store<Wide>(none, static_cast<OutT*>(a.du) + p.b * a.dus.b + t * a.dus.t + oc, at.n4);
    store<Wide>(none, static_cast<OutT*>(a.ddt) + p.b * a.ddts.b + t * a.ddts.t + oc, at.n4);
    if (a.z) store<Wide>(none, static_cast<OutT*>(a.dz) + p.b * a.dzs.b + t * a.dzs.t + oc, at.n4);
  }
  // dD and ddt_bias: over the token rows
  float2* lines = reinterpret_cast<float2*>(&tile[0][0][0]);
  if (steps == 0 || ((steps - 1) & 1) == 0) lines = reinterpret_cast<float2*>(&tile[1][0][0]);  // (finish may still be reading the other)
#pragma unroll
  for (int i = 0; i < 4; ++i) lines[at.row * CH + at.quad + i] = make_float2(dD[i], db[i]);
  __syncthreads();
  if (tid < p.nc) {
    float2 s = lines[tid];
#pragma unroll
    for (int r = 1; r < TT; ++r) {
      const float2 x = lines[r * CH + tid];
      s.x += x.x;
      s.y += x.y;
    }
    sums += static_cast<int64_t>(a.D) * a.N + p.c0 + tid;
    sums[0] = s.x;
    sums[a.D] = s.y;
  }
}

// dB and dC: the sum over the tiles of channels, in their order; V neighbouring states of a token a thread.
template <typename OutT, int V>
__global__ __launch_bounds__(256) void ttt_scan_bc_sum(ScanBcSumArgs a) {
  const int64_t id = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V, each = static_cast<int64_t>(a.T) * 2 * a.N;
  const int64_t bg = id / each;
  const int64_t e = id - bg * each;
  const int b = static_cast<int>(bg / a.G), g = static_cast<int>(bg % a.G);
  if (b >= a.B) return;
  const int64_t t = e / (2 * a.N);
  const int w = static_cast<int>(e / a.N % 2), n = static_cast<int>(e % a.N);
  const int len = a.lens ? max(0, min(a.lens[b], a.T)) : a.T;
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = 0.f;
  if (t < len) {
    const float* p = a.part + bg * a.tiles * each + e;
#pragma unroll 8
    for (int k = 0; k < a.tiles; ++k) {
      if constexpr (V == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + k * each);
        s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
      } else {
        s[0] += p[k * each];
      }
    }
  }
  OutT* o = w ? static_cast<OutT*>(a.dC) + b * a.dcs.b + g * a.dcs.h + t * a.dcs.t
              : static_cast<OutT*>(a.dB) + b * a.dbs.b + g * a.dbs.h + t * a.dbs.t;
#pragma unroll
  for (int i = 0; i < V; ++i) put(o + n + i, s[i]);
}

template <typename InT, typename OutT, int NS>
hipError_t go(bool states, const ScanArgs& a, hipStream_t s) {
  const int dg = a.D / a.G;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.G * ((dg + CH - 1) / CH) * a.nseg);
  if (states) {
    if (a.wide) ttt_scan_bwd_states<InT, OutT, NS, true><<<grid, 256, 0, s>>>(a);
    else ttt_scan_bwd_states<InT, OutT, NS, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (a.wide) ttt_scan_bwd<InT, OutT, NS, true><<<grid, 512, 0, s>>>(a);
    else ttt_scan_bwd<InT, OutT, NS, false><<<grid, 512, 0, s>>>(a);
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
  const bool four = a.N % 4 == 0;
  const unsigned grid = static_cast<unsigned>((n / (four ? 4 : 1) + 255) / 256);
  if (a.out_dtype == 0) {
    if (four) ttt_scan_bc_sum<float, 4><<<grid, 256, 0, s>>>(a);
    else ttt_scan_bc_sum<float, 1><<<grid, 256, 0, s>>>(a);
  } else {
    if (four) ttt_scan_bc_sum<uint16_t, 4><<<grid, 256, 0, s>>>(a);
    else ttt_scan_bc_sum<uint16_t, 1><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace ttt
