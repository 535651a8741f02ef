// Linear attention with a decay per head, token by token: the state carried in
// place, as generation needs it.
//
// Pages: [TTT] = news article "大模型最强架构TTT问世！斯坦福UCSD等5年磨一剑，一夜推翻Transformer"
// (aharts.cn / itmax.cn), part 03 §8 (linear attention as a state of d x d) and
// part 04 §3 (generation is sequential).
//
//   W <- lambda W + v_t k_t^T,   z_t = scale W q_t
// A token reads and writes the whole state, 8 d^2 bytes, against 4 d^2 flops: the
// kernel is a copy of the state with the arithmetic on the way.  One workgroup of
// 4d threads per (sequence, head); thread (i = tid / 4, n = tid % 4) owns W[i][16a +
// 4n .. 16a + 4n + 3], so that each load of a wave covers 16 rows x 64 bytes, and the
// row's product with q is finished by a quad sum.  q, k and v go through LDS as
// fp32; with rotary positions q and k are turned there, so that a generated token
// is one launch.  Measured on MI355X for B512 H32 d64 bf16 with rotary positions: 106 us, 5.15 TB/s of 545 MB
// (a copy of 512 MiB reaches 5.3 TB/s); B16 H32: 5.6 us, most of it the launch and three dependent loads.
#include <type_traits>

#include "args_attn.h"
#include "mfma_common.h"
#include "rope.h"

namespace ttt {
namespace {

constexpr int TT = 8;  // tokens staged at a time

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(uint16_t x) { return bf16_bits_to_f32(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = f32_to_bf16_bits(x); }

__device__ __forceinline__ float quad_sum(float x) {
  x += mfma::dpp_mov<0xB1>(x);
  x += mfma::dpp_mov<0x4E>(x);
  return x;
}

// element c of a row, turned to its position
template <typename InT>
__device__ __forceinline__ float rotated(const InT* p, int c, const Rope& r, int64_t pos) {
  const float x = as_f32(p[c]);
  if (!r.freqs || c >= r.rot) return x;
  const int half = r.rot / 2;
  const int i = r.interleaved ? c >> 1 : (c < half ? c : c - half);
  const bool second = r.interleaved ? (c & 1) : c >= half;
  const float other = as_f32(p[r.interleaved ? c ^ 1 : (second ? c - half : c + half)]);
  float cs, sn;
  rope_angle(pos, r.freqs[i], cs, sn);
  return r.scale * (second ? fmaf(other, sn, x * cs) : fmaf(-other, sn, x * cs));
}

template <int D, typename InT, typename OutT>
__global__ __launch_bounds__(4 * D) void ttt_attn_decode(AttnDecodeArgs a) {
  constexpr int NB = D / 16;
  __shared__ __align__(16) float qs[TT][D], ks[TT][D];
  __shared__ float vs[TT][D];
  const int tid = threadIdx.x, i = tid >> 2, n = tid & 3;
  const int chain = blockIdx.x;
  const int b = chain / a.H, h = chain % a.H, hk = h / a.group;
  // lambda x as m x + a x: near 1 as 1 + expm1(log lambda), so that thousands of tokens do not add up the
  // rounding of lambda
  const float lam = expf(a.log_decay[h]);
  const float m = lam > 0.5f ? 1.f : 0.f, em = lam > 0.5f ? expm1f(a.log_decay[h]) : lam;
  int len = a.T;
  if (a.lens) len = max(0, min(a.lens[b], a.T));
  const InT* q = static_cast<const InT*>(a.Q) + b * a.qs.b + h * a.qs.h;
  const InT* k = static_cast<const InT*>(a.K) + b * a.ks.b + hk * a.ks.h;
  const InT* v = static_cast<const InT*>(a.V) + b * a.vs.b + hk * a.vs.h;
  OutT* z = static_cast<OutT*>(a.Z) + b * a.os.b + h * a.os.h;
  float4* wp = reinterpret_cast<float4*>(a.W + (static_cast<int64_t>(chain) * D + i) * D + 4 * n);

  if (len > 0) {
    float4 w[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) w[c] = wp[4 * c];
    for (int t0 = 0; t0 < len; t0 += TT) {
      const int nt = min(TT, len - t0);
      if (t0) __syncthreads();
      for (int e = tid; e < nt * D; e += 4 * D) {
        const int t = e / D, c = e % D;
        const int64_t at = t0 + t;
        const int64_t pos = a.rope.freqs ? rope_pos(a.rope, b, t0 + t) : 0;
        qs[t][c] = rotated(q + at * a.qs.t, c, a.rope, pos) * a.scale;
        ks[t][c] = rotated(k + at * a.ks.t, c, a.rope, pos);
        vs[t][c] = as_f32(v[at * a.vs.t + c]);
      }
      __syncthreads();
      for (int t = 0; t < nt; ++t) {
        const float vi = vs[t][i];
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < NB; ++c) {
          const float4 kc = *reinterpret_cast<const float4*>(&ks[t][16 * c + 4 * n]);
          const float4 qc = *reinterpret_cast<const float4*>(&qs[t][16 * c + 4 * n]);
          w[c].x = fmaf(vi, kc.x, fmaf(w[c].x, em, w[c].x * m));
          w[c].y = fmaf(vi, kc.y, fmaf(w[c].y, em, w[c].y * m));
          w[c].z = fmaf(vi, kc.z, fmaf(w[c].z, em, w[c].z * m));
          w[c].w = fmaf(vi, kc.w, fmaf(w[c].w, em, w[c].w * m));
          sum = fmaf(w[c].x, qc.x, sum);
          sum = fmaf(w[c].y, qc.y, sum);
          sum = fmaf(w[c].z, qc.z, sum);
          sum = fmaf(w[c].w, qc.w, sum);
        }
        sum = quad_sum(sum);
        if (n == 0) put(z + (t0 + t) * a.os.t + i, sum);
      }
    }
#pragma unroll
    for (int c = 0; c < NB; ++c) wp[4 * c] = w[c];
  }
  for (int t = len + tid / D; t < a.T; t += 4)  // four rows of D a step
    put(z + t * a.os.t + tid % D, 0.f);
}

template <int D>
hipError_t go(const AttnDecodeArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H), block(4 * D);
  const bool inf = a.in_dtype == 0, outf = a.out_dtype == 0;
  if (inf && outf) ttt_attn_decode<D, float, float><<<grid, block, 0, s>>>(a);
  else if (inf) ttt_attn_decode<D, float, uint16_t><<<grid, block, 0, s>>>(a);
  else if (outf) ttt_attn_decode<D, uint16_t, float><<<grid, block, 0, s>>>(a);
  else ttt_attn_decode<D, uint16_t, uint16_t><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t s) {
  switch (a.d) {
    case 16: return go<16>(a, s);
    case 32: return go<32>(a, s);
    case 64: return go<64>(a, s);
    case 128: return go<128>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ttt
