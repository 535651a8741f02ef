// Linear attention with a decay per head: launch arguments and entry points.
#pragma once
#include "ttt_common.h"

namespace ttt {

// Elements between sequences, heads and tokens of a [B, heads, T, d] tensor.
struct Strides3 {
  int64_t b, h, t;
};

// Rotary positions: pair i of the first rot elements of a row turned by position * freqs[i], times scale.
struct Rope {
  const int64_t* pos;    // pos[b * pos_b + t * pos_t], or nullptr for 0
  int64_t pos_b, pos_t;  // (pos_t = 0: the position of the first token, the others follow it)
  int64_t pos0;          // added to every position
  const double* freqs;   // [rot / 2], radians per position
  int rot;
  bool interleaved;      // pairs (2i, 2i+1), else (i, i + rot / 2)
  float scale;
};

// One recurrence over the tokens of every (sequence, head):
//   S_t = lambda S_{t-1} + V_t Y_t^T,   O_t = scale S_t X_t      (S: d x d, row = element of V)
// The forward has X, Y, V = Q, K, V; dQ has X, Y, V = dZ, V, K (S is then W^T).
struct AttnArgs {
  int B, H, T, d;
  int group;             // query heads per key / value head
  int nseg, seglen;      // segments per sequence, tokens per segment (a multiple of the chunk)
  int x_dtype, in_dtype, out_dtype;
  const void* X;         // by query head
  const void* Y;         // by key / value head
  const void* V;         // by key / value head
  Strides3 xs, ys, vs, os;
  const float* log_decay;  // [H]
  float scale;
  const float* S0;       // initial state or nullptr (zero)
  int64_t s0_bstride;
  bool transposed;       // the walk reads S0 and loc as S^T
  const int32_t* lens;   // [B] or nullptr (every sequence has T tokens)
  float* loc;            // [B * H, nseg, d, d] (nseg > 1): end states of segments 0 .. nseg-2, then S0
  void* O;
  float* S_final;        // [B, H, d, d] or nullptr
};

// The reverse recurrence of the backward: with G_t the gradient of the state after token t,
//   G_{t-1} = lambda (G_t + scale dZ_t Q_t^T) ...,  dV_t = G_t K_t,  dK_t = G_t^T V_t
struct AttnBwdArgs {
  int B, H, T, d;
  int group;
  int nseg, seglen;
  int in_dtype, out_dtype;
  const void* Q;
  const void* K;
  const void* V;
  const void* dZ;
  Strides3 qs, ks, vs, zs;
  const float* log_decay;
  float scale;
  const float* W0;       // or nullptr
  int64_t w0_bstride;
  const int32_t* lens;
  const float* dWf;      // [B, H, d, d] or nullptr
  float* gloc;           // [B * H, nseg, 2, d, d]: each segment's G and dG/dlog_decay from zero (nseg > 1)
  double* dgpart;        // [B * H, nseg] (nseg > 1)
  void* dK;              // by key / value head, or fp32 [B, H, T, d] in the workspace where group > 1
  void* dV;
  Strides3 dks, dvs;
  bool parts;            // dK, dV go to the workspace, one fp32 part per query head
  float* dg;             // [B, H]
  float* dW0;            // [B, H, d, d]
};

// dK, dV of a shared head: the sum of its query heads' parts.
struct AttnSumArgs {
  int B, Hkv, T, d, group, out_dtype;
  const float* parts;    // [B, Hkv * group, T, d]
  void* out;
  Strides3 os;
};

// One or a few tokens, the state carried in place.
struct AttnDecodeArgs {
  int B, H, T, d;
  int group;
  int in_dtype, out_dtype;
  const void* Q;
  const void* K;
  const void* V;
  Strides3 qs, ks, vs, os;
  const float* log_decay;
  float scale;
  const int32_t* lens;
  float* W;
  void* Z;
  Rope rope;             // of q and k (rope.freqs == nullptr: none)
};

// q and k turned by their positions.
struct RotaryArgs {
  int B, H, Hkv, T, d;
  int dtype;
  const void* q;         // [B, H, T, d]
  const void* k;         // [B, Hkv, T, d] (Hkv may be 0)
  void* qo;
  void* ko;
  Strides3 qs, ks, qos, kos;
  Rope rope;
  bool inverse;          // turn back (the gradient)
  bool in_place;         // the rest of each row is where it belongs
};

constexpr int kAttnChunk = 32;  // tokens per chunk of the chunked form

bool attn_supported(int d);
int attn_segments(int64_t chains, int T, int d);
hipError_t launch_attn_states(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_bwd_states(const AttnBwdArgs& a, hipStream_t s);
hipError_t launch_attn_bwd(const AttnBwdArgs& a, hipStream_t s);
hipError_t launch_attn_bwd_dg(const AttnBwdArgs& a, hipStream_t s);
hipError_t launch_attn_sum(const AttnSumArgs& a, hipStream_t s);
hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t s);
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t s);

}  // namespace ttt
