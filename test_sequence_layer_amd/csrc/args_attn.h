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

// Forward: Z and the last state.
struct AttnArgs {
  int B, H, T, d;
  int group;             // query heads per key / value head
  int nseg, seglen;      // segments per sequence, tokens per segment (a multiple of the chunk)
  bool carried;          // loc holds the states themselves, else what each segment adds to them
  int in_dtype, out_dtype;
  const void* Q;         // by query head
  const void* K;         // by key / value head
  const void* V;
  Strides3 qs, ks, vs, zs;
  const float* log_decay;  // [H]
  float scale;
  const float* W0;       // initial state or nullptr (zero)
  int64_t w0_bstride;
  const int32_t* lens;   // [B] or nullptr (every sequence has T tokens)
  float* loc;            // [B * H, nseg, d, d] (nseg > 1): end states of segments 0 .. nseg-2, then W0
  void* Z;
  float* W_final;        // [B, H, d, d]
};

// Backward: three walks for each (sequence, head) segment, dQ from the first token to
// the last, dK and dV from the last to the first (their segments are counted from there).
struct AttnBwdArgs {
  int B, H, T, d;
  int group;
  int nseg, seglen;
  bool carried;
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
  float* loc;            // [B * H, nseg, 3, d, d] (nseg > 1): end values of segments 0 .. nseg-2 of W^T and
                         // dW^T/dlog_decay, and of G^T
  double* dgpart;        // [B * H, nseg] (nseg > 1)
  void* dQ;
  void* dK;              // by key / value head, or fp32 [B, H, T, d] in the workspace where group > 1
  void* dV;
  Strides3 dqs, dks, dvs;
  bool parts;            // dK, dV go to the workspace, one fp32 part per query head
  float* dg;             // [B, H]
  float* dW0;            // [B, H, d, d]
};

// Segments' own states -> the states at their ends, in place: s_c <- lambda^seglen s_{c-1} + s_c.
struct AttnCarryArgs {
  int64_t chains;
  int H, d, nseg, seglen;
  bool backward;           // three matrices a segment: W^T, dW^T/dlog_decay, G^T; else one
  const float* log_decay;
  float* loc;
};

// What the walks leave in parts: dK, dV of shared heads (the sum over their query heads) and the decay's
// gradient (the sum over segments).
struct AttnSumArgs {
  int B, Hkv, T, d, group, nseg, out_dtype;
  const float* dk_parts;  // [B, Hkv * group, T, d], or nullptr
  const float* dv_parts;
  void* dK;
  void* dV;
  Strides3 dks, dvs;
  const double* dgpart;   // [B * Hkv * group, nseg], or nullptr
  float* dg;
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
int attn_segments(int64_t chains, int T, int d, bool wide, bool backward);
hipError_t launch_attn_states(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_carry(const AttnCarryArgs& a, hipStream_t s);
hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_bwd_states(const AttnBwdArgs& a, hipStream_t s);
hipError_t launch_attn_bwd(const AttnBwdArgs& a, hipStream_t s);
hipError_t launch_attn_sum(const AttnSumArgs& a, hipStream_t s);
hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t s);
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t s);
const char* rotary_name(const RotaryArgs& a);  // the way launch_rotary takes

}  // namespace ttt
