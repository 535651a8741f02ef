// What stands around a layer's state (short convolution, selective scan, block norm): launch arguments and entry points.
#pragma once
#include "args_attn.h"

namespace ttt {

// Elements between sequences and tokens of a [B, T, D] tensor.
struct Strides2 {
  int64_t b, t;
};

struct ConvArgs {
  int B, T, D, K;
  int in_dtype, out_dtype;
  bool silu;
  bool wide;              // every address and stride is a multiple of 16 bytes, D of the elements in 16 bytes
  const void* X;          // [B, T, D]
  const float* w;         // [D, K]
  const float* bias;      // [D] or nullptr
  const void* state;      // [B, K-1, D] or nullptr (zeros)
  const int32_t* lens;    // [B] or nullptr
  void* Y;                // forward: output
  void* state_out;        // [B, K-1, D] or nullptr; decode: state itself
  Strides2 xs, ys;        // ys: Y or dY
  // backward
  const void* dY;
  const void* dstate_out; // or nullptr
  void* dX;
  void* dstate;           // or nullptr
  Strides2 dxs;
  int seg;                // tokens a thread walks
  float* part;            // [B * nparts, D * (K + 1)]: dw [D, K], then dbias [D]
  int nparts;             // partial rows a sequence
};

struct ScanArgs {
  int B, T, D, N, G;
  int in_dtype, out_dtype;
  bool softplus;
  bool wide;              // rows in pieces of 8 (or 4) elements: channels of a group and addresses fit, B and C in pieces of 4
  const void *u, *dt, *z; // [B, T, D] (z or nullptr)
  const void *Bm, *Cm;    // [B, G, T, N]
  const float* A;         // [D, N]
  const float* Dskip;     // [D] or nullptr
  const float* dt_bias;   // [D] or nullptr
  const float* h0;        // [B, D, N] or nullptr
  const int32_t* lens;
  void* y;
  float* h_final;         // [B, D, N]; decode: the state, in place
  Strides2 us, dts, zs, ys;
  Strides3 bs, cs;
  int nseg, seglen;       // segments of a sequence walked at the same time, tokens of each (a multiple of the tile)
  float* hseg;            // [B, nseg, D, N] (nseg > 1): slot 0 h0, slot s what segment s - 1 adds from a zero state
  float* sseg;            // [B, nseg, D] (nseg > 1): sum of dt of segment s
  // backward
  const void* dy;
  const float* dh_final;  // [B, D, N] or nullptr
  void *du, *ddt, *dz;
  Strides2 dus, ddts, dzs;
  float* dh0;             // [B, D, N] or nullptr
  float* gseg;            // [B, nseg, D, N] (nseg > 1): what the segment's dy add to the gradient of its start state
  float* ckpt;            // [B, chunks, D, N]: the state before each chunk
  float* bcpart;          // [B, G, tiles, T, 2, N]: dB, dC of each tile of channels
  float* part;            // [B * nseg, D * (N + 2)]: dA [D, N], dD [D], ddt_bias [D]
  int chunks;             // per sequence
};

// The sums behind the walks of ttt_selective_scan_bwd: dB, dC over the tiles of channels.
struct ScanBcSumArgs {
  int B, T, N, G, tiles, out_dtype;
  const int32_t* lens;
  const float* part;
  void *dB, *dC;
  Strides3 dbs, dcs;
};

struct NormArgs {
  int B, T, D;
  int in_dtype, res_dtype;
  bool layer, gate_first, wide;
  float eps;
  const void *X, *Z, *res;  // Z, res or nullptr
  const float *alpha, *gamma_post, *beta_post, *gamma_pre, *beta_pre;  // [D] or nullptr
  const int32_t* lens;
  void *S, *Y;              // forward, each or nullptr
  Strides2 xs, zs, rs, ss, ys;
  // backward: ss, ys are the strides of dS, dY
  const void *dS, *dY;      // each or nullptr
  void *dX, *dZ, *dres;     // dZ, dres or nullptr
  Strides2 dxs, dzs, drs;
  float* part;              // [blocks, 5 D]: dalpha, dgamma_post, dbeta_post, dgamma_pre, dbeta_pre
  int blocks;
};

// out[c] = sum over rows of part[row * ld + c], in up to five pieces of neighbouring columns.
struct RowSumArgs {
  const float* part;
  int64_t ld;
  int rows;
  int64_t n[5];             // columns of each piece
  float* out[5];            // or nullptr: not wanted
};

constexpr int kScanCh = 64;     // channels of a workgroup
constexpr int kScanTile = 32;   // tokens staged at a time

int scan_states(int N);         // states that each of a channel's four lanes holds; 0: not supported
int scan_chunk(int N);          // tokens between checkpoints
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_decode(const ConvArgs& a, hipStream_t s);
hipError_t launch_scan_states(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bwd_states(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bc_sum(const ScanBcSumArgs& a, hipStream_t s);
hipError_t launch_scan_decode(const ScanArgs& a, hipStream_t s);
int norm_max_d();
int norm_teams(int D);          // rows a workgroup of the backward works on at a time
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s);
hipError_t launch_row_sum(const RowSumArgs& a, hipStream_t s);

}  // namespace ttt
