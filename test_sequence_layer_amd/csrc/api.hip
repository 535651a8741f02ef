// C ABI of libttt.so: argument validation and kernel dispatch.
// The entry points and their contracts are documented in include/ttt.h.
#include <limits.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>

#include "../../include/ttt.h"
#include "ttt_internal.h"

// Scratch of ttt_linear_fwd_chunked_noalloc (chunk maps and start states):
// one copy per GPU the library runs on, held until the process ends.  In host
// code this name stands for a host-side shadow, not device memory: host code
// uses only the per-device address scratch_address() looks up.
__device__ __align__(256) unsigned char scratch[TTT_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_dev[kMaxDevices];  // device address of each GPU's `scratch` (nullptr: not looked up yet)

// The device address of `scratch` on the GPU that owns `stream`, looked up once
// per device (hipGetSymbolAddress with that device current) and kept.
hipError_t scratch_address(hipStream_t stream, void** out) {
  int dev = 0;
  hipError_t e = hipStreamGetDevice(stream, &dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_dev[dev]) {
    int cur = 0;
    if ((e = hipGetDevice(&cur)) != hipSuccess) return e;
    if (cur != dev && (e = hipSetDevice(dev)) != hipSuccess) return e;
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (cur != dev) {
      const hipError_t back = hipSetDevice(cur);
      if (e == hipSuccess) e = back;
    }
    if (e != hipSuccess) return e;
    if (!p) return hipErrorInvalidSymbol;
    g_scratch_dev[dev] = p;
  }
  *out = g_scratch_dev[dev];
  return hipSuccess;
}

struct Range {
  const void* p;
  int64_t bytes;
};

bool overlaps(Range a, Range b) {
  if (a.bytes <= 0 || b.bytes <= 0 || a.p == nullptr || b.p == nullptr) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// a*b*c*... <= limit without overflow (all factors >= 0)
bool mul_ok(int64_t& acc, int64_t f, int64_t limit = (int64_t(1) << 46)) {
  if (f < 0) return false;
  if (f != 0 && acc > limit / f) return false;
  acc *= f;
  return true;
}

int64_t dtype_size(int32_t dt) { return dt == TTT_BF16 ? 2 : 4; }
bool dtype_ok(int32_t dt) { return dt == TTT_F32 || dt == TTT_BF16; }

// element extent of eta (last index + 1) for B, H, T >= 1
int64_t eta_extent(int64_t B, int64_t H, int64_t T, int64_t sb, int64_t sh, int64_t st) {
  return (B - 1) * sb + (H - 1) * sh + (T - 1) * st + 1;
}

enum Kernel { K_NONE, K_GENERIC, K_MFMA, K_MFMA32, K_PRIMAL };

constexpr uint32_t kRowFlags = TTT_FLAG_ROWS1 | TTT_FLAG_ROWS2 | TTT_FLAG_ROWS4;

Kernel pick_linear(const ttt::LinearArgs& a, uint32_t flags) {
  if (flags & TTT_FLAG_PRIMAL) return ttt::linear_primal_supported(a.d) ? K_PRIMAL : K_NONE;
  if (flags & TTT_FLAG_GENERIC) return ttt::linear_generic_supported(a.d, a.b) ? K_GENERIC : K_NONE;
  if (ttt::linear_mfma_supported(a)) return K_MFMA;
  if (flags & kRowFlags) return K_NONE;  // row blocks exist only in the bf16 matrix-core kernel
  if (ttt::linear_mfma_f32_supported(a)) return K_MFMA32;
  if (ttt::linear_generic_supported(a.d, a.b)) return K_GENERIC;
  return K_NONE;
}

// Row blocks per (sequence, head, chunk) of the matrix-core forward: the
// flag's count, else 1 (see TTT_FLAG_ROWS1 in ttt.h for why).
int row_blocks(uint32_t flags) {
  if (flags & TTT_FLAG_ROWS4) return 4;
  if (flags & TTT_FLAG_ROWS2) return 2;
  return 1;
}

ttt::LinearArgs make_linear_args(const ttt_linear_desc* d, const void* Q, const void* K, const void* V,
                                 const float* W0, const float* eta, const void* Z, const float* Wf) {
  ttt::LinearArgs a;
  a.B = d->B; a.H = d->H; a.T = d->T; a.d = d->d; a.b = d->b;
  a.in_dtype = d->in_dtype; a.out_dtype = d->out_dtype;
  a.Q = Q; a.K = K; a.V = V; a.W0 = W0; a.w0_bstride = d->w0_batch_stride;
  a.eta = eta; a.esb = d->eta_stride_b; a.esh = d->eta_stride_h; a.est = d->eta_stride_t;
  a.Z = const_cast<void*>(Z); a.Wf = const_cast<float*>(Wf);
  a.nchunk = 1; a.mb1 = d->T / 16; a.Wstart = nullptr; a.maps = nullptr;
  a.gamma = nullptr; a.beta = nullptr; a.eps = 0.f;
  a.Esave = nullptr;
  a.rb = row_blocks(d->flags);
  return a;
}

ttt_status validate_linear(const ttt_linear_desc* d, const void* Q, const void* K, const void* V,
                           const float* W0, const float* eta, const void* Z, const float* Wf,
                           Kernel* which) {
  if (which) *which = K_NONE;
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->H < 0 || d->T < 0 || d->d < 1 || d->b < 1) return TTT_ERR_SHAPE;
  if (d->T % d->b != 0) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype)) return TTT_ERR_DTYPE;
  if (d->flags & ~(static_cast<uint32_t>(TTT_FLAG_GENERIC | TTT_FLAG_PRIMAL) | kRowFlags)) return TTT_ERR_FLAGS;
  if ((d->flags & TTT_FLAG_GENERIC) && (d->flags & TTT_FLAG_PRIMAL)) return TTT_ERR_FLAGS;
  {
    const uint32_t rows = d->flags & kRowFlags;
    if (rows & (rows - 1)) return TTT_ERR_FLAGS;  // more than one row-block count
    if (rows && (d->flags & (TTT_FLAG_GENERIC | TTT_FLAG_PRIMAL))) return TTT_ERR_FLAGS;
  }
  int64_t chains = 1, tok = 1, wel = 1;
  if (!mul_ok(chains, d->B) || !mul_ok(chains, d->H) || chains > INT_MAX) return TTT_ERR_SHAPE;
  if (chains * row_blocks(d->flags) > INT_MAX) return TTT_ERR_SHAPE;  // workgroups of one launch
  tok = chains;
  if (!mul_ok(tok, d->T) || !mul_ok(tok, d->d)) return TTT_ERR_SHAPE;
  wel = chains;
  if (!mul_ok(wel, d->d) || !mul_ok(wel, d->d)) return TTT_ERR_SHAPE;
  const int64_t hdd = static_cast<int64_t>(d->H) * d->d * d->d;
  if (d->w0_batch_stride != 0 && d->w0_batch_stride != hdd) return TTT_ERR_STRIDE;
  if (d->eta_stride_b < 0 || d->eta_stride_h < 0 || d->eta_stride_t < 0) return TTT_ERR_STRIDE;

  ttt::LinearArgs a = make_linear_args(d, Q, K, V, W0, eta, Z, Wf);
  const Kernel k = pick_linear(a, d->flags);
  if (k == K_NONE) return TTT_ERR_UNSUPPORTED;
  if (chains == 0) {
    if (which) *which = k;
    return TTT_OK;
  }

  // pointers
  if (!W0 || !Wf) return TTT_ERR_NULL;
  if (tok > 0 && (!Q || !K || !V || !Z || !eta)) return TTT_ERR_NULL;
  if (!aligned(W0, 16) || !aligned(Wf, 16)) return TTT_ERR_ALIGN;
  if (tok > 0 && (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(Z, 16) || !aligned(eta, 4)))
    return TTT_ERR_ALIGN;

  // extents and aliasing
  const int64_t in_b = tok * dtype_size(d->in_dtype);
  const int64_t z_b = tok * dtype_size(d->out_dtype);
  const int64_t wf_b = wel * 4;
  const int64_t w0_b = (d->w0_batch_stride == 0 ? hdd : wel) * 4;
  const int64_t eta_b =
      tok > 0 ? eta_extent(d->B, d->H, d->T, d->eta_stride_b, d->eta_stride_h, d->eta_stride_t) * 4 : 0;
  const Range rq{Q, in_b}, rk{K, in_b}, rv{V, in_b}, re{eta, eta_b}, rw0{W0, w0_b};
  const Range rz{Z, z_b}, rwf{Wf, wf_b};
  for (Range in : {rq, rk, rv, re, rw0})
    if (overlaps(rz, in)) return TTT_ERR_ALIAS;
  if (overlaps(rz, rwf)) return TTT_ERR_ALIAS;
  for (Range in : {rq, rk, rv, re})
    if (overlaps(rwf, in)) return TTT_ERR_ALIAS;
  if (overlaps(rwf, rw0)) {
    const bool inplace = static_cast<const void*>(Wf) == static_cast<const void*>(W0) && d->w0_batch_stride == hdd;
    if (!inplace) return TTT_ERR_ALIAS;
  }
  if (which) *which = k;
  return TTT_OK;
}

ttt::PrimalArgs make_primal_args_fwd(const ttt_linear_desc* d, const void* Q, const void* K, const void* V,
                                     const float* W0, const float* eta, void* Z, float* Wf) {
  ttt::PrimalArgs a;
  a.B = d->B; a.H = d->H; a.T = d->T; a.d = d->d; a.b = d->b;
  a.in_dtype = d->in_dtype; a.out_dtype = d->out_dtype;
  a.Q = Q; a.K = K; a.V = V;
  a.W_in = W0; a.Wb_in = W0; a.w_in_bstride = d->w0_batch_stride;
  a.eta = eta; a.esb = d->eta_stride_b; a.esh = d->eta_stride_h; a.est = d->eta_stride_t;
  a.Z = Z; a.W_out = Wf; a.Wb_out = nullptr; a.pos = 0;
  a.gamma = nullptr; a.beta = nullptr; a.eps = 0.f;
  return a;
}

ttt_status validate_decode(const ttt_linear_desc* d, const void* Q, const void* K, const void* V, const float* eta,
                           const void* Z, const float* W, const float* Wb, int64_t pos) {
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->H < 0 || d->T < 0 || d->d < 1 || d->b < 1) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype)) return TTT_ERR_DTYPE;
  if (d->flags != 0) return TTT_ERR_FLAGS;
  if (pos < 0) return TTT_ERR_POS;
  if (d->w0_batch_stride != 0) return TTT_ERR_STRIDE;
  if (d->eta_stride_b < 0 || d->eta_stride_h < 0 || d->eta_stride_t < 0) return TTT_ERR_STRIDE;
  int64_t chains = 1, tok = 1, wel = 1;
  if (!mul_ok(chains, d->B) || !mul_ok(chains, d->H) || chains > INT_MAX) return TTT_ERR_SHAPE;
  tok = chains;
  if (!mul_ok(tok, d->T) || !mul_ok(tok, d->d)) return TTT_ERR_SHAPE;
  wel = chains;
  if (!mul_ok(wel, d->d) || !mul_ok(wel, d->d)) return TTT_ERR_SHAPE;
  if (!ttt::linear_primal_supported(d->d)) return TTT_ERR_UNSUPPORTED;
  if (chains == 0) return TTT_OK;
  if (!W || !Wb) return TTT_ERR_NULL;
  if (tok > 0 && (!Q || !K || !V || !Z || !eta)) return TTT_ERR_NULL;
  if (!aligned(W, 16) || !aligned(Wb, 16)) return TTT_ERR_ALIGN;
  if (tok > 0 && (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(Z, 16) || !aligned(eta, 4)))
    return TTT_ERR_ALIGN;
  const int64_t in_b = tok * dtype_size(d->in_dtype);
  const int64_t z_b = tok * dtype_size(d->out_dtype);
  const int64_t w_b = wel * 4;
  const int64_t eta_b =
      tok > 0 ? eta_extent(d->B, d->H, d->T, d->eta_stride_b, d->eta_stride_h, d->eta_stride_t) * 4 : 0;
  const Range rq{Q, in_b}, rk{K, in_b}, rv{V, in_b}, re{eta, eta_b}, rz{Z, z_b}, rw{W, w_b}, rwb{Wb, w_b};
  for (Range out : {rz, rw, rwb})
    for (Range in : {rq, rk, rv, re})
      if (overlaps(out, in)) return TTT_ERR_ALIAS;
  if (overlaps(rz, rw) || overlaps(rz, rwb) || overlaps(rw, rwb)) return TTT_ERR_ALIAS;
  return TTT_OK;
}

// Layer-norm parameters: finite eps >= 0, gamma and beta [H, d] fp32, non-NULL,
// 4-byte aligned, overlapping none of the outputs.
ttt_status check_ln(int64_t chains, int64_t H, int64_t d, const float* gamma, const float* beta, float eps,
                    std::initializer_list<Range> outs) {
  if (!(eps >= 0.f) || eps > 1e30f) return TTT_ERR_SHAPE;
  if (chains == 0) return TTT_OK;
  if (!gamma || !beta) return TTT_ERR_NULL;
  if (!aligned(gamma, 4) || !aligned(beta, 4)) return TTT_ERR_ALIGN;
  const int64_t hd_b = H * d * 4;
  for (Range out : outs)
    for (Range in : {Range{gamma, hd_b}, Range{beta, hd_b}})
      if (overlaps(out, in)) return TTT_ERR_ALIAS;
  return TTT_OK;
}

ttt_status check_ln_params(const ttt_linear_desc* d, const float* gamma, const float* beta, float eps,
                           std::initializer_list<Range> outs) {
  return check_ln(static_cast<int64_t>(d->B) * d->H, d->H, d->d, gamma, beta, eps, outs);
}

ttt_status validate_ln_decode(const ttt_linear_desc* d, const void* Q, const void* K, const void* V,
                              const float* eta, const float* gamma, const float* beta, float eps, const void* Z,
                              const float* W, const float* Wb, int64_t pos) {
  const ttt_status st = validate_decode(d, Q, K, V, eta, Z, W, Wb, pos);
  if (st != TTT_OK) return st;
  const int64_t chains = static_cast<int64_t>(d->B) * d->H;
  const int64_t w_b = chains * d->d * d->d * 4;
  return check_ln_params(d, gamma, beta, eps,
                         {Range{Z, chains * d->T * d->d * dtype_size(d->out_dtype)}, Range{W, w_b}, Range{Wb, w_b}});
}

ttt::PrimalArgs make_decode_args(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                                 const float* eta, void* Z, float* W, float* Wb, int64_t pos) {
  ttt::PrimalArgs a;
  a.B = desc->B; a.H = desc->H; a.T = desc->T; a.d = desc->d; a.b = desc->b;
  a.in_dtype = desc->in_dtype; a.out_dtype = desc->out_dtype;
  a.Q = Q; a.K = K; a.V = V;
  a.W_in = W; a.Wb_in = Wb; a.w_in_bstride = static_cast<int64_t>(desc->H) * desc->d * desc->d;
  a.eta = eta; a.esb = desc->eta_stride_b; a.esh = desc->eta_stride_h; a.est = desc->eta_stride_t;
  a.Z = Z; a.W_out = W; a.Wb_out = Wb; a.pos = pos;
  a.gamma = nullptr; a.beta = nullptr; a.eps = 0.f;
  return a;
}

// ----------------------------------------------------------- backward --

enum BwdKernel { KB_NONE, KB_GENERIC, KB_MFMA };

ttt::BwdArgs make_bwd_args(const ttt_linear_desc* d, const void* Q, const void* K, const float* eta,
                           const float* Wf, const float* E, const void* dZ, const float* dWf, void* dQ, void* dK,
                           void* dV, float* deta, float* dW0) {
  ttt::BwdArgs a;
  a.B = d->B; a.H = d->H; a.T = d->T; a.d = d->d; a.b = d->b;
  a.in_dtype = d->in_dtype; a.out_dtype = d->out_dtype;
  a.Q = Q; a.K = K;
  a.eta = eta; a.esb = d->eta_stride_b; a.esh = d->eta_stride_h; a.est = d->eta_stride_t;
  a.Wf = Wf; a.E = E; a.dZ = dZ; a.dWf = dWf;
  a.dQ = dQ; a.dK = dK; a.dV = dV; a.deta = deta; a.dW0 = dW0;
  a.V = nullptr; a.gamma = nullptr; a.beta = nullptr; a.eps = 0.f; a.dgamma = nullptr; a.dbeta = nullptr;
  return a;
}

BwdKernel pick_bwd(const ttt::BwdArgs& a, uint32_t flags) {
  if (!(flags & TTT_FLAG_GENERIC) && ttt::linear_bwd_mfma_supported(a)) return KB_MFMA;
  if (ttt::linear_bwd_generic_supported(a.d, a.b)) return KB_GENERIC;
  return KB_NONE;
}

ttt_status validate_bwd(const ttt_linear_desc* d, const void* Q, const void* K, const float* eta, const float* Wf,
                        const float* E, const void* dZ, const float* dWf, const void* dQ, const void* dK,
                        const void* dV, const float* deta, const float* dW0, BwdKernel* which) {
  if (which) *which = KB_NONE;
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->H < 0 || d->T < 0 || d->d < 1 || d->b < 1) return TTT_ERR_SHAPE;
  if (d->T % d->b != 0) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype)) return TTT_ERR_DTYPE;
  if (d->flags & ~static_cast<uint32_t>(TTT_FLAG_GENERIC)) return TTT_ERR_FLAGS;
  if (d->w0_batch_stride != 0 && d->w0_batch_stride != static_cast<int64_t>(d->H) * d->d * d->d)
    return TTT_ERR_STRIDE;
  if (d->eta_stride_b < 0 || d->eta_stride_h < 0 || d->eta_stride_t < 0) return TTT_ERR_STRIDE;
  int64_t chains = 1, tok = 1, wel = 1;
  if (!mul_ok(chains, d->B) || !mul_ok(chains, d->H) || chains > INT_MAX) return TTT_ERR_SHAPE;
  tok = chains;
  if (!mul_ok(tok, d->T) || !mul_ok(tok, d->d)) return TTT_ERR_SHAPE;
  wel = chains;
  if (!mul_ok(wel, d->d) || !mul_ok(wel, d->d)) return TTT_ERR_SHAPE;
  const ttt::BwdArgs a = make_bwd_args(d, Q, K, eta, Wf, E, dZ, dWf, nullptr, nullptr, nullptr, nullptr, nullptr);
  const BwdKernel k = pick_bwd(a, d->flags);
  if (k == KB_NONE) return TTT_ERR_UNSUPPORTED;
  if (chains == 0) {
    if (which) *which = k;
    return TTT_OK;
  }
  if (!Wf || !dW0) return TTT_ERR_NULL;
  if (tok > 0 && (!Q || !K || !eta || !E || !dZ || !dQ || !dK || !dV || !deta)) return TTT_ERR_NULL;
  if (!aligned(Wf, 16) || !aligned(dW0, 16) || (dWf && !aligned(dWf, 16))) return TTT_ERR_ALIGN;
  if (tok > 0) {
    for (const void* p : {Q, K, static_cast<const void*>(E), dZ, dQ, dK, dV})
      if (!aligned(p, 16)) return TTT_ERR_ALIGN;
    if (!aligned(eta, 4) || !aligned(deta, 4)) return TTT_ERR_ALIGN;
  }
  const int64_t in_b = tok * dtype_size(d->in_dtype);
  const int64_t g_b = tok * dtype_size(d->out_dtype);
  const int64_t w_b = wel * 4;
  const int64_t eta_b =
      tok > 0 ? eta_extent(d->B, d->H, d->T, d->eta_stride_b, d->eta_stride_h, d->eta_stride_t) * 4 : 0;
  const int64_t deta_b = tok > 0 ? chains * d->T * 4 : 0;
  const Range ins[] = {{Q, in_b}, {K, in_b}, {eta, eta_b}, {Wf, w_b}, {E, tok * 4}, {dZ, g_b}, {dWf, w_b}};
  const Range outs[] = {{dQ, g_b}, {dK, g_b}, {dV, g_b}, {deta, deta_b}, {dW0, w_b}};
  for (int i = 0; i < 5; ++i) {
    for (const Range& in : ins)
      if (overlaps(outs[i], in)) return TTT_ERR_ALIAS;
    for (int j = i + 1; j < 5; ++j)
      if (overlaps(outs[i], outs[j])) return TTT_ERR_ALIAS;
  }
  if (which) *which = k;
  return TTT_OK;
}

// ---------------------------------------------------------------- MLP --

ttt::MlpArgs make_mlp_args(const ttt_mlp_desc* d, const void* Q, const void* K, const void* V, const float* W1,
                           const float* W2, const float* eta, const void* Z, const float* W1f, const float* W2f) {
  ttt::MlpArgs a;
  a.B = d->B; a.H = d->H; a.T = d->T; a.d = d->d; a.dh = d->dh; a.b = d->b;
  a.in_dtype = d->in_dtype; a.out_dtype = d->out_dtype;
  a.Q = Q; a.K = K; a.V = V; a.W1 = W1; a.W2 = W2; a.w_bstride = d->w_batch_stride;
  a.eta = eta; a.esb = d->eta_stride_b; a.esh = d->eta_stride_h; a.est = d->eta_stride_t;
  a.Z = const_cast<void*>(Z); a.W1f = const_cast<float*>(W1f); a.W2f = const_cast<float*>(W2f);
  a.gamma = nullptr; a.beta = nullptr; a.eps = 0.f;
  a.ckpt = nullptr;
  return a;
}

ttt_status validate_mlp(const ttt_mlp_desc* d, const void* Q, const void* K, const void* V, const float* W1,
                        const float* W2, const float* eta, const void* Z, const float* W1f, const float* W2f,
                        bool* ok_kernel) {
  if (ok_kernel) *ok_kernel = false;
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->H < 0 || d->T < 0 || d->d < 1 || d->dh < 1 || d->b < 1) return TTT_ERR_SHAPE;
  if (d->T % d->b != 0) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype)) return TTT_ERR_DTYPE;
  if ((d->flags & ~static_cast<uint32_t>(TTT_FLAG_PRIMAL)) != 0 || d->reserved != 0) return TTT_ERR_FLAGS;
  int64_t chains = 1, tok = 1, wel = 1;
  if (!mul_ok(chains, d->B) || !mul_ok(chains, d->H) || chains > INT_MAX) return TTT_ERR_SHAPE;
  tok = chains;
  if (!mul_ok(tok, d->T) || !mul_ok(tok, d->d)) return TTT_ERR_SHAPE;
  wel = chains;
  if (!mul_ok(wel, d->d) || !mul_ok(wel, d->dh)) return TTT_ERR_SHAPE;
  const int64_t hw = static_cast<int64_t>(d->H) * d->d * d->dh;
  if (d->w_batch_stride != 0 && d->w_batch_stride != hw) return TTT_ERR_STRIDE;
  if (d->eta_stride_b < 0 || d->eta_stride_h < 0 || d->eta_stride_t < 0) return TTT_ERR_STRIDE;
  ttt::MlpArgs a = make_mlp_args(d, Q, K, V, W1, W2, eta, Z, W1f, W2f);
  const bool supported =
      (d->flags & TTT_FLAG_PRIMAL) ? ttt::mlp_primal_supported(d->d, d->dh) : ttt::mlp_supported(a);
  if (!supported) return TTT_ERR_UNSUPPORTED;
  if (chains == 0) {
    if (ok_kernel) *ok_kernel = true;
    return TTT_OK;
  }
  if (!W1 || !W2 || !W1f || !W2f) return TTT_ERR_NULL;
  if (tok > 0 && (!Q || !K || !V || !Z || !eta)) return TTT_ERR_NULL;
  for (const void* p : {static_cast<const void*>(W1), static_cast<const void*>(W2),
                        static_cast<const void*>(W1f), static_cast<const void*>(W2f)})
    if (!aligned(p, 16)) return TTT_ERR_ALIGN;
  if (tok > 0 && (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(Z, 16) || !aligned(eta, 4)))
    return TTT_ERR_ALIGN;
  const int64_t in_b = tok * dtype_size(d->in_dtype);
  const int64_t z_b = tok * dtype_size(d->out_dtype);
  const int64_t wf_b = wel * 4;
  const int64_t w0_b = (d->w_batch_stride == 0 ? hw : wel) * 4;
  const int64_t eta_b =
      tok > 0 ? eta_extent(d->B, d->H, d->T, d->eta_stride_b, d->eta_stride_h, d->eta_stride_t) * 4 : 0;
  const Range rq{Q, in_b}, rk{K, in_b}, rv{V, in_b}, re{eta, eta_b}, rw1{W1, w0_b}, rw2{W2, w0_b};
  const Range rz{Z, z_b}, rf1{W1f, wf_b}, rf2{W2f, wf_b};
  for (Range out : {rz, rf1, rf2}) {
    for (Range in : {rq, rk, rv, re})
      if (overlaps(out, in)) return TTT_ERR_ALIAS;
  }
  if (overlaps(rz, rf1) || overlaps(rz, rf2) || overlaps(rf1, rf2)) return TTT_ERR_ALIAS;
  if (overlaps(rz, rw1) || overlaps(rz, rw2)) return TTT_ERR_ALIAS;
  const bool per_seq = d->w_batch_stride == hw;
  if (overlaps(rf1, rw1) && !(per_seq && static_cast<const void*>(W1f) == static_cast<const void*>(W1)))
    return TTT_ERR_ALIAS;
  if (overlaps(rf2, rw2) && !(per_seq && static_cast<const void*>(W2f) == static_cast<const void*>(W2)))
    return TTT_ERR_ALIAS;
  if (overlaps(rf1, rw2) || overlaps(rf2, rw1)) return TTT_ERR_ALIAS;
  if (ok_kernel) *ok_kernel = true;
  return TTT_OK;
}

}  // namespace

extern "C" {

int ttt_abi_version(void) { return TTT_ABI_VERSION; }

const char* ttt_status_str(int s) {
  switch (s) {
    case TTT_OK: return "ok";
    case TTT_ERR_NULL: return "a required pointer is NULL";
    case TTT_ERR_SHAPE: return "invalid shape (negative size, b < 1, T % b != 0 or size overflow)";
    case TTT_ERR_DTYPE: return "invalid dtype code";
    case TTT_ERR_UNSUPPORTED: return "no kernel is built for this (d, b, dtype) combination";
    case TTT_ERR_ALIAS: return "an output overlaps an input";
    case TTT_ERR_ALIGN: return "a pointer is misaligned (16 bytes for tensors, 4 for eta)";
    case TTT_ERR_HIP: return "the HIP runtime rejected the kernel launch";
    case TTT_ERR_STRIDE: return "invalid stride";
    case TTT_ERR_FLAGS: return "unknown flag or non-zero reserved field";
    case TTT_ERR_POS: return "negative decode position";
    case TTT_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case TTT_ERR_SCRATCH:
      return "the call needs more than the library's static scratch (TTT_NOALLOC_SCRATCH_BYTES); "
             "use ttt_linear_fwd_chunked with a workspace, or fewer chunks";
    default: return "unknown status";
  }
}

ttt_status ttt_linear_validate(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                               const float* W0, const float* eta, const void* Z, const float* W_final) {
  return validate_linear(desc, Q, K, V, W0, eta, Z, W_final, nullptr);
}

const char* ttt_linear_kernel_name(const ttt_linear_desc* d) {
  if (!d) return nullptr;
  ttt::LinearArgs a = make_linear_args(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  switch (pick_linear(a, d->flags)) {
    case K_MFMA: return ttt::linear_mfma_name(a);
    case K_MFMA32: return "ttt_linear_mfma_f32_d64b16";
    case K_GENERIC: return ttt::linear_generic_name(a.d);
    case K_PRIMAL: return ttt::linear_primal_name(a.d);
    default: return nullptr;
  }
}

ttt_status ttt_linear_fwd(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                          const float* W0, const float* eta, void* Z, float* W_final, void* stream) {
  Kernel k;
  const ttt_status st = validate_linear(desc, Q, K, V, W0, eta, Z, W_final, &k);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  const ttt::LinearArgs a = make_linear_args(desc, Q, K, V, W0, eta, Z, W_final);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (k == K_MFMA)
    e = ttt::launch_linear_mfma(a, s);
  else if (k == K_MFMA32)
    e = ttt::launch_linear_mfma_f32(a, s);
  else if (k == K_PRIMAL)
    e = ttt::launch_linear_primal(make_primal_args_fwd(desc, Q, K, V, W0, eta, Z, W_final), s);
  else
    e = ttt::launch_linear_generic(a, s);
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

namespace {

// Checks of a forward's saved-for-backward buffer (fp32, one value per token
// and output): non-NULL, 16-byte aligned, overlapping no input or output.
ttt_status check_saved(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V, const float* W0,
                       const float* eta, const void* Z, const float* W_final, const float* saved) {
  const int64_t chains = static_cast<int64_t>(desc->B) * desc->H;
  const int64_t tok = chains * desc->T * desc->d;
  if (tok == 0) return TTT_OK;
  if (!saved) return TTT_ERR_NULL;
  if (!aligned(saved, 16)) return TTT_ERR_ALIGN;
  const int64_t in_b = tok * dtype_size(desc->in_dtype), z_b = tok * dtype_size(desc->out_dtype);
  const int64_t hdd = static_cast<int64_t>(desc->H) * desc->d * desc->d;
  const int64_t w0_b = (desc->w0_batch_stride == 0 ? hdd : chains * desc->d * desc->d) * 4;
  const int64_t eta_b =
      eta_extent(desc->B, desc->H, desc->T, desc->eta_stride_b, desc->eta_stride_h, desc->eta_stride_t) * 4;
  const Range re{saved, tok * 4};
  for (Range r : {Range{Q, in_b}, Range{K, in_b}, Range{V, in_b}, Range{eta, eta_b}, Range{W0, w0_b},
                  Range{Z, z_b}, Range{W_final, chains * desc->d * desc->d * 4}})
    if (overlaps(re, r)) return TTT_ERR_ALIAS;
  return TTT_OK;
}

}  // namespace

ttt_status ttt_linear_fwd_save(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                               const float* W0, const float* eta, void* Z, float* W_final, float* E_saved,
                               void* stream) {
  Kernel k;
  ttt_status st = validate_linear(desc, Q, K, V, W0, eta, Z, W_final, &k);
  if (st != TTT_OK) return st;
  if (desc->flags & TTT_FLAG_PRIMAL) return TTT_ERR_FLAGS;
  const int64_t chains = static_cast<int64_t>(desc->B) * desc->H;
  if (chains == 0) return TTT_OK;
  st = check_saved(desc, Q, K, V, W0, eta, Z, W_final, E_saved);
  if (st != TTT_OK) return st;
  const int64_t tok = chains * desc->T * desc->d;
  ttt::LinearArgs a = make_linear_args(desc, Q, K, V, W0, eta, Z, W_final);
  a.Esave = tok > 0 ? E_saved : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = k == K_MFMA ? ttt::launch_linear_mfma(a, s) : ttt::launch_linear_generic(a, s);
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

ttt_status ttt_linear_bwd_validate(const ttt_linear_desc* desc, const void* Q, const void* K, const float* eta,
                                   const float* W_final, const float* E_saved, const void* dZ,
                                   const float* dW_final, const void* dQ, const void* dK, const void* dV,
                                   const float* deta, const float* dW0) {
  return validate_bwd(desc, Q, K, eta, W_final, E_saved, dZ, dW_final, dQ, dK, dV, deta, dW0, nullptr);
}

const char* ttt_linear_bwd_kernel_name(const ttt_linear_desc* d) {
  if (!d) return nullptr;
  const ttt::BwdArgs a = make_bwd_args(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                       nullptr, nullptr, nullptr, nullptr);
  switch (pick_bwd(a, d->flags)) {
    case KB_MFMA: return "ttt_linear_bwd_d64b16";
    case KB_GENERIC: return ttt::linear_bwd_generic_name(a.d);
    default: return nullptr;
  }
}

ttt_status ttt_linear_bwd(const ttt_linear_desc* desc, const void* Q, const void* K, const float* eta,
                          const float* W_final, const float* E_saved, const void* dZ, const float* dW_final,
                          void* dQ, void* dK, void* dV, float* deta, float* dW0, void* stream) {
  BwdKernel k;
  const ttt_status st =
      validate_bwd(desc, Q, K, eta, W_final, E_saved, dZ, dW_final, dQ, dK, dV, deta, dW0, &k);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  const ttt::BwdArgs a = make_bwd_args(desc, Q, K, eta, W_final, E_saved, dZ, dW_final, dQ, dK, dV, deta, dW0);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = k == KB_MFMA ? ttt::launch_linear_bwd_mfma(a, s) : ttt::launch_linear_bwd_generic(a, s);
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

namespace {

// Every check of the layer-norm forward (the plain forward's, then its own).
ttt_status validate_ln(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V, const float* W0,
                       const float* gamma, const float* beta, float eps, const float* eta, const void* Z,
                       const float* W_final) {
  Kernel k;
  const ttt_status st = validate_linear(desc, Q, K, V, W0, eta, Z, W_final, &k);
  if (st != TTT_OK) return st;
  const bool ok = (desc->flags == 0 && k == K_MFMA) || (desc->flags == TTT_FLAG_PRIMAL && k == K_PRIMAL);
  if (!ok) return TTT_ERR_UNSUPPORTED;
  const int64_t chains = static_cast<int64_t>(desc->B) * desc->H;
  const int64_t z_b = chains * desc->T * desc->d * dtype_size(desc->out_dtype);
  return check_ln_params(desc, gamma, beta, eps, {Range{Z, z_b}, Range{W_final, chains * desc->d * desc->d * 4}});
}

hipError_t launch_ln(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V, const float* W0,
                     const float* gamma, const float* beta, float eps, const float* eta, void* Z, float* W_final,
                     float* saved, void* stream) {
  if (desc->flags & TTT_FLAG_PRIMAL) {
    ttt::PrimalArgs p = make_primal_args_fwd(desc, Q, K, V, W0, eta, Z, W_final);
    p.gamma = gamma; p.beta = beta; p.eps = eps;
    return ttt::launch_linear_primal(p, static_cast<hipStream_t>(stream));
  }
  ttt::LinearArgs a = make_linear_args(desc, Q, K, V, W0, eta, Z, W_final);
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.rb = 1;
  a.Esave = saved;
  return ttt::launch_linear_mfma(a, static_cast<hipStream_t>(stream));
}

}  // namespace

const char* ttt_linear_ln_kernel_name(const ttt_linear_desc* d) {
  if (!d) return nullptr;
  ttt::LinearArgs a = make_linear_args(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  const Kernel k = pick_linear(a, d->flags);
  if (d->flags == 0 && k == K_MFMA) return "ttt_linear_mfma_d64b16 (layer norm)";
  if (d->flags == TTT_FLAG_PRIMAL && k == K_PRIMAL) return ttt::linear_primal_name(a.d, true);
  return nullptr;
}

ttt_status ttt_linear_ln_fwd(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                             const float* W0, const float* gamma, const float* beta, float eps, const float* eta,
                             void* Z, float* W_final, void* stream) {
  const ttt_status st = validate_ln(desc, Q, K, V, W0, gamma, beta, eps, eta, Z, W_final);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  const hipError_t e = launch_ln(desc, Q, K, V, W0, gamma, beta, eps, eta, Z, W_final, nullptr, stream);
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

ttt_status ttt_linear_ln_fwd_save(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                                  const float* W0, const float* gamma, const float* beta, float eps,
                                  const float* eta, void* Z, float* W_final, float* G_saved, void* stream) {
  ttt_status st = validate_ln(desc, Q, K, V, W0, gamma, beta, eps, eta, Z, W_final);
  if (st != TTT_OK) return st;
  if (desc->flags != 0) return TTT_ERR_UNSUPPORTED;  // the primal kernel saves nothing
  const int64_t chains = static_cast<int64_t>(desc->B) * desc->H;
  if (chains == 0) return TTT_OK;
  st = check_saved(desc, Q, K, V, W0, eta, Z, W_final, G_saved);
  if (st != TTT_OK) return st;
  const int64_t hd_b = static_cast<int64_t>(desc->H) * desc->d * 4;
  const Range rd{G_saved, chains * desc->T * desc->d * 4};
  if (overlaps(rd, Range{gamma, hd_b}) || overlaps(rd, Range{beta, hd_b})) return TTT_ERR_ALIAS;
  const bool any = chains * desc->T > 0;
  const hipError_t e =
      launch_ln(desc, Q, K, V, W0, gamma, beta, eps, eta, Z, W_final, any ? G_saved : nullptr, stream);
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

namespace {

// Every check of the layer-norm backward: the plain backward's (with the saved
// delta in E's place), then V, gamma, beta, eps and the two extra outputs.
ttt_status validate_ln_bwd(const ttt_linear_desc* d, const void* Q, const void* K, const void* V, const float* eta,
                           const float* gamma, const float* beta, float eps, const float* Wf, const float* Ds,
                           const void* dZ, const float* dWf, const void* dQ, const void* dK, const void* dV,
                           const float* deta, const float* dW0, const float* dgamma, const float* dbeta) {
  BwdKernel k;
  const ttt_status st = validate_bwd(d, Q, K, eta, Wf, Ds, dZ, dWf, dQ, dK, dV, deta, dW0, &k);
  if (st != TTT_OK) return st;
  ttt::BwdArgs a = make_bwd_args(d, Q, K, eta, Wf, Ds, dZ, dWf, nullptr, nullptr, nullptr, nullptr, nullptr);
  if ((d->flags & ~static_cast<uint32_t>(TTT_FLAG_GENERIC)) != 0 || !ttt::linear_ln_bwd_supported(a))
    return TTT_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || eps > 1e30f) return TTT_ERR_SHAPE;
  const int64_t chains = static_cast<int64_t>(d->B) * d->H;
  if (chains == 0) return TTT_OK;
  const int64_t tok = chains * d->T * d->d;
  if (!gamma || !beta || !dgamma || !dbeta || (tok > 0 && !V)) return TTT_ERR_NULL;
  if (!aligned(gamma, 4) || !aligned(beta, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4)) return TTT_ERR_ALIGN;
  if (tok > 0 && !aligned(V, 16)) return TTT_ERR_ALIGN;
  const int64_t in_b = tok * dtype_size(d->in_dtype), g_b = tok * dtype_size(d->out_dtype);
  const int64_t hd_b = static_cast<int64_t>(d->H) * d->d * 4, cd_b = chains * d->d * 4;
  const int64_t w_b = chains * d->d * d->d * 4;
  const int64_t eta_b = tok > 0 ? eta_extent(d->B, d->H, d->T, d->eta_stride_b, d->eta_stride_h, d->eta_stride_t) * 4 : 0;
  const Range ins[] = {{Q, in_b}, {K, in_b}, {V, in_b}, {eta, eta_b}, {gamma, hd_b}, {beta, hd_b}, {Wf, w_b},
                       {Ds, tok * 4}, {dZ, g_b}, {dWf, w_b}};
  const Range outs[] = {{dQ, g_b}, {dK, g_b}, {dV, g_b}, {deta, tok > 0 ? chains * d->T * 4 : 0}, {dW0, w_b},
                        {dgamma, cd_b}, {dbeta, cd_b}};
  for (int i = 0; i < 7; ++i) {
    for (const Range& in : ins)
      if (overlaps(outs[i], in)) return TTT_ERR_ALIAS;
    for (int j = i + 1; j < 7; ++j)
      if (overlaps(outs[i], outs[j])) return TTT_ERR_ALIAS;
  }
  return TTT_OK;
}

}  // namespace

ttt_status ttt_linear_ln_bwd_validate(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                                      const float* eta, const float* gamma, const float* beta, float eps,
                                      const float* W_final, const float* G_saved, const void* dZ,
                                      const float* dW_final, const void* dQ, const void* dK, const void* dV,
                                      const float* deta, const float* dW0, const float* dgamma,
                                      const float* dbeta) {
  return validate_ln_bwd(desc, Q, K, V, eta, gamma, beta, eps, W_final, G_saved, dZ, dW_final, dQ, dK, dV,
                         deta, dW0, dgamma, dbeta);
}

const char* ttt_linear_ln_bwd_kernel_name(const ttt_linear_desc* d) {
  if (!d || (d->flags & ~static_cast<uint32_t>(TTT_FLAG_GENERIC)) != 0) return nullptr;
  const ttt::BwdArgs a = make_bwd_args(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                       nullptr, nullptr, nullptr, nullptr);
  if (!ttt::linear_ln_bwd_supported(a)) return nullptr;
  return (d->flags & TTT_FLAG_GENERIC) ? "ttt_linear_ln_bwd_fp32" : "ttt_linear_ln_bwd_d64b16";
}

ttt_status ttt_linear_ln_bwd(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                             const float* eta, const float* gamma, const float* beta, float eps,
                             const float* W_final, const float* G_saved, const void* dZ, const float* dW_final,
                             void* dQ, void* dK, void* dV, float* deta, float* dW0, float* dgamma, float* dbeta,
                             void* stream) {
  const ttt_status st = validate_ln_bwd(desc, Q, K, V, eta, gamma, beta, eps, W_final, G_saved, dZ, dW_final,
                                        dQ, dK, dV, deta, dW0, dgamma, dbeta);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  ttt::BwdArgs a =
      make_bwd_args(desc, Q, K, eta, W_final, G_saved, dZ, dW_final, dQ, dK, dV, deta, dW0);
  a.V = V;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e =
      (desc->flags & TTT_FLAG_GENERIC) ? ttt::launch_linear_ln_bwd(a, s) : ttt::launch_linear_ln_bwd_mfma(a, s);
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

int64_t ttt_linear_chunked_workspace_bytes(const ttt_linear_desc* desc, int32_t nchunks) {
  if (!desc || nchunks < 1 || desc->B < 0 || desc->H < 0 || desc->d < 1) return -1;
  if (nchunks == 1) return 0;
  // maps (P, R) of chunks 1 .. n-2 and start states of chunks 1 .. n-1
  const int64_t per_chain = (static_cast<int64_t>(nchunks - 2) * 2 + (nchunks - 1)) * desc->d * desc->d * 4;
  return static_cast<int64_t>(desc->B) * desc->H * per_chain;
}

namespace {

// Argument checks of the chunked forward (everything but the workspace).
ttt_status validate_chunked(const ttt_linear_desc* desc, int32_t nchunks, const void* Q, const void* K,
                            const void* V, const float* W0, const float* eta, const void* Z, const float* W_final) {
  Kernel k;
  ttt_status st = validate_linear(desc, Q, K, V, W0, eta, Z, W_final, &k);
  if (st != TTT_OK) return st;
  if (nchunks < 1 || nchunks > desc->T / 16) {  // every chunk holds at least one mini-batch
    if (!(nchunks == 1 && desc->T == 0)) return TTT_ERR_SHAPE;
  }
  if ((desc->flags & ~kRowFlags) != 0 || k != K_MFMA) return TTT_ERR_UNSUPPORTED;
  // workgroups of the launches (nchunks - 1 units per chain, row blocks in the last)
  if (static_cast<int64_t>(desc->B) * desc->H * nchunks * row_blocks(desc->flags) > INT_MAX)
    return TTT_ERR_SHAPE;
  return TTT_OK;
}

// Mini-batches of chunk 0 of a chunked forward.  Its workgroup runs the plain
// forward in the first launch while the others compute two maps each, which
// measured ~10% slower per mini-batch on MI355X (219 against 198 us for 410
// mini-batches), so with maps in that launch chunk 0 gets ~1.1 shares of the
// sequence and the other chunks one each; every chunk keeps at least one.
int64_t chunk0_minibatches(int64_t nb, int32_t nchunks) {
  const double share = nchunks > 2 ? 1.1 : 1.0;
  int64_t mb1 = static_cast<int64_t>(static_cast<double>(nb) * share / (nchunks - 1 + share) + 0.5);
  if (mb1 < 1) mb1 = 1;
  if (mb1 > nb - (nchunks - 1)) mb1 = nb - (nchunks - 1);
  return mb1;
}

// The chunked forward's launches, after validate_chunked, nchunks > 1 and
// B*H > 0, with a workspace of at least the bytes it needs.
ttt_status run_chunked(const ttt_linear_desc* desc, int32_t nchunks, const void* Q, const void* K, const void* V,
                       const float* W0, const float* eta, void* Z, float* W_final, void* workspace,
                       void* stream);

}  // namespace

ttt_status ttt_linear_fwd_chunked(const ttt_linear_desc* desc, int32_t nchunks, const void* Q, const void* K,
                                  const void* V, const float* W0, const float* eta, void* Z, float* W_final,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  ttt_status st = validate_chunked(desc, nchunks, Q, K, V, W0, eta, Z, W_final);
  if (st != TTT_OK) return st;
  if (nchunks == 1) return ttt_linear_fwd(desc, Q, K, V, W0, eta, Z, W_final, stream);
  const int64_t chains = static_cast<int64_t>(desc->B) * desc->H;
  if (chains == 0) return TTT_OK;
  const int64_t need = ttt_linear_chunked_workspace_bytes(desc, nchunks);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return TTT_ERR_WORKSPACE;
  {
    const int64_t tok = chains * desc->T * desc->d;
    const int64_t in_b = tok * dtype_size(desc->in_dtype), z_b = tok * dtype_size(desc->out_dtype);
    const int64_t hdd = static_cast<int64_t>(desc->H) * desc->d * desc->d;
    const int64_t w0_b = (desc->w0_batch_stride == 0 ? hdd : chains * desc->d * desc->d) * 4;
    const int64_t eta_b = tok > 0 ? eta_extent(desc->B, desc->H, desc->T, desc->eta_stride_b, desc->eta_stride_h,
                                               desc->eta_stride_t) * 4 : 0;
    const Range rw{workspace, need};
    for (Range r : {Range{Q, in_b}, Range{K, in_b}, Range{V, in_b}, Range{eta, eta_b}, Range{W0, w0_b},
                    Range{Z, z_b}, Range{W_final, chains * desc->d * desc->d * 4}})
      if (overlaps(rw, r)) return TTT_ERR_ALIAS;
  }
  return run_chunked(desc, nchunks, Q, K, V, W0, eta, Z, W_final, workspace, stream);
}

ttt_status ttt_linear_fwd_chunked_noalloc(const ttt_linear_desc* desc, int32_t nchunks, const void* Q,
                                          const void* K, const void* V, const float* W0, const float* eta,
                                          void* Z, float* W_final, void* stream) {
  ttt_status st = validate_chunked(desc, nchunks, Q, K, V, W0, eta, Z, W_final);
  if (st != TTT_OK) return st;
  if (nchunks == 1) return ttt_linear_fwd(desc, Q, K, V, W0, eta, Z, W_final, stream);
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  if (ttt_linear_chunked_workspace_bytes(desc, nchunks) > TTT_NOALLOC_SCRATCH_BYTES) return TTT_ERR_SCRATCH;
  void* ws = nullptr;
  if (scratch_address(static_cast<hipStream_t>(stream), &ws) != hipSuccess) return TTT_ERR_HIP;
  // (the chunked passes write every map and start state before reading it, so
  // the scratch needs no clearing between calls)
  return run_chunked(desc, nchunks, Q, K, V, W0, eta, Z, W_final, ws, stream);
}

namespace {

ttt_status run_chunked(const ttt_linear_desc* desc, int32_t nchunks, const void* Q, const void* K, const void* V,
                       const float* W0, const float* eta, void* Z, float* W_final, void* workspace,
                       void* stream) {
  const int64_t chains = static_cast<int64_t>(desc->B) * desc->H;
  ttt::LinearArgs a = make_linear_args(desc, Q, K, V, W0, eta, Z, W_final);
  a.nchunk = nchunks;
  a.mb1 = chunk0_minibatches(desc->T / 16, nchunks);
  a.maps = static_cast<float*>(workspace);
  a.Wstart = a.maps + chains * (nchunks - 2) * 2 * desc->d * desc->d;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // chunk 0 and the maps of chunks 1 .. n-2 (one workgroup per unit; the row
  // block flag applies to the last launch only)
  ttt::LinearArgs a1 = a;
  a1.rb = 1;
  hipError_t e = ttt::launch_linear_mfma_head_maps(a1, s);
  if (e == hipSuccess && nchunks > 2) e = ttt::launch_linear_chunk_scan(a, s);
  if (e == hipSuccess) e = ttt::launch_linear_mfma(a, s);
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

}  // namespace

ttt_status ttt_linear_decode_validate(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                                      const float* eta, const void* Z, const float* W, const float* Wb,
                                      int64_t pos) {
  return validate_decode(desc, Q, K, V, eta, Z, W, Wb, pos);
}

ttt_status ttt_linear_decode(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                             const float* eta, void* Z, float* W, float* Wb, int64_t pos, void* stream) {
  const ttt_status st = validate_decode(desc, Q, K, V, eta, Z, W, Wb, pos);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  const hipError_t e =
      ttt::launch_linear_primal(make_decode_args(desc, Q, K, V, eta, Z, W, Wb, pos), static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

ttt_status ttt_linear_ln_decode_validate(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                                         const float* eta, const float* gamma, const float* beta, float eps,
                                         const void* Z, const float* W, const float* Wb, int64_t pos) {
  return validate_ln_decode(desc, Q, K, V, eta, gamma, beta, eps, Z, W, Wb, pos);
}

ttt_status ttt_linear_ln_decode(const ttt_linear_desc* desc, const void* Q, const void* K, const void* V,
                                const float* eta, const float* gamma, const float* beta, float eps, void* Z,
                                float* W, float* Wb, int64_t pos, void* stream) {
  const ttt_status st = validate_ln_decode(desc, Q, K, V, eta, gamma, beta, eps, Z, W, Wb, pos);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  ttt::PrimalArgs a = make_decode_args(desc, Q, K, V, eta, Z, W, Wb, pos);
  a.gamma = gamma; a.beta = beta; a.eps = eps;
  const hipError_t e = ttt::launch_linear_primal(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

ttt_status ttt_mlp_validate(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V,
                            const float* W1_0, const float* W2_0, const float* eta, const void* Z,
                            const float* W1_final, const float* W2_final) {
  return validate_mlp(desc, Q, K, V, W1_0, W2_0, eta, Z, W1_final, W2_final, nullptr);
}

const char* ttt_mlp_ln_kernel_name(const ttt_mlp_desc* d) {
  if (!d) return nullptr;
  if (d->flags & TTT_FLAG_PRIMAL)
    return ttt::mlp_primal_supported(d->d, d->dh) ? "ttt_mlp_ln_primal_d64h256" : nullptr;
  ttt::MlpArgs a = make_mlp_args(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                 nullptr);
  return ttt::mlp_supported(a) ? "ttt_mlp_fwd_d64h256b16 (layer norm)" : nullptr;
}

const char* ttt_mlp_kernel_name(const ttt_mlp_desc* d) {
  if (!d) return nullptr;
  if (d->flags & TTT_FLAG_PRIMAL) return ttt::mlp_primal_supported(d->d, d->dh) ? "ttt_mlp_primal_d64h256" : nullptr;
  ttt::MlpArgs a = make_mlp_args(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                 nullptr);
  return ttt::mlp_supported(a) ? ttt::mlp_name(a) : nullptr;
}

namespace {

ttt::MlpPrimalArgs make_mlp_primal_args(const ttt_mlp_desc* d, const void* Q, const void* K, const void* V,
                                        const float* eta, void* Z) {
  ttt::MlpPrimalArgs a;
  a.B = d->B; a.H = d->H; a.T = d->T; a.d = d->d; a.dh = d->dh; a.b = d->b;
  a.in_dtype = d->in_dtype; a.out_dtype = d->out_dtype;
  a.Q = Q; a.K = K; a.V = V;
  a.eta = eta; a.esb = d->eta_stride_b; a.esh = d->eta_stride_h; a.est = d->eta_stride_t;
  a.Z = Z;
  a.W1_in = a.W2_in = a.W1b_in = a.W2b_in = nullptr;
  a.W1_out = a.W2_out = a.W1b_out = a.W2b_out = nullptr;
  a.w_in_bstride = 0;
  a.pos = 0;
  a.gamma = nullptr; a.beta = nullptr; a.eps = 0.f;
  return a;
}

ttt_status validate_mlp_decode(const ttt_mlp_desc* d, const void* Q, const void* K, const void* V,
                               const float* eta, const void* Z, const float* W1, const float* W2, const float* W1b,
                               const float* W2b, int64_t pos) {
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->H < 0 || d->T < 0 || d->d < 1 || d->dh < 1 || d->b < 1) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype)) return TTT_ERR_DTYPE;
  if (d->flags != 0 || d->reserved != 0) return TTT_ERR_FLAGS;
  if (pos < 0) return TTT_ERR_POS;
  if (d->w_batch_stride != 0) return TTT_ERR_STRIDE;
  if (d->eta_stride_b < 0 || d->eta_stride_h < 0 || d->eta_stride_t < 0) return TTT_ERR_STRIDE;
  int64_t chains = 1, tok = 1, wel = 1;
  if (!mul_ok(chains, d->B) || !mul_ok(chains, d->H) || chains > INT_MAX) return TTT_ERR_SHAPE;
  tok = chains;
  if (!mul_ok(tok, d->T) || !mul_ok(tok, d->d)) return TTT_ERR_SHAPE;
  wel = chains;
  if (!mul_ok(wel, d->d) || !mul_ok(wel, d->dh)) return TTT_ERR_SHAPE;
  if (!ttt::mlp_primal_supported(d->d, d->dh)) return TTT_ERR_UNSUPPORTED;
  if (chains == 0) return TTT_OK;
  if (!W1 || !W2 || !W1b || !W2b) return TTT_ERR_NULL;
  if (tok > 0 && (!Q || !K || !V || !Z || !eta)) return TTT_ERR_NULL;
  for (const float* p : {W1, W2, W1b, W2b})
    if (!aligned(p, 16)) return TTT_ERR_ALIGN;
  if (tok > 0 && (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(Z, 16) || !aligned(eta, 4)))
    return TTT_ERR_ALIGN;
  const int64_t in_b = tok * dtype_size(d->in_dtype);
  const int64_t z_b = tok * dtype_size(d->out_dtype);
  const int64_t w_b = wel * 4;
  const int64_t eta_b =
      tok > 0 ? eta_extent(d->B, d->H, d->T, d->eta_stride_b, d->eta_stride_h, d->eta_stride_t) * 4 : 0;
  const Range ins[] = {{Q, in_b}, {K, in_b}, {V, in_b}, {eta, eta_b}};
  const Range outs[] = {{Z, z_b}, {W1, w_b}, {W2, w_b}, {W1b, w_b}, {W2b, w_b}};
  for (int i = 0; i < 5; ++i) {
    for (const Range& in : ins)
      if (overlaps(outs[i], in)) return TTT_ERR_ALIAS;
    for (int j = i + 1; j < 5; ++j)
      if (overlaps(outs[i], outs[j])) return TTT_ERR_ALIAS;
  }
  return TTT_OK;
}

ttt_status validate_mlp_ln_decode(const ttt_mlp_desc* d, const void* Q, const void* K, const void* V,
                                  const float* eta, const float* gamma, const float* beta, float eps, const void* Z,
                                  const float* W1, const float* W2, const float* W1b, const float* W2b,
                                  int64_t pos) {
  const ttt_status st = validate_mlp_decode(d, Q, K, V, eta, Z, W1, W2, W1b, W2b, pos);
  if (st != TTT_OK) return st;
  const int64_t chains = static_cast<int64_t>(d->B) * d->H;
  const int64_t w_b = chains * d->d * d->dh * 4;
  return check_ln(chains, d->H, d->d, gamma, beta, eps,
                  {Range{Z, chains * d->T * d->d * dtype_size(d->out_dtype)}, Range{W1, w_b}, Range{W2, w_b},
                   Range{W1b, w_b}, Range{W2b, w_b}});
}

ttt::MlpPrimalArgs make_mlp_decode_args(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V,
                                        const float* eta, void* Z, float* W1, float* W2, float* W1b, float* W2b,
                                        int64_t pos) {
  ttt::MlpPrimalArgs a = make_mlp_primal_args(desc, Q, K, V, eta, Z);
  a.W1_in = a.W1_out = W1;
  a.W2_in = a.W2_out = W2;
  a.W1b_in = a.W1b_out = W1b;
  a.W2b_in = a.W2b_out = W2b;
  a.w_in_bstride = static_cast<int64_t>(desc->H) * desc->d * desc->dh;
  a.pos = pos;
  return a;
}

}  // namespace

ttt_status ttt_mlp_decode_validate(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V,
                                   const float* eta, const void* Z, const float* W1, const float* W2,
                                   const float* W1b, const float* W2b, int64_t pos) {
  return validate_mlp_decode(desc, Q, K, V, eta, Z, W1, W2, W1b, W2b, pos);
}

ttt_status ttt_mlp_decode(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V, const float* eta,
                          void* Z, float* W1, float* W2, float* W1b, float* W2b, int64_t pos, void* stream) {
  const ttt_status st = validate_mlp_decode(desc, Q, K, V, eta, Z, W1, W2, W1b, W2b, pos);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  const hipError_t e = ttt::launch_mlp_primal(make_mlp_decode_args(desc, Q, K, V, eta, Z, W1, W2, W1b, W2b, pos),
                                              static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

ttt_status ttt_mlp_ln_decode_validate(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V,
                                      const float* eta, const float* gamma, const float* beta, float eps,
                                      const void* Z, const float* W1, const float* W2, const float* W1b,
                                      const float* W2b, int64_t pos) {
  return validate_mlp_ln_decode(desc, Q, K, V, eta, gamma, beta, eps, Z, W1, W2, W1b, W2b, pos);
}

ttt_status ttt_mlp_ln_decode(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V,
                             const float* eta, const float* gamma, const float* beta, float eps, void* Z, float* W1,
                             float* W2, float* W1b, float* W2b, int64_t pos, void* stream) {
  const ttt_status st = validate_mlp_ln_decode(desc, Q, K, V, eta, gamma, beta, eps, Z, W1, W2, W1b, W2b, pos);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  ttt::MlpPrimalArgs a = make_mlp_decode_args(desc, Q, K, V, eta, Z, W1, W2, W1b, W2b, pos);
  a.gamma = gamma; a.beta = beta; a.eps = eps;
  const hipError_t e = ttt::launch_mlp_primal(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

ttt_status ttt_mlp_fwd(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V, const float* W1_0,
                       const float* W2_0, const float* eta, void* Z, float* W1_final, float* W2_final,
                       void* stream) {
  bool ok;
  const ttt_status st = validate_mlp(desc, Q, K, V, W1_0, W2_0, eta, Z, W1_final, W2_final, &ok);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  if (desc->flags & TTT_FLAG_PRIMAL) {
    // token by token from W0 (the first token starts a mini-batch, so no
    // mini-batch-start state is read)
    ttt::MlpPrimalArgs p = make_mlp_primal_args(desc, Q, K, V, eta, Z);
    p.W1_in = p.W1b_in = W1_0;
    p.W2_in = p.W2b_in = W2_0;
    p.w_in_bstride = desc->w_batch_stride;
    p.W1_out = W1_final;
    p.W2_out = W2_final;
    const hipError_t e = ttt::launch_mlp_primal(p, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
  }
  const ttt::MlpArgs a = make_mlp_args(desc, Q, K, V, W1_0, W2_0, eta, Z, W1_final, W2_final);
  const hipError_t e = ttt::launch_mlp(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

ttt_status ttt_mlp_ln_fwd(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V,
                          const float* W1_0, const float* W2_0, const float* gamma, const float* beta, float eps,
                          const float* eta, void* Z, float* W1_final, float* W2_final, void* stream) {
  bool ok;
  ttt_status st = validate_mlp(desc, Q, K, V, W1_0, W2_0, eta, Z, W1_final, W2_final, &ok);
  if (st != TTT_OK) return st;
  const int64_t chains = static_cast<int64_t>(desc->B) * desc->H;
  const int64_t z_b = chains * desc->T * desc->d * dtype_size(desc->out_dtype);
  const int64_t w_b = chains * desc->d * desc->dh * 4;
  st = check_ln(chains, desc->H, desc->d, gamma, beta, eps,
                {Range{Z, z_b}, Range{W1_final, w_b}, Range{W2_final, w_b}});
  if (st != TTT_OK || chains == 0) return st;
  if (desc->flags & TTT_FLAG_PRIMAL) {
    ttt::MlpPrimalArgs p = make_mlp_primal_args(desc, Q, K, V, eta, Z);
    p.W1_in = p.W1b_in = W1_0;
    p.W2_in = p.W2b_in = W2_0;
    p.w_in_bstride = desc->w_batch_stride;
    p.W1_out = W1_final;
    p.W2_out = W2_final;
    p.gamma = gamma; p.beta = beta; p.eps = eps;
    const hipError_t e = ttt::launch_mlp_primal(p, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
  }
  ttt::MlpArgs a = make_mlp_args(desc, Q, K, V, W1_0, W2_0, eta, Z, W1_final, W2_final);
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  const hipError_t e = ttt::launch_mlp(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

int64_t ttt_mlp_bwd_workspace_bytes(const ttt_mlp_desc* d) {
  if (!d || d->B < 0 || d->H < 0 || d->T < 0 || d->d < 1 || d->dh < 1 || d->b < 1) return -1;
  int64_t n = 1;
  const int64_t nb = (static_cast<int64_t>(d->T) + d->b - 1) / d->b;
  for (int64_t f : {static_cast<int64_t>(d->B), static_cast<int64_t>(d->H), nb, int64_t{2},
                    static_cast<int64_t>(d->d), static_cast<int64_t>(d->dh), int64_t{4}})
    if (!mul_ok(n, f)) return -1;
  return n;
}

namespace {

// Every host-side check of the TTT-MLP backward.
ttt_status validate_mlp_bwd(const ttt_mlp_desc* d, const void* Q, const void* K, const void* V, const float* W1_0,
                            const float* W2_0, const float* eta, const float* dZ, const float* dW1f,
                            const float* dW2f, const void* ws, int64_t ws_bytes, const float* dQ, const float* dK,
                            const float* dV, const float* deta, const float* dW1, const float* dW2) {
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->H < 0 || d->T < 0 || d->d < 1 || d->dh < 1 || d->b < 1) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype)) return TTT_ERR_DTYPE;
  if ((d->flags & ~static_cast<uint32_t>(TTT_FLAG_PRIMAL)) != 0 || d->reserved != 0) return TTT_ERR_FLAGS;
  const int64_t hs = static_cast<int64_t>(d->H) * d->d * d->dh;
  if (d->w_batch_stride != 0 && d->w_batch_stride != hs) return TTT_ERR_STRIDE;
  if (d->eta_stride_b < 0 || d->eta_stride_h < 0 || d->eta_stride_t < 0) return TTT_ERR_STRIDE;
  int64_t chains = 1, tok = 1, wel = 1;
  if (!mul_ok(chains, d->B) || !mul_ok(chains, d->H) || chains > INT_MAX) return TTT_ERR_SHAPE;
  tok = chains;
  if (!mul_ok(tok, d->T) || !mul_ok(tok, d->d)) return TTT_ERR_SHAPE;
  wel = chains;
  if (!mul_ok(wel, d->d) || !mul_ok(wel, d->dh)) return TTT_ERR_SHAPE;
  const int64_t need = ttt_mlp_bwd_workspace_bytes(d);
  if (need < 0) return TTT_ERR_SHAPE;
  // dZ and every gradient are fp32; the Q/K/V dtype is in_dtype
  if (d->out_dtype != TTT_F32 || !ttt::mlp_bwd_supported(d->d, d->dh, d->b)) return TTT_ERR_UNSUPPORTED;
  if (chains == 0) return TTT_OK;
  if (!W1_0 || !W2_0 || !dW1 || !dW2) return TTT_ERR_NULL;
  if (tok > 0 && (!Q || !K || !V || !eta || !dZ || !dQ || !dK || !dV || !deta)) return TTT_ERR_NULL;
  for (const float* p : {W1_0, W2_0, dW1, dW2}) if (!aligned(p, 16)) return TTT_ERR_ALIGN;
  for (const float* p : {dW1f, dW2f}) if (p && !aligned(p, 16)) return TTT_ERR_ALIGN;
  if (tok > 0) {
    for (const void* p : {Q, K, V}) if (!aligned(p, static_cast<int>(dtype_size(d->in_dtype)))) return TTT_ERR_ALIGN;
    for (const float* p : {dQ, dK}) if (!aligned(p, 16)) return TTT_ERR_ALIGN;
    for (const float* p : {dZ, dV, deta, eta}) if (!aligned(p, 4)) return TTT_ERR_ALIGN;
  }
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 16))) return TTT_ERR_WORKSPACE;
  const int64_t in_b = tok * dtype_size(d->in_dtype), f_b = tok * 4;
  const int64_t w0_b = (d->w_batch_stride == 0 ? hs : wel) * 4, w_b = wel * 4;
  const int64_t eta_b =
      tok > 0 ? eta_extent(d->B, d->H, d->T, d->eta_stride_b, d->eta_stride_h, d->eta_stride_t) * 4 : 0;
  const Range ins[] = {{Q, in_b}, {K, in_b}, {V, in_b}, {W1_0, w0_b}, {W2_0, w0_b}, {eta, eta_b},
                       {dZ, f_b}, {dW1f, dW1f ? w_b : 0}, {dW2f, dW2f ? w_b : 0}};
  const Range outs[] = {{dQ, f_b}, {dK, f_b}, {dV, f_b}, {deta, chains * d->T * 4}, {dW1, w_b}, {dW2, w_b},
                        {ws, need}};
  for (int i = 0; i < 7; ++i) {
    for (const Range& in : ins)
      if (overlaps(outs[i], in)) return TTT_ERR_ALIAS;
    for (int j = i + 1; j < 7; ++j)
      if (overlaps(outs[i], outs[j])) return TTT_ERR_ALIAS;
  }
  return TTT_OK;
}

// The matrix-core (dual-form) backward takes the shape it supports with
// 16-byte aligned token and gradient tensors; everything else, and
// TTT_FLAG_PRIMAL, runs the primal kernel.
bool mlp_bwd_dual_shape(const ttt_mlp_desc* d) {
  return !(d->flags & TTT_FLAG_PRIMAL) && ttt::mlp_bwd_mfma_supported(d->d, d->dh, d->b, d->in_dtype, d->T);
}

}  // namespace

ttt_status ttt_mlp_bwd_validate(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V,
                                const float* W1_0, const float* W2_0, const float* eta, const float* dZ,
                                const float* dW1_final, const float* dW2_final, const void* workspace,
                                int64_t workspace_bytes, const float* dQ, const float* dK, const float* dV,
                                const float* deta, const float* dW1_0, const float* dW2_0) {
  return validate_mlp_bwd(desc, Q, K, V, W1_0, W2_0, eta, dZ, dW1_final, dW2_final, workspace, workspace_bytes, dQ,
                          dK, dV, deta, dW1_0, dW2_0);
}

ttt_status ttt_mlp_bwd(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V, const float* W1_0,
                       const float* W2_0, const float* eta, const float* dZ, const float* dW1_final,
                       const float* dW2_final, void* workspace, int64_t workspace_bytes, float* dQ, float* dK,
                       float* dV, float* deta, float* dW1_0, float* dW2_0, void* stream) {
  const ttt_status st = validate_mlp_bwd(desc, Q, K, V, W1_0, W2_0, eta, dZ, dW1_final, dW2_final, workspace,
                                         workspace_bytes, dQ, dK, dV, deta, dW1_0, dW2_0);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  ttt::MlpBwdArgs a;
  a.B = desc->B; a.H = desc->H; a.T = desc->T; a.d = desc->d; a.dh = desc->dh; a.b = desc->b;
  a.in_dtype = desc->in_dtype;
  a.Q = Q; a.K = K; a.V = V;
  a.W1_in = W1_0; a.W2_in = W2_0; a.w_in_bstride = desc->w_batch_stride;
  a.eta = eta; a.esb = desc->eta_stride_b; a.esh = desc->eta_stride_h; a.est = desc->eta_stride_t;
  a.dZ = dZ; a.dW1f = dW1_final; a.dW2f = dW2_final;
  a.ws = static_cast<float*>(workspace);
  a.dQ = dQ; a.dK = dK; a.dV = dV; a.deta = deta; a.dW1 = dW1_0; a.dW2 = dW2_0;
  a.gamma = nullptr; a.beta = nullptr; a.eps = 0.f; a.dgamma = nullptr; a.dbeta = nullptr;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  bool dual = mlp_bwd_dual_shape(desc);
  if (desc->T > 0)
    for (const void* p : {Q, K, V, static_cast<const void*>(dZ), static_cast<const void*>(dQ),
                          static_cast<const void*>(dK), static_cast<const void*>(dV)})
      dual = dual && aligned(p, 16);
  if (!dual) {
    const hipError_t e = ttt::launch_mlp_bwd(a, s);
    return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
  }
  if (desc->T > 0) {
    // pass 1: the forward kernel writes the state at every mini-batch start
    ttt::MlpArgs f = make_mlp_args(desc, Q, K, V, W1_0, W2_0, eta, nullptr, nullptr, nullptr);
    f.ckpt = a.ws;
    const hipError_t e1 = ttt::launch_mlp_ckpt(f, s);
    if (e1 != hipSuccess) return TTT_ERR_HIP;
  }
  const hipError_t e = ttt::launch_mlp_bwd_mfma(a, s);
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

const char* ttt_mlp_bwd_kernel_name(const ttt_mlp_desc* d) {
  if (!d) return nullptr;
  if (!ttt::mlp_bwd_supported(d->d, d->dh, d->b) || d->out_dtype != TTT_F32) return nullptr;
  return mlp_bwd_dual_shape(d) ? "ttt_mlp_bwd_d64h256b16" : "ttt_mlp_bwd_d64h256";
}

}  // extern "C"

namespace {

// ttt_mlp_bwd's checks, then the layer-norm parameters and their gradients:
// gamma, beta [H, d] and dgamma, dbeta [B, H, d] fp32, 4-byte aligned, the
// latter two outputs overlapping no input and no other output.
ttt_status validate_mlp_ln_bwd(const ttt_mlp_desc* d, const void* Q, const void* K, const void* V, const float* W1_0,
                               const float* W2_0, const float* gamma, const float* beta, float eps, const float* eta,
                               const float* dZ, const float* dW1f, const float* dW2f, const void* ws,
                               int64_t ws_bytes, const float* dQ, const float* dK, const float* dV, const float* deta,
                               const float* dW1, const float* dW2, const float* dgamma, const float* dbeta) {
  const ttt_status st = validate_mlp_bwd(d, Q, K, V, W1_0, W2_0, eta, dZ, dW1f, dW2f, ws, ws_bytes, dQ, dK, dV, deta,
                                         dW1, dW2);
  if (st != TTT_OK) return st;
  const int64_t chains = static_cast<int64_t>(d->B) * d->H;
  const int64_t tok = chains * d->T * d->d * 4, w_b = chains * d->d * d->dh * 4, cd_b = chains * d->d * 4;
  const int64_t need = ttt_mlp_bwd_workspace_bytes(d);
  const std::initializer_list<Range> all_outs = {{dQ, tok}, {dK, tok}, {dV, tok}, {deta, chains * d->T * 4},
                                                 {dW1, w_b}, {dW2, w_b}, {ws, need}, {dgamma, cd_b}, {dbeta, cd_b}};
  const ttt_status sl = check_ln(chains, d->H, d->d, gamma, beta, eps, all_outs);
  if (sl != TTT_OK) return sl;
  if (chains == 0) return TTT_OK;
  if (!dgamma || !dbeta) return TTT_ERR_NULL;
  if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return TTT_ERR_ALIGN;
  const int64_t in_b = tok / 4 * dtype_size(d->in_dtype);
  const int64_t w0_b = (d->w_batch_stride == 0 ? static_cast<int64_t>(d->H) * d->d * d->dh * 4 : w_b);
  const int64_t eta_b =
      d->T > 0 ? eta_extent(d->B, d->H, d->T, d->eta_stride_b, d->eta_stride_h, d->eta_stride_t) * 4 : 0;
  const Range ins[] = {{Q, in_b}, {K, in_b}, {V, in_b}, {W1_0, w0_b}, {W2_0, w0_b}, {eta, eta_b}, {dZ, tok},
                       {dW1f, dW1f ? w_b : 0}, {dW2f, dW2f ? w_b : 0}};
  // dgamma and dbeta are the last two outputs: each against every input and
  // every output before it (ttt_mlp_bwd's checks covered the others)
  const Range* outs = all_outs.begin();
  const int n_out = static_cast<int>(all_outs.size());
  for (int i = n_out - 2; i < n_out; ++i) {
    for (const Range& in : ins)
      if (overlaps(outs[i], in)) return TTT_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return TTT_ERR_ALIAS;
  }
  return TTT_OK;
}

}  // namespace

extern "C" {

ttt_status ttt_mlp_ln_bwd_validate(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V,
                                   const float* W1_0, const float* W2_0, const float* gamma, const float* beta,
                                   float eps, const float* eta, const float* dZ, const float* dW1_final,
                                   const float* dW2_final, const void* workspace, int64_t workspace_bytes,
                                   const float* dQ, const float* dK, const float* dV, const float* deta,
                                   const float* dW1_0, const float* dW2_0, const float* dgamma, const float* dbeta) {
  return validate_mlp_ln_bwd(desc, Q, K, V, W1_0, W2_0, gamma, beta, eps, eta, dZ, dW1_final, dW2_final, workspace,
                             workspace_bytes, dQ, dK, dV, deta, dW1_0, dW2_0, dgamma, dbeta);
}

ttt_status ttt_mlp_ln_bwd(const ttt_mlp_desc* desc, const void* Q, const void* K, const void* V, const float* W1_0,
                          const float* W2_0, const float* gamma, const float* beta, float eps, const float* eta,
                          const float* dZ, const float* dW1_final, const float* dW2_final, void* workspace,
                          int64_t workspace_bytes, float* dQ, float* dK, float* dV, float* deta, float* dW1_0,
                          float* dW2_0, float* dgamma, float* dbeta, void* stream) {
  const ttt_status st = validate_mlp_ln_bwd(desc, Q, K, V, W1_0, W2_0, gamma, beta, eps, eta, dZ, dW1_final,
                                            dW2_final, workspace, workspace_bytes, dQ, dK, dV, deta, dW1_0, dW2_0,
                                            dgamma, dbeta);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  ttt::MlpBwdArgs a;
  a.B = desc->B; a.H = desc->H; a.T = desc->T; a.d = desc->d; a.dh = desc->dh; a.b = desc->b;
  a.in_dtype = desc->in_dtype;
  a.Q = Q; a.K = K; a.V = V;
  a.W1_in = W1_0; a.W2_in = W2_0; a.w_in_bstride = desc->w_batch_stride;
  a.eta = eta; a.esb = desc->eta_stride_b; a.esh = desc->eta_stride_h; a.est = desc->eta_stride_t;
  a.dZ = dZ; a.dW1f = dW1_final; a.dW2f = dW2_final;
  a.ws = static_cast<float*>(workspace);
  a.dQ = dQ; a.dK = dK; a.dV = dV; a.deta = deta; a.dW1 = dW1_0; a.dW2 = dW2_0;
  a.gamma = gamma; a.beta = beta; a.eps = eps; a.dgamma = dgamma; a.dbeta = dbeta;
  const hipError_t e = ttt::launch_mlp_bwd(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TTT_OK : TTT_ERR_HIP;
}

const char* ttt_mlp_ln_bwd_kernel_name(const ttt_mlp_desc* d) {
  if (!d) return nullptr;
  if (!ttt::mlp_bwd_supported(d->d, d->dh, d->b) || d->out_dtype != TTT_F32) return nullptr;
  return "ttt_mlp_bwd_d64h256 (layer norm)";
}

}  // extern "C"

// ------------------------------------- linear attention, rotary positions --

namespace {

// A strided [B, H, T, d] tensor.
struct View {
  const void* p;
  int64_t B, H, T, d;
  ttt_strides s;
  int64_t size;  // bytes of an element
};

View view(const void* p, int64_t B, int64_t H, int64_t T, int64_t d, ttt_strides s, int32_t dtype) {
  // strides of dimensions of size 1 (or 0) carry nothing
  if (B <= 1) s.b = 0;
  if (H <= 1) s.h = 0;
  if (T <= 1) s.t = 0;
  return View{p, B, H, T, d, s, dtype_size(dtype)};
}

ttt::Strides3 strides(const View& v) { return ttt::Strides3{v.s.b, v.s.h, v.s.t}; }

bool empty(const View& v) { return v.B == 0 || v.H == 0 || v.T == 0; }

// elements from the first to behind the last
int64_t extent(const View& v) { return (v.B - 1) * v.s.b + (v.H - 1) * v.s.h + (v.T - 1) * v.s.t + v.d; }

Range range(const View& v) { return Range{v.p, empty(v) ? 0 : extent(v) * v.size}; }

// strides >= 0, no extent beyond 2^46 elements; an output's elements apart
bool strides_ok(const View& v, bool output) {
  if (v.s.b < 0 || v.s.h < 0 || v.s.t < 0) return false;
  if (empty(v)) return true;
  int64_t st[3] = {v.s.b, v.s.h, v.s.t}, n[3] = {v.B, v.H, v.T};
  int64_t span = v.d;
  for (int i = 0; i < 3; ++i) {
    int64_t e = 1;
    if (n[i] > 1 && (!mul_ok(e, n[i] - 1) || !mul_ok(e, st[i]))) return false;
  }
  if (!output) return true;
  for (int done = 0; done < 3; ++done) {  // smallest stride first
    int m = -1;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && (m < 0 || st[i] < st[m])) m = i;
    if (m < 0) break;
    if (st[m] < span) return false;
    span += (n[m] - 1) * st[m];
    n[m] = 1;
  }
  return true;
}

bool view_aligned(const View& v, int64_t bytes) {
  if (empty(v)) return true;
  return aligned(v.p, static_cast<uintptr_t>(bytes)) && v.s.b * v.size % bytes == 0 && v.s.h * v.size % bytes == 0 &&
         v.s.t * v.size % bytes == 0;
}

// Whether two tensors share memory.  Tensors whose ranges interleave are apart if they
// are slices of the same rows: with some of the dimensions b, h, t (any choice of them)
// of the same strides in both, what the other dimensions reach in the one ends before it
// begins in the other, and both together fit the pitch of the chosen ones, each of which
// holds all of the smaller.
bool views_overlap(const View& a, const View& b) {
  if (!overlaps(range(a), range(b))) return false;
  const View &lo = reinterpret_cast<uintptr_t>(a.p) <= reinterpret_cast<uintptr_t>(b.p) ? a : b;
  const View& hi = &lo == &a ? b : a;
  const int64_t bytes = static_cast<int64_t>(reinterpret_cast<uintptr_t>(hi.p) - reinterpret_cast<uintptr_t>(lo.p));
  if (lo.size != hi.size || bytes % lo.size != 0) return true;
  const int64_t off = bytes / lo.size;
  const int64_t ls[3] = {lo.s.b, lo.s.h, lo.s.t}, ln[3] = {lo.B, lo.H, lo.T};
  const int64_t hs[3] = {hi.s.b, hi.s.h, hi.s.t}, hn[3] = {hi.B, hi.H, hi.T};
  for (int rows = 1; rows < 8; ++rows) {  // the chosen dimensions
    int64_t low = lo.d, end = off + hi.d, n[3], s[3] = {0, 0, 0};
    bool ok = true;
    for (int i = 0; i < 3; ++i) {
      n[i] = 0;
      if (!(rows >> i & 1)) {
        low += (ln[i] - 1) * ls[i];
        end += (hn[i] - 1) * hs[i];
      } else if (ln[i] > 1 || hn[i] > 1) {  // (a dimension of size 1 has no stride)
        ok = ok && (ln[i] == 1 || hn[i] == 1 || ls[i] == hs[i]);
        n[i] = ln[i] > hn[i] ? ln[i] : hn[i];
        s[i] = ln[i] > 1 ? ls[i] : hs[i];
      }
    }
    if (!ok || off < low) continue;
    for (;;) {  // smallest pitch first
      int m = -1;
      for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (m < 0 || s[i] < s[m])) m = i;
      if (m < 0) return false;
      if (s[m] < end) break;
      end += (n[m] - 1) * s[m];
      n[m] = 0;
    }
  }
  return true;
}

bool same_view(const View& a, const View& b) {
  return a.p == b.p && a.s.b == b.s.b && a.s.h == b.s.h && a.s.t == b.s.t && a.size == b.size && a.H == b.H;
}

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 256;  // of a launch
bool finite(float x) { return x - x == 0.f; }

// sizes, types, flags; chains = B * H
ttt_status check_attn_desc(const ttt_linear_attn_desc* d, int64_t* chains) {
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->H < 0 || d->Hkv < 0 || d->T < 0 || d->d < 1 || d->T > kMaxTokens) return TTT_ERR_SHAPE;
  if (d->H > 0 && (d->Hkv < 1 || d->H % d->Hkv != 0)) return TTT_ERR_SHAPE;
  if (!finite(d->scale)) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype)) return TTT_ERR_DTYPE;
  if (d->flags != 0 || d->reserved != 0) return TTT_ERR_FLAGS;
  *chains = 1;
  if (!mul_ok(*chains, d->B) || !mul_ok(*chains, d->H) || *chains > INT_MAX) return TTT_ERR_SHAPE;
  int64_t tok = *chains, wel = *chains;
  if (!mul_ok(tok, d->T) || !mul_ok(tok, d->d) || !mul_ok(wel, d->d) || !mul_ok(wel, d->d)) return TTT_ERR_SHAPE;
  if (d->w0_batch_stride != 0 && d->w0_batch_stride != static_cast<int64_t>(d->H) * d->d * d->d) return TTT_ERR_STRIDE;
  if (!ttt::attn_supported(d->d)) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// From this many segments on a launch of its own carries their states on; below, each workgroup reads those before
// its own.  T2048, us with that launch and without: d128 10 segments of 24 chains 48.6 and 51.8, gradients 137 and
// 160; d64 16 segments of 24 chains 29.4 and 32.5, but 10 of 48 chains 34.3 and 31.8, gradients with 13 of 24 chains
// 57 and 60; 16 segments of 24 chains at d32 22.5 and 20.5, at d16 19.8 and 16.6.
int carry_from(int d, bool backward) { return d == 128 ? 8 : d == 64 ? (backward ? 8 : 16) : 24; }

struct AttnPlan {
  int nseg, seglen;
  int64_t loc, dgpart, dk, dv, bytes;  // workspace offsets
};

AttnPlan attn_plan(const ttt_linear_attn_desc* d, bool backward) {
  AttnPlan p;
  const int64_t chains = static_cast<int64_t>(d->B) * d->H, dd = static_cast<int64_t>(d->d) * d->d * 4;
  const int n = ttt::attn_segments(chains, d->T, d->d, d->in_dtype == TTT_F32 || d->d == 128, backward);
  const int c = ttt::kAttnChunk;
  p.seglen = ((d->T + n - 1) / n + c - 1) / c * c;
  if (p.seglen < c) p.seglen = c;
  p.nseg = d->T > 0 ? (d->T + p.seglen - 1) / p.seglen : 1;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  const bool split = p.nseg > 1;
  p.loc = take(split ? chains * p.nseg * dd * (backward ? 3 : 1) : 0);
  p.dgpart = take(split && backward ? chains * p.nseg * 8 : 0);
  const int64_t part = backward && d->H > d->Hkv ? chains * d->T * d->d * 4 : 0;
  p.dk = take(part);
  p.dv = take(part);
  p.bytes = at;
  return p;
}

ttt::AttnCarryArgs make_carry_args(const ttt_linear_attn_desc* d, const AttnPlan& p, const float* g, float* loc,
                                   bool backward) {
  ttt::AttnCarryArgs a;
  a.chains = static_cast<int64_t>(d->B) * d->H;
  a.H = d->H; a.d = d->d;
  a.nseg = p.nseg; a.seglen = p.seglen;
  a.backward = backward;
  a.log_decay = g; a.loc = loc;
  return a;
}

ttt_status check_rope(const ttt_rope* r, int32_t d, int64_t B, int64_t T, Range* pos, Range* freqs) {
  if (r->rot < 0 || r->rot % 2 != 0 || r->rot > d) return TTT_ERR_SHAPE;
  if (!finite(r->scale)) return TTT_ERR_SHAPE;
  if ((r->interleaved != 0 && r->interleaved != 1) || r->reserved != 0) return TTT_ERR_FLAGS;
  if (r->pos_stride_b < 0 || r->pos_stride_t < 0) return TTT_ERR_STRIDE;
  for (int i = 0; i < 2; ++i) {
    int64_t e = 1;
    if (!mul_ok(e, i ? T : B) || !mul_ok(e, i ? r->pos_stride_t : r->pos_stride_b)) return TTT_ERR_STRIDE;
  }
  if (r->rot > 0 && !r->freqs) return TTT_ERR_NULL;
  if (!aligned(r->pos, 8) || !aligned(r->freqs, 8)) return TTT_ERR_ALIGN;
  const int64_t n = B == 0 || T == 0 ? 0 : (B - 1) * r->pos_stride_b + (T - 1) * r->pos_stride_t + 1;
  *pos = Range{r->pos, n * 8};
  *freqs = Range{r->freqs, static_cast<int64_t>(r->rot) * 4};
  return TTT_OK;
}

ttt::Rope make_rope(const ttt_rope* r) {
  ttt::Rope o;
  o.pos = r ? r->pos : nullptr;
  o.pos_b = r ? r->pos_stride_b : 0;
  o.pos_t = r ? r->pos_stride_t : 0;
  o.pos0 = r ? r->pos_offset : 0;
  o.freqs = r && r->rot > 0 ? r->freqs : nullptr;
  o.rot = r ? r->rot : 0;
  o.interleaved = r && r->interleaved;
  o.scale = r ? r->scale : 1.f;
  return o;
}

// each output against every input and the outputs before it
ttt_status check_alias(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& in : ins)
      if (overlaps(*o, in)) return TTT_ERR_ALIAS;
    for (const Range* p = outs.begin(); p != o; ++p)
      if (overlaps(*o, *p)) return TTT_ERR_ALIAS;
  }
  return TTT_OK;
}

// q, k, v and z (Z or dZ) of the forward and the backward
ttt_status check_attn_views(const ttt_linear_attn_desc* d, const View& q, const View& k, const View& v, const View& z,
                            bool z_out, int64_t align) {
  const bool any = !empty(q);
  if (any && (!q.p || !k.p || !v.p || !z.p)) return TTT_ERR_NULL;
  for (const View* x : {&q, &k, &v})
    if (!strides_ok(*x, false)) return TTT_ERR_STRIDE;
  if (!strides_ok(z, z_out)) return TTT_ERR_STRIDE;
  for (const View* x : {&q, &k, &v, &z})
    if (!view_aligned(*x, align ? align : x->size)) return TTT_ERR_ALIGN;
  (void)d;
  return TTT_OK;
}

ttt_status check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (need == 0) return TTT_OK;
  if (!ws || !aligned(ws, 16) || bytes < need) return TTT_ERR_WORKSPACE;
  return TTT_OK;
}

struct AttnViews {
  View q, k, v, z;
  Range g, w0, lens;
  int64_t state_bytes;
};

AttnViews attn_views(const ttt_linear_attn_desc* d, const void* Q, const void* K, const void* V, const void* Z,
                     const float* g, const float* W0, const int32_t* lens) {
  AttnViews v;
  v.q = view(Q, d->B, d->H, d->T, d->d, d->q, d->in_dtype);
  v.k = view(K, d->B, d->Hkv, d->T, d->d, d->k, d->in_dtype);
  v.v = view(V, d->B, d->Hkv, d->T, d->d, d->v, d->in_dtype);
  v.z = view(Z, d->B, d->H, d->T, d->d, d->z, d->out_dtype);
  const int64_t hdd = static_cast<int64_t>(d->H) * d->d * d->d * 4;
  v.state_bytes = hdd * d->B;
  v.g = Range{g, static_cast<int64_t>(d->H) * 4};
  v.w0 = Range{W0, W0 ? (d->w0_batch_stride ? v.state_bytes : hdd) : 0};
  v.lens = Range{lens, lens ? static_cast<int64_t>(d->B) * 4 : 0};
  return v;
}

ttt_status validate_attn_fwd(const ttt_linear_attn_desc* d, const void* Q, const void* K, const void* V, const float* g,
                             const float* W0, const int32_t* lens, const void* Z, const float* Wf, const void* ws,
                             int64_t ws_bytes) {
  int64_t chains;
  ttt_status st = check_attn_desc(d, &chains);
  if (st != TTT_OK) return st;
  const AttnViews v = attn_views(d, Q, K, V, Z, g, W0, lens);
  const AttnPlan plan = attn_plan(d, false);
  if (chains * plan.nseg * 4 * d->d > kMaxThreads) return TTT_ERR_SHAPE;
  if (chains == 0) return TTT_OK;
  if (!g || !Wf) return TTT_ERR_NULL;
  if ((st = check_attn_views(d, v.q, v.k, v.v, v.z, true, 16)) != TTT_OK) return st;
  if (!aligned(g, 4) || !aligned(lens, 4) || !aligned(W0, 16) || !aligned(Wf, 16)) return TTT_ERR_ALIGN;
  if ((st = check_workspace(ws, ws_bytes, plan.bytes)) != TTT_OK) return st;
  const Range wf{Wf, v.state_bytes}, wsr{ws, plan.bytes}, z = range(v.z);
  if ((st = check_alias({wf, wsr}, {range(v.q), range(v.k), range(v.v), v.g, v.lens, z})) != TTT_OK) return st;
  if ((st = check_alias({z}, {v.g, v.lens})) != TTT_OK) return st;
  if (views_overlap(v.z, v.q) || views_overlap(v.z, v.k) || views_overlap(v.z, v.v)) return TTT_ERR_ALIAS;
  if (overlaps(z, v.w0) || overlaps(wsr, v.w0)) return TTT_ERR_ALIAS;
  if (overlaps(wf, v.w0) && !(Wf == W0 && d->w0_batch_stride != 0)) return TTT_ERR_ALIAS;
  return TTT_OK;
}

ttt_status validate_attn_bwd(const ttt_linear_attn_desc* d, const void* Q, const void* K, const void* V, const float* g,
                             const float* W0, const int32_t* lens, const void* dZ, const float* dWf, const void* dQ,
                             const void* dK, const void* dV, const float* dg, const float* dW0, const void* ws,
                             int64_t ws_bytes) {
  int64_t chains;
  ttt_status st = check_attn_desc(d, &chains);
  if (st != TTT_OK) return st;
  const AttnViews v = attn_views(d, Q, K, V, dZ, g, W0, lens);
  const View dq = view(dQ, d->B, d->H, d->T, d->d, d->dq, d->out_dtype);
  const View dk = view(dK, d->B, d->Hkv, d->T, d->d, d->dk, d->out_dtype);
  const View dv = view(dV, d->B, d->Hkv, d->T, d->d, d->dv, d->out_dtype);
  const AttnPlan plan = attn_plan(d, true);
  if (3 * chains * plan.nseg * 4 * d->d > kMaxThreads) return TTT_ERR_SHAPE;  // the walks
  if (d->H > d->Hkv && 2 * chains / (d->H / d->Hkv) * d->T * (d->d / 4) + chains > kMaxThreads) return TTT_ERR_SHAPE;  // the sums
  if (chains == 0) return TTT_OK;
  if (!g || !dg || !dW0) return TTT_ERR_NULL;
  if (!empty(dq) && (!dQ || !dK || !dV)) return TTT_ERR_NULL;
  if ((st = check_attn_views(d, v.q, v.k, v.v, v.z, false, 16)) != TTT_OK) return st;
  for (const View* x : {&dq, &dk, &dv}) {
    if (!strides_ok(*x, true)) return TTT_ERR_STRIDE;
    if (!view_aligned(*x, 16)) return TTT_ERR_ALIGN;
  }
  if (!aligned(g, 4) || !aligned(lens, 4) || !aligned(W0, 16) || !aligned(dWf, 16) || !aligned(dg, 4) ||
      !aligned(dW0, 16))
    return TTT_ERR_ALIGN;
  if ((st = check_workspace(ws, ws_bytes, plan.bytes)) != TTT_OK) return st;
  const Range wsr{ws, plan.bytes}, dgr{dg, chains * 4}, dw0r{dW0, v.state_bytes};
  const Range dwf{dWf, dWf ? v.state_bytes : 0};
  const Range dqr = range(dq), dkr = range(dk), dvr = range(dv);
  for (const Range& o : {dqr, dkr, dvr, dgr, dw0r, wsr})
    for (const Range& in : {v.g, v.w0, v.lens, dwf})
      if (overlaps(o, in)) return TTT_ERR_ALIAS;
  for (const View* in : {&v.q, &v.k, &v.v, &v.z}) {
    for (const View* o : {&dq, &dk, &dv})
      if (views_overlap(*o, *in)) return TTT_ERR_ALIAS;
    for (const Range& o : {dgr, dw0r, wsr})
      if (overlaps(o, range(*in))) return TTT_ERR_ALIAS;
  }
  if ((st = check_alias({dgr, dw0r, wsr}, {dqr, dkr, dvr})) != TTT_OK) return st;
  if (views_overlap(dq, dk) || views_overlap(dq, dv) || views_overlap(dk, dv)) return TTT_ERR_ALIAS;
  return TTT_OK;
}

ttt_status validate_attn_decode(const ttt_linear_attn_desc* d, const void* Q, const void* K, const void* V,
                                const float* g, const int32_t* lens, const ttt_rope* rope, const void* Z,
                                const float* W) {
  int64_t chains;
  ttt_status st = check_attn_desc(d, &chains);
  if (st != TTT_OK) return st;
  if (d->w0_batch_stride != 0) return TTT_ERR_STRIDE;
  if (chains * 4 * d->d > kMaxThreads) return TTT_ERR_SHAPE;
  Range pos{nullptr, 0}, freqs{nullptr, 0};
  if (rope && (st = check_rope(rope, d->d, d->B, d->T, &pos, &freqs)) != TTT_OK) return st;
  if (chains == 0) return TTT_OK;
  if (!g || !W) return TTT_ERR_NULL;
  const AttnViews v = attn_views(d, Q, K, V, Z, g, nullptr, lens);
  if ((st = check_attn_views(d, v.q, v.k, v.v, v.z, true, 0)) != TTT_OK) return st;
  if (!aligned(g, 4) || !aligned(lens, 4) || !aligned(W, 16)) return TTT_ERR_ALIGN;
  if (views_overlap(v.z, v.q) || views_overlap(v.z, v.k) || views_overlap(v.z, v.v)) return TTT_ERR_ALIAS;
  if ((st = check_alias({range(v.z)}, {v.g, v.lens, pos, freqs})) != TTT_OK) return st;
  return check_alias({Range{W, v.state_bytes}},
                     {range(v.q), range(v.k), range(v.v), range(v.z), v.g, v.lens, pos, freqs});
}

struct RotaryViews {
  View q, k, qo, ko;
};

RotaryViews rotary_views(const ttt_rotary_desc* d, const void* q, const void* k, const void* qo, const void* ko) {
  return RotaryViews{view(q, d->B, d->H, d->T, d->d, d->q, d->dtype), view(k, d->B, d->Hkv, d->T, d->d, d->k, d->dtype),
                     view(qo, d->B, d->H, d->T, d->d, d->q_out, d->dtype),
                     view(ko, d->B, d->Hkv, d->T, d->d, d->k_out, d->dtype)};
}

ttt_status validate_rotary(const ttt_rotary_desc* d, const ttt_rope* rope, const void* q, const void* k, const void* qo,
                           const void* ko) {
  if (!d || !rope) return TTT_ERR_NULL;
  if (d->B < 0 || d->H < 0 || d->Hkv < 0 || d->T < 0 || d->d < 1 || d->T > kMaxTokens) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->dtype)) return TTT_ERR_DTYPE;
  if ((d->flags & ~TTT_FLAG_INVERSE) || d->reserved != 0) return TTT_ERR_FLAGS;
  const int64_t heads = static_cast<int64_t>(d->H) + d->Hkv;
  int64_t n = 1;
  if (heads > INT_MAX || !mul_ok(n, d->B) || !mul_ok(n, d->T) || !mul_ok(n, d->d)) return TTT_ERR_SHAPE;
  if (n > kMaxThreads || !mul_ok(n, heads)) return TTT_ERR_SHAPE;
  Range pos, freqs;
  ttt_status st = check_rope(rope, d->d, d->B, d->T, &pos, &freqs);
  if (st != TTT_OK) return st;
  const RotaryViews v = rotary_views(d, q, k, qo, ko);
  if (empty(v.q) && empty(v.k)) return TTT_OK;
  if ((!empty(v.q) && (!q || !qo)) || (!empty(v.k) && (!k || !ko))) return TTT_ERR_NULL;
  for (const View* x : {&v.q, &v.k})
    if (!strides_ok(*x, false)) return TTT_ERR_STRIDE;
  for (const View* x : {&v.qo, &v.ko})
    if (!strides_ok(*x, true)) return TTT_ERR_STRIDE;
  for (const View* x : {&v.q, &v.k, &v.qo, &v.ko})
    if (!view_aligned(*x, x->size)) return TTT_ERR_ALIGN;
  if ((!same_view(v.q, v.qo) && views_overlap(v.q, v.qo)) || (!same_view(v.k, v.ko) && views_overlap(v.k, v.ko)))
    return TTT_ERR_ALIAS;
  if (views_overlap(v.qo, v.ko) || views_overlap(v.qo, v.k) || views_overlap(v.ko, v.q)) return TTT_ERR_ALIAS;
  for (const Range& o : {range(v.qo), range(v.ko)})
    if (overlaps(o, pos) || overlaps(o, freqs)) return TTT_ERR_ALIAS;
  return TTT_OK;
}

// a valid call's launch; false: nothing to do
bool rotary_args(const ttt_rotary_desc* desc, const ttt_rope* rope, const void* q, const void* k, void* q_out, void* k_out,
                 ttt::RotaryArgs* args) {
  const RotaryViews v = rotary_views(desc, q, k, q_out, k_out);
  if (empty(v.q) && empty(v.k)) return false;
  ttt::RotaryArgs& a = *args;
  a.B = desc->B; a.H = desc->H; a.Hkv = desc->Hkv; a.T = desc->T; a.d = desc->d;
  a.dtype = desc->dtype;
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
  a.qs = strides(v.q); a.ks = strides(v.k); a.qos = strides(v.qo); a.kos = strides(v.ko);
  a.rope = make_rope(rope);
  a.inverse = (desc->flags & TTT_FLAG_INVERSE) != 0;
  a.in_place = (desc->H == 0 || same_view(v.q, v.qo)) && (desc->Hkv == 0 || same_view(v.k, v.ko));
  return !(a.in_place && a.rope.rot == 0);
}

ttt_status hip_status(hipError_t e) { return e == hipSuccess ? TTT_OK : TTT_ERR_HIP; }

}  // namespace

extern "C" {

int64_t ttt_linear_attn_workspace_bytes(const ttt_linear_attn_desc* desc, int32_t backward) {
  int64_t chains;
  if (check_attn_desc(desc, &chains) != TTT_OK) return -1;
  return chains == 0 ? 0 : attn_plan(desc, backward != 0).bytes;
}

ttt_status ttt_linear_attn_fwd_validate(const ttt_linear_attn_desc* desc, const void* Q, const void* K, const void* V,
                                        const float* log_decay, const float* W0, const int32_t* lens, const void* Z,
                                        const float* W_final, const void* workspace, int64_t workspace_bytes) {
  return validate_attn_fwd(desc, Q, K, V, log_decay, W0, lens, Z, W_final, workspace, workspace_bytes);
}

ttt_status ttt_linear_attn_fwd(const ttt_linear_attn_desc* desc, const void* Q, const void* K, const void* V,
                               const float* log_decay, const float* W0, const int32_t* lens, void* Z, float* W_final,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  const ttt_status st =
      validate_attn_fwd(desc, Q, K, V, log_decay, W0, lens, Z, W_final, workspace, workspace_bytes);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  const AttnViews v = attn_views(desc, Q, K, V, Z, log_decay, W0, lens);
  const AttnPlan plan = attn_plan(desc, false);
  ttt::AttnArgs a;
  a.B = desc->B; a.H = desc->H; a.T = desc->T; a.d = desc->d;
  a.group = desc->H / desc->Hkv;
  a.nseg = plan.nseg; a.seglen = plan.seglen;
  a.in_dtype = desc->in_dtype; a.out_dtype = desc->out_dtype;
  a.Q = Q; a.K = K; a.V = V;
  a.qs = strides(v.q); a.ks = strides(v.k); a.vs = strides(v.v); a.zs = strides(v.z);
  a.log_decay = log_decay; a.scale = desc->scale;
  a.W0 = W0; a.w0_bstride = desc->w0_batch_stride;
  a.lens = lens;
  a.loc = static_cast<float*>(workspace);
  a.Z = Z; a.W_final = W_final;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  a.carried = plan.nseg >= carry_from(a.d, false);
  if (plan.nseg > 1 && ttt::launch_attn_states(a, s) != hipSuccess) return TTT_ERR_HIP;
  if (a.carried && ttt::launch_attn_carry(make_carry_args(desc, plan, log_decay, a.loc, false), s) != hipSuccess)
    return TTT_ERR_HIP;
  return hip_status(ttt::launch_attn_fwd(a, s));
}

ttt_status ttt_linear_attn_bwd_validate(const ttt_linear_attn_desc* desc, const void* Q, const void* K, const void* V,
                                        const float* log_decay, const float* W0, const int32_t* lens, const void* dZ,
                                        const float* dW_final, const void* dQ, const void* dK, const void* dV,
                                        const float* dlog_decay, const float* dW0, const void* workspace,
                                        int64_t workspace_bytes) {
  return validate_attn_bwd(desc, Q, K, V, log_decay, W0, lens, dZ, dW_final, dQ, dK, dV, dlog_decay, dW0, workspace,
                           workspace_bytes);
}

ttt_status ttt_linear_attn_bwd(const ttt_linear_attn_desc* desc, const void* Q, const void* K, const void* V,
                               const float* log_decay, const float* W0, const int32_t* lens, const void* dZ,
                               const float* dW_final, void* dQ, void* dK, void* dV, float* dlog_decay, float* dW0,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  const ttt_status st = validate_attn_bwd(desc, Q, K, V, log_decay, W0, lens, dZ, dW_final, dQ, dK, dV, dlog_decay, dW0,
                                          workspace, workspace_bytes);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0) return TTT_OK;
  const AttnViews v = attn_views(desc, Q, K, V, dZ, log_decay, W0, lens);
  const AttnPlan plan = attn_plan(desc, true);
  char* ws = static_cast<char*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int group = desc->H / desc->Hkv;

  ttt::AttnBwdArgs r;
  r.B = desc->B; r.H = desc->H; r.T = desc->T; r.d = desc->d;
  r.group = group;
  r.nseg = plan.nseg; r.seglen = plan.seglen;
  r.in_dtype = desc->in_dtype; r.out_dtype = desc->out_dtype;
  r.Q = Q; r.K = K; r.V = V; r.dZ = dZ;
  r.qs = strides(v.q); r.ks = strides(v.k); r.vs = strides(v.v); r.zs = strides(v.z);
  r.log_decay = log_decay; r.scale = desc->scale;
  r.W0 = W0; r.w0_bstride = desc->w0_batch_stride;
  r.lens = lens; r.dWf = dW_final;
  r.loc = reinterpret_cast<float*>(ws + plan.loc);
  r.dgpart = reinterpret_cast<double*>(ws + plan.dgpart);
  r.parts = group > 1;
  const ttt::Strides3 dks = strides(view(dK, desc->B, desc->Hkv, desc->T, desc->d, desc->dk, desc->out_dtype));
  const ttt::Strides3 dvs = strides(view(dV, desc->B, desc->Hkv, desc->T, desc->d, desc->dv, desc->out_dtype));
  const int64_t hs = static_cast<int64_t>(desc->T) * desc->d;
  const ttt::Strides3 packed{hs * desc->H, hs, desc->d};
  r.dQ = dQ;
  r.dK = r.parts ? ws + plan.dk : dK;
  r.dV = r.parts ? ws + plan.dv : dV;
  r.dqs = strides(view(dQ, desc->B, desc->H, desc->T, desc->d, desc->dq, desc->out_dtype));
  r.dks = r.parts ? packed : dks;
  r.dvs = r.parts ? packed : dvs;
  r.dg = dlog_decay; r.dW0 = dW0;
  r.carried = plan.nseg >= carry_from(r.d, true);
  if (plan.nseg > 1 && ttt::launch_attn_bwd_states(r, s) != hipSuccess) return TTT_ERR_HIP;
  if (r.carried && ttt::launch_attn_carry(make_carry_args(desc, plan, log_decay, r.loc, true), s) != hipSuccess)
    return TTT_ERR_HIP;
  if (ttt::launch_attn_bwd(r, s) != hipSuccess) return TTT_ERR_HIP;

  ttt::AttnSumArgs m;
  m.B = desc->B; m.Hkv = desc->Hkv; m.T = desc->T; m.d = desc->d;
  m.group = group; m.nseg = plan.nseg; m.out_dtype = desc->out_dtype;
  m.dk_parts = r.parts ? static_cast<const float*>(r.dK) : nullptr;
  m.dv_parts = r.parts ? static_cast<const float*>(r.dV) : nullptr;
  m.dK = dK; m.dV = dV;
  m.dks = dks; m.dvs = dvs;
  m.dgpart = plan.nseg > 1 ? r.dgpart : nullptr;
  m.dg = dlog_decay;
  return hip_status(ttt::launch_attn_sum(m, s));
}

ttt_status ttt_linear_attn_decode_validate(const ttt_linear_attn_desc* desc, const void* Q, const void* K,
                                           const void* V, const float* log_decay, const int32_t* lens,
                                           const ttt_rope* rope, const void* Z, const float* W) {
  return validate_attn_decode(desc, Q, K, V, log_decay, lens, rope, Z, W);
}

ttt_status ttt_linear_attn_decode(const ttt_linear_attn_desc* desc, const void* Q, const void* K, const void* V,
                                  const float* log_decay, const int32_t* lens, const ttt_rope* rope, void* Z, float* W,
                                  void* stream) {
  const ttt_status st = validate_attn_decode(desc, Q, K, V, log_decay, lens, rope, Z, W);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->H == 0 || desc->T == 0) return TTT_OK;
  const AttnViews v = attn_views(desc, Q, K, V, Z, log_decay, nullptr, lens);
  ttt::AttnDecodeArgs a;
  a.B = desc->B; a.H = desc->H; a.T = desc->T; a.d = desc->d;
  a.group = desc->H / desc->Hkv;
  a.in_dtype = desc->in_dtype; a.out_dtype = desc->out_dtype;
  a.Q = Q; a.K = K; a.V = V;
  a.qs = strides(v.q); a.ks = strides(v.k); a.vs = strides(v.v); a.os = strides(v.z);
  a.log_decay = log_decay; a.scale = desc->scale;
  a.lens = lens; a.W = W; a.Z = Z;
  a.rope = make_rope(rope);
  return hip_status(ttt::launch_attn_decode(a, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_rotary_validate(const ttt_rotary_desc* desc, const ttt_rope* rope, const void* q, const void* k,
                               const void* q_out, const void* k_out) {
  return validate_rotary(desc, rope, q, k, q_out, k_out);
}

const char* ttt_rotary_kernel_name(const ttt_rotary_desc* desc, const ttt_rope* rope, const void* q, const void* k,
                                   const void* q_out, const void* k_out) {
  ttt::RotaryArgs a;
  if (validate_rotary(desc, rope, q, k, q_out, k_out) != TTT_OK) return nullptr;
  if (!rotary_args(desc, rope, q, k, const_cast<void*>(q_out), const_cast<void*>(k_out), &a)) return nullptr;
  return ttt::rotary_name(a);
}

ttt_status ttt_rotary(const ttt_rotary_desc* desc, const ttt_rope* rope, const void* q, const void* k, void* q_out,
                      void* k_out, void* stream) {
  const ttt_status st = validate_rotary(desc, rope, q, k, q_out, k_out);
  if (st != TTT_OK) return st;
  ttt::RotaryArgs a;
  if (!rotary_args(desc, rope, q, k, q_out, k_out, &a)) return TTT_OK;
  return hip_status(ttt::launch_rotary(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ------------------------- short convolution, selective scan, block norm --

namespace {

// Strides, alignment to whole elements and overlap of a call's tensors (a null one is not there).  own: an output that may
// be exactly that input.
ttt_status check_tensors(std::initializer_list<View> ins, std::initializer_list<View> outs,
                         std::initializer_list<Range> flat_ins, std::initializer_list<Range> flat_outs,
                         const View* own_out = nullptr, const View* own_in = nullptr) {
  for (const View& v : ins) {
    if (!v.p) continue;
    if (!strides_ok(v, false)) return TTT_ERR_STRIDE;
    if (!view_aligned(v, v.size)) return TTT_ERR_ALIGN;
  }
  for (const View& v : outs) {
    if (!v.p) continue;
    if (!strides_ok(v, true)) return TTT_ERR_STRIDE;
    if (!view_aligned(v, v.size)) return TTT_ERR_ALIGN;
  }
  for (const View* o = outs.begin(); o != outs.end(); ++o) {
    if (!o->p) continue;
    for (const View& in : ins) {
      if (!in.p) continue;
      if (own_out && own_in && same_view(*o, *own_out) && same_view(in, *own_in) && same_view(*o, in)) continue;
      if (views_overlap(*o, in)) return TTT_ERR_ALIAS;
    }
    for (const View* p = outs.begin(); p != o; ++p)
      if (p->p && views_overlap(*o, *p)) return TTT_ERR_ALIAS;
    for (const Range& in : flat_ins)
      if (overlaps(range(*o), in)) return TTT_ERR_ALIAS;
    for (const Range& f : flat_outs)
      if (overlaps(range(*o), f)) return TTT_ERR_ALIAS;
  }
  for (const Range* f = flat_outs.begin(); f != flat_outs.end(); ++f) {
    for (const View& in : ins)
      if (in.p && overlaps(*f, range(in))) return TTT_ERR_ALIAS;
    for (const Range& in : flat_ins)
      if (overlaps(*f, in)) return TTT_ERR_ALIAS;
    for (const Range* g = flat_outs.begin(); g != f; ++g)
      if (overlaps(*f, *g)) return TTT_ERR_ALIAS;
  }
  return TTT_OK;
}

bool all_aligned(std::initializer_list<const void*> ps, uintptr_t n) {
  for (const void* p : ps)
    if (!aligned(p, n)) return false;
  return true;
}

bool all_wide(std::initializer_list<View> vs) {
  for (const View& v : vs)
    if (v.p && !view_aligned(v, 16)) return false;
  return true;
}

ttt::Strides2 strides2(const View& v) { return ttt::Strides2{v.s.b, v.s.t}; }

View rows_view(const void* p, int64_t B, int64_t T, int64_t D, ttt_strides s, int32_t dtype) {
  s.h = 0;
  return view(p, B, 1, T, D, s, dtype);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

Range floats(const float* p, int64_t n) { return Range{p, p ? n * 4 : 0}; }

// ---- short convolution

ttt_status check_conv_desc(const ttt_short_conv_desc* d) {
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->T < 0 || d->D < 1 || d->K < 1 || d->T > kMaxTokens) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype)) return TTT_ERR_DTYPE;
  if ((d->flags & ~TTT_FLAG_SILU) || d->reserved != 0) return TTT_ERR_FLAGS;
  int64_t n = 1;
  if (!mul_ok(n, d->B) || !mul_ok(n, d->T > 0 ? d->T : 1) || !mul_ok(n, d->D)) return TTT_ERR_SHAPE;
  if (d->K < 2 || d->K > 4) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

struct ConvPlan {
  int seg, nparts;  // tokens a thread walks, rows of partial sums a sequence
  int64_t bytes;
};

// The backward's segments: 8 of them to a workgroup, 16 to 128 tokens each, as long as there are 2^17 walks.  Shorter ones read
// and compute K - 1 tokens more often, longer ones leave fewer walks.  us, bf16 and K = 4 but for the last column:
//   B x T x D      1 x 512 x 1536  8 x 2048 x 1536  4 x 2048 x 4096  4 x 8192 x 4096  8 x 2048 x 1536 fp32
//   chosen              16: 23          24: 53           32: 64          128: 217              48: 79
//   8 tokens               16              50               68               248                  79
//   16                     23              41               65               211                  75
//   24                     30              51               58               200                  89
//   32                     37              52               61               197                  69
//   64                     64              79               95               216                  89
//   128                   123             147              172               212                 147
// How many workgroups come out for the 256 CUs, which the rule does not look at, decides as much as the length: the choice is 10 to
// 27% above the best of these, at 1 x 512 44%.
ConvPlan conv_plan(const ttt_short_conv_desc* d) {
  ConvPlan p;
  const int64_t pieces = ceil_div(d->D, d->in_dtype == TTT_BF16 ? 8 : 4);
  int64_t seg = static_cast<int64_t>(d->T) * d->B * pieces >> 17;
  p.seg = static_cast<int>(seg < 16 ? 16 : seg > 128 ? 128 : seg);
  p.nparts = static_cast<int>(d->T > 0 ? ceil_div(ceil_div(d->T, p.seg), 8) : 1);
  p.bytes = static_cast<int64_t>(d->B) * p.nparts * d->D * (d->K + 1) * 4;
  return p;
}

struct ConvViews {
  View x, y, dx;
  Range w, bias, lens;
  int64_t state_in, state_out;  // bytes
};

ConvViews conv_views(const ttt_short_conv_desc* d, const void* X, const float* w, const float* bias, const int32_t* lens,
                     const void* Y, const void* dX) {
  ConvViews v;
  v.x = rows_view(X, d->B, d->T, d->D, d->x, d->in_dtype);
  v.y = rows_view(Y, d->B, d->T, d->D, d->y, d->out_dtype);
  v.dx = rows_view(dX, d->B, d->T, d->D, d->dx, d->out_dtype);
  v.w = floats(w, static_cast<int64_t>(d->D) * d->K);
  v.bias = floats(bias, d->D);
  v.lens = Range{lens, lens ? static_cast<int64_t>(d->B) * 4 : 0};
  const int64_t n = static_cast<int64_t>(d->B) * (d->K - 1) * d->D;
  v.state_in = n * dtype_size(d->in_dtype);
  v.state_out = n * dtype_size(d->out_dtype);
  return v;
}

ttt_status validate_conv_fwd(const ttt_short_conv_desc* d, const void* X, const float* w, const float* bias,
                             const void* state, const int32_t* lens, const void* Y, const void* state_final, bool decode) {
  ttt_status st = check_conv_desc(d);
  if (st != TTT_OK) return st;
  const int64_t blocks = ceil_div(d->D, d->in_dtype == TTT_BF16 ? 8 * 64 : 4 * 64);  // waves of a row
  if (static_cast<int64_t>(d->B) * (decode ? 1 : ceil_div(d->T, 8) + 1) * blocks * 64 > kMaxThreads) return TTT_ERR_SHAPE;
  if (d->B == 0) return TTT_OK;
  if (!w || (decode && !state_final)) return TTT_ERR_NULL;
  if (d->T > 0 && (!X || !Y)) return TTT_ERR_NULL;
  const ConvViews v = conv_views(d, X, w, bias, lens, Y, nullptr);
  if (!all_aligned({w, bias, lens}, 4) || !all_aligned({state, state_final}, dtype_size(d->in_dtype))) return TTT_ERR_ALIGN;
  const Range s{state, state ? v.state_in : 0}, f{state_final, state_final ? v.state_in : 0};
  return check_tensors({v.x}, {v.y}, {v.w, v.bias, v.lens, s}, {f});
}

ttt_status validate_conv_bwd(const ttt_short_conv_desc* d, const void* X, const float* w, const float* bias,
                             const void* state, const int32_t* lens, const void* dY, const void* dstate_final,
                             const void* dX, const float* dw, const float* dbias, const void* dstate, const void* ws,
                             int64_t ws_bytes) {
  ttt_status st = check_conv_desc(d);
  if (st != TTT_OK) return st;
  const ConvPlan plan = conv_plan(d);
  const int64_t pieces = ceil_div(d->D, d->in_dtype == TTT_BF16 ? 8 : 4);
  if (static_cast<int64_t>(d->B) * plan.nparts * ceil_div(pieces, 32) * 256 > kMaxThreads) return TTT_ERR_SHAPE;
  if (static_cast<int64_t>(d->D) * (d->K + 1) > kMaxThreads / 16) return TTT_ERR_SHAPE;  // the sums
  if (!w || !dw) return TTT_ERR_NULL;
  if (static_cast<int64_t>(d->B) * d->T > 0 && (!X || !dY || !dX)) return TTT_ERR_NULL;
  const ConvViews v = conv_views(d, X, w, bias, lens, dY, dX);
  if (!all_aligned({w, bias, lens, dw, dbias}, 4) || !aligned(state, dtype_size(d->in_dtype)) ||
      !all_aligned({dstate, dstate_final}, dtype_size(d->out_dtype)))
    return TTT_ERR_ALIGN;
  if ((st = check_workspace(ws, ws_bytes, plan.bytes)) != TTT_OK) return st;
  const Range s{state, state ? v.state_in : 0}, df{dstate_final, dstate_final ? v.state_out : 0};
  return check_tensors({v.x, v.y}, {v.dx}, {v.w, v.bias, v.lens, s, df},
                       {floats(dw, static_cast<int64_t>(d->D) * d->K), floats(dbias, d->D),
                        Range{dstate, dstate ? v.state_out : 0}, Range{ws, plan.bytes}});
}

ttt::ConvArgs make_conv_args(const ttt_short_conv_desc* d, const ConvViews& v, const void* X, const float* w,
                             const float* bias, const void* state, const int32_t* lens) {
  ttt::ConvArgs a = {};
  a.B = d->B; a.T = d->T; a.D = d->D; a.K = d->K;
  a.in_dtype = d->in_dtype; a.out_dtype = d->out_dtype;
  a.silu = (d->flags & TTT_FLAG_SILU) != 0;
  a.X = X; a.w = w; a.bias = bias; a.state = state; a.lens = lens;
  a.xs = strides2(v.x); a.ys = strides2(v.y); a.dxs = strides2(v.dx);
  return a;
}

// ---- selective scan

ttt_status check_scan_desc(const ttt_selective_scan_desc* d) {
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->T < 0 || d->D < 1 || d->N < 1 || d->G < 1 || d->D % d->G != 0 || d->T > kMaxTokens)
    return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype)) return TTT_ERR_DTYPE;
  if (d->flags & ~TTT_FLAG_SOFTPLUS) return TTT_ERR_FLAGS;
  if (ttt::scan_states(d->N) == 0) return TTT_ERR_UNSUPPORTED;
  int64_t n = 1;
  if (!mul_ok(n, d->B) || !mul_ok(n, d->T > 0 ? d->T : 1) || !mul_ok(n, d->D) || !mul_ok(n, d->N)) return TTT_ERR_SHAPE;
  return TTT_OK;
}

struct ScanPlan {
  int nseg, seglen, chunks;
  int64_t tiles, blocks;  // of channels in a group; workgroups of one segment
  int64_t hseg, sseg, gseg, ckpt, bcpart, part, bytes;
};

// Tokens of a segment: those that take the least time by a model of it.  One workgroup runs on each of the 256 CUs, 64
// channels of one segment, and a launch takes as many rounds as that gives.  One segment of 2048 tokens takes 133 us, its
// gradients 635 to 687: 0.07 and 0.35 us a token.  More than one walk the tokens once more for their start states; what that
// costs (0.85 and 0.3 of a token, 8 us and 0.25 us a segment) is no measurement of its own but was set so that the choice
// comes near the best of 1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48 and 64 segments.  Measured, us, bf16, N = 16:
//   blocks, tokens          8, 2048   24, 2048   24, 8192   48, 2048   96, 2048   128, 2048   144, 2048   288, 2048
//   forward, one segment        133        132        513        133        133         134         136         268
//   forward, chosen              33         41        142         80        111         124         135         268
//   forward, best                31         44        126         70        110         126         136         268
//   gradients, one              635        653       2562        654        658         687         682        1362
//   gradients, chosen            63        146        377        203        349         523         574        1006
//   gradients, best              64        143        373        203        346         466         568        1006
// N and the type are not looked at.  With N = 4, 8 and 32 in bf16 and 4, 8, 16 and 32 in fp32, on all of these but 144, the choice
// is within 6% of the best in 68 cases of 98.  The others are up to 25% above it, in the forward at 8, 48 and 128 workgroups and at
// 8192 tokens, in the gradients at 128; worst are the gradients at 128 with N = 4 in bf16, 341 us for 237.
int64_t scan_seglen(int64_t blocks, int64_t T, bool backward) {
  const double token = backward ? 0.35 : 0.07, twice = backward ? 1.3 : 1.85;
  int64_t best = 0;
  double least = 0.0;
  for (int64_t n = 1; n <= 64 && (n == 1 || (n - 1) * 64 < T); ++n) {
    // segments are whole tiles, so n of them may come out as fewer
    const int64_t len = ceil_div(std::max<int64_t>(ceil_div(T, n), n > 1 ? 64 : 1), ttt::kScanTile) * ttt::kScanTile;
    const int64_t count = std::max<int64_t>(ceil_div(T, len), 1);
    const double rounds = static_cast<double>(ceil_div(blocks * count, 256));
    const double cost =
        rounds * static_cast<double>(len) * token * (count > 1 ? twice : 1.0) + (count > 1 ? 8.0 + 0.25 * count : 0.0);
    if (best == 0 || cost < least) {
      least = cost;
      best = len;
    }
  }
  return best;
}

ScanPlan scan_plan(const ttt_selective_scan_desc* d, bool backward) {
  ScanPlan p;
  p.tiles = ceil_div(d->D / d->G, ttt::kScanCh);
  p.blocks = static_cast<int64_t>(d->B) * d->G * p.tiles;
  p.seglen = static_cast<int>(scan_seglen(p.blocks, d->T, backward));
  p.nseg = static_cast<int>(d->T > 0 ? ceil_div(d->T, p.seglen) : 1);
  p.chunks = static_cast<int>(ceil_div(d->T, ttt::scan_chunk(d->N)));
  int64_t at = 0;
  auto take = [&](bool wanted, int64_t elements) {
    const int64_t o = at;
    if (wanted) at += ceil_div(elements * 4, 256) * 256;
    return o;
  };
  const int64_t bd = static_cast<int64_t>(d->B) * d->D, bdn = bd * d->N;
  p.hseg = take(p.nseg > 1, bdn * p.nseg);
  p.sseg = take(p.nseg > 1, bd * p.nseg);
  p.gseg = take(backward && p.nseg > 1, bdn * p.nseg);
  p.ckpt = take(backward, bdn * p.chunks);
  p.bcpart = take(backward, p.blocks * d->T * 2 * d->N);
  p.part = take(backward, static_cast<int64_t>(d->B) * p.nseg * d->D * (d->N + 2));
  p.bytes = at;
  return p;
}

struct ScanViews {
  View u, dt, z, y, Bm, Cm;
  Range A, D, bias, lens, h0;
  int64_t state;  // bytes
};

ScanViews scan_views(const ttt_selective_scan_desc* d, const void* u, const void* dt, const float* A, const void* Bm,
                     const void* Cm, const float* D, const void* z, const float* bias, const float* h0,
                     const int32_t* lens, const void* y) {
  ScanViews v;
  v.u = rows_view(u, d->B, d->T, d->D, d->u, d->in_dtype);
  v.dt = rows_view(dt, d->B, d->T, d->D, d->dt, d->in_dtype);
  v.z = rows_view(z, d->B, d->T, d->D, d->z, d->in_dtype);
  v.y = rows_view(y, d->B, d->T, d->D, d->y, d->out_dtype);
  v.Bm = view(Bm, d->B, d->G, d->T, d->N, d->Bm, d->in_dtype);
  v.Cm = view(Cm, d->B, d->G, d->T, d->N, d->Cm, d->in_dtype);
  v.A = floats(A, static_cast<int64_t>(d->D) * d->N);
  v.D = floats(D, d->D);
  v.bias = floats(bias, d->D);
  v.lens = Range{lens, lens ? static_cast<int64_t>(d->B) * 4 : 0};
  v.state = static_cast<int64_t>(d->B) * d->D * d->N * 4;
  v.h0 = Range{h0, h0 ? v.state : 0};
  return v;
}

ttt_status validate_scan_fwd(const ttt_selective_scan_desc* d, const void* u, const void* dt, const float* A,
                             const void* Bm, const void* Cm, const float* D, const void* z, const float* bias,
                             const float* h0, const int32_t* lens, const void* y, const float* h, const void* ws,
                             int64_t ws_bytes, bool decode) {
  ttt_status st = check_scan_desc(d);
  if (st != TTT_OK) return st;
  ScanPlan plan = scan_plan(d, false);
  if (decode) plan.bytes = 0;
  if (decode ? static_cast<int64_t>(d->B) * ceil_div(d->D, 16) * 64 > kMaxThreads : plan.blocks * plan.nseg * 512 > kMaxThreads)
    return TTT_ERR_SHAPE;
  if (d->B == 0) return TTT_OK;
  if (!A || !h) return TTT_ERR_NULL;
  if (d->T > 0 && (!u || !dt || !Bm || !Cm || !y)) return TTT_ERR_NULL;
  const ScanViews v = scan_views(d, u, dt, A, Bm, Cm, D, z, bias, h0, lens, y);
  if (!all_aligned({A, D, bias, h0, h, lens}, 4)) return TTT_ERR_ALIGN;
  if ((st = check_workspace(ws, ws_bytes, plan.bytes)) != TTT_OK) return st;
  const Range hf{h, v.state}, wsr{ws, plan.bytes};
  const Range other = h == h0 ? Range{nullptr, 0} : v.h0;  // (the state carried in place)
  if ((st = check_tensors({v.u, v.dt, v.z, v.Bm, v.Cm}, {v.y}, {v.A, v.D, v.bias, v.lens, other}, {hf, wsr})) != TTT_OK)
    return st;
  return TTT_OK;
}

ttt_status validate_scan_bwd(const ttt_selective_scan_desc* d, const void* u, const void* dt, const float* A,
                             const void* Bm, const void* Cm, const float* D, const void* z, const float* bias,
                             const float* h0, const int32_t* lens, const void* dy, const float* dhf, const void* du,
                             const void* ddt, const float* dA, const void* dB, const void* dC, const float* dD,
                             const void* dz, const float* dbias, const float* dh0, const void* ws, int64_t ws_bytes) {
  ttt_status st = check_scan_desc(d);
  if (st != TTT_OK) return st;
  const ScanPlan plan = scan_plan(d, true);
  if (plan.blocks * plan.nseg * 512 > kMaxThreads) return TTT_ERR_SHAPE;
  if (static_cast<int64_t>(d->B) * d->G * d->T * 2 * d->N > kMaxThreads) return TTT_ERR_SHAPE;  // the sums
  if (static_cast<int64_t>(d->D) * (d->N + 2) > kMaxThreads / 16) return TTT_ERR_SHAPE;
  if (!A || !dA) return TTT_ERR_NULL;
  if (static_cast<int64_t>(d->B) * d->T > 0) {
    if (!u || !dt || !Bm || !Cm || !dy || !du || !ddt || !dB || !dC) return TTT_ERR_NULL;
    if ((z != nullptr) != (dz != nullptr)) return TTT_ERR_NULL;
  }
  const ScanViews v = scan_views(d, u, dt, A, Bm, Cm, D, z, bias, h0, lens, dy);
  if (!all_aligned({A, D, bias, h0, lens, dhf, dA, dD, dbias, dh0}, 4)) return TTT_ERR_ALIGN;
  if ((st = check_workspace(ws, ws_bytes, plan.bytes)) != TTT_OK) return st;
  const View vdu = rows_view(du, d->B, d->T, d->D, d->du, d->out_dtype);
  const View vddt = rows_view(ddt, d->B, d->T, d->D, d->ddt, d->out_dtype);
  const View vdz = rows_view(dz, d->B, d->T, d->D, d->dz, d->out_dtype);
  const View vdB = view(dB, d->B, d->G, d->T, d->N, d->dBm, d->out_dtype);
  const View vdC = view(dC, d->B, d->G, d->T, d->N, d->dCm, d->out_dtype);
  return check_tensors({v.u, v.dt, v.z, v.Bm, v.Cm, v.y}, {vdu, vddt, vdz, vdB, vdC},
                       {v.A, v.D, v.bias, v.lens, v.h0, Range{dhf, dhf ? v.state : 0}},
                       {floats(dA, static_cast<int64_t>(d->D) * d->N), floats(dD, d->D), floats(dbias, d->D),
                        Range{dh0, dh0 ? v.state : 0}, Range{ws, plan.bytes}});
}

ttt::ScanArgs make_scan_args(const ttt_selective_scan_desc* d, const ScanViews& v, const void* u, const void* dt,
                             const float* A, const void* Bm, const void* Cm, const float* D, const void* z,
                             const float* bias, const float* h0, const int32_t* lens) {
  ttt::ScanArgs a = {};
  a.B = d->B; a.T = d->T; a.D = d->D; a.N = d->N; a.G = d->G;
  a.in_dtype = d->in_dtype; a.out_dtype = d->out_dtype;
  a.softplus = (d->flags & TTT_FLAG_SOFTPLUS) != 0;
  a.u = u; a.dt = dt; a.z = z; a.Bm = Bm; a.Cm = Cm;
  a.A = A; a.Dskip = D; a.dt_bias = bias; a.h0 = h0; a.lens = lens;
  a.us = strides2(v.u); a.dts = strides2(v.dt); a.zs = strides2(v.z); a.ys = strides2(v.y);
  a.bs = strides(v.Bm); a.cs = strides(v.Cm);
  const int64_t four = 4 * dtype_size(d->in_dtype);
  a.wide = d->D / d->G % 8 == 0 && d->N % 4 == 0 && view_aligned(v.Bm, four) && view_aligned(v.Cm, four) &&
           all_wide({v.u, v.dt, v.z, v.y});
  return a;
}

// ---- block norm

ttt_status check_norm_desc(const ttt_block_norm_desc* d) {
  if (!d) return TTT_ERR_NULL;
  if (d->B < 0 || d->T < 0 || d->D < 1 || d->T > kMaxTokens) return TTT_ERR_SHAPE;
  if (!finite(d->eps) || d->eps < 0.f) return TTT_ERR_SHAPE;
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->res_dtype)) return TTT_ERR_DTYPE;
  if ((d->flags & ~(TTT_FLAG_RMS | TTT_FLAG_GATE_FIRST)) || d->reserved != 0) return TTT_ERR_FLAGS;
  if (d->D > ttt::norm_max_d()) return TTT_ERR_UNSUPPORTED;
  int64_t n = 1;
  if (!mul_ok(n, d->B) || !mul_ok(n, d->T) || !mul_ok(n, d->D)) return TTT_ERR_SHAPE;
  return TTT_OK;
}

// Workgroups of the backward, each with a row of partial sums: as many as stay on the card, with a few rows each.  us, layer norm,
// bf16, with 128, 256, 512, 1024 and 2048 of them:
//   8 x 2048 x 768: 198, 108, 79, 84, 95;  x 2048: 383, 203, 155, 166, 194;  x 4096: 534, 308, 312, 342, 415;
//   x 8192: 1932, 1118, 1151, 1224, 1370;  2 x 512 x 768: 20, 17, 19, 19, 19
int norm_blocks(const ttt_block_norm_desc* d) {
  const int64_t rows = static_cast<int64_t>(d->B) * d->T, most = d->D <= 4096 ? 512 : 256;
  const int64_t n = ceil_div(rows, ttt::norm_teams(d->D));
  return static_cast<int>(n < 1 ? 1 : n < most ? n : most);
}

int64_t norm_bytes(const ttt_block_norm_desc* d) { return static_cast<int64_t>(norm_blocks(d)) * 5 * d->D * 4; }

struct NormViews {
  View x, z, res, s, y;
  Range alpha, gp, bp, gn, bn, lens;
};

NormViews norm_views(const ttt_block_norm_desc* d, const void* X, const void* Z, const void* res, const float* alpha,
                     const float* gp, const float* bp, const float* gn, const float* bn, const int32_t* lens,
                     const void* S, const void* Y) {
  NormViews v;
  v.x = rows_view(X, d->B, d->T, d->D, d->x, d->in_dtype);
  v.z = rows_view(Z, d->B, d->T, d->D, d->z, d->in_dtype);
  v.res = rows_view(res, d->B, d->T, d->D, d->res, d->res_dtype);
  v.s = rows_view(S, d->B, d->T, d->D, d->s, d->res_dtype);
  v.y = rows_view(Y, d->B, d->T, d->D, d->y, d->in_dtype);
  v.alpha = floats(alpha, d->D);
  v.gp = floats(gp, d->D);
  v.bp = floats(bp, d->D);
  v.gn = floats(gn, d->D);
  v.bn = floats(bn, d->D);
  v.lens = Range{lens, lens ? static_cast<int64_t>(d->B) * 4 : 0};
  return v;
}

ttt_status validate_norm_fwd(const ttt_block_norm_desc* d, const void* X, const void* Z, const void* res,
                             const float* alpha, const float* gp, const float* bp, const float* gn, const float* bn,
                             const int32_t* lens, const void* S, const void* Y) {
  const ttt_status st = check_norm_desc(d);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(d->B) * d->T == 0) return TTT_OK;
  if (!X || (!S && !Y) || (bp && !gp) || (Y && !gn) || (bn && !gn)) return TTT_ERR_NULL;
  if (!all_aligned({alpha, gp, bp, gn, bn, lens}, 4)) return TTT_ERR_ALIGN;
  const NormViews v = norm_views(d, X, Z, res, alpha, gp, bp, gn, bn, lens, S, Y);
  return check_tensors({v.x, v.z, v.res}, {v.s, v.y}, {v.alpha, v.gp, v.bp, v.gn, v.bn, v.lens}, {}, &v.s, &v.res);
}

ttt_status validate_norm_bwd(const ttt_block_norm_desc* d, const void* X, const void* Z, const void* res,
                             const float* alpha, const float* gp, const float* bp, const float* gn, const int32_t* lens,
                             const void* dS, const void* dY, const void* dX, const void* dZ, const void* dres,
                             const float* dalpha, const float* dgp, const float* dbp, const float* dgn, const float* dbn,
                             const void* ws, int64_t ws_bytes) {
  ttt_status st = check_norm_desc(d);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(d->B) * d->T > 0) {
    if (!X || !dX || (!dS && !dY) || (Z != nullptr) != (dZ != nullptr)) return TTT_ERR_NULL;
  }
  if ((bp && !gp) || (dY && !gn)) return TTT_ERR_NULL;
  if (!all_aligned({alpha, gp, bp, gn, lens, dalpha, dgp, dbp, dgn, dbn}, 4)) return TTT_ERR_ALIGN;
  const int64_t need = norm_bytes(d);
  if ((st = check_workspace(ws, ws_bytes, need)) != TTT_OK) return st;
  const NormViews v = norm_views(d, X, Z, res, alpha, gp, bp, gn, nullptr, lens, dS, dY);
  const View dx = rows_view(dX, d->B, d->T, d->D, d->dx, d->in_dtype);
  const View dz = rows_view(dZ, d->B, d->T, d->D, d->dz, d->in_dtype);
  const View dr = rows_view(dres, d->B, d->T, d->D, d->dres, d->res_dtype);
  return check_tensors({v.x, v.z, v.res, v.s, v.y}, {dx, dz, dr}, {v.alpha, v.gp, v.bp, v.gn, v.lens},
                       {floats(dalpha, d->D), floats(dgp, d->D), floats(dbp, d->D), floats(dgn, d->D), floats(dbn, d->D),
                        Range{ws, need}});
}

ttt::NormArgs make_norm_args(const ttt_block_norm_desc* d, const NormViews& v, const void* X, const void* Z,
                             const void* res, const float* alpha, const float* gp, const float* bp, const float* gn,
                             const float* bn, const int32_t* lens) {
  ttt::NormArgs a = {};
  a.B = d->B; a.T = d->T; a.D = d->D;
  a.in_dtype = d->in_dtype; a.res_dtype = d->res_dtype;
  a.layer = !(d->flags & TTT_FLAG_RMS);
  a.gate_first = Z && (d->flags & TTT_FLAG_GATE_FIRST);
  a.eps = d->eps;
  a.X = X; a.Z = Z; a.res = res;
  a.alpha = alpha; a.gamma_post = gp; a.beta_post = bp; a.gamma_pre = gn; a.beta_pre = bn;
  a.lens = lens;
  a.xs = strides2(v.x); a.zs = strides2(v.z); a.rs = strides2(v.res); a.ss = strides2(v.s); a.ys = strides2(v.y);
  a.wide = d->D % 8 == 0 && all_wide({v.x, v.z, v.res, v.s, v.y}) && all_aligned({alpha, gp, bp, gn, bn}, 16);
  return a;
}

}  // namespace

extern "C" {

int64_t ttt_short_conv_workspace_bytes(const ttt_short_conv_desc* desc) {
  if (check_conv_desc(desc) != TTT_OK) return -1;
  return conv_plan(desc).bytes;
}

ttt_status ttt_short_conv_fwd_validate(const ttt_short_conv_desc* desc, const void* X, const float* w, const float* bias,
                                       const void* state, const int32_t* lens, const void* Y, const void* state_final) {
  return validate_conv_fwd(desc, X, w, bias, state, lens, Y, state_final, false);
}

ttt_status ttt_short_conv_fwd(const ttt_short_conv_desc* desc, const void* X, const float* w, const float* bias,
                              const void* state, const int32_t* lens, void* Y, void* state_final, void* stream) {
  const ttt_status st = validate_conv_fwd(desc, X, w, bias, state, lens, Y, state_final, false);
  if (st != TTT_OK) return st;
  if (desc->B == 0 || (desc->T == 0 && !state_final)) return TTT_OK;
  const ConvViews v = conv_views(desc, X, w, bias, lens, Y, nullptr);
  ttt::ConvArgs a = make_conv_args(desc, v, X, w, bias, state, lens);
  a.wide = desc->D % (desc->in_dtype == TTT_BF16 ? 8 : 4) == 0 && all_wide({v.x, v.y}) &&
           all_aligned({w, bias, state, state_final}, 16);
  a.Y = Y; a.state_out = state_final;
  return hip_status(ttt::launch_conv_fwd(a, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_short_conv_decode_validate(const ttt_short_conv_desc* desc, const void* X, const float* w,
                                          const float* bias, const int32_t* lens, const void* Y, const void* state) {
  return validate_conv_fwd(desc, X, w, bias, nullptr, lens, Y, state, true);
}

ttt_status ttt_short_conv_decode(const ttt_short_conv_desc* desc, const void* X, const float* w, const float* bias,
                                 const int32_t* lens, void* Y, void* state, void* stream) {
  const ttt_status st = validate_conv_fwd(desc, X, w, bias, nullptr, lens, Y, state, true);
  if (st != TTT_OK) return st;
  if (desc->B == 0 || desc->T == 0) return TTT_OK;
  const ConvViews v = conv_views(desc, X, w, bias, lens, Y, nullptr);
  ttt::ConvArgs a = make_conv_args(desc, v, X, w, bias, nullptr, lens);
  a.wide = desc->D % (desc->in_dtype == TTT_BF16 ? 8 : 4) == 0 && all_wide({v.x, v.y}) && all_aligned({w, bias, state}, 16);
  a.Y = Y; a.state_out = state;
  return hip_status(ttt::launch_conv_decode(a, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_short_conv_bwd_validate(const ttt_short_conv_desc* desc, const void* X, const float* w, const float* bias,
                                       const void* state, const int32_t* lens, const void* dY, const void* dstate_final,
                                       const void* dX, const float* dw, const float* dbias, const void* dstate,
                                       const void* workspace, int64_t workspace_bytes) {
  return validate_conv_bwd(desc, X, w, bias, state, lens, dY, dstate_final, dX, dw, dbias, dstate, workspace,
                           workspace_bytes);
}

ttt_status ttt_short_conv_bwd(const ttt_short_conv_desc* desc, const void* X, const float* w, const float* bias,
                              const void* state, const int32_t* lens, const void* dY, const void* dstate_final, void* dX,
                              float* dw, float* dbias, void* dstate, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  const ttt_status st = validate_conv_bwd(desc, X, w, bias, state, lens, dY, dstate_final, dX, dw, dbias, dstate, workspace,
                                          workspace_bytes);
  if (st != TTT_OK) return st;
  const ConvPlan plan = conv_plan(desc);
  const ConvViews v = conv_views(desc, X, w, bias, lens, dY, dX);
  ttt::ConvArgs a = make_conv_args(desc, v, X, w, bias, state, lens);
  a.wide = desc->D % (desc->in_dtype == TTT_BF16 ? 8 : 4) == 0 && all_wide({v.x, v.y, v.dx}) &&
           all_aligned({w, bias, state, dstate, dstate_final}, 16);
  a.dY = dY; a.dstate_out = dstate_final;
  a.dX = dX; a.dstate = dstate;
  a.seg = plan.seg; a.nparts = plan.nparts;
  a.part = static_cast<float*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (desc->B > 0 && ttt::launch_conv_bwd(a, s) != hipSuccess) return TTT_ERR_HIP;
  ttt::RowSumArgs r = {};
  r.part = a.part;
  r.ld = static_cast<int64_t>(desc->D) * (desc->K + 1);
  r.rows = desc->B * plan.nparts;
  r.n[0] = static_cast<int64_t>(desc->D) * desc->K; r.out[0] = dw;
  r.n[1] = desc->D; r.out[1] = dbias;
  return hip_status(ttt::launch_row_sum(r, s));
}

int64_t ttt_selective_scan_workspace_bytes(const ttt_selective_scan_desc* desc, int32_t backward) {
  if (check_scan_desc(desc) != TTT_OK) return -1;
  return scan_plan(desc, backward != 0).bytes;
}

ttt_status ttt_selective_scan_fwd_validate(const ttt_selective_scan_desc* desc, const void* u, const void* dt,
                                           const float* A, const void* Bm, const void* Cm, const float* D, const void* z,
                                           const float* dt_bias, const float* h0, const int32_t* lens, const void* y,
                                           const float* h_final, const void* workspace, int64_t workspace_bytes) {
  return validate_scan_fwd(desc, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lens, y, h_final, workspace, workspace_bytes, false);
}

ttt_status ttt_selective_scan_fwd(const ttt_selective_scan_desc* desc, const void* u, const void* dt, const float* A,
                                  const void* Bm, const void* Cm, const float* D, const void* z, const float* dt_bias,
                                  const float* h0, const int32_t* lens, void* y, float* h_final, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  const ttt_status st = validate_scan_fwd(desc, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lens, y, h_final, workspace,
                                          workspace_bytes, false);
  if (st != TTT_OK) return st;
  if (desc->B == 0) return TTT_OK;
  const ScanPlan plan = scan_plan(desc, false);
  const ScanViews v = scan_views(desc, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lens, y);
  ttt::ScanArgs a = make_scan_args(desc, v, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lens);
  a.y = y; a.h_final = h_final;
  a.nseg = plan.nseg; a.seglen = plan.seglen;
  char* ws = static_cast<char*>(workspace);
  a.hseg = reinterpret_cast<float*>(ws + plan.hseg);
  a.sseg = reinterpret_cast<float*>(ws + plan.sseg);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (plan.nseg > 1 && ttt::launch_scan_states(a, s) != hipSuccess) return TTT_ERR_HIP;
  return hip_status(ttt::launch_scan_fwd(a, s));
}

ttt_status ttt_selective_scan_decode_validate(const ttt_selective_scan_desc* desc, const void* u, const void* dt,
                                              const float* A, const void* Bm, const void* Cm, const float* D,
                                              const void* z, const float* dt_bias, const int32_t* lens, const void* y,
                                              const float* h) {
  return validate_scan_fwd(desc, u, dt, A, Bm, Cm, D, z, dt_bias, nullptr, lens, y, h, nullptr, 0, true);
}

ttt_status ttt_selective_scan_decode(const ttt_selective_scan_desc* desc, const void* u, const void* dt, const float* A,
                                     const void* Bm, const void* Cm, const float* D, const void* z, const float* dt_bias,
                                     const int32_t* lens, void* y, float* h, void* stream) {
  const ttt_status st =
      validate_scan_fwd(desc, u, dt, A, Bm, Cm, D, z, dt_bias, nullptr, lens, y, h, nullptr, 0, true);
  if (st != TTT_OK) return st;
  if (desc->B == 0 || desc->T == 0) return TTT_OK;
  const ScanViews v = scan_views(desc, u, dt, A, Bm, Cm, D, z, dt_bias, nullptr, lens, y);
  ttt::ScanArgs a = make_scan_args(desc, v, u, dt, A, Bm, Cm, D, z, dt_bias, nullptr, lens);
  const int64_t four = 4 * dtype_size(desc->in_dtype);
  a.wide = desc->N % 4 == 0 && view_aligned(v.Bm, four) && view_aligned(v.Cm, four) && all_aligned({A, h}, 16);
  a.y = y; a.h_final = h;
  return hip_status(ttt::launch_scan_decode(a, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_selective_scan_bwd_validate(const ttt_selective_scan_desc* desc, const void* u, const void* dt,
                                           const float* A, const void* Bm, const void* Cm, const float* D, const void* z,
                                           const float* dt_bias, const float* h0, const int32_t* lens, const void* dy,
                                           const float* dh_final, const void* du, const void* ddt, const float* dA,
                                           const void* dBm, const void* dCm, const float* dD, const void* dz,
                                           const float* ddt_bias, const float* dh0, const void* workspace,
                                           int64_t workspace_bytes) {
  return validate_scan_bwd(desc, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lens, dy, dh_final, du, ddt, dA, dBm, dCm, dD, dz,
                           ddt_bias, dh0, workspace, workspace_bytes);
}

ttt_status ttt_selective_scan_bwd(const ttt_selective_scan_desc* desc, const void* u, const void* dt, const float* A,
                                  const void* Bm, const void* Cm, const float* D, const void* z, const float* dt_bias,
                                  const float* h0, const int32_t* lens, const void* dy, const float* dh_final, void* du,
                                  void* ddt, float* dA, void* dBm, void* dCm, float* dD, void* dz, float* ddt_bias,
                                  float* dh0, void* workspace, int64_t workspace_bytes, void* stream) {
  const ttt_status st = validate_scan_bwd(desc, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lens, dy, dh_final, du, ddt, dA, dBm,
                                          dCm, dD, dz, ddt_bias, dh0, workspace, workspace_bytes);
  if (st != TTT_OK) return st;
  const ScanPlan plan = scan_plan(desc, true);
  const ScanViews v = scan_views(desc, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lens, dy);
  ttt::ScanArgs a = make_scan_args(desc, v, u, dt, A, Bm, Cm, D, z, dt_bias, h0, lens);
  const View vdu = rows_view(du, desc->B, desc->T, desc->D, desc->du, desc->out_dtype);
  const View vddt = rows_view(ddt, desc->B, desc->T, desc->D, desc->ddt, desc->out_dtype);
  const View vdz = rows_view(dz, desc->B, desc->T, desc->D, desc->dz, desc->out_dtype);
  a.wide = a.wide && all_wide({vdu, vddt, vdz});
  a.dy = dy; a.dh_final = dh_final;
  a.du = du; a.ddt = ddt; a.dz = dz; a.dh0 = dh0;
  a.dus = strides2(vdu); a.ddts = strides2(vddt); a.dzs = strides2(vdz);
  a.nseg = plan.nseg; a.seglen = plan.seglen; a.chunks = plan.chunks;
  char* ws = static_cast<char*>(workspace);
  auto at = [&](int64_t o) { return reinterpret_cast<float*>(ws + o); };
  a.hseg = at(plan.hseg); a.sseg = at(plan.sseg); a.gseg = at(plan.gseg); a.ckpt = at(plan.ckpt);
  a.bcpart = at(plan.bcpart); a.part = at(plan.part);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (desc->B > 0) {
    if (plan.nseg > 1 && ttt::launch_scan_bwd_states(a, s) != hipSuccess) return TTT_ERR_HIP;
    if (ttt::launch_scan_bwd(a, s) != hipSuccess) return TTT_ERR_HIP;
    ttt::ScanBcSumArgs m = {};
    m.B = desc->B; m.T = desc->T; m.N = desc->N; m.G = desc->G;
    m.tiles = static_cast<int>(plan.tiles);
    m.out_dtype = desc->out_dtype;
    m.lens = lens;
    m.part = a.bcpart;
    m.dB = dBm; m.dC = dCm;
    m.dbs = strides(view(dBm, desc->B, desc->G, desc->T, desc->N, desc->dBm, desc->out_dtype));
    m.dcs = strides(view(dCm, desc->B, desc->G, desc->T, desc->N, desc->dCm, desc->out_dtype));
    if (ttt::launch_scan_bc_sum(m, s) != hipSuccess) return TTT_ERR_HIP;
  }
  ttt::RowSumArgs r = {};
  r.part = a.part;
  r.ld = static_cast<int64_t>(desc->D) * (desc->N + 2);
  r.rows = desc->B * plan.nseg;
  r.n[0] = static_cast<int64_t>(desc->D) * desc->N; r.out[0] = dA;
  r.n[1] = desc->D; r.out[1] = dD;
  r.n[2] = desc->D; r.out[2] = ddt_bias;
  return hip_status(ttt::launch_row_sum(r, s));
}

int64_t ttt_block_norm_workspace_bytes(const ttt_block_norm_desc* desc) {
  if (check_norm_desc(desc) != TTT_OK) return -1;
  return norm_bytes(desc);
}

ttt_status ttt_block_norm_fwd_validate(const ttt_block_norm_desc* desc, const void* X, const void* Z, const void* res,
                                       const float* alpha, const float* gamma_post, const float* beta_post,
                                       const float* gamma_pre, const float* beta_pre, const int32_t* lens, const void* S,
                                       const void* Y) {
  return validate_norm_fwd(desc, X, Z, res, alpha, gamma_post, beta_post, gamma_pre, beta_pre, lens, S, Y);
}

ttt_status ttt_block_norm_fwd(const ttt_block_norm_desc* desc, const void* X, const void* Z, const void* res,
                              const float* alpha, const float* gamma_post, const float* beta_post, const float* gamma_pre,
                              const float* beta_pre, const int32_t* lens, void* S, void* Y, void* stream) {
  const ttt_status st =
      validate_norm_fwd(desc, X, Z, res, alpha, gamma_post, beta_post, gamma_pre, beta_pre, lens, S, Y);
  if (st != TTT_OK) return st;
  if (static_cast<int64_t>(desc->B) * desc->T == 0) return TTT_OK;
  const NormViews v = norm_views(desc, X, Z, res, alpha, gamma_post, beta_post, gamma_pre, beta_pre, lens, S, Y);
  ttt::NormArgs a = make_norm_args(desc, v, X, Z, res, alpha, gamma_post, beta_post, gamma_pre, beta_pre, lens);
  a.S = S; a.Y = Y;
  return hip_status(ttt::launch_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

ttt_status ttt_block_norm_bwd_validate(const ttt_block_norm_desc* desc, const void* X, const void* Z, const void* res,
                                       const float* alpha, const float* gamma_post, const float* beta_post,
                                       const float* gamma_pre, const int32_t* lens, const void* dS, const void* dY,
                                       const void* dX, const void* dZ, const void* dres, const float* dalpha,
                                       const float* dgamma_post, const float* dbeta_post, const float* dgamma_pre,
                                       const float* dbeta_pre, const void* workspace, int64_t workspace_bytes) {
  return validate_norm_bwd(desc, X, Z, res, alpha, gamma_post, beta_post, gamma_pre, lens, dS, dY, dX, dZ, dres, dalpha,
                           dgamma_post, dbeta_post, dgamma_pre, dbeta_pre, workspace, workspace_bytes);
}

ttt_status ttt_block_norm_bwd(const ttt_block_norm_desc* desc, const void* X, const void* Z, const void* res,
                              const float* alpha, const float* gamma_post, const float* beta_post, const float* gamma_pre,
                              const int32_t* lens, const void* dS, const void* dY, void* dX, void* dZ, void* dres,
                              float* dalpha, float* dgamma_post, float* dbeta_post, float* dgamma_pre, float* dbeta_pre,
                              void* workspace, int64_t workspace_bytes, void* stream) {
  const ttt_status st =
      validate_norm_bwd(desc, X, Z, res, alpha, gamma_post, beta_post, gamma_pre, lens, dS, dY, dX, dZ, dres, dalpha,
                        dgamma_post, dbeta_post, dgamma_pre, dbeta_pre, workspace, workspace_bytes);
  if (st != TTT_OK) return st;
  const NormViews v = norm_views(desc, X, Z, res, alpha, gamma_post, beta_post, gamma_pre, nullptr, lens, dS, dY);
  ttt::NormArgs a = make_norm_args(desc, v, X, Z, res, alpha, gamma_post, beta_post, gamma_pre, nullptr, lens);
  const View dx = rows_view(dX, desc->B, desc->T, desc->D, desc->dx, desc->in_dtype);
  const View dz = rows_view(dZ, desc->B, desc->T, desc->D, desc->dz, desc->in_dtype);
  const View dr = rows_view(dres, desc->B, desc->T, desc->D, desc->dres, desc->res_dtype);
  a.wide = a.wide && all_wide({dx, dz, dr});
  a.dS = dS; a.dY = dY;
  a.dX = dX; a.dZ = dZ; a.dres = dres;
  a.dxs = strides2(dx); a.dzs = strides2(dz); a.drs = strides2(dr);
  a.blocks = norm_blocks(desc);
  a.part = static_cast<float*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (ttt::launch_norm_bwd(a, s) != hipSuccess) return TTT_ERR_HIP;
  ttt::RowSumArgs r = {};
  r.part = a.part;
  r.ld = static_cast<int64_t>(desc->D) * 5;
  r.rows = a.blocks;
  float* const out[5] = {dalpha, dgamma_post, dbeta_post, dgamma_pre, dbeta_pre};
  for (int k = 0; k < 5; ++k) {
    r.n[k] = desc->D;
    r.out[k] = out[k];
  }
  return hip_status(ttt::launch_row_sum(r, s));
}

}  // extern "C"
