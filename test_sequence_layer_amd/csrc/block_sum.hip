// The second launch of the backward passes around a layer's state: partial sums of the parameters' gradients, added in a
// fixed order, so that the same inputs give the same bits.
#include "block_common.h"

namespace ttt {
namespace {

// 64 columns by R groups of rows; each group's sum in 64 bits, the groups' in LDS.
template <int R>
__global__ __launch_bounds__(64 * R) void ttt_row_sum(RowSumArgs a) {
  __shared__ double sums[R][64];
  const int lane = threadIdx.x & 63, r = threadIdx.x >> 6;
  int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const bool on = c < a.ld;
  double s = 0.0;
  if (on) {
    const float* p = a.part + c;
    int row = r;
    for (; row + 3 * R < a.rows; row += 4 * R) {
      const float x0 = p[row * a.ld], x1 = p[(row + R) * a.ld], x2 = p[(row + 2 * R) * a.ld], x3 = p[(row + 3 * R) * a.ld];
      s += static_cast<double>(x0);
      s += static_cast<double>(x1);
      s += static_cast<double>(x2);
      s += static_cast<double>(x3);
    }
    for (; row < a.rows; row += R) s += static_cast<double>(p[row * a.ld]);
  }
  sums[r][lane] = s;
  __syncthreads();
  if (r != 0 || !on) return;
#pragma unroll
  for (int i = 1; i < R; ++i) s += sums[i][lane];
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    if (c >= 0 && c < a.n[k] && a.out[k]) a.out[k][c] = static_cast<float>(s);
    c -= a.n[k];
  }
}

}  // namespace

hipError_t launch_row_sum(const RowSumArgs& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.ld + 63) / 64);
  if (a.rows >= 32) ttt_row_sum<16><<<grid, 1024, 0, s>>>(a);
  else ttt_row_sum<4><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ttt
