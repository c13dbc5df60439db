// Product of 8-bit integers with a scale for each token and output channel:
//     y[t][o] = xscale[t] wscale[o] sum_k xq[t][k] wq[o][k]
// on the 16x16x64 int8 matrix step (int32 accumulators, exact).
//
// Few tokens: the m x n weight bytes are read once and bound the time.  A
// workgroup owns 16 output channels; its four waves take turns at blocks of 256
// inputs, so together they read 1 KB of each weight row at a time, and join
// their int32 sums in LDS.  Lane l of a step holds 16 inputs of row l % 16; the
// order of the inputs inside a block does not matter as long as both operands
// have the same one.
#include "head_common.h"
#include "head_launch.h"

using namespace lbh;

namespace {

__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// 16 codes of a row, zeros behind its end.
__device__ __forceinline__ i32x4 load_codes(const int8_t* p, long left) {
  if (left >= 16) return load_any<i32x4>(p);
  i32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < left) v[i >> 2] |= (int)((uint32_t)(uint8_t)p[i] << (8 * (i & 3)));
  return v;
}

template <typename Y, int NT>
__global__ __launch_bounds__(256) void lb_q8_skinny_kernel(const LbQ8LinearArgs A) {
  __shared__ i32x4 part[3][NT][64];
  const int w = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, c = lane >> 4;
  const int o0 = blockIdx.x * 16;
  const long t0 = (long)blockIdx.y * (16 * NT);
  const int8_t* wp = A.wq + (long)min(o0 + r, A.m - 1) * A.ldw;
  const int8_t* xp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xp[j] = A.xq + min(t0 + 16 * j + r, A.batch - 1) * A.ldx;
  i32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = i32x4{0, 0, 0, 0};
  for (int k0 = 256 * w; k0 < A.n; k0 += 1024) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = k0 + 64 * s + 16 * c;
      const i32x4 a = load_codes(wp + k, A.n - k);
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = mfma_i8(a, load_codes(xp[j] + k, A.n - k), acc[j]);
    }
  }
  if (w > 0) {
#pragma unroll
    for (int j = 0; j < NT; ++j) part[w - 1][j][lane] = acc[j];
  }
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    i32x4 v = acc[j];
#pragma unroll
    for (int i = 0; i < 3; ++i) v += part[i][j][lane];
    const long t = t0 + 16 * j + r;
    if (t >= A.batch) continue;
    const float xs = A.xscale[t];
    Y* y = (Y*)A.y + t * A.ldy;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = o0 + 4 * c + i;
      if (o < A.m) y[o] = (Y)((float)v[i] * (xs * A.wscale[o]));
    }
  }
}

template <typename Y>
void launch_linear(const LbQ8LinearArgs& a, hipStream_t stream) {
  const unsigned tiles = (a.m + 15) / 16;
  if (a.batch <= 16)
    hipLaunchKernelGGL((lb_q8_skinny_kernel<Y, 1>), dim3(tiles), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((lb_q8_skinny_kernel<Y, 4>), dim3(tiles, (unsigned)((a.batch + 63) / 64)), dim3(256), 0, stream,
                       a);
}

}  // namespace

hipError_t lb_launch_q8_linear(const LbQ8LinearArgs& a, int y_dtype, hipStream_t stream) {
  if (y_dtype == 0)
    launch_linear<float>(a, stream);
  else if (y_dtype == 1)
    launch_linear<f16>(a, stream);
  else
    launch_linear<bf16>(a, stream);
  return hipGetLastError();
}
