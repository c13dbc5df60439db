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

// Many tokens: a tile of BM channels x BN tokens a workgroup of 8 waves (2 x 4),
// each wave WM x WN matrix tiles of 16 x 16.  The reduction runs in chunks of
// 64 inputs, staged through four LDS buffers by direct global-to-LDS loads
// three chunks ahead (rows not aligned to 16 bytes pass through registers
// instead).  A staged row is 64 bytes, four 16-byte slots; slot s of row r
// holds inputs 16 (s ^ f(r)), f(r) = (r / 4 % 4) ^ (r & 2), so that any 8 or 16
// consecutive rows of one 16-input column lie in different banks.
//
// Per chunk a wave multiplies its first half of channel tiles, meets the
// others at the barrier that makes the next chunk visible, and multiplies
// the second half while the next chunk's operands are read: the second
// half's operands and the next first half's are always read one half ahead.
constexpr int kStages = 4;

struct TileAt {
  int bm, bt;
};
// Workgroups that share an XCD (every eighth) take neighbouring tiles: token
// tiles in groups of up to 8, fastest inside a group, so that 32 resident
// workgroups of an XCD read about 4 x 8 different blocks.
__device__ __forceinline__ TileAt tile_at(int tm, int tt) {
  const int n = tm * tt, L = (int)blockIdx.x;
  const int xcd = L & 7, idx = L >> 3, per = n >> 3, rem = n & 7;
  int P = xcd < rem ? xcd * (per + 1) + idx : rem * (per + 1) + (xcd - rem) * per + idx;
  const int group = P / (8 * tm);
  const int width = min(8, tt - 8 * group);
  P -= group * 8 * tm;
  TileAt t;
  t.bm = P / width;
  t.bt = 8 * group + P - t.bm * width;
  return t;
}

template <typename Y, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(512, 2) void lb_q8_tile_kernel(const LbQ8LinearArgs A, int tm, int tt) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the kernel's name only (and has no global-to-LDS loads)
  constexpr int BM = 32 * WM, BN = 64 * WN, HM = WM / 2;
  constexpr int kPieces = (BM + BN) / 16;       // 1 KB pieces (16 rows) of a stage
  constexpr int NL = (kPieces + 7) / 8;         // pieces a wave loads
  constexpr int kBytes = (BM + BN) * 64;
  static_assert(WM % 2 == 0, "two halves of channel tiles");
  __shared__ __align__(16) uint8_t stage0[kBytes], stage1[kBytes], stage2[kBytes], stage3[kBytes];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int r = lane & 15, c4 = lane >> 4;
  const int wm = w >> 2, wn = w & 3;
  const TileAt at = tile_at(tm, tt);
  const int o0 = at.bm * BM;
  const long t0 = (long)at.bt * BN;

  // pieces of this wave: lane l loads slot l % 4 of row l / 4 (rows behind the
  // last are read from the last; a wave without enough pieces repeats one)
  const int8_t* src[NL];
  int lds[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int piece = min(w * NL + i, kPieces - 1);
    const int row = 16 * piece + (lane >> 2);
    const int q = (lane & 3) ^ ((row >> 2) & 3) ^ (row & 2);
    if (row < BM)
      src[i] = A.wq + (long)min(o0 + row, A.m - 1) * A.ldw + 16 * q;
    else
      src[i] = A.xq + min(t0 + row - BM, A.batch - 1) * A.ldx + 16 * q;
    lds[i] = piece * 1024;
  }
  const int C = A.n >> 6;
  auto issue = [&](int c, uint8_t* S) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      if constexpr (DIRECT)
        __builtin_amdgcn_global_load_lds(src[i] + 64l * c,
                                         (__attribute__((address_space(3))) void*)(S + __builtin_amdgcn_readfirstlane(lds[i])),
                                         16, 0, 0);
      else
        *reinterpret_cast<i32x4*>(S + lds[i] + 16 * lane) = load_any<i32x4>(src[i] + 64l * c);
    }
  };
  const int slot = 16 * (c4 ^ ((r >> 2) & 3) ^ (r & 2));
  const int aoff = (16 * WM * wm + r) * 64 + slot;
  const int boff = (BM + 16 * WN * wn + r) * 64 + slot;
  auto read_a = [&](const uint8_t* S, int half, i32x4* a) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < HM; ++i) a[i] = *reinterpret_cast<const i32x4*>(S + aoff + 1024 * (half * HM + i));
  };
  auto read_b = [&](const uint8_t* S, i32x4* b) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < WN; ++j) b[j] = *reinterpret_cast<const i32x4*>(S + boff + 1024 * j);
  };
  i32x4 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto products = [&](int half, const i32x4* a, const i32x4* b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < HM; ++i)
#pragma unroll
      for (int j = 0; j < WN; ++j) acc[half * HM + i][j] = mfma_i8(a[i], b[j], acc[half * HM + i][j]);
  };
  // a wave's loads of the next chunk have landed (those of the two behind it may be
  // in flight) and its LDS reads too; then all meet
  auto sync = [&]() __attribute__((always_inline)) {
    if constexpr (DIRECT) {
      constexpr int kWait = 2 * NL;
      __builtin_amdgcn_s_waitcnt((kWait & 15) | ((kWait >> 4) << 14) | (7 << 4));
      __builtin_amdgcn_s_barrier();
      __asm__ volatile("" ::: "memory");
    } else {
      __syncthreads();
    }
  };
  if (C > 0) {
    i32x4 alo[HM], ahi[HM], b0[WN], b1[WN];
    auto body = [&](int c, const uint8_t* S, const uint8_t* Snext, uint8_t* Sfree, i32x4* b, i32x4* bn)
        __attribute__((always_inline)) {
      read_a(S, 1, ahi);
      issue(min(c + kStages - 1, C - 1), Sfree);  // past the end: the last chunk again, which nobody reads
      products(0, alo, b);
      sync();
      read_a(Snext, 0, alo);
      read_b(Snext, bn);
      products(1, ahi, b);
    };
    issue(0, stage0);
    issue(min(1, C - 1), stage1);
    issue(min(2, C - 1), stage2);
    sync();
    read_a(stage0, 0, alo);
    read_b(stage0, b0);
    int c = 0;
    for (; c + 4 <= C; c += 4) {
      body(c, stage0, stage1, stage3, b0, b1);
      body(c + 1, stage1, stage2, stage0, b1, b0);
      body(c + 2, stage2, stage3, stage1, b0, b1);
      body(c + 3, stage3, stage0, stage2, b1, b0);
    }
    if (c < C) body(c, stage0, stage1, stage3, b0, b1);
    if (c + 1 < C) body(c + 1, stage1, stage2, stage0, b1, b0);
    if (c + 2 < C) body(c + 2, stage2, stage3, stage1, b0, b1);
  }
  if (A.n & 63) {
    // the last inputs, straight from memory
    const int k = 64 * C + 16 * c4;
    i32x4 b[WN];
#pragma unroll
    for (int j = 0; j < WN; ++j)
      b[j] = load_codes(A.xq + min(t0 + 16 * (WN * wn + j) + r, A.batch - 1) * A.ldx + k, A.n - k);
#pragma unroll
    for (int i = 0; i < WM; ++i) {
      const i32x4 a = load_codes(A.wq + (long)min(o0 + 16 * (WM * wm + i) + r, A.m - 1) * A.ldw + k, A.n - k);
#pragma unroll
      for (int j = 0; j < WN; ++j) acc[i][j] = mfma_i8(a, b[j], acc[i][j]);
    }
  }
  // every load has landed and every wave is past its reads: the stages are free
  __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));
  __syncthreads();

  // Scaled outputs, 16 tokens at a time, through the wave's own part of the
  // stages: 4 channels a lane in, whole 16-byte pieces of a token's 16 WM
  // channels out.
  constexpr int RS = 16 * WM * sizeof(Y) + 16;  // bytes a token (16 more: banks staggered)
  static_assert(2 * 16 * RS <= kBytes, "two waves' tiles fit a stage");
  uint8_t* const st = (w >> 1 == 0 ? stage0 : w >> 1 == 1 ? stage1 : w >> 1 == 2 ? stage2 : stage3) + (w & 1) * (16 * RS);
  const int ob = o0 + 16 * WM * wm;
  float ws[WM][4];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) ws[i][e] = A.wscale[min(ob + 16 * i + 4 * c4 + e, A.m - 1)];
  constexpr int kPer = 16 / sizeof(Y);       // outputs a piece
  constexpr int kTok = 16 * WM / kPer;       // pieces a token
#pragma unroll
  for (int j = 0; j < WN; ++j) {
    const long tb = t0 + 16 * (WN * wn + j);
    const float xs = A.xscale[min(tb + r, A.batch - 1)];
#pragma unroll
    for (int i = 0; i < WM; ++i) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][e] * (xs * ws[i][e]);
      uint8_t* p = st + r * RS + (16 * i + 4 * c4) * sizeof(Y);
      if constexpr (sizeof(Y) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        u32x2 q;
        q[0] = Pair<Y>::pack(v[0], v[1]);
        q[1] = Pair<Y>::pack(v[2], v[3]);
        *reinterpret_cast<u32x2*>(p) = q;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int e = lane; e < 16 * kTok; e += 64) {
      const int t = e / kTok, piece = e % kTok;
      const u32x4 v = *reinterpret_cast<const u32x4*>(st + t * RS + 16 * piece);
      const int o = ob + piece * kPer;
      if (tb + t < A.batch && o < A.m) {
        Y* y = (Y*)A.y + (tb + t) * A.ldy + o;
        if (o + kPer <= A.m) {
          store_any(y, v);
        } else {
          for (int i = 0; o + i < A.m; ++i) y[i] = reinterpret_cast<const Y*>(st + t * RS + 16 * piece)[i];
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
#endif
}

template <typename Y, int WM, int WN>
void launch_tile(const LbQ8LinearArgs& a, hipStream_t stream) {
  const int tm = (a.m + 32 * WM - 1) / (32 * WM);
  const long tt = (a.batch + 64 * WN - 1) / (64 * WN);
  const bool direct = (((uintptr_t)a.xq | (uintptr_t)a.wq | (uintptr_t)a.ldx | (uintptr_t)a.ldw) & 15) == 0;
  const dim3 grid((unsigned)(tm * tt));
  if (direct)
    hipLaunchKernelGGL((lb_q8_tile_kernel<Y, WM, WN, true>), grid, dim3(512), 0, stream, a, tm, (int)tt);
  else
    hipLaunchKernelGGL((lb_q8_tile_kernel<Y, WM, WN, false>), grid, dim3(512), 0, stream, a, tm, (int)tt);
}

template <typename Y>
void launch_linear(const LbQ8LinearArgs& a, hipStream_t stream) {
  const unsigned tiles = (a.m + 15) / 16;
  if (a.batch <= 16)
    hipLaunchKernelGGL((lb_q8_skinny_kernel<Y, 1>), dim3(tiles), dim3(256), 0, stream, a);
  else if (a.batch <= 64)
    hipLaunchKernelGGL((lb_q8_skinny_kernel<Y, 4>), dim3(tiles, (unsigned)((a.batch + 63) / 64)), dim3(256), 0, stream,
                       a);
  else if (a.batch <= 512)
    launch_tile<Y, 2, 4>(a, stream);
  else
    launch_tile<Y, 8, 4>(a, stream);
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
