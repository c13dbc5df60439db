// Product of 8-bit integers with a scale for each token and output channel:
//     y[t][o] = xscale[t] wscale[o] sum_k xq[t][k] wq[o][k]
// on the 16x16x64 int8 matrix step (int32 accumulators, exact, so the order of
// the inputs is free).  Lane l of a step holds 16 inputs of row l % 16; which 16
// does not matter as long as both operands agree.
//
// Three kernels: up to 16 tokens the m x n weight bytes are the time, and
// lb_q8_stream_kernel reads them once without a pause (lb_q8_skinny_kernel where
// there are too few channels to stream, or the tokens do not fit LDS); more
// tokens are tiled, lb_q8_tile_kernel.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "head_common.h"
#include "head_launch.h"

using namespace lbh;

namespace {

typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(1)));  // at any byte

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

// Four channels from o on of token t, scaled and stored.
template <typename Y>
__device__ __forceinline__ void store_tile(const LbQ8LinearArgs& A, i32x4 v, int o, int t, float xs, float4 w4) {
  const float ws[4] = {w4.x, w4.y, w4.z, w4.w};
  if (t >= A.batch) return;
  Y* y = (Y*)A.y + (long)t * A.ldy + o;
  float f[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = (float)v[e] * (xs * ws[e]);
  if (o + 4 <= A.m) {
    if constexpr (sizeof(Y) == 4) {
      u32x4 q;
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = __builtin_bit_cast(uint32_t, f[e]);
      store_any(y, q);
    } else {
      u32x2 q;
      q[0] = Pair<Y>::pack(f[0], f[1]);
      q[1] = Pair<Y>::pack(f[2], f[3]);
      store_any(y, q);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (o + e < A.m) y[e] = (Y)f[e];
  }
}

// Up to 16 tokens, RT channel tiles of 16 a workgroup: its four waves take turns
// at blocks of 256 inputs, so together they read 1 KB of each weight row at a
// time, and join their int32 sums in LDS.  One tile where the channels are few
// (1 x 4096 -> 4096: 5.5 us, streaming 7.1); two where the tokens' codes are read
// from the cache for long rows (16 x 5120 -> 32000: 41 us, with one 47).
template <typename Y, int RT>
__global__ __launch_bounds__(256) void lb_q8_skinny_kernel(const LbQ8LinearArgs A) {
  __shared__ i32x4 part[3][RT][64];
  const int w = wave_id(), lane = threadIdx.x & 63;
  const int r = lane & 15, c = lane >> 4;
  const int o0 = blockIdx.x * (16 * RT);
  const int8_t* wp[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) wp[i] = A.wq + (long)min(o0 + 16 * i + r, A.m - 1) * A.ldw + 16 * c;
  const int8_t* const xp = A.xq + min((long)r, A.batch - 1) * A.ldx + 16 * c;
  i32x4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = i32x4{0, 0, 0, 0};
  const int whole = A.n >> 8;
  for (int k = w; k < whole; k += 4) {
    i32x4 a[RT][4], b[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int i = 0; i < RT; ++i) a[i][s] = load_any<i32x4>(wp[i] + 256 * k + 64 * s);
      b[s] = load_any<i32x4>(xp + 256 * k + 64 * s);
    }
    __builtin_amdgcn_sched_barrier(0);  // all loads are under way before the first product
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[i] = mfma_i8(a[i][s], b[s], acc[i]);
  }
  const int at = 256 * whole + 64 * w;  // what is left, 64 inputs a wave
  if (at < A.n) {
    const i32x4 b = load_codes(xp + at, A.n - at - 16 * c);
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = mfma_i8(load_codes(wp[i] + at, A.n - at - 16 * c), b, acc[i]);
  }
  if (w > 0) {
#pragma unroll
    for (int i = 0; i < RT; ++i) part[w - 1][i][lane] = acc[i];
  }
  __syncthreads();
  if (w > 0) return;
  const float xs = A.xscale[min((long)r, A.batch - 1)];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    i32x4 v = acc[i];
#pragma unroll
    for (int q = 0; q < 3; ++q) v += part[q][i][lane];
    const int o = o0 + 16 * i + 4 * c;
    float4 ws;
    ws.x = A.wscale[min(o, A.m - 1)];
    ws.y = A.wscale[min(o + 1, A.m - 1)];
    ws.z = A.wscale[min(o + 2, A.m - 1)];
    ws.w = A.wscale[min(o + 3, A.m - 1)];
    store_tile<Y>(A, v, o, r, xs, ws);
  }
}

// Up to 16 tokens, streaming: one workgroup of 16 waves a compute unit, the
// tokens' codes in LDS (read once a workgroup, zeros behind them), a tile of 16
// channels after another, its inputs dealt to the waves in units of 128.  A
// wave keeps kRing units (2 KB each) under way, across tiles, so the weights
// stream without a pause at a tile's end.  1 x 5120 -> 32000: 27 us of the 25 that a
// plain read of the weights takes (6.1 TB/s); 16 tokens 31 us.  (Two tiles at a
// time, 8 waves each: the same there, 20% slower for 8192 -> 28672.)
//
// A unit is two loads of 8 rows x 128 bytes, whole cache lines: lane l loads
// row l % 8 (second load: 8 + l % 8), and of its eight 16-byte chunks 2 (l / 16)
// or the one behind it, chosen so that after one exchange with lane l ^ 8 every
// lane holds chunks 2 (l / 16) and 2 (l / 16) + 1 of row l % 16, the operands of two
// matrix steps.  (16 rows x 64 bytes a load, which needs no exchange, reads half
// lines and was 12% slower for the weights and three times for the tokens.)
constexpr int kRing = 4;
constexpr int kStreamWaves = 16;
constexpr size_t kStreamLds = 155 * 1024;  // of the compute unit's 160 KB

__device__ __forceinline__ i32x4 lane_xor8(i32x4 v) {
  i32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (int)lane_xor<8>((uint32_t)v[i]);
  return o;
}

// steps: units a wave takes of a tile; xrow: bytes of a token's codes in LDS.
template <typename Y>
__global__ __launch_bounds__(64 * kStreamWaves) void lb_q8_stream_kernel(const LbQ8LinearArgs A, int tiles, int steps,
                                                                         int xrow, int max_rounds) {
  extern __shared__ __align__(16) uint8_t lds[];
  i32x4* const part = reinterpret_cast<i32x4*>(lds);  // [wave][lane]
  float* const wscale = reinterpret_cast<float*>(lds + kStreamWaves * 64 * 16);  // [round][16]
  const int lane = threadIdx.x & 63, w = wave_id();
  const int r = lane & 15, c = lane >> 4, hi = lane & 8;
  const float xscale = A.xscale[min((long)r, A.batch - 1)];
  const int tile0 = blockIdx.x, stride = gridDim.x;
  const int rounds = (tiles - tile0 + stride - 1) / stride;  // of the workgroup
  const int total = rounds * steps;
  uint8_t* const xs_codes = reinterpret_cast<uint8_t*>(wscale + 16 * max_rounds);

  // the loads' side of the stream
  const int cha = 16 * (2 * c + (hi ? 1 : 0)), chb = 16 * (2 * c + (hi ? 0 : 1));
  int it_tile = tile0, it_step = 0;
  const int8_t *pa, *pb;
  auto aim = [&]() {
    const int o = 16 * min(it_tile, tiles - 1) + (lane & 7);
    pa = A.wq + (long)min(o, A.m - 1) * A.ldw;
    pb = A.wq + (long)min(o + 8, A.m - 1) * A.ldw;
  };
  aim();
  i32x4 ra[kRing], rb[kRing];
  auto issue = [&](i32x4& a, i32x4& b) __attribute__((always_inline)) {
    const int k = 128 * (w + kStreamWaves * it_step);
    // behind the row, and behind the last tile, anything readable
    // does: it meets zeros, or nobody
    const bool live = it_tile < tiles;
    const int ka = k + cha, kb = k + chb;
    a = __builtin_nontemporal_load(reinterpret_cast<const i32x4_any*>(live && ka < A.n ? pa + ka : A.wq));
    b = __builtin_nontemporal_load(reinterpret_cast<const i32x4_any*>(live && kb < A.n ? pb + kb : A.wq));
    if (++it_step == steps) {
      it_step = 0;
      it_tile += stride;
      aim();
    }
  };
#pragma unroll
  for (int i = 0; i < kRing; ++i) issue(ra[i], rb[i]);
  for (int e = threadIdx.x; e < 16 * rounds; e += 64 * kStreamWaves) {
    const int o = 16 * (tile0 + e / 16 * stride) + e % 16;
    wscale[e] = A.wscale[min(o, A.m - 1)];
  }
  {
    // 16-byte chunks of the tokens' codes, zeros behind the last whole one (and one
    // chunk more a row than the units hold: it staggers the banks)
    const int chunks = xrow / 16, all = (int)A.batch * chunks;
    for (int e0 = threadIdx.x; e0 < all; e0 += 4 * 64 * kStreamWaves) {
      i32x4 v[4];
      int at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = e0 + i * 64 * kStreamWaves;
        const int t = e / chunks, k = 16 * (e - t * chunks);
        at[i] = e < all ? t * xrow + k : -1;
        v[i] = load_any<i32x4>(e < all && k < A.n ? A.xq + t * A.ldx + k : A.xq);
        if (k >= A.n) v[i] = i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at[i] >= 0) *reinterpret_cast<i32x4*>(xs_codes + at[i]) = v[i];
    }
  }
  auto meet = [&]() __attribute__((always_inline)) {
    // LDS accesses are done; loads stay under way
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
  };
  meet();

  const uint8_t* const xp = xs_codes + min(r, (int)A.batch - 1) * xrow + 32 * c;
  i32x4 acc = {0, 0, 0, 0};
  int tile = tile0, step = 0, turn = 0, round = 0;
  for (int f = 0; f < total; f += kRing) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      if (f + i >= total) break;
      const i32x4 a = ra[i], b = rb[i];
      i32x4 keep, send;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        keep[e] = hi ? b[e] : a[e];
        send[e] = hi ? a[e] : b[e];
      }
      const uint8_t* xk = xp + 128 * (w + kStreamWaves * step);
      acc = mfma_i8(keep, *reinterpret_cast<const i32x4*>(xk), acc);
      acc = mfma_i8(lane_xor8(send), *reinterpret_cast<const i32x4*>(xk + 16), acc);
      issue(ra[i], rb[i]);
      if (++step < steps) continue;
      // the tile is done: the waves' sums meet in LDS, one wave (in turn) joins them
      meet();  // the readers of the tile before are done
      part[w * 64 + lane] = acc;
      meet();
      if (w == turn) {
        i32x4 v = acc;
#pragma unroll 3
        for (int q = 1; q < kStreamWaves; ++q) v += part[((w + q) & (kStreamWaves - 1)) * 64 + lane];
        // (no global load here: the wait for it would be a wait for all weights under way)
        const float4 ws = *reinterpret_cast<const float4*>(wscale + 16 * round + 4 * c);
        store_tile<Y>(A, v, 16 * tile + 4 * c, r, xscale, ws);
      }
      turn = (turn + 1) & (kStreamWaves - 1);
      acc = i32x4{0, 0, 0, 0};
      step = 0;
      tile += stride;
      ++round;
    }
  }
}

// Many tokens: a tile of BM channels x BN tokens a workgroup of MW x NW waves,
// each wave WM x WN matrix tiles of 16 x 16.  The reduction runs in chunks of
// 128 inputs, staged through ST LDS buffers by direct global-to-LDS loads (rows
// not aligned to 16 bytes pass through registers instead).  A staged row is 128
// bytes, a whole cache line (staging 64 bytes a row, half lines, was 10 to 25%
// slower), in eight 16-byte slots; slot s of row r holds inputs 16 (s ^ (r / 2 % 8)),
// which leaves the 16 lanes that LDS serves at a time in different banks.
//
// Per chunk all waves meet, refill the buffer just left and multiply this
// chunk while the next one's operands are read.  The largest tile, whose
// operands do not fit the registers twice, goes by quarters of a chunk.
//
// What bounds it: 256 x 256 tiles run the matrix units 56% of the time at
// 1.9 GHz, the clock that the card's power leaves for random codes (2000 x 4096 ->
// 32000: 250 us, 2.1 POP/s; the vendor's int8 product of 8192 cubed reaches
// 2.07).  The smaller tiles are bound by what a compute unit loads, about 50
// bytes a ns, and by their start and end of about 5 us.
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

// body(I, c + I) for I = 0, 1, ... as long as c + I < end.
template <typename F, int... I>
__device__ __forceinline__ void chunks_while(F&& body, int c, int end, std::integer_sequence<int, I...>) {
  (void)((c + I < end ? (body(std::integral_constant<int, I>(), c + I), true) : false) && ...);
}

template <typename Y, int WM, int WN, int MW, int NW, int ST, bool DIRECT>
__global__ __launch_bounds__(64 * MW * NW, 2) void lb_q8_tile_kernel(const LbQ8LinearArgs A, int tm, int tt) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the kernel's name only (and has no global-to-LDS loads)
  constexpr int BM = 16 * WM * MW, BN = 16 * WN * NW;
  constexpr int kPieces = (BM + BN) / 8;                   // 1 KB pieces (8 rows) of a stage
  constexpr int NL = (kPieces + MW * NW - 1) / (MW * NW);  // pieces a wave loads
  constexpr int kBytes = (BM + BN) * 128;
  static_assert((ST - 1) * NL < 64, "loads under way a wave can wait for");
  __shared__ __align__(16) uint8_t stage0[kBytes], stage1[kBytes], stage2[ST > 2 ? kBytes : 16],
      stage3[ST > 3 ? kBytes : 16];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int r = lane & 15, c4 = lane >> 4;
  const int wm = w / NW, wn = w % NW;
  const TileAt at = tile_at(tm, tt);
  const int o0 = at.bm * BM;
  const long t0 = (long)at.bt * BN;

  // pieces of this wave: lane l loads slot l % 8 of row l / 8 (rows behind the
  // last are read from the last; a wave without enough pieces repeats one)
  const int8_t* src[NL];
  int lds[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int piece = min(w * NL + i, kPieces - 1);
    const int row = 8 * piece + (lane >> 3);
    const int q = (lane & 7) ^ ((row >> 1) & 7);
    if (row < BM)
      src[i] = A.wq + (long)min(o0 + row, A.m - 1) * A.ldw + 16 * q;
    else
      src[i] = A.xq + min(t0 + row - BM, A.batch - 1) * A.ldx + 16 * q;
    lds[i] = piece * 1024;
  }
  const int C = A.n >> 7;
  // chunk c into stage S (past the end: the last chunk again, which nobody reads)
  auto issue = [&](int c, uint8_t* S) __attribute__((always_inline)) {
    const long k = 128l * min(c, C - 1);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      uint8_t* const d = S + __builtin_amdgcn_readfirstlane(lds[i]);
      if constexpr (DIRECT)
        __builtin_amdgcn_global_load_lds(src[i] + k, (__attribute__((address_space(3))) void*)d, 16, 0, 0);
      else
        *reinterpret_cast<i32x4*>(d + 16 * lane) = load_any<i32x4>(src[i] + k);
    }
  };
  const int turn = 16 * (c4 ^ ((r >> 1) & 7));
  const int aoff = (16 * WM * wm + r) * 128 + turn;
  const int boff = (BM + 16 * WN * wn + r) * 128 + turn;
  i32x4 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  // a wave's loads have landed but for those of `ahead` chunks, and its LDS reads too;
  // then all meet
  auto sync = [&](auto ahead) __attribute__((always_inline)) {
    if constexpr (DIRECT) {
      constexpr int kWait = decltype(ahead)::value * NL;
      __builtin_amdgcn_s_waitcnt((kWait & 15) | ((kWait >> 4) << 14) | (7 << 4));
      __builtin_amdgcn_s_barrier();
      __asm__ volatile("" ::: "memory");
    } else {
      __syncthreads();
    }
  };
  auto stage = [&](int i) __attribute__((always_inline)) {
    return i % ST == 0 ? stage0 : i % ST == 1 ? stage1 : i % ST == 2 ? stage2 : stage3;
  };
  if constexpr (WM * WN >= 32) {
    // quarter by quarter: half the channel tiles on 64 inputs, the operands of the
    // next quarter read meanwhile
    constexpr int HM = WM / 2;
    if (C > 0) {
      i32x4 lo[HM], hi[HM], b0[WN], b1[WN];
      auto read_a = [&](const uint8_t* S, int k, int half, i32x4 (&a)[HM]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < HM; ++i)
          a[i] = *reinterpret_cast<const i32x4*>(S + (aoff ^ (64 * k)) + 2048 * (half * HM + i));
      };
      auto read_b = [&](const uint8_t* S, int k, i32x4 (&b)[WN]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < WN; ++j) b[j] = *reinterpret_cast<const i32x4*>(S + (boff ^ (64 * k)) + 2048 * j);
      };
      auto products = [&](int half, const i32x4 (&a)[HM], const i32x4 (&b)[WN]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < HM; ++i)
#pragma unroll
          for (int j = 0; j < WN; ++j) acc[half * HM + i][j] = mfma_i8(a[i], b[j], acc[half * HM + i][j]);
      };
      auto body = [&](auto ic, int c) __attribute__((always_inline)) {
        constexpr int I = decltype(ic)::value;
        read_a(stage(I), 0, 1, hi);
        products(0, lo, b0);
        read_a(stage(I), 1, 0, lo);
        read_b(stage(I), 1, b1);
        products(1, hi, b0);
        read_a(stage(I), 1, 1, hi);
        products(0, lo, b1);
        sync(std::integral_constant<int, ST - 2>());
        issue(c + ST, stage(I));
        read_a(stage(I + 1), 0, 0, lo);
        read_b(stage(I + 1), 0, b0);
        products(1, hi, b1);
      };
      for (int i = 0; i < ST; ++i) issue(i, stage(i));
      sync(std::integral_constant<int, ST - 1>());
      read_a(stage0, 0, 0, lo);
      read_b(stage0, 0, b0);
      int c = 0;
      for (; c + ST <= C; c += ST) chunks_while(body, c, c + ST, std::make_integer_sequence<int, ST>());
      chunks_while(body, c, C, std::make_integer_sequence<int, ST - 1>());
    }
  } else if (C > 0) {
    i32x4 a[2][2][WM], b[2][2][WN];
    auto read = [&](const uint8_t* S, i32x4 (&ra)[2][WM], i32x4 (&rb)[2][WN]) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int j = 0; j < WN; ++j) rb[k][j] = *reinterpret_cast<const i32x4*>(S + (boff ^ (64 * k)) + 2048 * j);
#pragma unroll
        for (int i = 0; i < WM; ++i) ra[k][i] = *reinterpret_cast<const i32x4*>(S + (aoff ^ (64 * k)) + 2048 * i);
      }
    };
    auto products = [&](const i32x4 (&ra)[2][WM], const i32x4 (&rb)[2][WN], int k) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
          for (int j = 0; j < WN; ++j) acc[i][j] = mfma_i8(ra[k][i], rb[k][j], acc[i][j]);
    };
    auto body = [&](auto ic, int c) __attribute__((always_inline)) {
      constexpr int I = decltype(ic)::value;
      sync(std::integral_constant<int, ST - 2>());
      issue(c + ST, stage(I));
      read(stage(I + 1), a[(I + 1) & 1], b[(I + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
      products(a[I & 1], b[I & 1], 0);
      products(a[I & 1], b[I & 1], 1);
      __builtin_amdgcn_sched_barrier(0);
    };
    // a turn of the loop ends where the stages and the two register buffers both start again
    constexpr int kTurn = ST % 2 ? 2 * ST : ST;
    static_assert(kTurn % ST == 0 && kTurn % 2 == 0, "chunk c is in stage c % ST and in registers c % 2");
    for (int i = 0; i < ST; ++i) issue(i, stage(i));
    sync(std::integral_constant<int, ST - 1>());
    read(stage0, a[0], b[0]);
    int c = 0;
    for (; c + kTurn <= C; c += kTurn) chunks_while(body, c, c + kTurn, std::make_integer_sequence<int, kTurn>());
    chunks_while(body, c, C, std::make_integer_sequence<int, kTurn - 1>());
  }
  if (A.n & 127) {
    // the last inputs, straight from memory
    for (int k0 = 128 * C; k0 < A.n; k0 += 64) {
      const int k = k0 + 16 * c4;
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
  }
  // every load has landed and every wave is past its reads: the stages are free
  __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));
  __syncthreads();

  // Scaled outputs, 16 tokens at a time, through the wave's own part of the
  // stages: 4 channels a lane in, whole 16-byte pieces of a token's 16 WM
  // channels out.
  constexpr int RS = 16 * WM * sizeof(Y) + 16;  // bytes a token (16 more: banks staggered)
  constexpr int kWaves = MW * NW, kShare = kWaves / 2;  // waves a stage (two stages hold all)
  static_assert(kShare * 16 * RS <= kBytes, "half the waves' tiles fit a stage");
  uint8_t* const st = (w / kShare == 0 ? stage0 : stage1) + (w % kShare) * (16 * RS);
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

template <typename Y, int WM, int WN, int MW, int NW, int ST>
void launch_tile(const LbQ8LinearArgs& a, hipStream_t stream) {
  constexpr int BM = 16 * WM * MW, BN = 16 * WN * NW;
  const int tm = (a.m + BM - 1) / BM;
  const long tt = (a.batch + BN - 1) / BN;
  const bool direct = (((uintptr_t)a.xq | (uintptr_t)a.wq | (uintptr_t)a.ldx | (uintptr_t)a.ldw) & 15) == 0;
  const dim3 grid((unsigned)(tm * tt)), block(64 * MW * NW);
  if (direct)
    hipLaunchKernelGGL((lb_q8_tile_kernel<Y, WM, WN, MW, NW, ST, true>), grid, block, 0, stream, a, tm, (int)tt);
  else
    // through registers a chunk's loads are waited for at once: a third stage gains nothing, and its turn of six chunks
    // costs (512 x 4096 -> 11008 with rows of 4104 bytes: 58 us in two stages, 111 in three)
    hipLaunchKernelGGL((lb_q8_tile_kernel<Y, WM, WN, MW, NW, ST == 3 ? 2 : ST, false>), grid, block, 0, stream, a, tm, (int)tt);
}

// Compute units of the current device (256 where it cannot be asked).
int cu_count() {
  int dev = 0, ncu = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&ncu, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || ncu <= 0)
    return 256;
  return ncu;
}

// Up to 16 tokens.
template <typename Y>
void launch_few(const LbQ8LinearArgs& a, int ncu, hipStream_t stream) {
  const int tiles = (a.m + 15) / 16;
  if (tiles <= ncu) {
    hipLaunchKernelGGL((lb_q8_skinny_kernel<Y, 1>), dim3(tiles), dim3(256), 0, stream, a);
    return;
  }
  const int units = (a.n + 127) / 128, steps = (units + kStreamWaves - 1) / kStreamWaves;
  const int xrow = steps * kStreamWaves * 128 + 16, rounds = (tiles + ncu - 1) / ncu;
  const size_t bytes = kStreamWaves * 1024 + (size_t)rounds * 64 + (size_t)a.batch * xrow;
  if (bytes <= kStreamLds && a.n % 16 == 0)
    hipLaunchKernelGGL((lb_q8_stream_kernel<Y>), dim3(ncu), dim3(64 * kStreamWaves), bytes, stream, a, tiles, steps,
                       xrow, rounds);
  else
    hipLaunchKernelGGL((lb_q8_skinny_kernel<Y, 2>), dim3((tiles + 1) / 2), dim3(256), 0, stream, a);
}

// The tile shape whose rounds of workgroups over the compute units take the
// least, counted in hundredths of a us a chunk as measured with one workgroup
// a compute unit.  Against all shapes on fourteen sizes (24 to 2000 tokens, 4096 to
// 32000 channels, weights from HBM) this choice was the fastest or within 4%: 64 x 5120 ->
// 32000 in 128 x 64 36 us (64 x 64 41, 128 x 128 38), 300 x 5120 -> 5120 in 64 x 128 18 (22,
// 26), 201 x 5120 -> 13824 in 128 x 128 31 (64 x 128 38, 128 x 256 44), 512 x 4096 -> 11008
// in 128 x 256 35 (128 x 128 45, 64 x 128 47, 256 x 256 58).  Starts and ends, some 5 us a
// shape, are not counted; on nine sizes with 256 or 512 inputs (64 to 2000 tokens, 5120 to
// 32000 channels) the choice was the fastest all the same: 300 x 512 -> 5120 5.2 us in 64 x
// 128 (128 x 64 5.3, 64 x 64 5.5).  Rows off 16 bytes are 1.3 to 2 times slower in all shapes
// (201 x 5120 -> 13824 54 us, 2000 x 4096 -> 32000 319, against 31 and 245) and take the
// same choice, there the fastest or within 6% on five sizes.
template <typename Y>
void launch_linear(const LbQ8LinearArgs& a, hipStream_t stream) {
  const int ncu = cu_count();
  if (a.batch <= 16) {
    launch_few<Y>(a, ncu, stream);
    return;
  }
  static const struct {
    int bm, bn, cost;
  } shapes[] = {{32, 64, 11}, {64, 64, 14}, {64, 128, 23}, {128, 64, 24}, {128, 128, 39}, {128, 256, 68}, {256, 256, 133}};
  int best = 0;
  long least = 0;
  for (int i = 0; i < 7; ++i) {
    const long wgs = (long)((a.m + shapes[i].bm - 1) / shapes[i].bm) * ((a.batch + shapes[i].bn - 1) / shapes[i].bn);
    const long cost = (wgs + ncu - 1) / ncu * shapes[i].cost;
    if (i == 0 || cost < least) {
      best = i;
      least = cost;
    }
  }
  switch (best) {
    case 0: launch_tile<Y, 2, 1, 1, 4, 4>(a, stream); break;
    case 1: launch_tile<Y, 2, 1, 2, 4, 4>(a, stream); break;
    case 2: launch_tile<Y, 2, 2, 2, 4, 4>(a, stream); break;
    case 3: launch_tile<Y, 4, 1, 2, 4, 4>(a, stream); break;
    case 4: launch_tile<Y, 4, 2, 2, 4, 4>(a, stream); break;
    case 5: launch_tile<Y, 4, 4, 2, 4, 3>(a, stream); break;
    default: launch_tile<Y, 8, 4, 2, 4, 2>(a, stream); break;
  }
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
