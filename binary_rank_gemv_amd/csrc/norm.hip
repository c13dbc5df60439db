// Residual root-mean-square norm, its backward pass, and the row quantiser.
//
// Forward, per row:  h = round(x + res);  s2 = sum h^2;  a = max |h w|
//     r = 1/sqrt(s2/n + eps);  y = (h w) r;  scale = a r / 127;
//     q = rint(y / scale) = rint((h w) * 127 / a)
// The largest |y| is a r, so both reductions run over the same values in one
// exchange: the row is read once, held in registers, and the 8-bit codes need
// no second reduction.  A group of G threads owns a row, thread t of it the
// vectors t, t + G, ... of eight elements.  Memory bounds it: 2047 x 8192 bf16
// with its residual, to 8 bits, 26.4 us in a replayed graph (4.4 TB/s; a copy reaches 5.2).
#include "head_common.h"
#include "head_launch.h"

using namespace lbh;

namespace {

constexpr float kBig = 0x1p100f;

// What a row's codes rint(127 v / a) are formed with.  Where a is tiny or huge, values are
// multiplied by `up` first (exact, a power of two), so that nothing leaves the range.
struct Q8Scale {
  float up, a, hi, lo;  // 127 / (a up) = hi + lo
};
__device__ __forceinline__ Q8Scale q8_scale(float a) {
  Q8Scale s;
  s.up = a < 1e-30f ? kBig : a > 1e30f ? 1.0f / kBig : 1.0f;
  s.a = a * s.up;
  // a row of zeros has codes 0
  s.hi = (s.a > 0.0f && s.a < INFINITY) ? 127.0f / s.a : 0.0f;
  s.lo = s.hi > 0.0f ? fmaf(-s.hi, s.a, 127.0f) / s.a : 0.0f;
  return s;
}

// Eight codes (their last 8 bits), those of the exact quotients, a half to the even code;
// leaves v scaled by `up`.  A product of two 2-byte values is exact in fp32, so v and a
// are.  A product with 127 / a alone would put a few codes in ten million on the other
// side, and halves on either.
template <bool SHORT>
__device__ __forceinline__ void q8_codes(float (&v)[8], const Q8Scale& s, int (&c)[8]) {
  if (s.up != 1.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s.up;
  }
  if constexpr (SHORT) {
    // v has 17 bits at most: 127 v is exact, and so is the rest 127 v - c a, which is compared with
    // a / 2 itself.  (Where c is 1 and the quotient below a half, the rest may be
    // rounded to -a / 2, which gives code 0 too.)  Short values hit a half often.
    const uint32_t half = __builtin_bit_cast(uint32_t, 0.5f * s.a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // rounded to a whole number by the addition, whose last bits are then the code's
      const float near = fmaf(v[i], s.hi, 0x1.8p23f), rest = fmaf(0x1.8p23f - near, s.a, 127.0f * v[i]);
      c[i] = __builtin_bit_cast(int, near);
      // an odd code gives a half away: one unit less than a / 2 is allowed for it
      const float most = __builtin_bit_cast(float, half - (uint32_t)(c[i] & 1));
      const int step = __builtin_bit_cast(int, rest) >> 31 | 1;
      c[i] += fabsf(rest) > most ? step : 0;
    }
  } else {
    // the rest as a share of a, off by less than 2^-23: what is that near to a half (a few
    // in a million, more where the weight is 1) is decided by 127 v - (c +- 1/2) a, exact in 64 bits
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = v[i], q = rintf(w * s.hi), rest = fmaf(w, s.lo, fmaf(w, s.hi, -q));
      most = fmaxf(most, fabsf(rest));
      c[i] = (int)(q + rintf(rest));
    }
    if (most > 0.5f - 0x1p-22f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = v[i], q = rintf(w * s.hi), rest = fmaf(w, s.lo, fmaf(w, s.hi, -q));
        const bool above = rest > 0.0f;
        const double off = fma(-(double)(q + (above ? 0.5f : -0.5f)), (double)s.a, 127.0 * (double)w);
        c[i] = (int)q;
        if (off == 0.0 ? (c[i] & 1) != 0 : (off > 0.0) == above) c[i] += above ? 1 : -1;
      }
    }
  }
}

// `fine`: the row is finite (otherwise its codes are 0).
template <bool SHORT>
__device__ __forceinline__ void q8_store(int8_t* p, long left, float (&v)[8], const Q8Scale& s, bool fine) {
  int c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (fine) q8_codes<SHORT>(v, s, c);
  if (left >= 8) {
    u32x2 w;
#pragma unroll
    for (int d = 0; d < 2; ++d)
      w[d] = (uint32_t)(c[4 * d] & 255) | (uint32_t)(c[4 * d + 1] & 255) << 8 | (uint32_t)(c[4 * d + 2] & 255) << 16 |
             (uint32_t)(c[4 * d + 3] & 255) << 24;
    store_any(p, w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (int8_t)c[i];
  }
}

// Sum of `s` and maximum of `a` over a group of G threads (G = 64: a wave;
// otherwise the whole workgroup).  A NaN reaches the sum and the maximum.
template <int G>
__device__ __forceinline__ void group_reduce(float& s, float& a) {
  s = wave_sum(s);
  a = wave_max(a);
  if constexpr (G > 64) {
    __shared__ float part[2][G / 64];
    const int w = wave_id(), lane = threadIdx.x & 63;
    if (lane == 0) {
      part[0][w] = s;
      part[1][w] = a;
    }
    __syncthreads();
    s = part[0][0];
    a = part[1][0];
#pragma unroll
    for (int i = 1; i < G / 64; ++i) {
      s += part[0][i];
      a = max_nan(a, part[1][i]);
    }
  }
}

// The power of two that a row is multiplied by where its sum of squares leaves the
// range of fp32 (values of bf16 beyond some 1e19; below 1e-14, where eps does not
// cover them): y = h r has none of it, and the sums are formed again. The question
// costs 0.2 of the 26.4 us of 2047 x 8192 forward and 0.6 of the 17 of 2048 x 4096 backward.
template <typename T>
__device__ __forceinline__ float row_power(float s2, float eps) {
  if constexpr (__is_same(T, bf16)) {
    if (s2 == INFINITY) return 0x1p-80f;
    if (s2 < 0x1p-90f && eps < 0x1p-100f) return 0x1p70f;
  }
  return 1.0f;
}

// QUANT: the row quantiser alone (no residual, weight or norm).
template <typename T, int G, int V, bool QUANT>
__global__ __launch_bounds__(G < 256 ? 256 : G) void lb_norm_kernel(const LbNormArgs A) {
  constexpr int kPer = G < 256 ? 256 / G : 1;  // rows a workgroup
  const int t = threadIdx.x % G;
  const long row = (long)blockIdx.x * kPer + threadIdx.x / G;
  if (row >= A.rows) return;  // whole waves only: G is a wave or the workgroup
  const T* x = (const T*)A.x + row * A.ldx;
  float h[V][8], hw[V][8];
  float s2 = 0.0f, a = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = 8 * (t + i * G);
    const long left = A.n - k;
    if (left > 0) {
      load8(x + k, left, 0.0f, h[i]);
      if constexpr (!QUANT) {
        if (A.residual) {
          float r[8];
          load8((const T*)A.residual + row * A.ldr + k, left, 0.0f, r);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[i][e] = (float)(T)(h[i][e] + r[e]);
        }
        load8((const T*)A.weight + k, left, 0.0f, hw[i]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = hw[i][e] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (QUANT) {
        hw[i][e] = h[i][e];
      } else {
        hw[i][e] *= h[i][e];
        s2 += h[i][e] * h[i][e];
      }
      a = max_nan(a, fabsf(hw[i][e]));
    }
  }
  if constexpr (!QUANT) {
    if (A.hidden) {
      T* hp = (T*)A.hidden + row * A.ldh;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int k = 8 * (t + i * G);
        store8(hp + k, (long)A.n - k, h[i]);
      }
    }
  }
  group_reduce<G>(s2, a);
  float r = 1.0f;
  if constexpr (!QUANT) {
    float eps = A.eps;
    const float up = row_power<T>(s2, eps);
    if (up != 1.0f) {  // all threads of the row
      const T* hp = A.hidden ? (const T*)A.hidden + row * A.ldh : x;
      eps = eps * up * up;  // in this order: up^2 alone can leave the range
      s2 = a = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int k = 8 * (t + i * G);
        const long left = A.n - k;
        float wt[8];
        load8(hp + k, left > 0 ? left : 0, 0.0f, h[i]);
        load8((const T*)A.weight + k, left > 0 ? left : 0, 0.0f, wt);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float he = h[i][e] * up;
          hw[i][e] = he * wt[e];
          s2 += he * he;
          a = max_nan(a, fabsf(hw[i][e]));
        }
      }
      if constexpr (G > 64) __syncthreads();  // the first sums have been read
      group_reduce<G>(s2, a);
    }
    r = 1.0f / sqrtf(s2 / (float)A.n + eps);
  }
  // NaN where the row or the weight has one, or an infinity meets a 0
  const float top = QUANT ? a : a * r;
  const bool fine = top < INFINITY;  // false for NaN too
  if constexpr (!QUANT) {
    if (A.y) {
      T* yp = (T*)A.y + row * A.ldy;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int k = 8 * (t + i * G);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = hw[i][e] * r;
        store8(yp + k, (long)A.n - k, y);
      }
    }
  }
  if (A.q) {
    const Q8Scale sc = q8_scale(a);
    int8_t* qp = A.q + row * A.ldq;
    constexpr bool kShort = sizeof(T) == 2 && (QUANT || __is_same(T, bf16));  // else 22 or 24 bits
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = 8 * (t + i * G);
      q8_store<kShort>(qp + k, (long)A.n - k, hw[i], sc, fine);
    }
    if (t == 0) A.scale[row] = fine ? top / 127.0f : NAN;
  }
}

template <typename T, int G, int V, bool QUANT>
void launch_one(const LbNormArgs& a, hipStream_t stream) {
  constexpr int per = G < 256 ? 256 / G : 1;
  const long blocks = (a.rows + per - 1) / per;
  hipLaunchKernelGGL((lb_norm_kernel<T, G, V, QUANT>), dim3((unsigned)blocks), dim3(G < 256 ? 256 : G), 0, stream, a);
}

// Threads a row by its length, and more of them, with fewer vectors each, while
// there are few rows.  To 8 bits, bf16, one vector a thread against two: of 5120,
// 1 row 3.8 and 4.0 us, 256 rows 5.4 and 5.9, 384 rows 7.4 and 7.2, 1024 rows 12.7 and
// 12.1, 2048 rows 22.5 and 20.2; of 8192, 256 rows 6.2 and 6.4, 1024 rows 15.2 and 15.1,
// 2048 rows 26.3 and 25.3; of 4096, 1 row 3.2 and 4.0, 512 rows 6.2 and 6.8, 1024 rows 9.8
// and 9.9, 2048 rows 14.8 and 15.2 (dense 14.2 and 13.2).
template <typename T, bool QUANT>
void launch_norm(const LbNormArgs& a, hipStream_t stream) {
  if (a.n <= 512)
    launch_one<T, 64, 1, QUANT>(a, stream);
  else if (a.n <= 2048)
    launch_one<T, 256, 1, QUANT>(a, stream);
  else if (a.n <= 4096 && a.rows > 512)
    launch_one<T, 256, 2, QUANT>(a, stream);
  else if (a.n <= 4096)
    launch_one<T, 512, 1, QUANT>(a, stream);
  else if (a.n <= 8192 && a.rows > 256)
    launch_one<T, 512, 2, QUANT>(a, stream);
  else if (a.n <= 8192)
    launch_one<T, 1024, 1, QUANT>(a, stream);
  else if (a.n <= 16384)
    launch_one<T, 1024, 2, QUANT>(a, stream);
  else
    launch_one<T, 1024, 4, QUANT>(a, stream);
}

// -------------------------------------------------------------------- backward
// With u = w dy:  dx = dhidden + r u - h (r^3 / n) sum(u h);  both sums
// (h^2 for r, and u h) run over the row in one exchange, so r need not be kept
// from the forward pass.  dweight = sum over rows of dy h r: a thread keeps the
// sum of its columns over its rows in registers, the R rows that a workgroup
// holds at a time join theirs in LDS at the end, and a second kernel adds the
// workgroups, all in a fixed order.  The next row's loads are under way while a
// row is reduced.  2048 x 4096 bf16: 15.1 us (4.7 TB/s with the partial sums) and 3
// to 4 for the sum of the workgroups in a kernel trace, both 17.0 in a replayed
// graph; with one row at a time and twice the workgroups it was 16.6 and 5.2.
template <typename T, int V>
struct RowIn {
  u32x4 h[V], dy[V], dh[V];
};
// Eight 2-byte elements as they lie in memory, zeros behind the row.
template <typename T>
__device__ __forceinline__ u32x4 raw8(const T* p, long left) {
  if (left >= 8) return load_any<u32x4>(p);
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = i < left ? p[i] : (T)0.0f;
  u32x4 w;
  __builtin_memcpy(&w, e, sizeof w);
  return w;
}
template <typename T>
__device__ __forceinline__ float part_of(const u32x4& w, int e) {
  return e & 1 ? Pair<T>::hi(w[e >> 1]) : Pair<T>::lo(w[e >> 1]);
}

// A value that all lanes of the wave hold.
__device__ __forceinline__ float wave_value(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

template <typename T, int G, int R, int V>
__global__ __launch_bounds__(G * R) void lb_norm_bwd_kernel(const LbNormBwdArgs A) {
  constexpr int kW = G / 64;
  constexpr bool kAhead = V == 1;  // registers for the next row
  // the longest rows: the columns' sums (128 KB) in LDS, no registers for them (512 x
  // 32768: 70 us with both kernels, registers still spill; reading dhidden and the
  // weight where they are used instead of holding them: 80)
  constexpr bool kInLds = V == 4;
  __shared__ float part[3][2][R][kW];  // two in turn, one for rows out of range
  __shared__ float join[kInLds ? G * V * 8 : R > 1 ? (R - 1) * G * V * 8 : 1];
  const int t = threadIdx.x % G, rg = threadIdx.x / G, w = wave_id() % kW, lane = threadIdx.x & 63;
  u32x4 wt[V];
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = 8 * (t + i * G);
    wt[i] = raw8((const T*)A.weight + k, (long)A.n - k);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[i][e] = 0.0f;
      if constexpr (kInLds) join[(i * 8 + e) * G + t] = 0.0f;  // this thread's alone
    }
  }
  const long stride = (long)gridDim.x * R;
  const long rounds = (A.rows + stride - 1) / stride;
  auto load = [&](long row, RowIn<T, V>& in) __attribute__((always_inline)) {
    const bool real = row < A.rows;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = 8 * (t + i * G);
      const long left = real ? (long)A.n - k : 0;
      in.h[i] = raw8((const T*)A.hidden + row * A.ldh + k, left);
      in.dy[i] = raw8((const T*)A.dy + row * A.lddy + k, left);
      in.dh[i] = raw8((const T*)A.dhidden + row * A.lddh + k, A.dhidden ? left : 0);
    }
  };
  RowIn<T, V> next;
  long row = (long)blockIdx.x * R + rg;
  load(row, next);
  for (long j = 0; j < rounds; ++j, row += stride) {
    if (!kAhead && j > 0) load(row, next);
    const RowIn<T, V> in = next;
    if (kAhead && j + 1 < rounds) load(row + stride, next);
    float s2 = 0.0f, uh = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float h = part_of<T>(in.h[i], e);
        s2 += h * h;
        uh += part_of<T>(wt[i], e) * part_of<T>(in.dy[i], e) * h;
      }
    }
    s2 = wave_sum(s2);
    uh = wave_sum(uh);
    [[maybe_unused]] const int flip = j & 1;
    if constexpr (kW > 1) {
      if (lane == 0) {
        part[flip][0][rg][w] = s2;
        part[flip][1][rg][w] = uh;
      }
      __syncthreads();  // two buffers in turn: one barrier a row is enough
      s2 = part[flip][0][rg][0];
      uh = part[flip][1][rg][0];
#pragma unroll
      for (int i = 1; i < kW; ++i) {
        s2 += part[flip][0][rg][i];
        uh += part[flip][1][rg][i];
      }
    }
    const float up = wave_value(row < A.rows ? row_power<T>(s2, A.eps) : 1.0f);
    if constexpr (__is_same(T, bf16)) {
      bool again = up != 1.0f;
      if constexpr (R > 1 && kW > 1) {
        // the same answer in the whole workgroup, for the barrier: from all its waves' sums,
        // sixteen at most to a row (a row that is in range has the same sums again)
        const float q = lane < R * kW ? part[flip][0][lane / kW][lane % kW] : 1.0f;
        again = __ballot(!(q < 0x1p120f) || (q < 0x1p-90f && A.eps < 0x1p-100f)) != 0;
      }
      if (again) {
        s2 = uh = 0.0f;
        auto add = [&](const u32x4& hv, const u32x4& dyv, const u32x4& wv) __attribute__((always_inline)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float h = part_of<T>(hv, e) * up;
            s2 += h * h;
            uh += part_of<T>(wv, e) * part_of<T>(dyv, e) * h;
          }
        };
        if constexpr (V < 4) {
#pragma unroll
          for (int i = 0; i < V; ++i) add(in.h[i], in.dy[i], wt[i]);
        } else {  // read again: the usual way needs the registers
#pragma unroll 1
          for (int k = 8 * t; k < A.n && row < A.rows; k += 8 * G) {
            const long left = (long)A.n - k;
            add(raw8((const T*)A.hidden + row * A.ldh + k, left), raw8((const T*)A.dy + row * A.lddy + k, left),
                raw8((const T*)A.weight + k, left));
          }
        }
        s2 = wave_sum(s2);
        uh = wave_sum(uh);
        if constexpr (kW > 1) {
          if (lane == 0) {
            part[2][0][rg][w] = s2;
            part[2][1][rg][w] = uh;
          }
          __syncthreads();
          s2 = uh = 0.0f;
#pragma unroll
          for (int i = 0; i < kW; ++i) {
            s2 += part[2][0][rg][i];
            uh += part[2][1][rg][i];
          }
        }
      }
    }
    const float ru = 1.0f / sqrtf(s2 / (float)A.n + A.eps * up * up), r = ru * up;
    const float c = (uh * ru) / (float)A.n * r;
    const bool real = row < A.rows;  // behind the last row there are zeros; with eps = 0 their r is infinite
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = 8 * (t + i * G);
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float hr = part_of<T>(in.h[i], e) * r, dy = part_of<T>(in.dy[i], e);
        d[e] = part_of<T>(in.dh[i], e) + (r * (part_of<T>(wt[i], e) * dy) - hr * c);
        if constexpr (kInLds) {
          if (real) join[(i * 8 + e) * G + t] += dy * hr;
        } else {
          if (real) dw[i][e] += dy * hr;
        }
      }
      store8((T*)A.dx + row * A.lddx + k, real ? (long)A.n - k : 0, d);
    }
  }
  if constexpr (R > 1) {
    if (rg > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) join[((rg - 1) * V * 8 + i * 8 + e) * G + t] = dw[i][e];
    }
    __syncthreads();
    if (rg > 0) return;
#pragma unroll
    for (int q = 0; q < R - 1; ++q)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] += join[(q * V * 8 + i * 8 + e) * G + t];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int k = 8 * (t + i * G);
    if constexpr (kInLds) {
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[i][e] = join[(i * 8 + e) * G + t];
    }
    store8(A.partial + (long)blockIdx.x * A.n + k, (long)A.n - k, dw[i]);
  }
}

// dweight = sum of the groups' partial sums: 32 columns x 32 slices of groups
// a workgroup, slices joined in order.
__global__ __launch_bounds__(1024) void lb_norm_dweight_kernel(const float* __restrict__ partial, int groups, int n,
                                                               float* __restrict__ dweight) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, p = threadIdx.x >> 5;
  const int k = blockIdx.x * 32 + c;
  float v = 0.0f;
  if (k < n) {
    int g = p;
    for (; g + 32 * 7 < groups; g += 32 * 8) {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = partial[(long)(g + 32 * i) * n + k];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += q[i];
    }
    for (; g < groups; g += 32) v += partial[(long)g * n + k];
  }
  s[p][c] = v;
  __syncthreads();
  if (p == 0 && k < n) {
    v = s[0][c];
    for (int i = 1; i < 32; ++i) v += s[i][c];
    dweight[k] = v;
  }
}

// Threads a row and rows a workgroup holds at a time.
struct BwdShape {
  int g, r, v;
};
BwdShape bwd_shape(int64_t n) {
  if (n <= 512) return {64, 16, 1};
  if (n <= 2048) return {256, 4, 1};
  if (n <= 4096) return {512, 2, 1};
  if (n <= 8192) return {1024, 1, 1};
  return {1024, 1, n <= 16384 ? 2 : 4};
}

template <typename T, int G, int R, int V>
void launch_bwd_one(const LbNormBwdArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((lb_norm_bwd_kernel<T, G, R, V>), dim3((unsigned)a.groups), dim3(G * R), 0, stream, a);
}

template <typename T>
void launch_bwd(const LbNormBwdArgs& a, hipStream_t stream) {
  const BwdShape s = bwd_shape(a.n);
  if (s.g == 64)
    launch_bwd_one<T, 64, 16, 1>(a, stream);
  else if (s.g == 256)
    launch_bwd_one<T, 256, 4, 1>(a, stream);
  else if (s.g == 512)
    launch_bwd_one<T, 512, 2, 1>(a, stream);
  else if (s.v == 1)
    launch_bwd_one<T, 1024, 1, 1>(a, stream);
  else if (s.v == 2)
    launch_bwd_one<T, 1024, 1, 2>(a, stream);
  else
    launch_bwd_one<T, 1024, 1, 4>(a, stream);
}

}  // namespace

hipError_t lb_launch_norm(const LbNormArgs& a, int dtype, hipStream_t stream) {
  if (dtype == 1)
    launch_norm<f16, false>(a, stream);
  else
    launch_norm<bf16, false>(a, stream);
  return hipGetLastError();
}

hipError_t lb_launch_q8_quantize(const LbNormArgs& a, int dtype, hipStream_t stream) {
  if (dtype == 0)
    launch_norm<float, true>(a, stream);
  else if (dtype == 1)
    launch_norm<f16, true>(a, stream);
  else
    launch_norm<bf16, true>(a, stream);
  return hipGetLastError();
}

// Workgroups of the backward pass: one a compute unit of this architecture (a fixed
// number, so that the sums and the workspace are the same on every part), fewer
// for few rows.
int lb_norm_bwd_groups(int64_t rows, int64_t n) {
  const int64_t r = bwd_shape(n).r, groups = (rows + r - 1) / r;
  return (int)(groups < 256 ? groups : 256);
}

hipError_t lb_launch_norm_bwd(const LbNormBwdArgs& a, int dtype, hipStream_t stream) {
  if (a.rows > 0) {
    if (dtype == 1)
      launch_bwd<f16>(a, stream);
    else
      launch_bwd<bf16>(a, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(lb_norm_dweight_kernel, dim3((a.n + 31) / 32), dim3(1024), 0, stream, a.partial, a.groups, a.n,
                     a.dweight);
  return hipGetLastError();
}
