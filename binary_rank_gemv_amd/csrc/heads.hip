// Heads of queries, keys and values: the norm of each head with the position
// rotation (dense, or on the way into a paged cache), its backward pass, and the
// move of a tree's accepted rows inside a cache.
//
// Per head x of dim channels, r = 1 / sqrt(mean x^2 + eps):  y = x r w, and of y
//     (a, b) -> (a cos - b sin, b cos + a sin)      angle_j = position inv_freq_j
// One pass: a head lies in the registers of LG lanes, 16 channels a lane, which are
// eight pairs; the sum of squares takes log2 LG moves between lanes.  A wave has one
// token and 64 / LG heads at a time.  Its lanes compute one pair's turn each, in turns (64
// bits, so that far positions keep their digits), and share them in LDS.  No wave
// waits for another.  Memory bounds it.
#include "attn_common.h"

using namespace lbh;

namespace {

constexpr int kMaxPairs = LB_HEAD_MAX_DIM / 2;

// cos and sin of the token's pairs, for the lanes of this wave.
template <int LG>
__device__ __forceinline__ void turns(float2* cs, int position, const float* __restrict__ inv_freq, int pairs, float sign) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < (LG == 16 ? 2 : 1); ++i) {
    const int j = lane + 64 * i;
    if (j < pairs) {
      const double t = (double)position * (double)inv_freq[j] * 0.15915494309189533577;  // 1 / 2 pi
      const float f = (float)(t - rint(t));
      float s, c;
      sincospif(2.0f * f, &s, &c);
      cs[j] = float2{c, sign * s};
    }
  }
}

// Sixteen channels of a head as they lie in memory, eight pairs (a, b): eight and eight
// in rows, or one after the other (INTER).  VEC: dim is a multiple of 16 and, unless INTER, the
// rotated half of 8, so that they are two wide loads; else they are read one by one.
// What is not rotated is paired as it lies.
template <typename T>
struct Raw {
  u32x4 lo, hi;
};

template <bool INTER>
__device__ __forceinline__ int first_of(int pair, int half) {
  if (INTER) return 2 * pair;
  return pair < half ? pair : 2 * pair;
}
template <bool INTER>
__device__ __forceinline__ int second_of(int pair, int half) {
  if (INTER) return 2 * pair + 1;
  return pair < half ? pair + half : 2 * pair + 1;
}
// Where the second eight channels lie, and the first.
template <bool INTER>
__device__ __forceinline__ int vec_lo(int u, int half) {
  if (INTER) return 16 * u;
  return 8 * u < half ? 8 * u : 16 * u;
}
template <bool INTER>
__device__ __forceinline__ int vec_hi(int u, int half) {
  if (INTER) return 16 * u + 8;
  return 8 * u < half ? 8 * u + half : 16 * u + 8;
}

template <typename T, bool INTER, bool VEC>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int u, int dim, int half, bool there) {
  Raw<T> r;
  r.lo = r.hi = u32x4{0, 0, 0, 0};
  if (!there) return r;
  if constexpr (VEC) {
    r.lo = load_any<u32x4>(p + vec_lo<INTER>(u, half));
    r.hi = load_any<u32x4>(p + vec_hi<INTER>(u, half));
  } else {
    T e[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = 8 * u + i;
      const bool in = pair < dim / 2;
      const T a = in ? p[first_of<INTER>(pair, half)] : (T)0.0f;
      const T b = in ? p[second_of<INTER>(pair, half)] : (T)0.0f;
      e[INTER ? 2 * i : i] = a;
      e[INTER ? 2 * i + 1 : 8 + i] = b;
    }
    __builtin_memcpy(&r, e, sizeof r);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ float element(const Raw<T>& r, int e) {
  const uint32_t w = e < 8 ? r.lo[e >> 1] : r.hi[(e - 8) >> 1];
  return e & 1 ? Pair<T>::hi(w) : Pair<T>::lo(w);
}
// The eight pairs of a lane, apart.
template <typename T, bool INTER>
__device__ __forceinline__ void pairs_of(const Raw<T>& r, float (&a)[8], float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = element(r, INTER ? 2 * i : i);
    b[i] = element(r, INTER ? 2 * i + 1 : 8 + i);
  }
}

template <typename T, bool INTER, bool VEC>
__device__ __forceinline__ void store_pairs(T* p, int u, int dim, int half, const float (&a)[8], const float (&b)[8]) {
  if constexpr (VEC) {
    u32x4 lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (INTER) {
        lo[i] = Pair<T>::pack(a[i], b[i]);
        hi[i] = Pair<T>::pack(a[4 + i], b[4 + i]);
      } else {
        lo[i] = Pair<T>::pack(a[2 * i], a[2 * i + 1]);
        hi[i] = Pair<T>::pack(b[2 * i], b[2 * i + 1]);
      }
    }
    store_any(p + vec_lo<INTER>(u, half), lo);
    store_any(p + vec_hi<INTER>(u, half), hi);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = 8 * u + i;
      if (pair < dim / 2) {
        p[first_of<INTER>(pair, half)] = (T)a[i];
        p[second_of<INTER>(pair, half)] = (T)b[i];
      }
    }
  }
}

// The same sixteen channels stored as they were read.
template <typename T, bool INTER, bool VEC>
__device__ __forceinline__ void store_raw(T* p, int u, int dim, int half, const Raw<T>& r) {
  if constexpr (VEC) {
    store_any(p + vec_lo<INTER>(u, half), r.lo);
    store_any(p + vec_hi<INTER>(u, half), r.hi);
  } else {
    T e[16];
    __builtin_memcpy(e, &r, sizeof r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = 8 * u + i;
      if (pair < dim / 2) {
        p[first_of<INTER>(pair, half)] = e[INTER ? 2 * i : i];
        p[second_of<INTER>(pair, half)] = e[INTER ? 2 * i + 1 : 8 + i];
      }
    }
  }
}

// Pairs from `half` on stay (not multiplied by 1 and 0: an infinity beside them would reach them).
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float2* cs, int u, int half) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (8 * u + i < half) {
      const float2 t = cs[8 * u + i];
      const float x = a[i], y = b[i];
      a[i] = x * t.x - y * t.y;
      b[i] = y * t.x + x * t.y;
    }
  }
}

template <int LG>
__device__ __forceinline__ float head_sum(float v) {
  v += lane_xor<1>(v);
  v += lane_xor<2>(v);
  if constexpr (LG > 4) v += lane_xor<4>(v);
  if constexpr (LG > 8) v += lane_xor<8>(v);
  return v;
}

// The power of two that a head is multiplied by where its sum of squares leaves fp32's
// range (values of bf16 beyond some 1e18; below 1e-14, where eps does not cover them).
template <typename T>
__device__ __forceinline__ float head_power(float s2, float eps) {
  if constexpr (__is_same(T, bf16)) {
    if (s2 == INFINITY) return 0x1p-80f;
    if (s2 < 0x1p-90f && eps < 0x1p-100f) return 0x1p70f;
  }
  return 1.0f;
}

// r of the head, and the power that its values take with it: y = (x up) r w.
template <typename T, int LG>
__device__ __forceinline__ float head_scale(const float (&a)[8], const float (&b)[8], int dim, float eps, float* power) {
  float s2 = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s2 += a[i] * a[i] + b[i] * b[i];
  s2 = head_sum<LG>(s2);
  const float up = head_power<T>(s2, eps);
  *power = up;
  if constexpr (__is_same(T, bf16)) {
    if (__ballot(up != 1.0f)) {  // every lane of the wave, for the moves between them
      s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s2 += (a[i] * up) * (a[i] * up) + (b[i] * up) * (b[i] * up);
      s2 = head_sum<LG>(s2);
      eps = eps * up * up;
    }
  }
  return 1.0f / sqrtf(s2 / (float)dim + eps);
}

// ------------------------------------------------------------------------ forward

// A wave: one token, `span` steps of 64 / LG heads; the queries' steps first, then the
// keys', then the values'.  APPEND: keys and values go to their page.  Bytes bound it.  With inputs from memory (six sets
// in turn, more than the caches hold): 4000 tokens of 64 and 8 heads of 128, bf16, normed, 33 us, 4.5 TB/s (a large copy
// reaches 5.1); 2039 into a cache, interleaved, 20 us, 4.1 TB/s; one token of 40 heads 3.8 us, latency.
template <typename T, int LG, bool INTER, bool VEC, bool APPEND>
__global__ __launch_bounds__(256) void lb_rope_kernel(const LbRopeArgs A) {
  __shared__ float2 cs_all[4][kMaxPairs];
  constexpr int kHeads = 64 / LG;
  const int w = wave_id(), lane = threadIdx.x & 63;
  const int u = lane % LG, sub = lane / LG;
  const uint32_t item = blockIdx.x * 4 + w;
  const uint32_t token = item / (uint32_t)A.blocks, block = item - token * A.blocks;
  if (token >= A.tokens) return;  // whole waves, and no barrier follows
  const int half = A.rot / 2;
  const int n0 = (A.heads[0] + kHeads - 1) / kHeads, n1 = n0 + (A.heads[1] + kHeads - 1) / kHeads;
  const int n2 = n1 + (A.heads[2] + kHeads - 1) / kHeads;
  const int from = block * A.span, to = min(from + A.span, n2);
  auto part_of = [&](int it) __attribute__((always_inline)) { return it < n0 ? 0 : it < n1 ? 1 : 2; };
  auto head_at = [&](int it, int part) __attribute__((always_inline)) {
    return (it - (part == 0 ? 0 : part == 1 ? n0 : n1)) * kHeads + sub;
  };
  auto fetch = [&](int it) __attribute__((always_inline)) {
    const int part = part_of(it), h = head_at(it, part);
    const T* x = (const T*)A.x[part] + token * A.xt[part] + h * A.xh[part];
    return load_raw<T, INTER, VEC>(x, u, A.dim, half, h < A.heads[part] && 16 * u < A.dim);
  };
  Raw<T> next = fetch(from), weight;
  int weight_part = -1;
  float2* const cs = cs_all[w];
  long at = -1;  // bytes from the cache's beginning to the token's slot
  if (half) turns<LG>(cs, A.positions[token], A.inv_freq, half, A.turn);
  if constexpr (APPEND) {
    const int seq = sequence_of(A.pages, token);
    const Span s = span_of(A.pages, max(seq, 0), A.tokens);
    if (seq < 0 || (int)token >= s.start + s.rows) return;  // a row of no sequence
    if (to > n0) {
      const int key = s.base + (int)token - s.start;
      const int page = key < s.keys ? page_of(A.pages, seq, key) : -1;
      if (page >= 0) at = page * A.pages.page + (key & ((1 << A.pages.shift) - 1)) * A.pages.slot;
    }
  }
  __builtin_amdgcn_wave_barrier();  // the turns are in LDS: this wave's accesses keep their order
  for (int it = from; it < to; ++it) {
    const Raw<T> in = next;
    if (it + 1 < to) next = fetch(it + 1);
    const int part = part_of(it), h = head_at(it, part);
    const bool there = h < A.heads[part] && 16 * u < A.dim;
    T* y;
    if (APPEND && part > 0)
      y = (T*)((part == 1 ? A.pages.k : A.pages.v) + at + h * A.pages.head);
    else
      y = (T*)A.y[part] + token * A.yt[part] + h * A.yh[part];
    const bool write = there && (!APPEND || part == 0 || at >= 0);
    const void* const weights = part < 2 ? A.weight[part] : nullptr;
    if (part == 2 || (!weights && !half)) {
      if (write) store_raw<T, INTER, VEC>(y, u, A.dim, half, in);
      continue;
    }
    float a[8], b[8];
    pairs_of<T, INTER>(in, a, b);
    if (weights) {
      if (part != weight_part) weight = load_raw<T, INTER, VEC>((const T*)weights, u, A.dim, half, 16 * u < A.dim);
      weight_part = part;
      float up, wa[8], wb[8];
      pairs_of<T, INTER>(weight, wa, wb);
      const float r = head_scale<T, LG>(a, b, A.dim, A.eps, &up);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = a[i] * up * r * wa[i];
        b[i] = b[i] * up * r * wb[i];
      }
    }
    rotate(a, b, cs, u, half);
    if (write) store_pairs<T, INTER, VEC>(y, u, A.dim, half, a, b);
  }
}

template <typename T, int LG, bool INTER, bool VEC, bool APPEND>
void launch_one(LbRopeArgs& a, hipStream_t stream) {
  constexpr int kHeads = 64 / LG;
  int steps = 0;
  for (int i = 0; i < 3; ++i) steps += (a.heads[i] + kHeads - 1) / kHeads;
  // one step a wave while there are few tokens, so that a call is short; with more, a wave takes some of
  // its token's heads and computes the turns, and to a cache the slot, once for them.  With inputs from
  // memory, bf16, normed, 2, 3, 5 and 9 steps: 4000 tokens of 64 and 8 heads 34.0, 33.5, 34.8 and 34.8 us, 2039 to a cache
  // 22.1, 23.2, 20.9 and 21.0.  (500 of 40 and 40 heads 8.4, 8.9, 10.9 and 10.8.)
  const long most = APPEND ? 5 : 3;
  a.blocks = a.tokens * steps <= 2048 ? steps : (steps + most - 1) / most;
  while (a.tokens * a.blocks > 1 << 25) a.blocks = (a.blocks + 1) / 2;  // a grid holds fewer than 2^32 threads
  a.span = (steps + a.blocks - 1) / a.blocks;
  const long groups = (a.tokens * a.blocks + 3) / 4;
  hipLaunchKernelGGL((lb_rope_kernel<T, LG, INTER, VEC, APPEND>), dim3((unsigned)groups), dim3(256), 0, stream, a);
}

template <typename T, int LG, bool INTER, bool APPEND>
void launch_vec(LbRopeArgs& a, hipStream_t stream) {
  if (a.dim % 16 == 0 && (INTER || a.rot % 16 == 0))
    launch_one<T, LG, INTER, true, APPEND>(a, stream);
  else
    launch_one<T, LG, INTER, false, APPEND>(a, stream);
}

template <typename T, bool INTER, bool APPEND>
void launch_lanes(LbRopeArgs& a, hipStream_t stream) {
  if (a.dim <= 64)
    launch_vec<T, 4, INTER, APPEND>(a, stream);
  else if (a.dim <= 128)
    launch_vec<T, 8, INTER, APPEND>(a, stream);
  else
    launch_vec<T, 16, INTER, APPEND>(a, stream);
}

template <typename T>
void launch_rope(LbRopeArgs& a, hipStream_t stream) {
  if (a.append) {
    if (a.interleaved)
      launch_lanes<T, true, true>(a, stream);
    else
      launch_lanes<T, false, true>(a, stream);
  } else {
    if (a.interleaved)
      launch_lanes<T, true, false>(a, stream);
    else
      launch_lanes<T, false, false>(a, stream);
  }
}

// ----------------------------------------------------------------------- backward
// dz is dy turned back; with u = w dz:  dx = r u - x (r^3 / dim) sum(u x), and
// dweight = sum over tokens and heads of dz x r.  A wave takes consecutive (token, heads)
// steps and keeps dweight of its lanes' channels in registers; the heads of a wave, the waves
// of a workgroup and, in a second kernel, the workgroups are added in a fixed order.
// Workgroups are for the queries or for the keys.  Bytes bound it: 4000 tokens of 64 and 8 heads of 128, bf16, 44 us,
// 5.0 TB/s; 37 of 40 and 40 7 us, latency.
template <typename T, int LG, bool INTER, bool VEC>
__global__ __launch_bounds__(256) void lb_rope_bwd_kernel(const LbRopeBwdArgs A) {
  __shared__ float2 cs_all[4][kMaxPairs];
  __shared__ float join[4][16 * LG];
  constexpr int kHeads = 64 / LG;
  const int w = wave_id(), lane = threadIdx.x & 63;
  const int u = lane % LG, sub = lane / LG;
  const int half = A.rot / 2;
  const int part = (int)blockIdx.x < A.groups[0] ? 0 : 1;
  const int group = blockIdx.x - (part ? A.groups[0] : 0);
  const int heads = A.heads[part];
  const uint32_t steps = (heads + kHeads - 1) / kHeads;
  const long total = A.tokens * steps, waves = 4l * A.groups[part];
  const long each = (total + waves - 1) / waves;
  const long from = (group * 4l + w) * each, to = from + each < total ? from + each : total;
  const bool lane_in = 16 * u < A.dim;
  const void* const weight = A.weight[part];
  float2* const cs = cs_all[w];
  float wa[8], wb[8], da[8], db[8];
  pairs_of<T, INTER>(load_raw<T, INTER, VEC>((const T*)weight, u, A.dim, half, weight && lane_in), wa, wb);
#pragma unroll
  for (int i = 0; i < 8; ++i) da[i] = db[i] = 0.0f;
  struct In {
    Raw<T> dy, x;
  };
  auto fetch = [&](uint32_t token, uint32_t step) __attribute__((always_inline)) {
    const int h = step * kHeads + sub;
    const bool there = h < heads && lane_in;
    In in;
    in.dy = load_raw<T, INTER, VEC>((const T*)A.dy[part] + token * A.dyt[part] + h * A.dyh[part], u, A.dim, half, there);
    in.x = load_raw<T, INTER, VEC>((const T*)A.x[part] + token * A.xt[part] + h * A.xh[part], u, A.dim, half,
                                   there && weight);
    return in;
  };
  uint32_t token = (uint32_t)(from / steps), step = (uint32_t)(from - token * (long)steps);
  int turned = -1;
  In next;
  if (from < to) next = fetch(token, step);
  for (long j = from; j < to; ++j) {
    const In in = next;
    const uint32_t t = token, st = step;
    if (++step == steps) {
      step = 0;
      ++token;
    }
    if (j + 1 < to) next = fetch(token, step);
    if (half && (int)t != turned) {
      turned = t;
      __builtin_amdgcn_wave_barrier();
      turns<LG>(cs, A.positions[t], A.inv_freq, half, -1.0f);
      __builtin_amdgcn_wave_barrier();
    }
    const int h = st * kHeads + sub;
    float a[8], b[8];
    pairs_of<T, INTER>(in.dy, a, b);
    rotate(a, b, cs, u, half);
    if (weight) {
      float xa[8], xb[8], up;
      pairs_of<T, INTER>(in.x, xa, xb);
      const float ru = head_scale<T, LG>(xa, xb, A.dim, A.eps, &up);
      float along = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xa[i] = xa[i] * up * ru;  // x r
        xb[i] = xb[i] * up * ru;
        along += wa[i] * a[i] * xa[i] + wb[i] * b[i] * xb[i];
      }
      along = head_sum<LG>(along) / (float)A.dim;
      const float r = ru * up;
      const bool there = h < heads;  // behind the last head there are zeros; with eps = 0 their r is infinite
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (there) {
          da[i] += a[i] * xa[i];
          db[i] += b[i] * xb[i];
        }
        a[i] = r * (wa[i] * a[i] - xa[i] * along);
        b[i] = r * (wb[i] * b[i] - xb[i] * along);
      }
    }
    if (h < heads && lane_in)
      store_pairs<T, INTER, VEC>((T*)A.dx[part] + t * A.dxt[part] + h * A.dxh[part], u, A.dim, half, a, b);
  }
  if (!weight) return;  // the whole workgroup
  auto over_heads = [&](float v) __attribute__((always_inline)) {
    if constexpr (LG <= 4) v += lane_xor<4>(v);
    if constexpr (LG <= 8) v += lane_xor<8>(v);
    v += lane_xor<16>(v);
    return v + lane_xor<32>(v);
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    da[i] = over_heads(da[i]);
    db[i] = over_heads(db[i]);
    if (sub == 0) {
      join[w][16 * u + i] = da[i];
      join[w][16 * u + 8 + i] = db[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * LG; i += 256) {
    const int pair = 8 * (i >> 4) + (i & 7);
    if (pair < A.dim / 2) {
      const int d = i & 8 ? second_of<INTER>(pair, half) : first_of<INTER>(pair, half);
      // VEC pairs what is not rotated by eights
      const int dv = i & 8 ? vec_hi<INTER>(i >> 4, half) : vec_lo<INTER>(i >> 4, half);
      const int channel = VEC && !INTER ? dv + (i & 7) : d;
      A.partial[(long)blockIdx.x * A.dim + channel] = (join[0][i] + join[1][i]) + (join[2][i] + join[3][i]);
    }
  }
}

// dweight = sum of the workgroups' partial sums: 16 columns x 64 slices of workgroups,
// joined in order.  Latency bounds it, 3 to 5 us.
__global__ __launch_bounds__(1024) void lb_rope_dweight_kernel(const LbRopeBwdArgs A) {
  __shared__ float s[64][17];
  const int part = blockIdx.y;
  if (!A.dweight[part]) return;
  const float* partial = A.partial + (part ? (long)A.groups[0] * A.dim : 0);
  const int groups = A.groups[part];
  const int c = threadIdx.x & 15, p = threadIdx.x >> 4;
  const int k = blockIdx.x * 16 + c;
  float v = 0.0f;
  if (k < A.dim) {
#pragma unroll 8
    for (int g = p; g < groups; g += 64) v += partial[(long)g * A.dim + k];
  }
  s[p][c] = v;
  __syncthreads();
  if (p == 0 && k < A.dim) {
    v = s[0][c];
#pragma unroll 16
    for (int i = 1; i < 64; ++i) v += s[i][c];
    A.dweight[part][k] = v;
  }
}

template <typename T, int LG, bool INTER>
void launch_bwd_vec(const LbRopeBwdArgs& a, hipStream_t stream) {
  const dim3 grid(a.groups[0] + a.groups[1]);
  if (a.dim % 16 == 0 && (INTER || a.rot % 16 == 0))
    hipLaunchKernelGGL((lb_rope_bwd_kernel<T, LG, INTER, true>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((lb_rope_bwd_kernel<T, LG, INTER, false>), grid, dim3(256), 0, stream, a);
}

template <typename T, bool INTER>
void launch_bwd_lanes(const LbRopeBwdArgs& a, hipStream_t stream) {
  if (a.dim <= 64)
    launch_bwd_vec<T, 4, INTER>(a, stream);
  else if (a.dim <= 128)
    launch_bwd_vec<T, 8, INTER>(a, stream);
  else
    launch_bwd_vec<T, 16, INTER>(a, stream);
}

template <typename T>
void launch_bwd(const LbRopeBwdArgs& a, hipStream_t stream) {
  if (a.interleaved)
    launch_bwd_lanes<T, true>(a, stream);
  else
    launch_bwd_lanes<T, false>(a, stream);
}

// ------------------------------------------------------------------ accepted rows
// A workgroup: the accepted rows of one head's keys or values, all in registers before the first is written: at
// most PIECES 16-byte pieces a thread, eight for 64 rows of 256 channels.  Latency bounds it, and, of many
// sequences, how many workgroups run at once: 48 trees, 40 heads of 128, 9 rows each, 15 us with room for 8 pieces a thread,
// 4.8 with one; one tree 2.9.
template <int PIECES>
__global__ __launch_bounds__(256) void lb_accept_kernel(const LbPages P, int dim, const int32_t* __restrict__ path,
                                                        int columns) {
  const int seq = blockIdx.y, head = blockIdx.x >> 1;
  char* const cache = (blockIdx.x & 1 ? P.v : P.k) + head * P.head;
  const int pieces = dim / 8;
  // rows of the sequence are named as the call that appended them had them: all rows that starts gives
  const Span s = span_of(P, seq, 0x7FFFFFFF);
  auto slot = [&](int row) __attribute__((always_inline)) {
    const int key = s.base + row;
    const int page = row >= 0 && row < s.rows && key < s.keys ? page_of(P, seq, key) : -1;
    return page < 0 ? -1l : page * P.page + (key & ((1 << P.shift) - 1)) * P.slot;
  };
  u32x4 r[PIECES];
  long to[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const uint32_t item = threadIdx.x + 256 * i;
    const int j = item / (uint32_t)pieces, c = item - j * pieces;
    to[i] = -1;
    r[i] = u32x4{0, 0, 0, 0};
    if (j < columns) {
      const int from = path[(long)seq * columns + j];
      if (from >= 0 && from != j) {
        const long src = slot(from), dst = slot(j);
        if (src >= 0 && dst >= 0) {
          r[i] = *(const u32x4*)(cache + src + 16 * c);
          to[i] = dst + 16 * c;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PIECES; ++i) __asm__ volatile("" : "+v"(r[i]));  // a use: every load of this wave has come back
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
    if (to[i] >= 0) *(u32x4*)(cache + to[i]) = r[i];
}

}  // namespace

hipError_t lb_launch_rope(LbRopeArgs& a, int dtype, hipStream_t stream) {
  if (dtype == 1)
    launch_rope<f16>(a, stream);
  else
    launch_rope<bf16>(a, stream);
  return hipGetLastError();
}

// Workgroups of the backward pass, a function of the sizes alone (the sums and the workspace are the same on
// every part): one step a wave up to four workgroups a compute unit (with the second kernel, inputs from memory: 512, 1024
// and 2048 workgroups 64, 58 and 57 us for 4000 tokens of 64 and 8 heads, bf16, 33, 30 and 33 for 8000 of 8 and 8).
void lb_rope_bwd_groups(int64_t tokens, int heads, int kv_heads, int dim, int* groups) {
  const int per = 64 / (dim <= 64 ? 4 : dim <= 128 ? 8 : 16);
  const int64_t a = tokens * ((heads + per - 1) / per), b = tokens * ((kv_heads + per - 1) / per);
  const int64_t all = a + b;
  const int64_t total = all <= 4 ? 1 : all / 4 < 1024 ? all / 4 : 1024;
  int64_t ga = all ? (a * total + all - 1) / all : 0, gb = all ? (b * total + all - 1) / all : 0;
  groups[0] = (int)ga;
  groups[1] = (int)gb;
}

hipError_t lb_launch_rope_bwd(const LbRopeBwdArgs& a, int dtype, hipStream_t stream) {
  if (a.groups[0] + a.groups[1] > 0) {
    if (dtype == 1)
      launch_bwd<f16>(a, stream);
    else
      launch_bwd<bf16>(a, stream);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.dweight[0] && !a.dweight[1])) return e;
  hipLaunchKernelGGL(lb_rope_dweight_kernel, dim3((a.dim + 15) / 16, 2), dim3(1024), 0, stream, a);
  return hipGetLastError();
}

hipError_t lb_launch_accept(const LbPages& p, int heads, int dim, const int32_t* path, int columns, hipStream_t stream) {
  const dim3 grid(2 * heads, p.seqs);
  const int items = columns * (dim / 8);
  if (items <= 256)
    hipLaunchKernelGGL(lb_accept_kernel<1>, grid, dim3(256), 0, stream, p, dim, path, columns);
  else if (items <= 512)
    hipLaunchKernelGGL(lb_accept_kernel<2>, grid, dim3(256), 0, stream, p, dim, path, columns);
  else
    hipLaunchKernelGGL(lb_accept_kernel<8>, grid, dim3(256), 0, stream, p, dim, path, columns);
  return hipGetLastError();
}
