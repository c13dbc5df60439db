// Log probabilities of given tokens, entropy and top alternatives of a row of
// logits, and the gradient of the logits.
//
// Forward: one pass over the row.  Each thread keeps a running maximum m and
//     s = sum exp(x - m),   e = sum exp(x - m) (x - m)
// (moved to a new maximum by s' = s exp(m - m'), e' = (e + (m - m') s) exp(m - m')),
// and log p = (x - m) - log s, entropy = log s - e / s.  Few rows are split over
// several workgroups, whose parts a second kernel joins.
//
// Alternatives: a logit and its place make one 64-bit key (order of the value,
// then the lower place), so no two are equal and the order is total.  Each
// wave holds its 64 largest keys so far, lane i the i-th; only logits above
// the top-th of them are looked at (a comparison of the thread's maximum of
// 16 against it), are collected in LDS and, 64 at a time, sorted and merged
// in.
#include "head_common.h"
#include "head_launch.h"

using namespace lbh;

namespace {

constexpr int kThreads = 256;
constexpr int kEpt = 16;                    // elements a thread holds of a chunk
constexpr int kChunk = kThreads * kEpt;     // 4096
constexpr float kLow = -3.402823466e+38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -1e30f;              // below any distance whose exp is not 0
constexpr int kBuf = 128;                   // collected keys a wave (64 merged at a time)

typedef unsigned long long u64;

__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// exp(d) for d <= 0; a d of -infinity or below any representable exp gives 0
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

struct Stat {
  float m, s, e;
};
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  Stat r;
  r.m = max_nan(a.m, b.m);
  const float da = max_nan(a.m - r.m, kFar), db = max_nan(b.m - r.m, kFar);
  const float ea = exp_of(da), eb = exp_of(db);
  r.s = a.s * ea + b.s * eb;
  r.e = (a.e + da * a.s) * ea + (b.e + db * b.s) * eb;
  return r;
}
__device__ __forceinline__ Stat wave_join(Stat a) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    Stat b;
    b.m = __shfl_xor(a.m, m, 64);
    b.s = __shfl_xor(a.s, m, 64);
    b.e = __shfl_xor(a.e, m, 64);
    a = join(a, b);
  }
  return a;
}

// ---------------------------------------------------------------- ordered keys
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;                                // NaN ranks first
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);     // -0 is 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  if (o == 0xFFFFFFFFu) return NAN;
  return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ u64 key_of(float x, uint32_t place) { return (u64)order_of(x) << 32 | (uint32_t)~place; }

__device__ __forceinline__ u64 shfl_xor64(u64 v, int m) {
  const uint32_t lo = __shfl_xor((uint32_t)v, m, 64), hi = __shfl_xor((uint32_t)(v >> 32), m, 64);
  return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 lane64(u64 v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
  return (u64)hi << 32 | lo;
}

// One exchange of a bitonic network: the lane whose bit `m` is clear keeps the
// larger key if `down`, the smaller otherwise.
__device__ __forceinline__ u64 exchange(u64 v, int m, bool down, int lane) {
  const u64 o = shfl_xor64(v, m);
  const bool keep_larger = ((lane & m) == 0) == down;
  return (v > o) == keep_larger ? v : o;
}
__device__ inline u64 sort64(u64 v, int lane) {  // lane 0 the largest
#pragma unroll
  for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
    for (int m = k >> 1; m > 0; m >>= 1) v = exchange(v, m, (lane & k) == 0, lane);
  return v;
}
// The 64 largest of two sorted lists, sorted.
__device__ inline u64 merge64(u64 a, u64 b, int lane) {
  const uint32_t lo = __shfl((uint32_t)b, 63 - lane, 64), hi = __shfl((uint32_t)(b >> 32), 63 - lane, 64);
  const u64 r = (u64)hi << 32 | lo;
  u64 v = a > r ? a : r;
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = exchange(v, m, true, lane);
  return v;
}

// The wave's LDS accesses stand in program order (the hardware keeps a wave's
// order; this keeps the compiler's).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wave's largest keys: `list` sorted over the lanes (0 where there are fewer
// than 64), `pending` more in its part of LDS.
struct Tops {
  u64 list;
  int pending;
  float bar;  // value of the top-th key; NaN while there are fewer
};

__device__ __forceinline__ void tops_flush(Tops& T, u64* buf, int top, int lane, int take) {
  // `take` keys (at most 64) from the front; the rest moves up
  u64 k = lane < take ? buf[lane] : 0;
  const int rest = T.pending - take;
  const u64 moved = lane < rest ? buf[take + lane] : 0;
  wave_fence();
  if (lane < rest) buf[lane] = moved;
  wave_fence();
  T.pending = rest;
  k = sort64(k, lane);
  T.list = merge64(T.list, k, lane);
  const u64 b = lane64(T.list, top - 1);
  T.bar = b ? value_of((uint32_t)(b >> 32)) : NAN;
}

// Collects the chunk's logits that can be among the `top` largest.  `v` holds
// kEpt of them, the first `valid` inside the row, `most` their maximum;
// place(i) is where the i-th stands.
template <typename PLACE>
__device__ __forceinline__ void tops_chunk(Tops& T, u64* buf, int top, int lane, const float (&v)[kEpt], int valid,
                                           float most, PLACE place) {
  // a chunk comes after all that is in the list, so an equal value is no better
  const bool some = valid > 0 && !(most <= T.bar);
  const u64 lanes = __ballot(some);
  if (lanes == 0) return;
  u64 least = 0;
  if (__popcll(lanes) > 32) {
    // many at once (the first chunk): the top-th of the lanes' own largest is a bar too
    u64 mine = 0;
#pragma unroll
    for (int i = 0; i < kEpt; ++i)
      if (i < valid) {
        const u64 k = key_of(v[i], place(i));
        mine = k > mine ? k : mine;
      }
    least = lane64(sort64(mine, lane), top - 1);
  }
  // places inside the chunk are in no order over the lanes, so what the list
  // takes in meanwhile raises `least` (a whole key), not the bar on values
  const float bar = T.bar;
  const float floor = least ? value_of((uint32_t)(least >> 32)) : NAN;
  uint32_t todo = 0;
#pragma unroll
  for (int i = 0; i < kEpt; ++i)
    if (i < valid && !(v[i] <= bar) && !(v[i] < floor)) todo |= 1u << i;
  u64 rest;
  while ((rest = __ballot(todo != 0)) != 0) {
    const int i = todo ? __builtin_ctz(todo) : 0;
    todo &= todo - 1;
    float x = v[0];
#pragma unroll
    for (int j = 1; j < kEpt; ++j) x = i == j ? v[j] : x;
    const u64 k = key_of(x, place(i));
    const bool in = (rest >> lane & 1) && k >= least;
    const u64 ins = __ballot(in);
    if (in) buf[T.pending + __popcll(ins & ((1ull << lane) - 1))] = k;
    wave_fence();
    T.pending += __popcll(ins);
    if (T.pending >= 64) {
      tops_flush(T, buf, top, lane, 64);
      const u64 b = lane64(T.list, top - 1);
      least = b > least ? b : least;
    }
  }
}

// ------------------------------------------------------------------- the parts
// What one workgroup leaves of its span of a row, when a row is split.
__host__ __device__ inline size_t part_bytes(int top) { return 16 + 8 * (size_t)top; }

__device__ __forceinline__ void write_row(const LbLogprobsArgs& A, long row, const Stat& S, float xt, int64_t target) {
  const float logs = logf(S.s);
  A.lse[row] = S.m;
  A.lse[A.rows + row] = logs;
  if (A.logprob) {
    float p = 0.0f;
    if (target >= A.vocab)
      p = NAN;
    else if (target >= 0)
      p = S.s == 0.0f ? -INFINITY : (xt - S.m) - logs;
    A.logprob[row] = p;
  }
  if (A.entropy) A.entropy[row] = S.s == 0.0f ? 0.0f : logs - S.e / S.s;
}

__device__ __forceinline__ void write_top(const LbLogprobsArgs& A, long row, const Stat& S, u64 key, int lane) {
  if (lane >= A.top) return;
  const float x = value_of((uint32_t)(key >> 32));
  A.top_index[row * A.top + lane] = (int64_t)(uint32_t)~(uint32_t)key;
  A.top_logprob[row * A.top + lane] = S.s == 0.0f ? (x != x ? x : -INFINITY) : (x - S.m) - logf(S.s);
}

template <typename T>
__device__ __forceinline__ float target_logit(const LbLogprobsArgs& A, long row, int64_t target) {
  if (target < 0 || target >= A.vocab) return 0.0f;
  return (float)((const T*)A.logits)[row * A.ld + target];
}

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void lb_logprobs_kernel(const LbLogprobsArgs A) {
  constexpr int kWaves = kThreads / 64;
  __shared__ u64 buf[TOP ? kWaves : 1][kBuf];
  __shared__ Stat stat[kWaves];
  const int t = threadIdx.x, w = wave_id(), lane = t & 63;
  const long row = blockIdx.x / A.splits;
  const int split = (int)(blockIdx.x - row * A.splits);
  const int begin = split * A.span;
  const int end = (int)min((long)A.vocab, (long)begin + A.span);
  const T* x = (const T*)A.logits + row * A.ld;
  Stat S = {kLow, 0.0f, 0.0f};
  Tops P = {0, 0, NAN};
  for (long c = begin; c < end; c += kChunk) {
    float v[kEpt];
    const long k0 = c + 8 * t, k1 = k0 + 8 * kThreads;
    float lo[8], hi[8];
    load8(x + k0, end - k0, -INFINITY, lo);
    load8(x + k1, end - k1, -INFINITY, hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = lo[i];
      v[8 + i] = hi[i];
    }
    float most = v[0];
#pragma unroll
    for (int i = 1; i < kEpt; ++i) most = max_nan(most, v[i]);
    const float m = max_nan(S.m, most);
    const float dm = max_nan(S.m - m, kFar), em = exp_of(dm);
    float s = S.s * em, e = (S.e + dm * S.s) * em;
#pragma unroll
    for (int i = 0; i < kEpt; ++i) {
      const float d = max_nan(v[i] - m, kFar);
      const float p = exp_of(d);
      s += p;
      e += p * d;
    }
    S.m = m;
    S.s = s;
    S.e = e;
    if constexpr (TOP) {
      const long left0 = end - k0, left1 = end - k1;
      const int n0 = left0 >= 8 ? 8 : left0 > 0 ? (int)left0 : 0, n1 = left1 >= 8 ? 8 : left1 > 0 ? (int)left1 : 0;
      const int valid = n1 > 0 ? 8 + n1 : n0;  // the first eight are whole where the second have any
      tops_chunk(P, buf[w], A.top, lane, v, valid, most,
                 [&](int i) { return (uint32_t)(i < 8 ? k0 + i : k1 + i - 8); });
    }
  }
  S = wave_join(S);
  if (lane == 0) stat[w] = S;
  if constexpr (TOP) {
    if (P.pending > 0) tops_flush(P, buf[w], A.top, lane, P.pending);
    __syncthreads();
    buf[w][lane] = P.list;
  }
  __syncthreads();
  if (w != 0) return;
  S = stat[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) S = join(S, stat[i]);
  u64 list = P.list;
  if constexpr (TOP) {
#pragma unroll
    for (int i = 1; i < kWaves; ++i) list = merge64(list, buf[i][lane], lane);
  }
  if (A.splits == 1) {
    if (lane == 0) {
      const int64_t target = A.targets ? A.targets[row] : -1;
      write_row(A, row, S, target_logit<T>(A, row, target), target);
    }
    if constexpr (TOP) write_top(A, row, S, list, lane);
  } else {
    char* part = (char*)A.ws + (size_t)blockIdx.x * part_bytes(A.top);
    if (lane == 0) *(Stat*)part = S;
    if constexpr (TOP)
      if (lane < A.top) ((u64*)(part + 16))[lane] = list;
  }
}

// Joins the parts of a row: one wave a row.
template <typename T>
__global__ __launch_bounds__(64) void lb_logprobs_join_kernel(const LbLogprobsArgs A) {
  const int lane = threadIdx.x;
  const long row = blockIdx.x;
  const size_t bytes = part_bytes(A.top);
  const char* parts = (const char*)A.ws + (size_t)row * A.splits * bytes;
  Stat S = {kLow, 0.0f, 0.0f};
  for (int i = lane; i < A.splits; i += 64) S = join(S, *(const Stat*)(parts + i * bytes));
  S = wave_join(S);
  if (A.top > 0) {
    u64 list = lane < A.top ? ((const u64*)(parts + 16))[lane] : 0;
    for (int i = 1; i < A.splits; ++i) {
      const u64 k = lane < A.top ? ((const u64*)(parts + i * bytes + 16))[lane] : 0;
      list = merge64(list, k, lane);
    }
    write_top(A, row, S, list, lane);
  }
  if (lane == 0) {
    const int64_t target = A.targets ? A.targets[row] : -1;
    write_row(A, row, S, target_logit<T>(A, row, target), target);
  }
}

// -------------------------------------------------------------------- backward
// d = p (a + b (log p + H)) + direct gradients, with a = -(dlogprob + sum
// dtop) and b = -dentropy.  Each logit is read once and its gradient written
// once.  The places with a direct gradient (the target and the alternatives)
// are marked in a bitmap of the workgroup's vectors of eight, and only a
// marked vector looks them up.
constexpr int kBwdVecs = 4;                          // vectors of eight a thread
constexpr int kBwdSpan = kThreads * kBwdVecs * 8;    // 8192 logits a workgroup

template <typename T>
__global__ __launch_bounds__(kThreads) void lb_logprobs_bwd_kernel(const LbLogprobsBwdArgs A, int spans) {
  __shared__ uint32_t marked[kBwdSpan / 8 / 32];
  __shared__ int place[LBH_MAX_DIRECT];
  __shared__ float direct[LBH_MAX_DIRECT];
  const int t = threadIdx.x;
  const long row = blockIdx.x / spans;
  const int begin = (int)(blockIdx.x - row * spans) * kBwdSpan;
  const T* x = (const T*)A.logits + row * A.ld;
  T* out = (T*)A.dlogits + row * A.ldd;
  float v[kBwdVecs][8];
#pragma unroll
  for (int i = 0; i < kBwdVecs; ++i) {
    const long k = begin + 8l * (t + i * kThreads);
    load8(x + k, A.vocab - k, 0.0f, v[i]);
  }
  const float m = A.lse[row], logs = A.lse[A.rows + row];  // log p = (x - m) - logs
  const float H = A.entropy ? A.entropy[row] : 0.0f;
  float a = 0.0f;
  const int64_t target = A.targets ? A.targets[row] : -1;
  const float glp = target >= A.vocab ? NAN : target >= 0 ? A.dlogprob[row] : 0.0f;
  a -= glp;
  for (int j = 0; j < A.top; ++j) a -= A.dtop[row * A.top + j];
  const float b = A.dentropy ? -A.dentropy[row] : 0.0f;
  const bool empty = logs == -INFINITY;  // nothing but masked logits
  if (t < kBwdSpan / 8 / 32) marked[t] = 0;
  __syncthreads();
  if (t <= A.top) {
    const int64_t p = t == 0 ? target : A.top_index[row * A.top + t - 1];
    const bool here = !empty && p >= begin && p < (long)begin + kBwdSpan && p < A.vocab;
    place[t] = here ? (int)p : -1;
    direct[t] = t == 0 ? glp : A.dtop[row * A.top + t - 1];
    if (here) {
      const int vec = (int)(p - begin) >> 3;
      atomicOr(&marked[vec >> 5], 1u << (vec & 31));
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBwdVecs; ++i) {
    const int vec = t + i * kThreads;
    const long k = begin + 8l * vec;
    if (k >= A.vocab) break;
    float d[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = max_nan((v[i][e] - m) - logs, kFar);
      const float p = exp_of(y);
      d[e] = empty ? 0.0f : p * (a + b * (y + H));
    }
    if (marked[vec >> 5] >> (vec & 31) & 1) {
      for (int j = 0; j <= A.top; ++j) {
        const int at = place[j] - (int)k;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at == e) d[e] += direct[j];
      }
    }
    store8(out + k, A.vocab - k, d);
  }
}

template <typename T>
void launch_fwd(const LbLogprobsArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.rows * a.splits));
  if (a.top > 0)
    hipLaunchKernelGGL((lb_logprobs_kernel<T, true>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((lb_logprobs_kernel<T, false>), grid, dim3(kThreads), 0, stream, a);
  if (a.splits > 1)
    hipLaunchKernelGGL((lb_logprobs_join_kernel<T>), dim3((unsigned)a.rows), dim3(64), 0, stream, a);
}

template <typename T>
void launch_bwd(const LbLogprobsBwdArgs& a, hipStream_t stream) {
  const int spans = (a.vocab + kBwdSpan - 1) / kBwdSpan;
  hipLaunchKernelGGL((lb_logprobs_bwd_kernel<T>), dim3((unsigned)(a.rows * spans)), dim3(kThreads), 0, stream, a, spans);
}

}  // namespace

// Workgroups a row: one where the rows alone fill the card, else as many as
// give about 1024 workgroups, each with a whole chunk at least.
int lb_logprobs_splits(int64_t rows, int64_t vocab, int dtype, int* span) {
  (void)dtype;
  const int64_t chunks = (vocab + kChunk - 1) / kChunk;
  int64_t splits = rows > 0 ? 1024 / rows : 1;
  if (splits > chunks) splits = chunks;
  if (splits < 1) splits = 1;
  const int64_t per = (chunks + splits - 1) / splits;
  *span = (int)(per * kChunk < vocab ? per * kChunk : (vocab + 7) / 8 * 8);
  return (int)((chunks + per - 1) / per);
}

size_t lb_logprobs_partial_bytes(int64_t rows, int splits, int top) {
  return splits > 1 ? (size_t)rows * splits * part_bytes(top) : 0;
}

hipError_t lb_launch_logprobs(const LbLogprobsArgs& a, int dtype, hipStream_t stream) {
  if (dtype == 0)
    launch_fwd<float>(a, stream);
  else if (dtype == 1)
    launch_fwd<f16>(a, stream);
  else
    launch_fwd<bf16>(a, stream);
  return hipGetLastError();
}

hipError_t lb_launch_logprobs_bwd(const LbLogprobsBwdArgs& a, int dtype, hipStream_t stream) {
  if (dtype == 0)
    launch_bwd<float>(a, stream);
  else if (dtype == 1)
    launch_bwd<f16>(a, stream);
  else
    launch_bwd<bf16>(a, stream);
  return hipGetLastError();
}
