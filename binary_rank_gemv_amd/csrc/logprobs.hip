// Log probabilities of given tokens, entropy and top alternatives of a row of
// logits, and the gradient of the logits.
//
// Forward: one pass over the row.  Each thread keeps a running maximum m and
//     s = sum exp(x - m),   e = sum exp(x - m) (x - m)
// (moved to a new maximum by s' = s exp(m - m'), e' = (e + (m - m') s) exp(m - m')),
// and log p = (x - m) - log s, entropy = log s - e / s.  Few rows are split over
// several workgroups, whose parts a second kernel joins.
//
// What bounds it: memory, for long texts (2048 x 32000 fp16: 30.5 us without
// alternatives, 4.3 TB/s, of which about 5 are the start and the end, where all
// rows are at the same point; 34.5 with one alternative, 37 with 20; its vector
// instructions alone would take 20); latency, for few rows (one row of 32000: 9 us).
// The gradient reads and writes at 5 TB/s (1021 x 32000 bf16: 26 us).
//
// Alternatives: a logit and its place make one 64-bit key (order of the value,
// then the lower place), so no two are equal and the order is total.  The pass
// keeps each thread's maximum, nothing else.  The threads of equal lane are a
// group; the top-th largest of the 64 groups' maxima is a bound that at
// least `top` logits reach and few others do (24 expected for top 20, in a row
// without ties), so only threads whose maximum reaches it read their part of
// the row again and collect what reaches it in LDS, where the keys are
// sorted, 64 at a time, over the lanes.
#include "head_common.h"
#include "head_launch.h"

using namespace lbh;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kEpt = 16;                    // elements a thread holds of a chunk
constexpr int kChunk = kThreads * kEpt;     // 4096
constexpr float kLow = -3.402823466e+38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -1e4f;               // below any distance whose exp is not 0 (and far from overflow in sums)
constexpr int kBuf = 128;                   // collected keys a wave (64 merged at a time)
constexpr int kKept = 8;                    // groups of chunks whose maxima a thread keeps for the second look
constexpr int kWork = 256;                  // entries of the second look's list

typedef unsigned long long u64;

// exp(d) for d <= 0; a d of -infinity or below any representable exp gives 0
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

struct Stat {
  float m, s, e;
};
struct Part {
  Stat s;
  float xt;  // the target's logit, in the part that holds it
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
template <int M>
__device__ __forceinline__ Stat join_lane(const Stat& a) {
  Stat b;
  b.m = lane_xor<M>(a.m);
  b.s = lane_xor<M>(a.s);
  b.e = lane_xor<M>(a.e);
  return join(a, b);
}
__device__ __forceinline__ Stat wave_join(Stat a) {
  a = join_lane<1>(a);
  a = join_lane<2>(a);
  a = join_lane<4>(a);
  a = join_lane<8>(a);
  a = join_lane<16>(a);
  return join_lane<32>(a);
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

template <int M>
__device__ __forceinline__ uint32_t other(uint32_t v) { return lane_xor<M>(v); }
template <int M>
__device__ __forceinline__ u64 other(u64 v) {
  return (u64)lane_xor<M>((uint32_t)(v >> 32)) << 32 | lane_xor<M>((uint32_t)v);
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ u64 lane_of(u64 v, int lane) {
  return (u64)lane_of((uint32_t)(v >> 32), lane) << 32 | lane_of((uint32_t)v, lane);
}

// One exchange of a bitonic network over the lanes: the lane whose bit M is
// clear keeps the larger key if `down`, the smaller otherwise.
template <int M, typename K>
__device__ __forceinline__ K exchange(K v, bool down, int lane) {
  const K o = other<M>(v);
  const bool keep_larger = ((lane & M) == 0) == down;
  return (v > o) == keep_larger ? v : o;
}
template <typename K>
__device__ __forceinline__ K falling64(K v, int lane) {  // of a bitonic sequence
  v = exchange<32>(v, true, lane);
  v = exchange<16>(v, true, lane);
  v = exchange<8>(v, true, lane);
  v = exchange<4>(v, true, lane);
  v = exchange<2>(v, true, lane);
  return exchange<1>(v, true, lane);
}
template <typename K>
__device__ __forceinline__ K sort64(K v, int lane) {  // lane 0 the largest
  bool d = (lane & 2) == 0;
  v = exchange<1>(v, d, lane);
  d = (lane & 4) == 0;
  v = exchange<2>(v, d, lane);
  v = exchange<1>(v, d, lane);
  d = (lane & 8) == 0;
  v = exchange<4>(v, d, lane);
  v = exchange<2>(v, d, lane);
  v = exchange<1>(v, d, lane);
  d = (lane & 16) == 0;
  v = exchange<8>(v, d, lane);
  v = exchange<4>(v, d, lane);
  v = exchange<2>(v, d, lane);
  v = exchange<1>(v, d, lane);
  d = (lane & 32) == 0;
  v = exchange<16>(v, d, lane);
  v = exchange<8>(v, d, lane);
  v = exchange<4>(v, d, lane);
  v = exchange<2>(v, d, lane);
  v = exchange<1>(v, d, lane);
  return falling64(v, lane);
}
// The 64 largest of two falling lists, falling.
__device__ __forceinline__ u64 merge64(u64 a, u64 b, int lane) {
  const u64 r = other<32>(other<16>(other<15>(b)));  // b backwards
  return falling64(a > r ? a : r, lane);
}

// The wave's LDS accesses stand in program order (the hardware keeps a wave's
// order; this keeps the compiler's).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wave's largest keys: `list` falling over the lanes (0 where there are fewer
// than 64), `pending` more in its part of LDS.
struct Tops {
  u64 list;
  u64 least;  // the top-th of the list: a key has to be larger (0: any)
  int pending;
};

// Moves `take` keys (at most 64) from the front of the buffer into the list.
__device__ __forceinline__ void tops_flush(Tops& T, u64* buf, int top, int lane, int take) {
  const u64 k = lane < take ? buf[lane] : 0;
  const int rest = T.pending - take;
  const u64 moved = lane < rest ? buf[take + lane] : 0;
  wave_fence();
  if (lane < rest) buf[lane] = moved;
  wave_fence();
  T.pending = rest;
  T.list = merge64(T.list, sort64(k, lane), lane);
  T.least = lane_of(T.list, top - 1);
}

// v[i] for an i of the lane's own: all in registers (out of an array the compiler
// makes an indexed read of scratch memory of it).
typedef float f32xe __attribute__((ext_vector_type(kEpt)));
__device__ __forceinline__ float pick(f32xe v, int i) { return v[i]; }

// Collects the chunk's logits of at least `floor` (NaN: all) that can be among
// the `top` largest.  `v` holds kEpt of them, the first `valid` inside the row;
// place(i) is where the i-th stands.
template <typename PLACE>
__device__ __forceinline__ void tops_chunk(Tops& T, u64* buf, int top, int lane, const float (&v)[kEpt], int valid,
                                           float floor, PLACE place) {
  uint32_t todo = 0;
  f32xe all;
#pragma unroll
  for (int i = 0; i < kEpt; ++i) {
    all[i] = v[i];
    if (i < valid && !(v[i] < floor)) todo |= 1u << i;
  }
  while (__ballot(todo != 0) != 0) {
    const int i = todo ? __builtin_ctz(todo) : 0;
    const u64 k = key_of(pick(all, i), place(i));
    const bool in = todo && k > T.least;
    const u64 ins = __ballot(in);
    if (in) buf[T.pending + __popcll(ins & ((1ull << lane) - 1))] = k;
    todo &= todo - 1;
    wave_fence();
    T.pending += __popcll(ins);
    if (T.pending >= 64) tops_flush(T, buf, top, lane, 64);
  }
}

// ------------------------------------------------------------------- the parts
// What one workgroup leaves of its span of a row, when a row is split: one
// Part, and behind those of all rows `top` keys a part.
__host__ __device__ inline size_t part_keys_at(long parts) { return (size_t)parts * sizeof(Part); }

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

// The 64 largest of `count` keys, falling, in wave 0; `keys` in LDS or global
// memory, `room` LDS for the waves' lists.  Whole workgroup.
__device__ __forceinline__ u64 block_top(const u64* keys, int count, u64 (*room)[64], int w, int lane) {
  u64 list = 0;
  for (int at = 64 * w; at < count; at += 64 * kWaves) {
    u64 k = at + lane < count ? keys[at + lane] : 0;
    if (count > 1) k = sort64(k, lane);
    list = at == 64 * w ? k : merge64(list, k, lane);
  }
  if (count > 64) {
    room[w][lane] = list;
    __syncthreads();
    if (w == 0) {
      const int lists = min(kWaves, (count + 63) / 64);
      for (int i = 1; i < lists; ++i) list = merge64(list, room[i][lane], lane);
    }
  }
  return list;
}

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));  // at any byte

template <typename T>
struct Chunk {
  u32x4 w[kEpt * sizeof(T) / 16];
};
// 16-byte words of two vectors of eight; what lies behind the row is -infinity.
template <typename T>
__device__ __forceinline__ void chunk_load(Chunk<T>& C, const T* x, long c, long end, int t) {
  constexpr int kW = sizeof(T) / 2;  // 16-byte words a vector
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long k = c + 8 * (t + h * kThreads), left = end - k;
    if (left >= 8) {
#pragma unroll
      for (int j = 0; j < kW; ++j) C.w[h * kW + j] = load_any<u32x4>((const char*)(x + k) + 16 * j);
    } else {
      T e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = i < left ? x[k + i] : (T)-INFINITY;
      __builtin_memcpy(&C.w[h * kW], e, sizeof e);
    }
  }
}
template <typename T>
__device__ __forceinline__ void chunk_load_whole(Chunk<T>& C, const T* x, int t) {
  constexpr int kW = sizeof(T) / 2;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < kW; ++j)
      C.w[h * kW + j] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_any*>((const char*)(x + 8 * (t + h * kThreads)) + 16 * j));
}
template <typename T>
__device__ __forceinline__ void chunk_values(const Chunk<T>& C, float (&v)[kEpt]) {
#pragma unroll
  for (int i = 0; i < kEpt; ++i) {
    if constexpr (sizeof(T) == 4)
      v[i] = __builtin_bit_cast(float, (uint32_t)C.w[i >> 2][i & 3]);
    else
      v[i] = i & 1 ? Pair<T>::hi(C.w[i >> 3][(i >> 1) & 3]) : Pair<T>::lo(C.w[i >> 3][(i >> 1) & 3]);
  }
}

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void lb_logprobs_kernel(const LbLogprobsArgs A) {
  __shared__ u64 buf[TOP ? kWaves : 1][kBuf];
  __shared__ u64 keys[TOP ? kWaves * 64 : 1];
  __shared__ uint32_t group[TOP ? kWaves : 1][64];
  __shared__ float kept[TOP ? kKept : 1][TOP ? kThreads : 1];
  __shared__ uint32_t work[TOP ? kWork : 1];
  __shared__ int listed, counts[kWaves];
  __shared__ Stat stat[kWaves];
  const int t = threadIdx.x, w = wave_id(), lane = t & 63;
  const long row = blockIdx.x / A.splits;
  const int split = (int)(blockIdx.x - row * A.splits);
  const long begin = (long)split * A.span;
  const long end = min((long)A.vocab, begin + A.span);
  const T* x = (const T*)A.logits + row * A.ld;
  const int64_t target = A.targets ? A.targets[row] : -1;
  const float xt = target >= begin && target < end ? (float)x[target] : 0.0f;
  Stat S = {kLow, 0.0f, 0.0f};
  float largest = -INFINITY;
  const int per = (int)((end - begin + kKept * kChunk - 1) / (kKept * kChunk));  // chunks a kept maximum
  int slot = 0, in_slot = 0;
  auto take = [&](const Chunk<T>& chunk) __attribute__((always_inline)) {
    float v[kEpt];
    chunk_values(chunk, v);
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
      largest = max_nan(largest, most);
      kept[slot][t] = in_slot == 0 ? most : max_nan(kept[slot][t], most);  // this thread's alone
      if (++in_slot == per) {
        in_slot = 0;
        ++slot;
      }
    }
  };
  // whole chunks, the next one's loads (of the last: itself again) under way while
  // one is taken; then what is left
  const int whole = (int)((end - begin) / kChunk);
  Chunk<T> chunk, next;
  const T* at = x + begin;
  if (whole > 0) chunk_load_whole<T>(chunk, at, t);
  for (int j = 0; j < whole; ++j) {
    if (j + 1 < whole) at += kChunk;
    chunk_load_whole<T>(next, at, t);
    __builtin_amdgcn_sched_barrier(0);
    take(chunk);
    chunk = next;
  }
  if (begin + (long)whole * kChunk < end) {
    chunk_load<T>(chunk, x, begin + (long)whole * kChunk, end, t);
    take(chunk);
  }
  S = wave_join(S);
  if (lane == 0) stat[w] = S;
  int count = 0;
  if constexpr (TOP) {
    // (a thread without a part of the row counts for nothing)
    const uint32_t mine = begin + 8 * t < end ? order_of(largest) : 0;
    group[w][lane] = mine;
    if (t == 0) listed = 0;
    __syncthreads();
    uint32_t g = group[0][lane];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) g = max(g, group[i][lane]);
    uint32_t bound;
    if (A.top == 1) {
      g = max(g, other<1>(g));
      g = max(g, other<2>(g));
      g = max(g, other<4>(g));
      g = max(g, other<8>(g));
      g = max(g, other<16>(g));
      bound = lane_of(max(g, other<32>(g)), 0);
    } else {
      bound = lane_of(sort64(g, lane), A.top - 1);
    }
    const float floor = bound ? value_of(bound) : NAN;
    Tops P = {0, 0, 0};
    const bool any = mine && mine >= bound;
    const int slots = (int)((end - begin + (long)per * kChunk - 1) / ((long)per * kChunk));
    if (__ballot(any) != 0) {
      u64 hit[kKept];
      int hits = 0, at = 0;
#pragma unroll
      for (int j = 0; j < kKept; ++j) {
        hit[j] = __ballot(any && j < slots && !(kept[j][t] < floor));
        hits += __popcll(hit[j]);
      }
      if (lane == 0) at = atomicAdd(&listed, hits);
      at = lane_of((uint32_t)at, 0);
#pragma unroll
      for (int j = 0; j < kKept; ++j) {
        const int p = at + __popcll(hit[j] & ((1ull << lane) - 1));
        if ((hit[j] >> lane & 1) && p < kWork) work[p] = (uint32_t)j << 16 | t;
        at += __popcll(hit[j]);
      }
    }
    __syncthreads();
    const int entries = listed;
    // a lane an entry; with more entries than the list takes (many equal
    // logits) every thread looks through its own
    const bool by_list = entries <= kWork;
    const int entry = 64 * w + lane;
    const uint32_t what = by_list ? (entry < entries ? work[entry] : 0) : t;
    const int from = what & 0xFFFF;
    const long first_c = begin + (long)(what >> 16) * per * kChunk;
    const long last_c = by_list ? first_c + (long)per * kChunk : end;
    const bool mine_too = by_list ? entry < entries : any;
    if (__ballot(mine_too) != 0) {
      const int rounds = by_list ? per : slots * per;
      for (int i = 0; i < rounds; ++i) {
        const long c = first_c + (long)i * kChunk;
        const long stop = mine_too && c < last_c ? end : c;
        const long k0 = c + 8 * from, k1 = k0 + 8 * kThreads;
        const long left0 = stop - k0, left1 = stop - k1;
        const int n0 = left0 >= 8 ? 8 : left0 > 0 ? (int)left0 : 0, n1 = left1 >= 8 ? 8 : left1 > 0 ? (int)left1 : 0;
        const int valid = n1 > 0 ? 8 + n1 : n0;  // the first eight are whole where the second have any
        float v[kEpt];
        Chunk<T> part;
        chunk_load<T>(part, x, c, stop, from);
        chunk_values(part, v);
        tops_chunk(P, buf[w], A.top, lane, v, valid, floor,
                   [&](int i) { return (uint32_t)(i < 8 ? k0 + i : k1 + i - 8); });
      }
    }
    // a wave that merged before brings the `top` first of its list, one that did not what it collected
    const u64 first = lane_of(P.list, 0);
    if (first && P.pending > 0) tops_flush(P, buf[w], A.top, lane, P.pending);
    const int mine_n = first ? A.top : P.pending;
    if (lane == 0) counts[w] = mine_n;
    __syncthreads();
    int at = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      at += i < w ? counts[i] : 0;
      count += counts[i];
    }
    if (lane < mine_n) keys[at + lane] = first ? P.list : buf[w][lane];
  }
  __syncthreads();
  u64 list = 0;
  if constexpr (TOP) list = block_top(keys, count, reinterpret_cast<u64(*)[64]>(&buf[0][0]), w, lane);
  if (w != 0) return;
  S = lane < kWaves ? stat[lane] : Stat{kLow, 0.0f, 0.0f};
  S = join_lane<1>(S);
  S = join_lane<2>(S);
  S.m = __builtin_bit_cast(float, lane_of(__builtin_bit_cast(uint32_t, S.m), 0));
  S.s = __builtin_bit_cast(float, lane_of(__builtin_bit_cast(uint32_t, S.s), 0));
  S.e = __builtin_bit_cast(float, lane_of(__builtin_bit_cast(uint32_t, S.e), 0));
  if (A.splits == 1) {
    if (lane == 0) write_row(A, row, S, xt, target);
    if constexpr (TOP) write_top(A, row, S, list, lane);
  } else {
    if (lane == 0) reinterpret_cast<Part*>(A.ws)[blockIdx.x] = Part{S, xt};
    if constexpr (TOP)
      if (lane < A.top)
        reinterpret_cast<u64*>((char*)A.ws + part_keys_at(A.rows * A.splits))[(long)blockIdx.x * A.top + lane] = list;
  }
}

// Joins the parts of a row.
__global__ __launch_bounds__(kThreads) void lb_logprobs_join_kernel(const LbLogprobsArgs A) {
  __shared__ u64 room[kWaves][64];
  const int w = wave_id(), lane = threadIdx.x & 63;
  const long row = blockIdx.x;
  const int64_t target = A.targets ? A.targets[row] : -1;
  const Part* parts = reinterpret_cast<const Part*>(A.ws) + row * A.splits;
  Stat S = {kLow, 0.0f, 0.0f};
  float xt = 0.0f;
  for (int i = lane; i < A.splits; i += 64) {
    const Part p = parts[i];
    S = join(S, p.s);
    if (target >= (long)i * A.span && target < (long)(i + 1) * A.span) xt = p.xt;
  }
  u64 list = 0;
  if (A.top > 0) {
    const u64* keys = reinterpret_cast<const u64*>((const char*)A.ws + part_keys_at(A.rows * A.splits));
    list = block_top(keys + row * A.splits * A.top, A.splits * A.top, room, w, lane);
  }
  if (w != 0) return;
  S = wave_join(S);
  const u64 owner = __ballot(xt != 0.0f);  // at most one lane (none where the logit is 0)
  if (owner) xt = __builtin_bit_cast(float, lane_of(__builtin_bit_cast(uint32_t, xt), __builtin_ctzll(owner)));
  if (A.top > 0) write_top(A, row, S, list, lane);
  if (lane == 0) write_row(A, row, S, xt, target);
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
  if (a.splits > 1) hipLaunchKernelGGL(lb_logprobs_join_kernel, dim3((unsigned)a.rows), dim3(kThreads), 0, stream, a);
}

template <typename T>
void launch_bwd(const LbLogprobsBwdArgs& a, hipStream_t stream) {
  const int spans = (a.vocab + kBwdSpan - 1) / kBwdSpan;
  hipLaunchKernelGGL((lb_logprobs_bwd_kernel<T>), dim3((unsigned)(a.rows * spans)), dim3(kThreads), 0, stream, a, spans);
}

}  // namespace

// Workgroups a row.  A row of up to 16 chunks is one workgroup's: splitting it
// saves 3 to 4 us on the card (17 x 50257 fp32 with 4 alternatives: 13.3 us
// whole, 10.3 in 8 parts; 128 x 32000 fp16: 10.8 whole, 12.1 in 2), which the
// second launch and its workspace cost on the host.  A longer one is split
// into parts of two chunks at least while the card has fewer than 512
// workgroups (1 x 128256 bf16 with 5 alternatives: 26.8 us whole, 10.9 in 8;
// 61 x 100003 with 20: 23.9 and 14.4; 512 x 128256: 37.8, and 35.5 in 2).
int lb_logprobs_splits(int64_t rows, int64_t vocab, int* span) {
  const int64_t chunks = (vocab + kChunk - 1) / kChunk;
  int64_t splits = rows > 0 && chunks > 16 ? 512 / rows : 1;
  if (splits > (chunks + 1) / 2) splits = (chunks + 1) / 2;
  if (splits < 1) splits = 1;
  const int64_t per = (chunks + splits - 1) / splits;
  if (per >= chunks) {
    *span = (int)((vocab + 7) / 8 * 8);
    return 1;
  }
  *span = (int)(per * kChunk);
  return (int)((chunks + per - 1) / per);
}

size_t lb_logprobs_partial_bytes(int64_t rows, int splits, int top) {
  return splits > 1 ? part_keys_at(rows * splits) + (size_t)rows * splits * top * sizeof(u64) : 0;
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
