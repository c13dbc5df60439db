// Attention over a paged cache, of single tokens, prompts and trees of drafted tokens:
//     out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q k_j - m)
// over the keys that a row sees, in one pass over keys and values: m is a maximum so
// far, and sum and output are scaled down where it grows.
//
// The rows of a key head's group (tokens x heads that share it) are the columns of the
// matrix steps, the keys their rows: S^T = K Q^T.  A lane then holds a few keys of one row, so
// the row's maximum takes moves between few lanes, and what it holds after the exponential is its
// operand of O^T = V^T P^T as it stands, with no move at all: which key a step's k-th place stands
// for is free as long as both operands agree.  V^T is read from LDS through the transposing
// read.
//
// Work is spread by the keys that there are: span_of all sequences gives the keys a workgroup takes, so
// that about `target` workgroups share them, whatever the lengths; a sequence's parts
// are joined by a second kernel.  All of that is computed on the device, so that a captured call
// serves any lengths.
#include <type_traits>

#include "attn_common.h"

using namespace lbh;

namespace {

typedef f16 h8 __attribute__((ext_vector_type(8)));
typedef bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kMinSpan = 256;   // keys a workgroup takes at least, where a sequence has them
constexpr float kSlack = 8.0f;  // log2: how far a maximum may grow before the sums are scaled down

template <typename T>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (__is_same(T, f16))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}

// Of 16 lanes' 8 bytes each, four rows of 16 elements: lane i gets column i % 16, four rows.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* lds) {
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)lds);
  return __builtin_bit_cast(u32x2, v);
}

// Whether a word of two elements has a NaN or an infinity, and the word without them.
template <typename T>
__device__ __forceinline__ bool odd_word(uint32_t w) {
  constexpr uint32_t m = __is_same(T, f16) ? 0x7C00u : 0x7F80u;
  return (w & m) == m || (w >> 16 & m) == m;
}
template <typename T>
__device__ __forceinline__ uint32_t even_word(uint32_t w) {
  constexpr uint32_t m = __is_same(T, f16) ? 0x7C00u : 0x7F80u;
  return ((w & m) == m ? 0u : w & 0xFFFFu) | ((w >> 16 & m) == m ? 0u : w & 0xFFFF0000u);
}

// ------------------------------------------------------------------- who does what

// A workgroup's place: of sequence `seq` the block of rows and the part of the keys.
struct Place {
  int seq;        // -1: none
  Span s;
  int blocks;     // blocks of rows of the sequence
  int parts;      // parts of its keys
  int span;       // keys a part
  int local;      // of the sequence's blocks x parts
  long slot;      // of its results, where there are several parts
};

// Wave sums over 64 lanes of what each lane has, and what the lanes before it have.
__device__ __forceinline__ int scan64(int v, int* total) {
  const int lane = threadIdx.x & 63;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(s, d);
    s += lane >= d ? o : 0;
  }
  *total = __builtin_amdgcn_readlane(s, 63);
  return s - v;
}

struct Share {
  int span, blocks, parts;
  Span s;
};
__device__ __forceinline__ int blocks_of(const Span& s, int group, int rows) { return (s.rows * group + rows - 1) / rows; }
__device__ __forceinline__ int parts_of(int keys, int span) { return max(1, (keys + span - 1) / span); }

// The keys a part has.  The sum is in floating point, in one order everywhere: every
// workgroup of the call, and the join, gets the same.
template <int STEP>
__device__ __forceinline__ int span_for(const LbAttnArgs& A, int rows) {
  const int lane = threadIdx.x & 63;
  float units = 0.0f;
  for (int i = lane; i < A.pages.seqs; i += 64) {
    const Span s = span_of(A.pages, i, (int)A.tokens);
    units += (float)s.keys * (float)blocks_of(s, A.group, rows);
  }
  units = wave_sum(units) * (float)A.kv_heads / (float)A.target;
  const int want = max(kMinSpan, units < 1e9f ? (int)units + 1 : 1 << 30);
  return __builtin_amdgcn_readfirstlane((want + STEP - 1) / STEP * STEP);
}

// The place of item `item` (BY_ROW false), or of the sequence `item` (BY_ROW true: local is 0).
template <int STEP, bool BY_ROW>
__device__ __forceinline__ Place place_of(const LbAttnArgs& A, int rows, int item) {
  const int lane = threadIdx.x & 63;
  Place p;
  p.seq = -1;
  p.span = span_for<STEP>(A, rows);
  int items = 0, slots = 0;
  for (int from = 0; from < A.pages.seqs; from += 64) {
    const int i = from + lane;
    const Span s = span_of(A.pages, min(i, A.pages.seqs - 1), (int)A.tokens);
    const int blocks = i < A.pages.seqs ? blocks_of(s, A.group, rows) : 0;
    const int parts = parts_of(s.keys, p.span);
    int all, all_slots;
    const int before = items + scan64(blocks * parts, &all);
    const int slots_before = slots + scan64(parts > 1 ? blocks * parts : 0, &all_slots);
    const bool mine = BY_ROW ? i == item : blocks > 0 && item >= before && item < before + blocks * parts;
    const uint64_t b = __ballot(mine);
    if (b) {
      const int l = __builtin_ctzll(b);
      p.seq = from + l;
      p.s.start = __builtin_amdgcn_readlane(s.start, l);
      p.s.rows = __builtin_amdgcn_readlane(s.rows, l);
      p.s.keys = __builtin_amdgcn_readlane(s.keys, l);
      p.s.base = __builtin_amdgcn_readlane(s.base, l);
      p.blocks = __builtin_amdgcn_readlane(blocks, l);
      p.parts = __builtin_amdgcn_readlane(parts, l);
      p.local = BY_ROW ? 0 : item - __builtin_amdgcn_readlane(before, l);
      p.slot = __builtin_amdgcn_readlane(slots_before, l) + p.local;
      return p;
    }
    items += all;
    slots += all_slots;
  }
  return p;
}

// Keys that the rows of a block see, all of them together and each of them: those below `most`,
// and below `full`.
struct Sight {
  int most, full;
};
__device__ __forceinline__ Sight sight_of(const LbAttnArgs& A, const Span& s, int first_row, int rows) {
  const int last = min(first_row + rows, s.rows * A.group) - 1;
  Sight v;
  if (A.tree) {
    v.most = s.keys;
    v.full = s.base;
  } else {
    v.most = min(s.keys, s.base + last / A.group + 1);
    v.full = s.base + first_row / A.group + 1;
  }
  v.most = max(v.most, 0);
  v.full = max(min(v.full, v.most), 0);
  return v;
}

// Four channels of a row's result: scaled by the sum, or, of a part, as they are.
template <typename T>
__device__ __forceinline__ void store_result(const LbAttnArgs& A, const Span& s, int kv_head, int row, int d, f32x4 o,
                                             float m, float l) {
  const int t = row / A.group, h = kv_head * A.group + row - t * A.group;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (d < A.dim) {
    T* out = (T*)A.out + (s.start + t) * A.ot + h * A.oh + d;
    u32x2 w;
    w[0] = Pair<T>::pack(l == 0.0f ? 0.0f : o[0] * inv, l == 0.0f ? 0.0f : o[1] * inv);
    w[1] = Pair<T>::pack(l == 0.0f ? 0.0f : o[2] * inv, l == 0.0f ? 0.0f : o[3] * inv);
    store_any(out, w);
  }
  if (d == 0 && A.lse) A.lse[(long)(s.start + t) * A.heads + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------------ few rows
// 16 NT rows a workgroup; its W waves have the same rows and take turns at steps of 32 keys, each
// with its own stages in LDS, filled by direct loads: the next step's keys are under way
// from the products with this one's on, its values from their products on.  No wave waits for another until the
// end, when the waves' sums are joined in LDS.  Bytes bound it.
//
// A stage holds 32 rows of DP channels.  16-byte piece c of row r lies at place c ^ swizzle(r), so that
// the 16 rows of a read, and the transposing read's 16 rows x 32 bytes, fall on all banks.
template <int DP>
__device__ __forceinline__ int swizzle(int row) {
  return DP == 64 ? (row >> 1) & 7 : row & 15;
}

template <typename T, int DP, int NT, int W>
__global__ __launch_bounds__(64 * W) void lb_attn_stream_kernel(const LbAttnArgs A) {
  constexpr int kRowBytes = 2 * DP, kPieces = DP / 8, kStage = 32 * kRowBytes;
  constexpr int kPer = 1024 / kRowBytes;   // keys of one load of the wave
  constexpr int kLoads = 32 / kPer;
  constexpr int kRows = 16 * NT;
  __shared__ __attribute__((aligned(1024))) uint8_t k_stages[W][kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t v_stages[W][kStage];
  __shared__ float2 ml[W][16];
  const int w = wave_id(), lane = threadIdx.x & 63;
  const int r16 = lane & 15, g = lane >> 4;
  const int kv_head = blockIdx.x % A.kv_heads;
  const Place p = place_of<32 * W, false>(A, kRows, blockIdx.x / A.kv_heads);
  if (p.seq < 0) return;  // the whole workgroup: all waves computed the same
  // causal rows: the last block, which sees the most, first
  const int block = p.blocks - 1 - p.local / p.parts, part = p.local % p.parts;
  const int first_row = block * kRows, all_rows = p.s.rows * A.group;
  const Sight sight = sight_of(A, p.s, first_row, kRows);
  const int parts = parts_of(sight.most, p.span);
  if (part >= parts) return;
  const int from = part * p.span, to = min(from + p.span, sight.most);

  const LbPages& P = A.pages;
  const char* const k_head = P.k + kv_head * P.head;
  const char* const v_head = P.v + kv_head * P.head;
  uint8_t* const ks = k_stages[w];
  uint8_t* const vs = v_stages[w];
  const bool padded = A.dim < DP;
  if (padded) {  // pieces that no load fills
    for (int i = lane; i < kStage / 16; i += 64) {
      *(u32x4*)(ks + 16 * i) = u32x4{0, 0, 0, 0};
      *(u32x4*)(vs + 16 * i) = u32x4{0, 0, 0, 0};
    }
    __syncthreads();
  }

  // the rows' queries, operands of S^T = K Q^T: row r16 of a tile, channels 32 s + 8 g + (0..7)
  u32x4 q[NT][DP / 32];
  int sees[NT];       // keys of the row's sight (without a tree)
  uint64_t word[NT];  // its word of the tree
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = first_row + 16 * n + r16;
    const bool in = row < all_rows;
    const int t = in ? row / A.group : 0, h = kv_head * A.group + (in ? row - t * A.group : 0);
    const T* src = (const T*)A.q + (p.s.start + t) * A.qt + h * A.qh;
#pragma unroll
    for (int s = 0; s < DP / 32; ++s) {
      const int d = 32 * s + 8 * g;
      q[n][s] = in && d < A.dim ? load_any<u32x4>(src + d) : u32x4{0, 0, 0, 0};
    }
    word[n] = A.tree && in ? (uint64_t)A.tree[p.s.start + t] : 0;
    sees[n] = in ? A.tree ? sight.most : min(sight.most, p.s.base + t + 1) : 0;
  }
  // the keys of a step of 32 that row n sees, a bit each
  auto below = [](int n) __attribute__((always_inline)) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
  auto seen = [&](int n, int key, int good) __attribute__((always_inline)) {
    uint32_t v = below(sees[n] - key);
    if (A.tree) {
      const int before = p.s.base - key;  // keys of the step before the rows' own
      const uint32_t drafted = before >= 32 ? 0u : before >= 0 ? (uint32_t)(word[n] << before)
                               : before > -64 ? (uint32_t)(word[n] >> -before) : 0u;
      v &= below(before) | drafted;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v &= good >> i & 1 ? ~0u : ~(0xFFu << (8 * i));
    return v;
  };

  // pages of a step's keys, by eights, and which of them are pages (a bit each)
  struct Pages {
    int id[4];
    int good;
  };
  const int mask = (1 << P.shift) - 1;
  typedef const __attribute__((address_space(4))) int32_t* Table;  // read by the scalar unit: not counted with the loads
  const Table table = (Table)(uintptr_t)(P.table + p.seq * P.table_stride);
  auto lookup = [&](int key) __attribute__((always_inline)) {
    Pages t;
#pragma unroll
    for (int i = 0; i < 4; ++i) t.id[i] = table[min((key + 8 * i) >> P.shift, P.columns - 1)];
    t.good = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) t.good |= ((uint32_t)t.id[i] < (uint32_t)P.pages ? 1 : 0) << i;
    return t;
  };
  const int load_row = lane / kPieces, load_piece = lane % kPieces;
  const int lane_at = load_row * (int)P.slot;
  // a step of keys or values into its stage; `whole`: every key is there
  auto issue = [&](const char* head, uint8_t* stage, int key, const Pages& t, bool whole) __attribute__((always_inline)) {
    auto direct = [&](auto check) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const char* const src = head + t.id[kPer * i / 8] * P.page + ((key + kPer * i) & mask) * P.slot;
        const int piece = load_piece ^ swizzle<DP>(kPer * i + load_row);
        if (!decltype(check)::value || 8 * piece < A.dim)
          __builtin_amdgcn_global_load_lds(src + (uint32_t)(lane_at + 16 * piece),
                                           (__attribute__((address_space(3))) void*)(stage + 1024 * i), 16, 0, 0);
      }
    };
    if (whole && !padded) {
      direct(std::false_type());
    } else if (whole) {
      direct(std::true_type());
    } else {
#pragma unroll 1
      for (int i = 0; i < kLoads; ++i) {
        const int row = kPer * i + load_row, piece = load_piece ^ swizzle<DP>(row), eight = kPer * i / 8;
        const int page = eight == 0 ? t.id[0] : eight == 1 ? t.id[1] : eight == 2 ? t.id[2] : t.id[3];
        const char* const src = head + page * P.page + ((key + kPer * i) & mask) * P.slot + lane_at + 16 * piece;
        const bool in = key + row < sight.most && (t.good >> eight & 1) && 8 * piece < A.dim;
        *(u32x4*)(stage + 1024 * i + 16 * lane) = in ? *(const u32x4*)src : u32x4{0, 0, 0, 0};
      }
    }
  };
  auto is_whole = [&](int key, const Pages& t) __attribute__((always_inline)) {
    return key + 32 <= sight.most && t.good == 15;
  };
  // this wave's loads have landed but for the last `kLeft`, and its LDS reads have come back
  auto landed = [&](bool more) __attribute__((always_inline)) {
    if (more)
      __builtin_amdgcn_s_waitcnt((kLoads & 15) | ((kLoads >> 4) << 14) | (7 << 4));
    else
      __builtin_amdgcn_s_waitcnt((7 << 4));
    __asm__ volatile("" ::: "memory");
  };
  auto reads_done = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __asm__ volatile("" ::: "memory");
  };

  f32x4 o[NT][DP / 16];
  float m[NT], l[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) o[n][d] = f32x4{0, 0, 0, 0};
  }
  int key = from + 32 * w;
  const uint8_t* const k_at = ks + r16 * kRowBytes + 16 * (g ^ swizzle<DP>(r16));
  const int v_row = 4 * g + (r16 >> 2);
  const uint8_t* const v_at = vs + v_row * kRowBytes + 16 * (((lane & 3) >> 1) ^ swizzle<DP>(v_row)) + 8 * (lane & 1);
  if (key < to) {
    Pages here = lookup(key);
    bool whole = is_whole(key, here);
    issue(k_head, ks, key, here, whole);
    issue(v_head, vs, key, here, whole);
    // the queries and what the tree says have come back: the loop waits for no loads but its own
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int s = 0; s < DP / 32; ++s) __asm__ volatile("" : "+v"(q[n][s]));
      __asm__ volatile("" : "+v"(word[n]));
    }
    for (; key < to; key += 32 * W) {
      const bool more = key + 32 * W < to;
      const Pages next = lookup(more ? key + 32 * W : key);
      const bool next_whole = is_whole(key + 32 * W, next);
      landed(true);  // the keys; the values may be under way
      f32x4 st[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) st[n][0] = st[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < DP / 32; ++s) {
        const uint8_t* const at = ks + (((int)(k_at - ks)) ^ (64 * s));
        const u32x4 k0 = *(const u32x4*)at, k1 = *(const u32x4*)(at + 16 * kRowBytes);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          st[n][0] = mfma16<T>(k0, q[n][s], st[n][0]);
          st[n][1] = mfma16<T>(k1, q[n][s], st[n][1]);
        }
      }
      reads_done();
      if (more) issue(k_head, ks, key + 32 * W, next, next_whole);
      const bool masked = key + 32 > sight.full || !whole;
      u32x4 pr[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = st[n][i >> 2][i & 3] * A.scale;
        if (masked) {
          const uint32_t v = seen(n, key, here.good) >> (4 * g);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(v >> (16 * (i >> 2) + (i & 3)) & 1)) x[i] = -INFINITY;
        }
        float most = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) most = fmaxf(most, x[i]);
        most = fmaxf(most, lane_xor<16>(most));
        most = fmaxf(most, lane_xor<32>(most));
        if (__ballot(most > m[n] + kSlack)) {
          const float up = fmaxf(m[n], most);
          const float a = m[n] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[n] - up);
          m[n] = up;
          l[n] *= a;
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) o[n][d] *= a;
        }
        const float at = m[n] == -INFINITY ? 0.0f : m[n];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = __builtin_amdgcn_exp2f(x[i] - at);
          l[n] += x[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[n][i] = Pair<T>::pack(x[2 * i], x[2 * i + 1]);
      }
      landed(more);  // the values; the next keys may be under way
      if (masked) {
        // a NaN or an infinity among the values of a key that some rows do not see: its product with their 0
        // would be one too.  It is added to the rows that see it, and taken out of the stage.
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const u32x4 v = *(const u32x4*)(vs + 1024 * i + 16 * lane);
          const uint64_t b = __ballot(odd_word<T>(v[0]) || odd_word<T>(v[1]) || odd_word<T>(v[2]) || odd_word<T>(v[3]));
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (b >> (j * kPieces) & (kPieces == 64 ? ~0ull : (1ull << kPieces) - 1)) odd |= 1u << (kPer * i + j);
        }
        if (odd) {
          for (uint32_t left = odd; left; left &= left - 1) {
            const int row = __builtin_ctz(left);
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
              const u32x2 v = *(const u32x2*)(vs + row * kRowBytes + 16 * ((2 * d + (g >> 1)) ^ swizzle<DP>(row)) + 8 * (g & 1));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t e16 = v[e >> 1] >> (16 * (e & 1)) & 0xFFFFu;
                const float f = Pair<T>::lo(e16);
                if (!odd_word<T>(e16)) continue;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  if (seen(n, key, here.good) >> row & 1) o[n][d][e] += f;
              }
            }
          }
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            u32x4 v = *(const u32x4*)(vs + 1024 * i + 16 * lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = even_word<T>(v[e]);
            *(u32x4*)(vs + 1024 * i + 16 * lane) = v;
          }
        }
      }
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) {
        const uint8_t* const at = vs + (((int)(v_at - vs)) ^ (32 * d));
        const u32x2 v0 = read_transposed(at), v1 = read_transposed(at + 16 * kRowBytes);
        const u32x4 v = {v0[0], v0[1], v1[0], v1[1]};
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][d] = mfma16<T>(v, pr[n], o[n][d]);
      }
      reads_done();
      if (more) issue(v_head, vs, key + 32 * W, next, next_whole);
      here = next;
      whole = next_whole;
    }
  }

  // the waves' results joined, 16 rows at a time; four channels d of row r lie at place (d / 4) ^ r
  f32x4* const join = (f32x4*)&k_stages[0][0];
  static_assert(sizeof(k_stages) == W * 16 * DP * 4, "the joined rows fit the keys' stages");
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] += lane_xor<16>(l[n]);
    l[n] += lane_xor<32>(l[n]);
    __syncthreads();  // every wave has read its stages, or the rows before
    if (g == 0) ml[w][r16] = float2{m[n], l[n]};
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) join[(w * 16 + r16) * (DP / 4) + ((4 * d + g) ^ r16)] = o[n][d];
    __syncthreads();
    for (int i = threadIdx.x; i < 4 * DP; i += 64 * W) {
      const int r = i / (DP / 4), c = i % (DP / 4);
      const int row = first_row + 16 * n + r;
      if (row >= all_rows) break;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < W; ++j) top = fmaxf(top, ml[j][r].x);
      f32x4 sum = {0, 0, 0, 0};
      float total = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float2 v = ml[j][r];
        const float a = v.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(v.x - top);
        // a wave without a key of this row has no maximum; with a NaN for its only score, a NaN sum
        total += v.x == -INFINITY ? v.y : a * v.y;
        sum += a * join[(j * 16 + r) * (DP / 4) + (c ^ r)];
      }
      if (parts == 1) {
        store_result<T>(A, p.s, kv_head, row, 4 * c, sum, top, total);
      } else if (4 * c < A.dim) {
        const long at = (p.slot * A.kv_heads + kv_head) * kRows + row - first_row;
        *(f32x4*)(A.partial + at * A.dim + 4 * c) = sum;
        if (c == 0) ((float2*)(A.partial + A.slots * A.kv_heads * kRows * A.dim))[at] = float2{top, total};
      }
    }
  }
}

// ------------------------------------------------------------------------- the join
// A wave a token and key head; the parts' maxima and sums first, then four channels a lane.
template <typename T, int STEP>
__global__ __launch_bounds__(256) void lb_attn_join_kernel(const LbAttnArgs A, int rows) {
  const int w = wave_id(), lane = threadIdx.x & 63;
  const long item = blockIdx.x * 4l + w;
  const int token = (int)(item / A.kv_heads), kv_head = (int)(item - (long)token * A.kv_heads);
  if (token >= A.tokens) return;
  const int seq = sequence_of(A.pages, token);
  if (seq < 0) return;
  const Place p = place_of<STEP, true>(A, rows, seq);
  const int t = token - p.s.start;
  if (t >= p.s.rows) return;
  const float2* const ml = (const float2*)(A.partial + A.slots * A.kv_heads * rows * A.dim);
  for (int row = t * A.group; row < (t + 1) * A.group; ++row) {
    const int block = row / rows;
    const int parts = parts_of(sight_of(A, p.s, block * rows, rows).most, p.span);
    if (parts == 1) continue;
    const long slot = p.slot + (long)(p.blocks - 1 - block) * p.parts;
    auto at = [&](int j) __attribute__((always_inline)) { return ((slot + j) * A.kv_heads + kv_head) * rows + row % rows; };
    float top = -INFINITY, total = 0.0f;
    for (int j = 0; j < parts; ++j) top = fmaxf(top, ml[at(j)].x);
    f32x4 sum = {0, 0, 0, 0};
    for (int j = 0; j < parts; ++j) {
      const float2 v = ml[at(j)];
      const float a = v.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(v.x - top);
      total += v.x == -INFINITY ? v.y : a * v.y;
      if (4 * lane < A.dim) sum += a * *(const f32x4*)(A.partial + at(j) * A.dim + 4 * lane);
    }
    store_result<T>(A, p.s, kv_head, row, 4 * lane, sum, top, total);
  }
}

template <typename T, int DP, int NT, int W>
void launch_stream(const LbAttnArgs& a, const LbAttnPlan& plan, hipStream_t stream) {
  hipLaunchKernelGGL((lb_attn_stream_kernel<T, DP, NT, W>), dim3((unsigned)plan.grid), dim3(64 * W), 0, stream, a);
  const long waves = a.tokens * a.kv_heads;
  hipLaunchKernelGGL((lb_attn_join_kernel<T, 32 * W>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a,
                     plan.rows);
}

template <typename T, int DP, int W>
void launch_rows(const LbAttnArgs& a, const LbAttnPlan& plan, hipStream_t stream) {
  if (plan.rows == 16)
    launch_stream<T, DP, 1, W>(a, plan, stream);
  else if (DP == 256 || plan.rows == 32)
    launch_stream<T, DP, 2, W>(a, plan, stream);
  else if constexpr (DP < 256)
    launch_stream<T, DP, 4, W>(a, plan, stream);
}

template <typename T>
void launch_attn(const LbAttnArgs& a, const LbAttnPlan& plan, hipStream_t stream) {
  if (a.dim <= 64)
    launch_rows<T, 64, 4>(a, plan, stream);
  else if (a.dim <= 128)
    launch_rows<T, 128, 4>(a, plan, stream);
  else
    launch_rows<T, 256, 2>(a, plan, stream);
}

}  // namespace

// Rows of a workgroup by the rows that a sequence has on average.  A sequence of n rows has at most
// n group / rows + 1 blocks, and `target` / kv_heads parts are added over all of them; a
// sequence with several parts has at most twice its share of them.
LbAttnPlan lb_attn_plan(int64_t tokens, int seqs, int heads, int kv_heads, int dim) {
  LbAttnPlan p;
  const int64_t group = heads / kv_heads, mean = (tokens * group + seqs - 1) / seqs;
  p.rows = mean <= 16 ? 16 : mean <= 32 || dim > 128 ? 32 : 64;
  p.target = 1024;
  const int64_t share = (p.target + kv_heads - 1) / kv_heads;
  p.slots = 2 * share + 8;
  p.grid = (share + tokens * group / p.rows + seqs + 8) * kv_heads;
  return p;
}

size_t lb_attn_workspace(const LbAttnPlan& plan, int kv_heads, int dim) {
  return (size_t)plan.slots * kv_heads * plan.rows * (dim + 2) * sizeof(float);
}

hipError_t lb_launch_attn(const LbAttnArgs& a, const LbAttnPlan& plan, int dtype, hipStream_t stream) {
  if (dtype == 1)
    launch_attn<f16>(a, plan, stream);
  else
    launch_attn<bf16>(a, plan, stream);
  return hipGetLastError();
}
