// Attention over a paged cache, of single tokens, prompts and trees of drafted tokens:
//     out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q k_j - m)
// over the keys that a row sees, in one pass over keys and values: m is a maximum so
// far, and sum and output are scaled down where it grows.
//
// The rows of a key head's group (tokens x heads that share it) are the columns of the
// matrix steps, the keys their rows: S^T = K Q^T.  A lane then holds a few keys of one row, so
// the row's maximum takes moves between few lanes, and what it holds after the exponential is its
// operand of O^T = V^T P^T as it stands: which key a step's k-th place stands for is free as long as
// both operands agree.  V^T is read from LDS through the transposing read.
// That operand is rounded to the values' type, since the matrix units take both in one.  Of few rows, what the rounding
// leaves is multiplied too.  Of many rows, whose matrix steps bound them, it is lost: half a step of each probability,
// relative, in fp16 up to 2^-32 of the row's largest one; their sum is of the unrounded ones, in fp32 like all else.
//
// Work is spread by the keys that there are, whatever the lengths: from all sequences' keys follows how many a
// workgroup takes, so that those that run at once have as many each; a sequence's parts are joined by a second
// kernel.  All of that is computed on the device, so that a captured call serves any lengths.
#include <algorithm>
#include <type_traits>

#include "attn_common.h"
#include "attn_split.h"

using namespace lbh;

namespace {

typedef f16 h8 __attribute__((ext_vector_type(8)));
typedef bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kPartKeys = 512;  // what beginning, writing and joining a part of many rows costs, in keys
// The exponent that probabilities are relative to, in log2: kAhead below a row's largest score when it was last raised, and
// it is raised when that has grown by more than kSlack since.  bf16 has fp32's range.  In fp16 a probability is at most
// 2^15, half of what the type holds, and what is lost below its smallest step is 2^-32 of the row's largest one, of few rows
// (whose matrix steps wait for memory) 2^-38.  (Of many rows, 12 ahead and 3 of slack: 2000 tokens on 2000 of 16 / 4 heads of
// 256 165 -> 182 us, 4000 on 4100 of 64 / 8 heads of 128 814 -> 820.)
template <typename T, bool MANY>
constexpr float kAhead = __is_same(T, f16) ? MANY ? 7.0f : 14.0f : 0.0f;
template <typename T, bool MANY>
constexpr float kSlack = __is_same(T, f16) ? 15.0f - kAhead<T, MANY> : 8.0f;
// Whether a row's largest score asks for it, and the one after that: not below the score by more than the two together
// (of scores beyond 2^26, where neighbours are that far apart, it is the score itself).
template <typename T, bool MANY>
__device__ __forceinline__ bool grows(float most, float m) {
  return most - m > kAhead<T, MANY> + kSlack<T, MANY>;
}
template <typename T, bool MANY>
__device__ __forceinline__ float raised(float most, float m) {
  const float up = most - kAhead<T, MANY>;
  return fmaxf(m, grows<T, MANY>(most, up) ? most : up);
}

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

// The first n of 32 bits.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// The keys of a step of 32, from `key` on, that a row sees, a bit each: of those that are there, those before `sees`,
// and, of a tree, those before the rows' own and those of its word.
__device__ __forceinline__ uint32_t seen_of(const LbAttnArgs& A, int base, int key, uint32_t there, int sees, uint64_t word) {
  uint32_t v = below(sees - key) & there;
  if (A.tree) {
    const int before = base - key;
    const uint32_t drafted = before >= 32 ? 0u : before >= 0 ? (uint32_t)(word << before)
                             : before > -64 ? (uint32_t)(word >> -before) : 0u;
    v &= below(before) | drafted;
  }
  return v;
}

// The larger of the sizes of two pairs of elements: of a NaN or an infinity, as bits, `kOdd` at least.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 size_max(u16x2 a, uint32_t w) {
  return __builtin_elementwise_max(a, __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu));
}
template <typename T>
__device__ __forceinline__ bool is_odd(u16x2 size) {
  constexpr unsigned short odd = __is_same(T, f16) ? 0x7C00 : 0x7F80;
  return size[0] >= odd || size[1] >= odd;
}

// Queries with the scale's sign, or 0 where it is 0: the scale that is left is positive, so that the largest score
// is found before it is scaled, and -infinity stays what it is.
__device__ __forceinline__ u32x4 with_sign(const LbAttnArgs& A, u32x4 q) { return (q ^ A.sign) & A.keep; }

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
  int slot;       // of its results, where there are several parts
};

// What the lanes before this one have together, and all of them.
__device__ __forceinline__ int scan64(int v, int* total) {
  int s = v;
  s += __builtin_amdgcn_update_dpp(0, s, 0x111, 0xF, 0xF, false);  // one to the right in a row of 16, two, four, eight
  s += __builtin_amdgcn_update_dpp(0, s, 0x112, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x114, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x118, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x142, 0xA, 0xF, false);  // a row's last to the next row
  s += __builtin_amdgcn_update_dpp(0, s, 0x143, 0xC, 0xF, false);  // the lower half's last to the upper half
  *total = __builtin_amdgcn_readlane(s, 63);
  return s - v;
}

__device__ __forceinline__ Span read_span(const LbAttnArgs& A, int seq) {
  Span s = span_of(A.pages, min(seq, A.pages.seqs - 1), (int)A.tokens);
  if (seq >= A.pages.seqs) s.rows = 0;
  return s;
}
// Keys of a part, from the sums over all sequences of the blocks, and of the blocks' keys.
template <bool MANY>
__device__ __forceinline__ int span_of_sums(const LbAttnArgs& A, float blocks, float units, bool* whole) {
  *whole = __builtin_amdgcn_readfirstlane(is_whole<MANY>(blocks * (float)A.kv_heads, (float)A.round));
  return __builtin_amdgcn_readfirstlane(span_from<MANY>(blocks, units, A.kv_heads, A.round, A.target, A.least));
}

// The place of item `item`.  A part has the keys, in steps of STEP, that spread all sequences' keys (times their
// blocks of rows) over the workgroups that run at once, `round` of them, and no fewer than `least`; the parts of a
// sequence are as long as each other.  Parts are rounded up, at most one for each block, so that `round` less the
// blocks is what is shared out.  Where blocks are many: of few rows, they are shared out over several rounds, so
// that the last parts are short beside the whole; of many rows (MANY), whose parts cost more to join, not at all,
// and the blocks that see the most come first.  Where blocks of many rows are few, lengths of parts are compared by the
// rounds they take (2 sequences of 64 rows over 16000 keys of 64 / 8 heads of 128: 92 -> 71 us, 500 tokens on 4000 of 16 / 4
// heads of 256 104 -> 73; 3 of 200 over 20000 of 32 / 8 heads, though, 213 -> 221).  Every workgroup finds its place by
// itself, up to 64 sequences at once; of more than kFewSeqs, a kernel before this one has added them up (`groups`).
template <int STEP, bool MANY>
__device__ __forceinline__ Place place_of(const LbAttnArgs& A, int rows, int item) {
  const int lane = threadIdx.x & 63;
  const int seqs = A.pages.seqs;
  int begin = 0, end = seqs, items = 0, slots = 0, span;
  bool whole = false;
  if (A.groups) {
    // the last 64 sequences that begin at or before the item
    int first = 0, count = (seqs + 63) >> 6;
    while (count > 1) {
      const int step = (count + 63) >> 6, at = lane * step;
      const uint64_t b = __ballot(at < count && A.groups[2 + 2 * (first + min(at, count - 1))] <= item);
      const int last = b ? 63 - __builtin_clzll(b) : 0;
      first += last * step;
      count = min(step, count - last * step);
    }
    span = A.groups[0];
    items = A.groups[2 + 2 * first];
    slots = A.groups[3 + 2 * first];
    begin = 64 * first;
    end = min(begin + 64, seqs);
  }
  const Span first = read_span(A, begin + lane);
  if (!A.groups) {
    // in floating point, in one order everywhere: all workgroups get the same
    const int own_blocks = blocks_of(first.rows, A.group, rows);
    float blocks = (float)own_blocks, units = units_of(first.keys, own_blocks);
    for (int from = 64; from < seqs; from += 64) {
      const Span s = read_span(A, from + lane);
      const int b = blocks_of(s.rows, A.group, rows);
      blocks += (float)b;
      units += units_of(s.keys, b);
    }
    blocks = wave_sum(blocks);
    span = span_of_sums<MANY>(A, blocks, wave_sum(units), &whole);
  }
  if (MANY && !whole && seqs <= 64) {
    // a lane each: the longest sequence in lane + 1 parts, and the others in parts of that length
    const int longest = __builtin_amdgcn_readfirstlane((int)wave_max(first.rows > 0 ? (float)first.keys : 0.0f));
    const int even = (longest / (lane + 1) + STEP) / STEP * STEP, mine = lane ? even : 1 << 30;
    const int own_blocks = blocks_of(first.rows, A.group, rows);
    int all = 0, joined = 0;
    for (uint64_t left = __ballot(own_blocks > 0); left; left &= left - 1) {
      const int l = __builtin_ctzll(left);
      const int b = __builtin_amdgcn_readlane(own_blocks, l), parts = parts_of(__builtin_amdgcn_readlane(first.keys, l), mine);
      all += b * parts;
      joined += parts > 1 ? b * parts : 0;
    }
    const bool fits = all <= (int)(gridDim.x / A.kv_heads) && joined <= A.slots;
    const float rounds = ceilf((float)all * (float)A.kv_heads / (float)A.round);
    const float cost = lane == 0 || fits ? rounds * (float)(even + kPartKeys) : INFINITY;
    const uint64_t best = __ballot(cost == -wave_max(-cost));
    span = __builtin_amdgcn_readlane(mine, __builtin_ctzll(best | 1ull << 63));
  }
  Place p;
  p.seq = -1;
  for (int from = begin; from < end; from += 64) {
    const Span s = from > begin ? read_span(A, from + lane) : first;
    const int blocks = blocks_of(s.rows, A.group, rows);
    const int own = part_keys<STEP>(s.keys, span);
    const int parts = parts_of(s.keys, own);
    int all, all_slots;
    int before = items + scan64(blocks * parts, &all);
    const int slots_before = slots + scan64(parts > 1 ? blocks * parts : 0, &all_slots);
    uint64_t b = __ballot(item >= before && item < before + blocks * parts);
    if (MANY && whole && seqs <= 64 && item < all) {
      // by the blocks' place in their sequence, the last ones of the longest first.  Where a single round of two a compute
      // unit holds them all, its second half goes the other way round, so that each unit has as much (2048 tokens of
      // 32 / 32 heads of 128 69 -> 66 us, 4000 of 16 / 4 heads of 64 84 -> 80).
      const int half = A.round / 2 / A.kv_heads;
      int left = A.round == 512 && all * A.kv_heads <= A.round && item >= half ? all - 1 - (item - half) : item;
      int level = __builtin_amdgcn_readfirstlane((int)wave_max((float)blocks));
      uint64_t at;
      do {
        --level;
        at = __ballot(blocks > level);
        left -= __builtin_popcountll(at);
      } while (left >= 0);
      left += __builtin_popcountll(at);
      const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(at >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)at, 0));
      b = __ballot(blocks > level && rank == left);
      before = item - (blocks - 1 - level);
    }
    if (b) {
      const int l = __builtin_ctzll(b);
      p.seq = from + l;
      p.s.start = __builtin_amdgcn_readlane(s.start, l);
      p.s.rows = __builtin_amdgcn_readlane(s.rows, l);
      p.s.keys = __builtin_amdgcn_readlane(s.keys, l);
      p.s.base = __builtin_amdgcn_readlane(s.base, l);
      p.blocks = __builtin_amdgcn_readlane(blocks, l);
      p.parts = __builtin_amdgcn_readlane(parts, l);
      p.span = __builtin_amdgcn_readlane(own, l);
      p.local = item - __builtin_amdgcn_readlane(before, l);
      p.slot = __builtin_amdgcn_readlane(slots_before, l) + p.local;
      return p;
    }
    items += all;
    slots += all_slots;
  }
  return p;
}

// Of many sequences, what every workgroup would add up, once: [0] the keys of a part, [2 + 2 g] and [3 + 2 g] the items and
// the slots before the 64 sequences from 64 g on.  One workgroup; latency bounds it.  One token
// of each sequence, 64 / 8 heads of 128, bf16, without and with it: 256 over 1000 keys 215 and 211 us, 1024 906 and 782, 4096
// over 500 4780 and 1590 (5.3 TB/s).
constexpr int kFewSeqs = 128;
template <int STEP, bool MANY>
__global__ __launch_bounds__(1024) void lb_attn_groups_kernel(const LbAttnArgs A, int* __restrict__ out, int rows) {
  __shared__ float2 sums[16];
  __shared__ int2 totals[1024], waves[16];
  const int w = wave_id(), lane = threadIdx.x & 63, t = threadIdx.x;
  const int groups = (A.pages.seqs + 63) >> 6;
  float blocks = 0.0f, units = 0.0f;
  for (int g = w; g < groups; g += 16) {
    const Span s = read_span(A, 64 * g + lane);
    const int b = blocks_of(s.rows, A.group, rows);
    blocks += (float)b;
    units += units_of(s.keys, b);
  }
  blocks = wave_sum(blocks);
  units = wave_sum(units);
  if (lane == 0) sums[w] = float2{blocks, units};
  __syncthreads();
  blocks = units = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    blocks += sums[i].x;
    units += sums[i].y;
  }
  bool whole;
  const int span = span_of_sums<MANY>(A, blocks, units, &whole);
  for (int g = w; g < groups; g += 16) {
    const Span s = read_span(A, 64 * g + lane);
    const int b = blocks_of(s.rows, A.group, rows), parts = parts_of(s.keys, part_keys<STEP>(s.keys, span));
    int2 all;
    scan64(b * parts, &all.x);
    scan64(parts > 1 ? b * parts : 0, &all.y);
    if (lane == 0) totals[g] = all;
  }
  __syncthreads();
  int2 all, before = t < groups ? totals[t] : int2{0, 0};
  before.x = scan64(before.x, &all.x);
  before.y = scan64(before.y, &all.y);
  if (lane == 0) waves[w] = all;
  __syncthreads();
  for (int i = 0; i < w; ++i) {
    before.x += waves[i].x;
    before.y += waves[i].y;
  }
  if (t < groups) *(int2*)(out + 2 + 2 * t) = before;
  if (t == 0) out[0] = span;
}

// Keys that the rows of a block see, all of them together and each of them: those below `most`,
// and below `full`.
struct Sight {
  int most, full;
};
__device__ __forceinline__ Sight sight_of(const LbAttnArgs& A, const Span& s, int first_row, int rows) {
  const int last = max(min(first_row + rows, s.rows * A.group), 1) - 1;
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

// Four channels of a row's result, scaled by the sum.
template <typename T>
__device__ __forceinline__ void store_result(const LbAttnArgs& A, int token, int head, int d, f32x4 o, float m, float l) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (d < A.dim) {
    T* out = (T*)A.out + token * A.ot + head * A.oh + d;
    u32x2 w;
    w[0] = Pair<T>::pack(l == 0.0f ? 0.0f : o[0] * inv, l == 0.0f ? 0.0f : o[1] * inv);
    w[1] = Pair<T>::pack(l == 0.0f ? 0.0f : o[2] * inv, l == 0.0f ? 0.0f : o[3] * inv);
    store_any(out, w);
  }
  if (d == 0 && A.lse) A.lse[(long)token * A.heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Where the parts of a row's result lie: part j in row first + j * step of the workspace.
// One for each row of the call, written by its first part.  A key head's parts are fewer than 2^16 (see the plan's
// target), and so are the sequences.
struct Parts {
  int first;
  uint32_t count;  // of the parts, and the sequence in the upper half
};
struct Workspace {
  float* sums;    // [slots][kv_heads][rows][dim]
  float2* ml;     // [slots][kv_heads][rows]: maximum, sum
  Parts* parts;   // [tokens][heads]
};
__device__ __forceinline__ Workspace workspace_of(const LbAttnArgs& A, int rows) {
  const long all = A.slots * A.kv_heads * rows;
  Workspace w;
  w.sums = A.partial;
  w.ml = (float2*)(A.partial + all * A.dim);
  w.parts = (Parts*)(w.ml + all);
  return w;
}

// Four channels of row `row` of a sequence (row `in_block` of its block): the result itself, or of one of several parts.
template <typename T>
__device__ __forceinline__ void store_part(const LbAttnArgs& A, const Place& p, int kv_head, int rows, int part, int parts,
                                           int row, int in_block, int d, f32x4 o, float m, float l) {
  const int t = (uint32_t)row / (uint32_t)A.group, token = p.s.start + t, head = kv_head * A.group + row - t * A.group;
  if (parts == 1) {
    store_result<T>(A, token, head, d, o, m, l);
  }
  if (parts > 1 || d == 0) {
    const Workspace w = workspace_of(A, rows);
    const int at = (p.slot * A.kv_heads + kv_head) * rows + in_block;
    if (parts > 1 && d < A.dim) *(f32x4*)(w.sums + (long)at * A.dim + d) = o;
    if (d == 0) {
      if (parts > 1) w.ml[at] = float2{m, l};
      if (part == 0 && A.slots > 0) w.parts[(long)token * A.heads + head] = Parts{at, (uint32_t)p.seq << 16 | (uint32_t)parts};
    }
  }
}

// A stage holds rows of DP channels.  16-byte piece c of row r lies at place c ^ swizzle(r): the 16 rows of a
// read fall on all banks, and so do the four rows of a transposing read, whose pieces are two or four in
// a row: the row's last bits move them by fours.
template <int DP>
__device__ __forceinline__ int swizzle(int row) {
  if constexpr (DP == 64) return (row & 2) << 1 | (row >> 2 & 3);  // two rows of 128 bytes fill the banks
  return (row & 3) << 2 | (row >> 2 & 3);
}

// 16 bytes a lane from base + offset to LDS, 1 KB from `lds` on.  In assembly, so that the compiler does not wait for it
// before reads of other stages; the kernels wait themselves.  Nothing is loaded into registers.
__device__ __forceinline__ void load_to_lds(uint32_t lds, const void* base, uint32_t offset) {
  // scalars, whatever the compiler knows of them
  const uint64_t p = (uint64_t)(uintptr_t)base;
  const uint32_t low = __builtin_amdgcn_readfirstlane((uint32_t)p), high = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
  const uint64_t from = (uint64_t)high << 32 | low;  // (the builtin's int, or'ed as it is, would spread its sign)
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
                   "v"(offset), "s"(from)
                   : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// Values of a key that some rows see and others do not may be NaN or infinite: their product with a 0 would be one
// too.  Such values are cleared in the stage, and added at the end to the rows that see them (`odd` says that
// there are any; the sums do not change by what was cleared, and nothing that is added to them is finite).
// Clears those of the kLoads KB that this lane's wave has loaded.
template <typename T, int LOADS>
__device__ __forceinline__ bool clear_odd(uint8_t* stage) {
  const int lane = threadIdx.x & 63;
  u16x2 size = {0, 0};
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const u32x4 v = *(const u32x4*)(stage + 1024 * i + 16 * lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) size = size_max(size, v[e]);
  }
  if (__builtin_expect(__ballot(is_odd<T>(size)) == 0, 1)) return false;
#pragma unroll 1
  for (int i = 0; i < LOADS; ++i) {
    u32x4 v = *(const u32x4*)(stage + 1024 * i + 16 * lane);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = even_word<T>(v[e]);
    *(u32x4*)(stage + 1024 * i + 16 * lane) = v;
  }
  return true;
}
// 0 where a key at `p` has an infinity or a NaN, else 1.  A finite score has a probability, however small, and an infinite
// value with it is infinite; with such a key the score is none, or infinite: 0 or more times infinity, or a row without a sum.
template <typename T>
__device__ __forceinline__ float is_even(const char* p, int dim) {
  const int d = 4 * (threadIdx.x & 63);
  const u32x2 k = d < dim ? *(const u32x2*)(p + 2 * d) : u32x2{0, 0};
  return __ballot(odd_word<T>(k[0]) || odd_word<T>(k[1])) ? 0.0f : 1.0f;
}
// The four values of channels d to d + 3 of a row at `p` that are odd, 0 in the place of the others.
template <typename T>
__device__ __forceinline__ f32x4 odd_values(const char* p, int d, int dim, bool there) {
  f32x4 f = {0, 0, 0, 0};
  if (there && d < dim) {
    const u32x2 v = *(const u32x2*)(p + 2 * d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = v[e >> 1] >> (16 * (e & 1)) & 0xFFFFu;
      f[e] = odd_word<T>(w) ? Pair<T>::lo(w) : 0.0f;
    }
  }
  return f;
}

// ------------------------------------------------------------------------ few rows
// Two probabilities in two operands: cut off to the type, and what that leaves, which is at least `least`.  (Where an
// infinite value meets it, it must be neither negative nor 0.)
template <typename T>
__device__ __forceinline__ void split(float a, float b, float least, uint32_t& w, uint32_t& rest) {
  float ra, rb;
  if constexpr (__is_same(T, f16)) {
    w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
    // a mixed fma takes the halves as they are; the compiler converts them first
    __asm__("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(ra) : "v"(w), "v"(a));
    __asm__("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(rb) : "v"(w), "v"(b));
  } else {
    const uint32_t x = __builtin_bit_cast(uint32_t, a), y = __builtin_bit_cast(uint32_t, b);
    w = __builtin_amdgcn_perm(y, x, 0x07060302);  // the upper halves
    ra = a - __builtin_bit_cast(float, x & 0xFFFF0000u);
    rb = b - __builtin_bit_cast(float, y & 0xFFFF0000u);
  }
  rest = Pair<T>::pack(fmaxf(ra, least), fmaxf(rb, least));
}

// 16 NT rows a workgroup; its W waves have the same rows and take turns at steps of 32 keys, each
// with its own stages in LDS, filled by direct loads: the next step's keys are under way
// from the products with this one's on, its values from their products on.  No wave waits for another until the
// end, when the waves' sums are joined in LDS.  The matrix steps wait for memory: a second product takes what the
// rounding of the probabilities left, so that they count with twice the type's digits (0.2 us of a call of 20 in blocks of
// 16 rows, 3% in blocks of 32: 16 sequences of 9 rows over 2000 keys of 64 / 8 heads of 128 40 -> 41).  A step's keys, and
// its values, are all in registers before their products; the next values are asked for then.  Bytes bound it: 32
// sequences of one token over 1 to 8000 keys of 64 / 8 heads of 128, bf16, 113 us, 5.2 TB/s (a large copy reaches 5.1); one
// over 4000 keys of 40 heads, fp16, 18 us, of which some 5 are the way to the first keys.
template <typename T, int DP, int NT, int W>
__global__ __launch_bounds__(64 * W, DP * NT <= 256 ? 2 : 1) void lb_attn_stream_kernel(const LbAttnArgs A) {
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
  // the latter: starts that name rows twice, whose sums may wrap as well
  if (part >= parts || (parts > 1 && (uint32_t)p.slot >= (uint64_t)A.slots)) return;
  const int from = part * p.span, to = min(from + p.span, sight.most);

  const LbPages& P = A.pages;
  const char* const k_head = P.k + kv_head * P.head;
  const char* const v_head = P.v + kv_head * P.head;
  uint8_t* const ks = k_stages[w];
  uint8_t* const vs = v_stages[w];
  const uint32_t k_lds = lds_address(ks), v_lds = lds_address(vs);
  // pages of a step's keys, by eights (0 where there is none), and which of its keys are there
  struct Pages {
    int id[4];
    uint32_t there;
  };
  const int mask = (1 << P.shift) - 1;
  typedef const __attribute__((address_space(4))) int32_t* Table;  // read by the scalar unit: not counted with the loads
  const Table table = (Table)(uintptr_t)(P.table + p.seq * P.table_stride);
  auto lookup = [&](int key) __attribute__((always_inline)) {
    Pages t;
#pragma unroll
    for (int i = 0; i < 4; ++i) t.id[i] = table[min((key + 8 * i) >> P.shift, P.columns - 1)];
    t.there = below(sight.most - key);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((uint32_t)t.id[i] >= (uint32_t)P.pages) {
        t.id[i] = 0;
        t.there &= ~(0xFFu << (8 * i));
      }
    }
    return t;
  };
  int key = from + 32 * w;
  Pages here = lookup(key);
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
    const int t = in ? (uint32_t)row / (uint32_t)A.group : 0, h = kv_head * A.group + (in ? row - t * A.group : 0);
    const T* src = (const T*)A.q + (p.s.start + t) * A.qt + h * A.qh;
#pragma unroll
    for (int s = 0; s < DP / 32; ++s) {
      const int d = 32 * s + 8 * g;
      q[n][s] = in && d < A.dim ? with_sign(A, load_any<u32x4>(src + d)) : u32x4{0, 0, 0, 0};
    }
    word[n] = A.tree && in ? (uint64_t)A.tree[p.s.start + t] : 0;
    sees[n] = in ? A.tree ? sight.most : min(sight.most, p.s.base + t + 1) : 0;
  }
  auto seen = [&](int n, int key, uint32_t there) __attribute__((always_inline)) {
    return seen_of(A, p.s.base, key, there, sees[n], word[n]);
  };

  // a step of keys or values into its stage.  Memory that holds no key of the sequence is read too, but no other
  // than the cache's: what is masked, or cleared, afterwards.
  const int load_row = lane / kPieces, load_piece = lane % kPieces;
  const int lane_at = load_row * (int)P.slot;
  auto issue = [&](const char* head, uint32_t stage, int key, const Pages& t) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const char* const src = head + t.id[kPer * i / 8] * P.page + ((key + kPer * i) & mask) * P.slot;
      const int piece = load_piece ^ swizzle<DP>(kPer * i + load_row);
      if (!padded || 8 * piece < A.dim) load_to_lds(stage + 1024 * i, src, lane_at + 16 * piece);
    }
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

  bool odd = false;
  f32x4 o[NT][DP / 16];
  float m[NT], l[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) o[n][d] = f32x4{0, 0, 0, 0};
  }
  const uint8_t* const k_at = ks + r16 * kRowBytes + 16 * (g ^ swizzle<DP>(r16));
  const int v_row = 4 * g + (r16 >> 2);
  const uint8_t* const v_at = vs + v_row * kRowBytes + 16 * (((lane & 3) >> 1) ^ swizzle<DP>(v_row)) + 8 * (lane & 1);
  if (key < to) {
    issue(k_head, k_lds, key, here);
    issue(v_head, v_lds, key, here);
    for (; key < to; key += 32 * W) {
      const bool more = key + 32 * W < to;
      const Pages next = lookup(more ? key + 32 * W : key);
      landed(true);  // the keys; the values may be under way
      f32x4 st[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) st[n][0] = st[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s0 = 0; s0 < DP / 32; s0 += 4) {
        u32x4 kf[4][2];
#pragma unroll
        for (int s = 0; s < 4 && s0 + s < DP / 32; ++s) {
          const uint8_t* const at = ks + (((int)(k_at - ks)) ^ (64 * (s0 + s)));
          kf[s][0] = *(const u32x4*)at;
          kf[s][1] = *(const u32x4*)(at + 16 * kRowBytes);
        }
#pragma unroll
        for (int s = 0; s < 4 && s0 + s < DP / 32; ++s)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            st[n][0] = mfma16<T>(kf[s][0], q[n][s0 + s], st[n][0]);
            st[n][1] = mfma16<T>(kf[s][1], q[n][s0 + s], st[n][1]);
          }
      }
      reads_done();
      if (more) issue(k_head, k_lds, key + 32 * W, next);
      const bool masked = key + 32 > sight.full || here.there != ~0u;
      // values of a step that not all rows see are cleared below; where they are not, all its keys are seen, or their values 0
      const bool cleared = min(key + 32, sight.most) > sight.full;
      const float least = cleared ? 0.0f : __is_same(T, f16) ? 0x1p-24f : 0x1p-126f;
      u32x4 pr[NT], rest[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = st[n][i >> 2][i & 3];
        if (masked) {
          const uint32_t v = seen(n, key, here.there) >> (4 * g);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(v >> (16 * (i >> 2) + (i & 3)) & 1)) x[i] = -INFINITY;
        }
        float most = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) most = fmaxf(most, x[i]);
        most = fmaxf(most, lane_xor<16>(most));
        most = fmaxf(most, lane_xor<32>(most)) * A.scale;
        if (__ballot(grows<T, false>(most, m[n]))) {
          const float up = raised<T, false>(most, m[n]);
          const float a = m[n] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[n] - up);
          m[n] = up;
          l[n] *= a;
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) o[n][d] *= a;
        }
        const float at = m[n] == -INFINITY ? 0.0f : m[n];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], A.scale, -at));
          l[n] += x[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a, b;
          split<T>(x[2 * i], x[2 * i + 1], least, a, b);
          pr[n][i] = a;
          rest[n][i] = b;
        }
      }
      landed(more);  // the values; the next keys may be under way
      if (__builtin_expect(here.there != ~0u, 0)) {  // values that are none
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (!(here.there >> (kPer * i + load_row) & 1)) *(u32x4*)(vs + 1024 * i + 16 * lane) = u32x4{0, 0, 0, 0};
      }
      if (cleared) odd |= clear_odd<T, kLoads>(vs);
      constexpr int kTogether = 8;  // operands of a step's products, all read before the last of them
      static_assert(DP / 16 % kTogether == 0 || DP / 16 < kTogether, "whole sets");
#pragma unroll
      for (int d0 = 0; d0 < DP / 16; d0 += kTogether) {
        u32x4 v[kTogether < DP / 16 ? kTogether : DP / 16];
#pragma unroll
        for (int d = 0; d < kTogether && d0 + d < DP / 16; ++d) {
          const uint8_t* const at = vs + (((int)(v_at - vs)) ^ (32 * (d0 + d)));
          const u32x2 v0 = read_transposed(at), v1 = read_transposed(at + 16 * kRowBytes);
          v[d] = u32x4{v0[0], v0[1], v1[0], v1[1]};
        }
        if (d0 + kTogether >= DP / 16) {
          reads_done();
          if (more) issue(v_head, v_lds, key + 32 * W, next);
        }
#pragma unroll
        for (int d = 0; d < kTogether && d0 + d < DP / 16; ++d)
#pragma unroll
          for (int n = 0; n < NT; ++n) o[n][d0 + d] = mfma16<T>(v[d], pr[n], o[n][d0 + d]);
#pragma unroll
        for (int d = 0; d < kTogether && d0 + d < DP / 16; ++d)
#pragma unroll
          for (int n = 0; n < NT; ++n) o[n][d0 + d] = mfma16<T>(v[d], rest[n], o[n][d0 + d]);
      }
      here = next;
    }
  }

  if (__builtin_expect(odd, 0)) {
    const int seen_whole = (max(sight.full, from) - from) / 32 * 32;  // steps before are this wave's or not, but seen whole
#pragma unroll 1
    for (int at = from + seen_whole; at < to; at += 32) {
      if ((at - from) / 32 % W != w) continue;
      const Pages t = lookup(at);
#pragma unroll 1
      for (int r = 0; r < 32; ++r) {
        const int eight = r >> 3, id = eight == 0 ? t.id[0] : eight == 1 ? t.id[1] : eight == 2 ? t.id[2] : t.id[3];
        const long src = id * P.page + ((at + r) & mask) * P.slot;
        const float one = is_even<T>(k_head + src, A.dim);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const bool mine = seen(n, at, t.there) >> r & 1;
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) o[n][d] += one * odd_values<T>(v_head + src, 16 * d + 4 * g, A.dim, mine);
        }
      }
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
      store_part<T>(A, p, kv_head, kRows, part, parts, row, row - first_row, 4 * c, sum, top, total);
    }
  }
}

// ----------------------------------------------------------------------- many rows
// A workgroup of W waves has 32 W rows of a sequence and key head, each wave 32 of them as the columns of 32 x 32
// matrix steps, and all its keys in tiles of KT x 32, which the waves load into LDS together and all read.  The products
// bound it, and the exponentials beside them: a wave's instructions are laid out so that the two run side by side.
// While step j's scores become probabilities, the products of step j + 1's keys are formed; while the maxima of
// step j + 1 are taken, those of step j's values.
//
// Keys have two stages, values three: a tile's values are read until one step after its keys.  One barrier a tile,
// where the next tile has landed; the one after it is then asked for.
//
// bf16, 64 / 8 heads of 128: a prompt of 4000 tokens over 4100 cached ones 765 to 805 us by the card's clock, 0.99 to 1.05
// PFLOP/s (1.06 for 16384 tokens of 32 / 8), where a large library product runs at 1.23 and a loop of this kernel's
// instructions alone, without barriers, at 1.32.  Slower, each beside this form's 804 to 823 us of the same day, were halves of
// the waves a step apart (916), tiles asked for two ahead (833), and the compiler's own order of a step (850 to 870).
template <typename T>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (__is_same(T, f16))
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}

template <typename T, int DP, int KT, int W>
__global__ __launch_bounds__(64 * W, DP == 256 ? 1 : 2) void lb_attn_tile_kernel(const LbAttnArgs A) {
  constexpr int kRowBytes = 2 * DP, kPieces = DP / 8, kKeys = 32 * KT, kStage = kKeys * kRowBytes;
  constexpr int kPer = 1024 / kRowBytes;       // keys of one load of a wave
  constexpr int kLoads = kStage / 1024 / W;    // loads of a wave for a tile's keys, and for its values
  constexpr int kRows = 32 * W, kS = DP / 16, kD = DP / 32;
  static_assert(kPer <= 8 && kLoads * 1024 * W == kStage, "a load lies in one page");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[5 * kStage];
  const int w = wave_id(), lane = threadIdx.x & 63;
  const int r32 = lane & 31, h = lane >> 5;
  const int kv_head = blockIdx.x % A.kv_heads;
  const Place p = place_of<kKeys, true>(A, kRows, blockIdx.x / A.kv_heads);
  if (p.seq < 0) return;  // the whole workgroup: all waves computed the same
  // causal rows: the last block, which sees the most, first
  const int block = p.blocks - 1 - p.local / p.parts, part = p.local % p.parts;
  const int all_rows = p.s.rows * A.group;
  const Sight sight = sight_of(A, p.s, block * kRows, kRows);
  const int parts = parts_of(sight.most, p.span);
  // the latter: starts that name rows twice, whose sums may wrap as well
  if (part >= parts || (parts > 1 && (uint32_t)p.slot >= (uint64_t)A.slots)) return;
  const int from = part * p.span, to = min(from + p.span, sight.most);
  const int first_row = block * kRows + 32 * w;
  // this wave's own rows: their keys end earlier, and may be seen by all of them later
  const bool has_rows = first_row < all_rows;
  const Sight own = sight_of(A, p.s, first_row, 32);
  const int steps = has_rows ? (max(min(own.most, to) - from, 0) + 31) / 32 : 0;
  const int tiles = (max(to - from, 0) + kKeys - 1) / kKeys;

  const LbPages& P = A.pages;
  const char* const k_head = P.k + kv_head * P.head;
  const char* const v_head = P.v + kv_head * P.head;
  const bool padded = A.dim < DP;
  if (padded) {  // pieces that no load fills
    for (int i = threadIdx.x; i < 5 * kStage / 16; i += 64 * W) *(u32x4*)(lds + 16 * i) = u32x4{0, 0, 0, 0};
    __syncthreads();
  }

  // the row's query, operand of S^T = K Q^T: channels 16 s + 8 h + (0..7)
  u32x4 q[kS];
  const int row = first_row + r32;
  const bool in = row < all_rows;
  const int t = in ? (uint32_t)row / (uint32_t)A.group : 0, head = kv_head * A.group + (in ? row - t * A.group : 0);
  const T* src = (const T*)A.q + (p.s.start + t) * A.qt + head * A.qh;
#pragma unroll
  for (int s = 0; s < kS; ++s) {
    const int d = 16 * s + 8 * h;
    q[s] = in && d < A.dim ? with_sign(A, load_any<u32x4>(src + d)) : u32x4{0, 0, 0, 0};
  }
  const uint64_t word = A.tree && in ? (uint64_t)A.tree[p.s.start + t] : 0;
  const int sees = in ? A.tree ? sight.most : min(sight.most, p.s.base + t + 1) : 0;

  typedef const __attribute__((address_space(4))) int32_t* Table;
  const Table table = (Table)(uintptr_t)(P.table + p.seq * P.table_stride);
  const int mask = (1 << P.shift) - 1;
  auto page_at = [&](int key) __attribute__((always_inline)) { return table[min(key >> P.shift, P.columns - 1)]; };
  auto is_page = [&](int page) __attribute__((always_inline)) { return (uint32_t)page < (uint32_t)P.pages; };
  bool good = true;  // every key has a page
  // this wave's part of tile t's keys and values into their stages
  const int load_row = lane / kPieces, load_piece = lane % kPieces;
  auto fill = [&](int t) __attribute__((always_inline)) {
    const int key0 = from + t * kKeys;
    const uint32_t k_to = lds_address(lds) + (t & 1) * kStage, v_to = lds_address(lds) + (2 + t % 3) * kStage;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = kPer * (kLoads * w + i), row = at + load_row, piece = load_piece ^ swizzle<DP>(row);
      const int page = page_at(key0 + at);
      const long src = (is_page(page) ? page : 0) * P.page + ((key0 + at) & mask) * P.slot;
      const uint32_t offset = load_row * (int)P.slot + 16 * piece;
      if (!padded || 8 * piece < A.dim) {
        load_to_lds(k_to + at * kRowBytes, k_head + src, offset);
        load_to_lds(v_to + at * kRowBytes, v_head + src, offset);
      }
    }
  };
  bool odd = false;
  // tile t, that was asked for, has landed in all waves, and every wave is past the stages that come next
  auto meet = [&](int t) __attribute__((always_inline)) {
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int key0 = from + t * kKeys;
    if (__builtin_expect(!good || key0 + kKeys > sight.most, 0)) {  // values that are none
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = kPer * (kLoads * w + i);
        if (key0 + at + load_row >= sight.most || !is_page(page_at(key0 + at)))
          *(u32x4*)(lds + (2 + t % 3) * kStage + at * kRowBytes + 16 * lane) = u32x4{0, 0, 0, 0};
      }
    }
    if (min(key0 + kKeys, sight.most) > sight.full)
      odd |= clear_odd<T, kLoads>(lds + (2 + t % 3) * kStage + kPer * kLoads * w * kRowBytes);
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
  };

  // which of a step's keys the row sees
  auto seen = [&](int key, uint32_t there) __attribute__((always_inline)) {
    return seen_of(A, p.s.base, key, there, sees, word);
  };
  // keys of a step that have a page, a bit each
  auto paged = [&](int key) __attribute__((always_inline)) {
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) v |= is_page(page_at(key + 8 * i)) ? 0xFFu << (8 * i) : 0u;
    return v;
  };

  f32x16 st[2], o[kD];
  u32x4 pr[2];
  float m = -INFINITY, l = 0.0f;
  pr[0] = pr[1] = u32x4{0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < kD; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  const int k_at = r32 * kRowBytes + 16 * (h ^ swizzle<DP>(r32));
  const int v_row = 4 * h + ((lane & 15) >> 2);
  const int v_at = v_row * kRowBytes + 16 * ((2 * (lane >> 4 & 1) + ((lane & 3) >> 1)) ^ swizzle<DP>(v_row)) + 8 * (lane & 1);
  // where step j's keys and values begin in LDS
  auto k_of = [&](int j) __attribute__((always_inline)) { return (j / KT & 1) * kStage + j % KT * 32 * kRowBytes; };
  auto v_of = [&](int j) __attribute__((always_inline)) { return (2 + j / KT % 3) * kStage + j % KT * 32 * kRowBytes; };

  auto scores = [&](int j, f32x16& s) __attribute__((always_inline)) {
    const int at = k_of(j) + k_at;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
    for (int c = 0; c < kS; ++c) {
      const u32x4 k = *(const u32x4*)(lds + (at ^ (32 * c)));
      s = mfma32<T>(k, q[c], s);
    }
  };
  auto products = [&](int j) __attribute__((always_inline)) {
    const int at = v_of(j) + v_at;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int d = 0; d < kD; ++d) {
        const u32x2 v0 = read_transposed(lds + (at ^ (64 * d)) + 16 * s * kRowBytes);
        const u32x2 v1 = read_transposed(lds + (at ^ (64 * d) ^ 32) + (16 * s + 8) * kRowBytes);
        const u32x4 v = {v0[0], v0[1], v1[0], v1[1]};
        o[d] = mfma32<T>(v, pr[s], o[d]);
      }
    }
  };
  // the row's largest score
  auto maximum = [&](const f32x16& s) __attribute__((always_inline)) {
    float a = s[0], b = s[1];
#pragma unroll
    for (int i = 2; i < 16; i += 2) {
      a = fmaxf(a, s[i]);
      b = fmaxf(b, s[i + 1]);
    }
    a = fmaxf(a, b);
    return fmaxf(a, lane_xor<32>(a)) * A.scale;
  };
  auto rescale = [&](float most) __attribute__((always_inline)) {
    if (__ballot(grows<T, true>(most, m))) {
      const float up = raised<T, true>(most, m);
      const float a = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - up);
      m = up;
      l *= a;
#pragma unroll
      for (int d = 0; d < kD; ++d) o[d] *= a;
    }
  };
  auto probabilities = [&](const f32x16& s) __attribute__((always_inline)) {
    const float at = m == -INFINITY ? 0.0f : m;
    float x[16], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = __builtin_amdgcn_exp2f(fmaf(s[i], A.scale, -at));
      sum[i & 1] += x[i];
    }
    l += sum[0] + sum[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) pr[i >> 2][i & 3] = Pair<T>::pack(x[2 * i], x[2 * i + 1]);
  };
  // before step j is left: where the next one begins a tile, that has landed in all waves, and the one after it is asked for
  auto advance = [&](int j) __attribute__((always_inline)) {
    const int t = (j + 1) / KT;
    if ((j + 1) % KT == 0 && t < tiles) {
      meet(t);
      if (t + 1 < tiles) fill(t + 1);
    }
  };

  if (tiles > 0) {
    fill(0);
    // most steps do not ask again whether their keys have a page
    for (int c = (from >> P.shift) + lane; c <= (to - 1) >> P.shift; c += 64) good = good && is_page(P.table[p.seq * P.table_stride + c]);
    good = __ballot(!good) == 0;
    const int clear = good ? min(steps, (min(own.full, to) - from) >> 5) : 0;  // steps that all rows see whole
    meet(0);
    if (tiles > 1) fill(1);
    int j = 0;
    if (clear > 0) {
      scores(0, st[0]);
      rescale(maximum(st[0]));
      // A step's instructions in the order they are wanted: reads well ahead of their products, and between the products
      // the exponentials and the maxima.  Nothing is moved across a fence.
      auto fence = []() __attribute__((always_inline)) { __builtin_amdgcn_sched_barrier(0); };
      auto body = [&](auto parity, int j) __attribute__((always_inline)) {
        constexpr int B = decltype(parity)::value;
        advance(j);
        u32x4 kf[kS], vf[2 * kD];
        const int k_from = k_of(j + 1) + k_at, v_from = v_of(j) + v_at;
        auto read_v = [&](int c) __attribute__((always_inline)) {
          const int s = c / kD, d = c % kD;
          const u32x2 v0 = read_transposed(lds + (v_from ^ (64 * d)) + 16 * s * kRowBytes);
          const u32x2 v1 = read_transposed(lds + (v_from ^ (64 * d) ^ 32) + (16 * s + 8) * kRowBytes);
          vf[c] = u32x4{v0[0], v0[1], v1[0], v1[1]};
        };
#pragma unroll
        for (int c = 0; c < kS; ++c) kf[c] = *(const u32x4*)(lds + (k_from ^ (32 * c)));
        fence();
        const float at = m == -INFINITY ? 0.0f : m;
        float x[16], sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] = fmaf(st[B][i], A.scale, -at);
          st[1 - B][i] = 0.0f;
        }
        fence();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int c = 0; c < kS; ++c) {
          st[1 - B] = mfma32<T>(kf[c], q[c], st[1 - B]);
          fence();
#pragma unroll
          for (int i = 16 * c / kS; i < 16 * (c + 1) / kS; ++i) x[i] = __builtin_amdgcn_exp2f(x[i]);
          if (c > 0) {
#pragma unroll
            for (int i = 16 * (c - 1) / kS; i < 16 * c / kS; ++i) {
              sum[i & 1] += x[i];
              if (i & 1) pr[i >> 3][(i >> 1) & 3] = Pair<T>::pack(x[i - 1], x[i]);
            }
          }
#pragma unroll
          for (int v = 2 * kD * c / kS; v < 2 * kD * (c + 1) / kS; ++v) read_v(v);
          fence();
        }
#pragma unroll
        for (int i = 16 * (kS - 1) / kS; i < 16; ++i) {
          sum[i & 1] += x[i];
          if (i & 1) pr[i >> 3][(i >> 1) & 3] = Pair<T>::pack(x[i - 1], x[i]);
        }
        l += sum[0] + sum[1];
        fence();
        __builtin_amdgcn_s_setprio(0);
        float a[2];
#pragma unroll
        for (int c = 0; c < 2 * kD; ++c) {
          o[c % kD] = mfma32<T>(vf[c], pr[c / kD], o[c % kD]);
          fence();
          if (c >= kD) {  // the scores are there: their maxima
#pragma unroll
            for (int i = 16 * (c - kD) / kD; i < 16 * (c - kD + 1) / kD; ++i)
              a[i & 1] = i < 2 ? st[1 - B][i] : fmaxf(a[i & 1], st[1 - B][i]);
            fence();
          }
        }
        const float top = fmaxf(a[0], a[1]);
        rescale(fmaxf(top, lane_xor<32>(top)) * A.scale);
      };
      // no way round a step's products in here: the outputs stay where they are
      for (; j + 2 < clear; j += 2) {
        body(std::integral_constant<int, 0>(), j);
        body(std::integral_constant<int, 1>(), j + 1);
      }
      if (j + 1 < clear) {
        body(std::integral_constant<int, 0>(), j);
        ++j;
        st[0] = st[1];
      }
      advance(j);
      probabilities(st[0]);
      products(j);
      ++j;
    }
    // the last keys, which not all rows see (all of them, where a page is missing), one step after the other
#pragma unroll 1
    for (; j < steps; ++j) {
      const int key = from + 32 * j;
      const uint32_t there = paged(key);
      scores(j, st[0]);
      const uint32_t v = seen(key, there) >> (4 * h);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!(v >> (8 * (i >> 2) + (i & 3)) & 1)) st[0][i] = -INFINITY;
      rescale(maximum(st[0]));
      probabilities(st[0]);
      products(j);
      advance(j);
    }
    for (; j < tiles * KT; ++j) advance(j);
    __syncthreads();  // the stages have been read
    int* const odd_waves = (int*)lds;
    if (lane == 0) odd_waves[w] = odd;
    __syncthreads();
    odd = false;
#pragma unroll
    for (int i = 0; i < W; ++i) odd = odd || odd_waves[i];
    if (__builtin_expect(odd, 0)) {
      // from the first tile on in which some were cleared
#pragma unroll 1
      for (int at = from + (max(sight.full, from) - from) / kKeys * kKeys; at < to; at += 32) {
        const uint32_t there = paged(at);
#pragma unroll 1
        for (int r = 0; r < 32; ++r) {
          const int page = page_at(at + r);
          const long src = (is_page(page) ? page : 0) * P.page + ((at + r) & mask) * P.slot;
          const float one = is_even<T>(k_head + src, A.dim);
          const bool mine = seen(at, there) >> r & 1;
#pragma unroll
          for (int d = 0; d < kD; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const f32x4 f = one * odd_values<T>(v_head + src, 32 * d + 8 * i + 4 * h, A.dim, mine);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[d][4 * i + e] += f[e];
            }
        }
      }
    }
  }
  l += lane_xor<32>(l);
  if (in) {
#pragma unroll
    for (int d = 0; d < kD; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 v = {o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        store_part<T>(A, p, kv_head, kRows, part, parts, row, row - block * kRows, 32 * d + 8 * i + 4 * h, v, m, l);
      }
  }
}

// ------------------------------------------------------------------------- the join
// Rows of the call whose keys were taken in parts.  A wave looks at `per` rows' records at once and joins those
// with several parts, one after the other: eight times 64 / LD parts at once, four channels a lane.  A part in which a
// row saw nothing has no maximum, and a sum of 0 (or NaN).  Latency bounds it, 4 us; of 15600 rows in
// some four parts of 128 channels 16 us, 3.4 TB/s.
template <typename T, int LD>
__global__ __launch_bounds__(256) void lb_attn_join_kernel(const LbAttnArgs A, int rows, int per) {
  constexpr int kSets = 64 / LD;
  const int w = wave_id(), lane = threadIdx.x & 63;
  const long all_rows = A.tokens * A.heads;
  const long row0 = (blockIdx.x * 4l + w) * per;
  if (row0 >= all_rows) return;
  const Workspace ws = workspace_of(A, rows);
  const long mine = row0 + lane;
  Parts r = {0, 0};
  if (lane < per && mine < all_rows) r = ws.parts[mine];
  const long limit = A.slots * A.kv_heads * rows;
  const int step = A.kv_heads * rows, count_of = r.count & 0xFFFF, seq = r.count >> 16 & 0xFFFF;
  bool several = lane < per && mine < all_rows && count_of > 1 && seq < A.pages.seqs;
  several = several && r.first >= 0 && r.first + (count_of - 1l) * step < limit;
  typedef const __attribute__((address_space(4))) int32_t* Ints;  // read by the scalar unit
  const Ints starts = (Ints)(uintptr_t)A.pages.starts, lens = (Ints)(uintptr_t)A.pages.lens;
  const int set = lane / LD, d = 4 * (lane % LD);
  const bool in = d < A.dim;
  for (uint64_t left = __ballot(several); left; left &= left - 1) {
    const int l = __builtin_ctzll(left);
    const int first = __builtin_amdgcn_readlane(r.first, l), count = __builtin_amdgcn_readlane(count_of, l);
    // A row of no sequence has no record, and what lies in its place may be an earlier call's: a record stands if its
    // sequence has the row in this call, which has written it then.  Asked for here, looked at behind the sums.
    const int of = __builtin_amdgcn_readlane(seq, l), start = starts[of], end = starts[of + 1], len = lens[of];
    float top = -INFINITY, total = 0.0f;
    f32x4 sum = {0, 0, 0, 0};
    // eight sets' loads at a time; behind the last part it again, with factor 0
#pragma unroll 1
    for (int j = 0; j < count; j += 8 * kSets) {
      float2 v[8];
      f32x4 o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = first + min(j + kSets * i + set, count - 1) * step;
        v[i] = ws.ml[at];
        o[i] = in ? *(const f32x4*)(ws.sums + (long)at * A.dim + d) : f32x4{0, 0, 0, 0};
      }
      float most = top;
#pragma unroll
      for (int i = 0; i < 8; ++i) most = fmaxf(most, v[i].x);
      if constexpr (LD <= 16) most = fmaxf(most, lane_xor<16>(most));
      if constexpr (LD <= 32) most = fmaxf(most, lane_xor<32>(most));
      const float before = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - most);
      top = most;
      if (j > 0) {  // what has been added so far: of parts without a maximum it is 0 or NaN, and stays that
        total *= before;
        sum *= before;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool real = j + kSets * i + set < count;
        const float a = v[i].x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(v[i].x - top);
        if (real) {
          total += v[i].x == -INFINITY ? v[i].y : a * v[i].y;
          sum += a * o[i];
        }
      }
    }
    if constexpr (LD <= 16) {
      total += lane_xor<16>(total);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += lane_xor<16>(sum[e]);
    }
    if constexpr (LD <= 32) {
      total += lane_xor<32>(total);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += lane_xor<32>(sum[e]);
    }
    const long row = row0 + l;
    const int t = (int)(row / A.heads);
    const Span s = span_of(A.pages, start, end, len, (int)A.tokens);
    if (set == 0 && t >= s.start && t < s.start + s.rows) {
      store_result<T>(A, t, (int)(row - (long)t * A.heads), d, sum, top, total);
    }
  }
}

template <typename T, int LD>
void launch_join(const LbAttnArgs& a, const LbAttnPlan& plan, hipStream_t stream) {
  if (!plan.join) return;
  // a row a wave while there are few, so that they are joined side by side
  const long rows = a.tokens * a.heads;
  const int per = rows <= 8192 ? 1 : rows <= 65536 ? 4 : 64;
  hipLaunchKernelGGL((lb_attn_join_kernel<T, LD>), dim3((unsigned)((rows + 4 * per - 1) / (4 * per))), dim3(256), 0, stream, a,
                     plan.rows, per);
}

template <int STEP, bool MANY>
void launch_groups(const LbAttnArgs& a, const LbAttnPlan& plan, hipStream_t stream) {
  if (a.groups) hipLaunchKernelGGL((lb_attn_groups_kernel<STEP, MANY>), dim3(1), dim3(1024), 0, stream, a, a.groups, plan.rows);
}

template <typename T, int DP, int NT, int W>
void launch_stream(const LbAttnArgs& a, const LbAttnPlan& plan, hipStream_t stream) {
  launch_groups<32 * W, false>(a, plan, stream);
  hipLaunchKernelGGL((lb_attn_stream_kernel<T, DP, NT, W>), dim3((unsigned)plan.grid), dim3(64 * W), 0, stream, a);
  launch_join<T, DP / 4>(a, plan, stream);
}

template <typename T, int DP, int KT, int W>
void launch_tile(const LbAttnArgs& a, const LbAttnPlan& plan, hipStream_t stream) {
  launch_groups<32 * KT, true>(a, plan, stream);
  hipLaunchKernelGGL((lb_attn_tile_kernel<T, DP, KT, W>), dim3((unsigned)plan.grid), dim3(64 * W), 0, stream, a);
  launch_join<T, DP / 4>(a, plan, stream);
}

template <typename T, int DP, int W>
void launch_rows(const LbAttnArgs& a, const LbAttnPlan& plan, hipStream_t stream) {
  if (plan.rows == 256) {
    if constexpr (DP == 128) launch_tile<T, DP, 2, 8>(a, plan, stream);
  } else if (plan.rows == 128)
    launch_tile<T, DP, DP == 256 ? 1 : 2, 4>(a, plan, stream);
  else if (plan.rows == 16)
    launch_stream<T, DP, 1, W>(a, plan, stream);
  else
    launch_stream<T, DP, 2, W>(a, plan, stream);
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

// Rows of a workgroup by the rows that a sequence has on average.  bf16, some 2000 keys: 36 rows (64 / 8 heads of 128,
// 16 sequences) in blocks of 16, 32 and 256 take 33, 34 and 45 us, 75 rows 45 and 45 in 32 and 256, 100 rows 59 and 46;
// 24 rows of 40 heads in 16 and 32 take 29 and 26; 75 rows of 8 heads of 256, 54 and 94 us in 32 and 128, of 16 heads of 64,
// 31 and 41 in 32 and 256.  (64 rows a workgroup of few rows leave no registers: 51 us for the first.)
// Of many rows, blocks of 128, two at a time on a compute unit, read the keys twice as often as those of 256, and keep
// fewer waves waiting where keys end soon: heads of 128, 3 prompts of 1500 81 and 91 us, one of 512 21 and 26, 4000 tokens on
// 4100 keys 848 and 814, 100 on 8000 126 and 111; heads of 64, 4000 tokens 77 and 85, 16000 2500 and 2610.
// A sequence of n rows has at most n group / rows + 1 blocks, and `target` / kv_heads parts at most are added over all
// of them; sequences with several parts have at most twice their share of them.
LbAttnPlan lb_attn_plan(int64_t tokens, int seqs, int64_t capacity, int heads, int kv_heads, int dim) {
  LbAttnPlan p;
  const int64_t group = heads / kv_heads, mean = (tokens * group + seqs - 1) / seqs;
  p.rows = mean <= 16 ? 16 : mean <= (dim > 64 && dim <= 128 ? 80 : 112) ? 32 : 128;
  if (p.rows == 128 && dim > 64 && dim <= 128 && (mean > 4096 || capacity > 4096)) p.rows = 256;
  // workgroups at once: by their LDS and registers
  p.round = p.rows == 256 || (p.rows == 128 && dim > 128) ? 256 : dim <= 64 && p.rows == 16 ? 1024 : 512;
  p.least = p.rows > 32 ? 1024 : 256;
  // blocks of all sequences, at most, and what is shared out for so many; an empty workgroup costs a nanosecond (6000 of
  // them for one token 5 us)
  const int64_t blocks = std::min(tokens * group / p.rows + seqs, tokens * group);
  const int64_t most = p.rows > 32 ? 2 * p.round : p.rows == 16 ? 1536 : 1024;
  p.target = p.rows > 32 ? (int)most : (int)std::min<int64_t>(most, p.round * (1 + 4 * blocks * kv_heads / p.round));
  const int64_t parts = (capacity + p.least - 1) / p.least;
  p.join = parts > 1;
  const int64_t share = (p.target + kv_heads - 1) / kv_heads + 1;
  p.slots = p.join ? std::min(2 * share + 2, blocks * parts) : 0;
  p.groups = seqs > kFewSeqs ? (seqs + 63) / 64 : 0;
  p.grid = std::min(share + blocks + 2, blocks * parts) * kv_heads;
  return p;
}

size_t lb_attn_groups_at(const LbAttnPlan& plan, int64_t tokens, int heads, int kv_heads, int dim) {
  if (!plan.join) return 0;
  return (size_t)plan.slots * kv_heads * plan.rows * (dim + 2) * sizeof(float) + (size_t)tokens * heads * 2 * sizeof(int);
}

size_t lb_attn_workspace(const LbAttnPlan& plan, int64_t tokens, int heads, int kv_heads, int dim) {
  return lb_attn_groups_at(plan, tokens, heads, kv_heads, dim) + (plan.groups ? (plan.groups + 1) * 2 * sizeof(int) : 0);
}

hipError_t lb_launch_attn(const LbAttnArgs& a, const LbAttnPlan& plan, int dtype, hipStream_t stream) {
  if (dtype == 1)
    launch_attn<f16>(a, plan, stream);
  else
    launch_attn<bf16>(a, plan, stream);
  return hipGetLastError();
}
