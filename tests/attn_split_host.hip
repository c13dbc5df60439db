// The attention's split of a batch, on the host: the items and the joined parts of one key head that the kernels
// number (csrc/attn.hip, place_of), with their own arithmetic, beside what the plan has room for.
#include <stdint.h>

#include <algorithm>
#include <vector>

#include "attn_launch.h"
#include "attn_split.h"

namespace {

template <int STEP, bool MANY>
void split(const LbAttnPlan& p, int seqs, int group, int kv_heads, const int32_t* rows, const int32_t* keys, int64_t* out) {
  float blocks = 0.0f, units = 0.0f;
  int longest = 0;
  for (int i = 0; i < seqs; ++i) {
    const int b = lbh::blocks_of(rows[i], group, p.rows);
    blocks += (float)b;
    units += lbh::units_of(keys[i], b);
    if (rows[i] > 0) longest = std::max(longest, keys[i]);
  }
  int span = lbh::span_from<MANY>(blocks, units, kv_heads, p.round, p.target, p.least);
  auto count = [&](bool even, int length, int64_t* all, int64_t* joined) {
    *all = *joined = 0;
    for (int i = 0; i < seqs; ++i) {
      const int64_t b = lbh::blocks_of(rows[i], group, p.rows);
      const int64_t parts = lbh::parts_of(keys[i], even ? length : lbh::part_keys<STEP>(keys[i], length));
      *all += b * parts;
      *joined += parts > 1 ? b * parts : 0;
    }
  };
  if (MANY && !lbh::is_whole<MANY>(blocks * (float)kv_heads, (float)p.round) && seqs <= 64) {
    float best = INFINITY;
    for (int lane = 0; lane < 64; ++lane) {
      const int even = (longest / (lane + 1) + STEP) / STEP * STEP, mine = lane ? even : 1 << 30;
      int64_t all, joined;
      count(true, mine, &all, &joined);
      if (lane > 0 && (all > p.grid / kv_heads || joined > p.slots)) continue;
      const float cost = ceilf((float)all * (float)kv_heads / (float)p.round) * (float)(even + 512);
      if (cost < best) {
        best = cost;
        span = mine;
      }
    }
  }
  count(false, span, &out[0], &out[1]);
}

}  // namespace

// out: items, items of sequences with several parts, workgroups, slots, the height of a block
extern "C" void attn_split(int64_t tokens, int32_t seqs, int64_t capacity, int32_t heads, int32_t kv_heads, int32_t dim,
                           const int32_t* rows, const int32_t* keys, int64_t* out) {
  const LbAttnPlan p = lb_attn_plan(tokens, seqs, capacity, heads, kv_heads, dim);
  const int group = heads / kv_heads;
  out[2] = p.grid / kv_heads;
  out[3] = p.slots;
  out[4] = p.rows;
  if (p.rows > 32)
    dim > 128 ? split<32, true>(p, seqs, group, kv_heads, rows, keys, out)
              : split<64, true>(p, seqs, group, kv_heads, rows, keys, out);
  else
    dim > 128 ? split<64, false>(p, seqs, group, kv_heads, rows, keys, out)
              : split<128, false>(p, seqs, group, kv_heads, rows, keys, out);
}
