// How the attention cuts sequences into blocks of rows and parts of keys: the arithmetic that its kernels
// do on the device, on plain numbers, so that it can be held to the plan's grid and workspace on the host too.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>

namespace lbh {

#define LB_SPLIT __host__ __device__ __forceinline__

// Blocks of `height` rows of a sequence's rows, times the heads of a group.
LB_SPLIT int blocks_of(int rows, int group, int height) { return (rows * group + height - 1) / height; }
LB_SPLIT int parts_of(int keys, int span) {
  const int parts = (keys + span - 1) / span;
  return parts > 1 ? parts : 1;
}
// Keys of a part of a sequence, at most `span` in whole steps: all its parts as long as each other.
template <int STEP>
LB_SPLIT int part_keys(int keys, int span) {
  const int parts = parts_of(keys, span), even = (keys + parts - 1) / parts;
  const int own = (even + STEP - 1) / STEP * STEP;
  return own > STEP ? own : STEP;
}
// What a sequence adds to the sum that the length of a part follows from: its keys for each of its blocks.  All of
// them, as the parts are cut from all: then sum of blocks x ceil(keys / span) is at most share + blocks, which is what
// the grid holds, and of the sequences with several parts at most twice the share, which the workspace holds.  (Causal
// blocks see half of their own rows' keys; a span from that half would cut up to twice the share.)
LB_SPLIT float units_of(int keys, int blocks) { return (float)keys * (float)blocks; }
// Whether blocks of many rows (of all key heads together) are taken with all their keys.
template <bool MANY>
LB_SPLIT bool is_whole(float blocks, float round) {
  return MANY && blocks > 0.5f * round;
}
// Keys of a part, from the sums over all sequences of the blocks and of the blocks' keys.
template <bool MANY>
LB_SPLIT int span_from(float blocks, float units, int kv_heads, int round_of, int target, int least) {
  const float round = (float)round_of;
  blocks *= (float)kv_heads;
  if (is_whole<MANY>(blocks, round)) return 1 << 30;
  const float rounds = MANY ? 2.0f : 1.0f + floorf(4.0f * blocks / round);
  const float share = fminf(fmaxf(round * rounds - blocks, 0.5f * round), (float)target);
  units *= (float)kv_heads / share;
  const int span = units < 1e9f ? (int)units + 1 : 1 << 30;
  return span > least ? span : least;
}

}  // namespace lbh
