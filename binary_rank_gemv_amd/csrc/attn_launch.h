// Host-side launchers of the operators between the projections (arguments
// already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "littlebit_attn.h"

// A cache and the sequences of a call, as the kernels read them.
struct LbPages {
  char* k;
  char* v;
  long page, head, slot;   // strides in bytes
  int pages, shift;        // page_size = 1 << shift
  const int32_t* starts;
  const int32_t* lens;
  const int32_t* table;
  long table_stride;
  int seqs, columns;
};

// Three kinds of heads (queries, keys, values), any of them absent (heads 0).
struct LbRopeArgs {
  const void* x[3];
  void* y[3];              // of keys and values to a cache: unused
  long xt[3], xh[3], yt[3], yh[3];
  int heads[3];
  const void* weight[2];
  const int32_t* positions;
  const float* inv_freq;
  int rot, interleaved;
  float eps;
  float turn;              // 1, or -1 to turn back
  long tokens;
  int dim;
  int blocks, span;        // waves a token, and heads' steps a wave
  bool append;
  LbPages pages;
};

struct LbRopeBwdArgs {
  const void* dy[2];
  const void* x[2];
  void* dx[2];
  long dyt[2], dyh[2], xt[2], xh[2], dxt[2], dxh[2];
  int heads[2];
  const void* weight[2];
  float* dweight[2];
  float* partial;          // [groups[0] + groups[1]][dim]
  int groups[2];
  const int32_t* positions;
  const float* inv_freq;
  int rot, interleaved;
  float eps;
  long tokens;
  int dim;
};

struct LbAttnArgs {
  LbPages pages;
  const void* q; long qt, qh;
  void* out; long ot, oh;
  const int64_t* tree;
  float* lse;
  float* partial;          // the workspace
  int* groups;             // in it, of many sequences: what every 64 of them have before them; or null
  long slots;
  long tokens;
  int heads, kv_heads, group, dim;
  float scale;             // its size, with the factor to base 2; 1 where it is 0
  uint32_t sign, keep;     // what of it goes into the queries' bits
  int round, target, least;  // as in the plan
};

// The attention's shape for a call, a function of its sizes alone.
struct LbAttnPlan {
  int rows;                // rows (tokens x heads of a group) of a workgroup
  int round;               // workgroups that run at once
  int target;              // and that the keys are spread over, at most
  int least;               // keys of a part, at least
  bool join;               // whether a sequence can have several parts
  long slots;              // workgroups whose results may have to be joined
  int groups;              // 64 sequences each, where a kernel adds them up first; or 0
  long grid;
};

void lb_rope_bwd_groups(int64_t tokens, int heads, int kv_heads, int dim, int* groups);
hipError_t lb_launch_rope(LbRopeArgs& a, int dtype, hipStream_t stream);
hipError_t lb_launch_rope_bwd(const LbRopeBwdArgs& a, int dtype, hipStream_t stream);
hipError_t lb_launch_accept(const LbPages& p, int heads, int dim, const int32_t* path, int columns, hipStream_t stream);
LbAttnPlan lb_attn_plan(int64_t tokens, int seqs, int64_t capacity, int heads, int kv_heads, int dim);
size_t lb_attn_groups_at(const LbAttnPlan& plan, int64_t tokens, int heads, int kv_heads, int dim);
size_t lb_attn_workspace(const LbAttnPlan& plan, int64_t tokens, int heads, int kv_heads, int dim);
hipError_t lb_launch_attn(const LbAttnArgs& a, const LbAttnPlan& plan, int dtype, hipStream_t stream);
