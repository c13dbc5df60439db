// Host-side launchers of the dense operators (arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct LbNormArgs {
  const void* x; long ldx;
  const void* residual; long ldr;
  const void* weight;
  void* hidden; long ldh;
  void* y; long ldy;
  int8_t* q; long ldq;
  float* scale;
  long rows;
  int n;
  float eps;
};

struct LbNormBwdArgs {
  const void* dy; long lddy;
  const void* dhidden; long lddh;
  const void* hidden; long ldh;
  const void* weight;
  void* dx; long lddx;
  float* dweight;
  float* partial;   // [groups][n]
  int groups;
  long rows;
  int n;
  float eps;
};

struct LbQ8LinearArgs {
  const int8_t* xq; long ldx;
  const float* xscale;
  const int8_t* wq; long ldw;
  const float* wscale;
  long batch;
  int m, n;
  void* y; long ldy;
};

struct LbLogprobsArgs {
  const void* logits; long ld;
  const int64_t* targets;
  float* logprob;
  float* entropy;
  float* lse;
  float* top_logprob;
  int64_t* top_index;
  void* ws;
  long rows;
  int vocab;
  int top;
  int splits;       // workgroups a row
  int span;         // elements of a split (a multiple of 8)
};

struct LbLogprobsBwdArgs {
  const void* logits; long ld;
  const int64_t* targets;
  const float* lse;
  const float* entropy;
  const float* dlogprob;
  const float* dentropy;
  const int64_t* top_index;
  const float* dtop;
  void* dlogits; long ldd;
  long rows;
  int vocab;
  int top;
};

int lb_norm_bwd_groups(int64_t rows, int64_t n);
hipError_t lb_launch_norm(const LbNormArgs& a, int dtype, hipStream_t stream);
hipError_t lb_launch_norm_bwd(const LbNormBwdArgs& a, int dtype, hipStream_t stream);
hipError_t lb_launch_q8_quantize(const LbNormArgs& a, int dtype, hipStream_t stream);
hipError_t lb_launch_q8_linear(const LbQ8LinearArgs& a, int y_dtype, hipStream_t stream);
int lb_logprobs_splits(int64_t rows, int64_t vocab, int* span);
size_t lb_logprobs_partial_bytes(int64_t rows, int splits, int top);
hipError_t lb_launch_logprobs(const LbLogprobsArgs& a, int dtype, hipStream_t stream);
hipError_t lb_launch_logprobs_bwd(const LbLogprobsBwdArgs& a, int dtype, hipStream_t stream);
