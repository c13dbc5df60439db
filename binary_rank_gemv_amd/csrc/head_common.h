// Shared device helpers of the dense operators (norm, 8-bit product, token
// log probabilities): element types, unaligned vector access, wave sums.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

typedef _Float16 f16;
typedef __bf16 bf16;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

#define LBH_MAX_DIRECT 65  // places with a direct gradient: the target and 64 alternatives

namespace lbh {

__device__ inline int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Wide access at any element alignment: global memory takes unaligned 8- and
// 16-byte accesses on this architecture, so these stay single instructions.
template <typename V>
__device__ __forceinline__ V load_any(const void* p) {
  V v;
  __builtin_memcpy(&v, p, sizeof(V));
  return v;
}
template <typename V>
__device__ __forceinline__ void store_any(void* p, V v) {
  __builtin_memcpy(p, &v, sizeof(V));
}

// Two elements of a packed word as fp32, and back (rounded to nearest even).
template <typename T>
struct Pair;
template <>
struct Pair<f16> {
  typedef f16 h2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(h2, w)[0]; }
  static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(h2, w)[1]; }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    h2 v;
    v[0] = (f16)a;
    v[1] = (f16)b;
    return __builtin_bit_cast(uint32_t, v);
  }
};
template <>
struct Pair<bf16> {
  typedef bf16 b2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ float lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    b2 v;
    v[0] = (bf16)a;
    v[1] = (bf16)b;
    return __builtin_bit_cast(uint32_t, v);
  }
};

// Eight consecutive elements as fp32.  `left` is how many of them the row
// still has: 8 or more is the whole vector, fewer are read one by one, and
// what lies behind the row is never touched.
template <typename T>
__device__ __forceinline__ void load8(const T* p, long left, float fill, float (&v)[8]) {
  if (left >= 8) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4 w = load_any<u32x4>(p + 4 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * j + i] = __builtin_bit_cast(float, (uint32_t)w[i]);
      }
    } else {
      const u32x4 w = load_any<u32x4>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = Pair<T>::lo(w[i]);
        v[2 * i + 1] = Pair<T>::hi(w[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? (float)p[i] : fill;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, long left, const float (&v)[8]) {
  if (left >= 8) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, v[4 * j + i]);
        store_any(p + 4 * j, w);
      }
    } else {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = Pair<T>::pack(v[2 * i], v[2 * i + 1]);
      store_any(p, w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (T)v[i];
  }
}

// The value of lane (lane ^ M), without a trip through LDS: cross-lane moves
// inside a row of 16, and the row swaps of this architecture for 16 and 32.
template <int M>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
  if constexpr (M == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
  if constexpr (M == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
  if constexpr (M == 4)  // i ^ 7, then i ^ 3
    return __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true), 0x1B, 0xF, 0xF, true);
  if constexpr (M == 8) return __builtin_amdgcn_mov_dpp(v, 0x128, 0xF, 0xF, true);
  if constexpr (M == 15) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);
#ifdef __HIP_DEVICE_COMPILE__
  // the swap exchanges the odd rows (upper half) of its first operand with the
  // even rows (lower half) of its second: with v as both, the even rows find
  // their partner in the second result, the odd rows in the first
  if constexpr (M == 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return threadIdx.x & 16 ? s[0] : s[1];
  }
  if constexpr (M == 32) {
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return threadIdx.x & 32 ? s[0] : s[1];
  }
#endif
  return v;
}
template <int M>
__device__ __forceinline__ float lane_xor(float v) {
  return __builtin_bit_cast(float, lane_xor<M>(__builtin_bit_cast(uint32_t, v)));
}

__device__ __forceinline__ float wave_sum(float v) {
  v += lane_xor<1>(v);
  v += lane_xor<2>(v);
  v += lane_xor<4>(v);
  v += lane_xor<8>(v);
  v += lane_xor<16>(v);
  return v + lane_xor<32>(v);
}
// The larger value, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float wave_max(float v) {
  v = max_nan(v, lane_xor<1>(v));
  v = max_nan(v, lane_xor<2>(v));
  v = max_nan(v, lane_xor<4>(v));
  v = max_nan(v, lane_xor<8>(v));
  v = max_nan(v, lane_xor<16>(v));
  return max_nan(v, lane_xor<32>(v));
}

}  // namespace lbh
