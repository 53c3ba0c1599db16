// block.h -- helpers shared by the operators around the routed experts:
// element types, row loads and stores, workgroup reductions.
#pragma once

#include "../common.h"

namespace moe {

template <typename T>
struct ElemType;
template <>
struct ElemType<float> {
  static constexpr int id = MOE_TYPE_F32;
};
template <>
struct ElemType<__bf16> {
  static constexpr int id = MOE_TYPE_BF16;
};

inline bool type_ok(int t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_BF16; }
inline size_t type_size(int t) { return t == MOE_TYPE_F32 ? 4 : 2; }

// 8 consecutive elements of a row, in registers as loaded (a bf16 row uses
// the first 16 bytes), so that several rows' loads are in flight before the
// first is converted.
template <typename T>
struct Raw8 {
  u32x4 a[sizeof(T) / 2];
};

template <typename T>
__device__ inline Raw8<T> load8_vec(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.a[i] = ((const u32x4*)p)[i];
  return r;
}
// the first n of 8 elements (any alignment); the rest 0
template <typename T>
__device__ inline Raw8<T> load8_part(const T* p, int n) {
  Raw8<T> r;
  T v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : (T)0.f;
  __builtin_memcpy(&r, v, sizeof(r));
  return r;
}
template <typename T>
__device__ inline void to_f32(const Raw8<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.a[i >> 2][i & 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.a[0][i] << 16);
      v[2 * i + 1] = __uint_as_float(r.a[0][i] & 0xFFFF0000u);
    }
  }
}

// Sum (or max) over the wave, in every lane's register as one value.
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

int norm_args_check(const moe_norm_t* N);

}  // namespace moe
