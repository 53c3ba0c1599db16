// block.h -- helpers shared by the operators around the routed experts:
// element types, row loads and stores, workgroup reductions.
#pragma once

#include "../common.h"

namespace moe {

inline bool type_ok(int t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_BF16; }
inline size_t type_size(int t) { return t == MOE_TYPE_F32 ? 4 : 2; }

// 8 consecutive elements of a row, in registers as loaded (a bf16 row uses
// the first 16 bytes), so that several rows' loads are in flight before the
// first is converted.  Rows need their elements' alignment alone: the memory
// instructions take 16 bytes at any address.
template <typename T>
struct Raw8 {
  u32x4 a[sizeof(T) / 2];
};

template <typename T>
__device__ inline Raw8<T> load8(const T* p) {
  Raw8<T> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
// the first n < 8 of 8 elements; the rest 0
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

// Sum over the wave in a fixed order, as a wave-uniform value (the DPP steps of
// wave_max; lanes that a row broadcast does not reach add 0).
template <int CTRL, int ROWS>
__device__ inline float dpp_or_0(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                              ROWS, 0xF, false));
}
__device__ inline float wave_sum(float v) {
  v += dpp_mov<0xB1>(v);         // quad_perm [1,0,3,2]
  v += dpp_mov<0x4E>(v);         // quad_perm [2,3,0,1]
  v += dpp_mov<0x141>(v);        // row_half_mirror
  v += dpp_mov<0x140>(v);        // row_mirror
  v += dpp_or_0<0x142, 0xA>(v);  // row_bcast:15 into rows 1, 3
  v += dpp_or_0<0x143, 0xC>(v);  // row_bcast:31 into rows 2, 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

template <int CTRL>
__device__ inline double dpp_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

}  // namespace moe
