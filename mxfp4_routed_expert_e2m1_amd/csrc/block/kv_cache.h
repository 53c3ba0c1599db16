// kv_cache.h -- the 4-bit cache's order in memory, and the checks that its calls share.
//
// A page of one head is one piece of page * (D + D/16) bytes (D = head_dim, NB = D/32 blocks of 32
// channels), pages of a head n_heads pieces apart:
//   K codes   [page][D/2]           a token's codes, channel 2i in the low nibble of byte i
//   K scales  [page][NB]
//   V codes   [page/4][16][4][NB]   4 tokens, 16 runs of D/16 channels, token, codes of the run
//   V scales  [page/4][NB][4]
// Both orders are those of the matrix core's operands.  In scores = K Q^T the contraction runs
// over channels: a lane wants whole runs of a token's channels.  In out = V^T P it runs over
// tokens: a lane wants the same channels of several tokens, and with 4 tokens side by side it
// has them in one 4 NB-byte load.  No byte holds codes of two tokens, so that writing a token
// touches no other.
#pragma once

#include "block.h"

namespace moe {

template <int D>
struct KvUnit {
  static constexpr int NB = D / 32;
  int page;
  __host__ __device__ int64_t bytes() const { return (int64_t)page * (D + D / 16); }
  __host__ __device__ int k_scales() const { return page * (D / 2); }
  __host__ __device__ int v_codes() const { return page * (D / 2 + NB); }
  __host__ __device__ int v_scales() const { return page * (D + NB); }
};

// 8 consecutive elements of a row, rounded once; PAST: past the L2s, for results of large calls.
template <typename T, bool PAST>
__device__ inline void store8(T* p, const float (&v)[8]) {
  T o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (T)v[i];
  if constexpr (PAST) {
    typedef u32x4 piece __attribute__((aligned(2)));  // (rows need their elements' alignment alone)
    u32x4 w[sizeof(o) / 16];
    __builtin_memcpy(w, o, sizeof(o));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(o) / 16); ++i) __builtin_nontemporal_store(w[i], (piece*)p + i);
  } else {
    __builtin_memcpy(p, o, sizeof(o));
  }
}

// The largest scale byte that a write leaves; what lies above reads as NaN.
constexpr uint32_t kMaxScaleByte = 252;

inline bool kv_sizes_ok(const moe_kv_cache_t* C) {
  const bool dim = C->head_dim == 64 || C->head_dim == 128 || C->head_dim == 256;
  const bool page = C->page >= 16 && C->page <= 256 && (C->page & (C->page - 1)) == 0;
  return dim && page && C->n_heads >= 1 && C->n_heads <= 1024 && C->n_pages >= 1 &&
         (int64_t)C->n_pages * C->page < ((int64_t)1 << 31);
}

inline int kv_cache_check(const moe_kv_cache_t* C) {
  if (!C) return MOE_ERR_INVALID_ARG;
  if (!kv_sizes_ok(C)) return MOE_ERR_SHAPE;
  if (!C->data) return MOE_ERR_INVALID_ARG;
  return aligned(C->data, 16) ? MOE_OK : MOE_ERR_ALIGNMENT;
}

// Strides of [rows][heads][dim]: rows of heads, or heads of rows, without overlap.
inline bool head_strides_ok(int64_t ld, int64_t hs, int rows, int heads, int dim) {
  constexpr int64_t kMost = (int64_t)1 << 40;
  if (rows > 1 && (ld < dim || ld > kMost)) return false;
  if (heads > 1 && (hs < dim || hs > kMost)) return false;
  if (rows <= 1 || heads <= 1) return true;
  return (ld - dim) / (heads - 1) >= hs || (hs - dim) / (rows - 1) >= ld;
}

}  // namespace moe
