// attn_plan.h -- how a call of the attention over the 4-bit cache is cut into work: the host's choice
// of a kernel, its tiles and its pieces, and the length of the pieces, which the kernels find from the
// lengths on the GPU.
#pragma once

#include "block.h"

namespace moe {

constexpr int kStep = 64;  // tokens to which pieces and the start of a pass are aligned

// A sequence's work: steps of kStep tokens, of each tile.  (Up to 2^24 of both.)
__host__ __device__ __forceinline__ int64_t steps_of(int tiles, int span) {
  return (int64_t)tiles * ((span + kStep - 1) / kStep);
}

// The tokens of a piece, the same for every sequence: the batch's `work` over `target` pieces where that makes no more than `target` of them, or over fewer by half a piece, or
// a whole one, for each of all its tiles, which leaves room for a last piece of each that is not full:
// at most `all` + target.  Work of more than 2^31 steps is counted in units of a power of two, rounded
// up.  `count`: the pieces that a cut makes.
template <typename Count>
__host__ __device__ __forceinline__ int choose_cut(int64_t work, int64_t all, int target, int quantum,
                                                   bool may_count, Count count) {
  const int unit = work >> 31 ? 33 - __builtin_clzll((uint64_t)work) : 0;
  const uint32_t w = (uint32_t)((work + ((int64_t)1 << unit) - 1) >> unit);
  for (int k = may_count ? 0 : 2;; ++k) {
    int over = all < target ? target - (int)all * k / 2 : 0;
    over = over > target / 2 ? over : (target + 1) / 2;
    int64_t c = (int64_t)((w + (uint32_t)over - 1) / (uint32_t)over) << unit;
    c = (c < (1 << 24) ? c : 1 << 24) * kStep;
    const int64_t up = (c + quantum - 1) & ~(int64_t)(quantum - 1);
    const int cut = (int)(up < quantum ? quantum : up > 0x40000000 ? 0x40000000 : up);
    if (k == 2 || count(cut) <= target) return cut;
  }
}
__host__ __device__ __forceinline__ int pieces_of(int span, int cut) {
  return span <= cut ? 1 : (span + cut - 1) / cut;
}

// Workgroups of 4 waves that a CU holds (by their registers and LDS):
constexpr int resident(bool f32, int dim, int nq) {
  if (dim == 256) return nq == 1 ? 2 : 1;
  if (dim == 128) return nq == 1 ? 3 : 2;
  return f32 || nq == 2 ? 3 : 4;
}

// How a call runs: the kernel and the rows of its tiles, the pieces to cut into.
struct AttnPlan {
  bool chunk;  // attn_chunk_kernel, or attn_rows_kernel
  int nq;      // of attn_rows_kernel
  bool shared, wide, halves;
  int tile_rows, quantum;
  int64_t tiles;   // at most, over all sequences
  int target;      // 0: tokens are not cut
  int64_t items;   // of the grid
};

inline int64_t tiles_of(int64_t rows, int64_t group, int64_t n_seqs, int tile_rows) {
  return (rows * group + tile_rows - 1) / tile_rows + n_seqs;
}

inline AttnPlan attn_plan(const moe_attn_t* A, const moe_kv_cache_t* C, bool f32, int64_t rows,
                          int64_t n_seqs, int64_t tokens, int cus) {
  AttnPlan p;
  const int64_t group = A->n_heads / C->n_heads;
  const int64_t each = (rows * group + n_seqs - 1) / n_seqs;  // rows of a sequence, on average
  p.shared = each <= 64;
  p.nq = f32 || each <= 16 ? 1 : 2;
  p.chunk = !f32 && !p.shared;
  p.tile_rows = p.shared ? 16 * p.nq : f32 ? 64 : 128;
  p.quantum = p.shared ? 128 : 64;
  // workgroups that the chip holds at once
  int64_t full = (p.chunk ? 2 : resident(f32, C->head_dim, p.nq)) * cus;
  const auto tiles_of_256 = [&] {
    p.tile_rows = 256;
    full = cus;
  };
  if (p.chunk && C->head_dim < 256 && tiles_of(rows, group, n_seqs, 256) * C->n_heads >= cus)
    tiles_of_256();
  p.tiles = tiles_of(rows, group, n_seqs, p.tile_rows);
  // Cutting shortens a workgroup's pass by the chip's idle part of it, and costs the joining launch
  // (5 us: the time of 900 tokens for few rows, of 2048 for many, which also have more to join).
  // Below, few tiles get workgroups of twice the waves.  One request of 8 key heads of 128 with 4
  // query heads each, us with 4 waves, 8 waves, cut:
  //   bf16   512 tokens 8.0, 7.4, 9.8   1000: 11.4, 9.3, 10.0   1500: 14.7, 11.5, 10.0
  //   f32    512 tokens 8.9, 8.3, 9.7   768: 11.3, 9.9, 9.6     1000: 13.8, 11.7, 9.8
  int64_t groups = p.tiles * C->n_heads;
  // Tokens that a tile's rows see at most, as far as the window goes.  (With a prefix, rows in front of
  // its end see up to it, so a window and a long prefix are planned as shorter than they are.)
  int64_t span = tokens;
  if (A->window > 0 && A->window + p.tile_rows / group + 1 < span)
    span = A->window + p.tile_rows / group + 1;
  p.wide = p.shared && span > 256 && span <= (f32 ? 768 : 1024) && groups <= cus;
  const bool cut = !p.wide && groups < full &&
                   span * (full - groups) / full >= (p.chunk ? 2048 : f32 ? 700 : 900);
  // Tiles of 256 rows once there is work for all CUs, by their number or since they are cut: 200 and
  // 512 new rows over 8192 tokens, 32 query heads on 8 of 128, 61.0 and 96.6 us in tiles of 128, 55.7
  // and 89.5 in those.
  if (cut && p.chunk && C->head_dim < 256 && each > 128 && p.tile_rows == 128) {
    tiles_of_256();
    p.tiles = tiles_of(rows, group, n_seqs, 256);
    groups = p.tiles * C->n_heads;
  }
  // Few tiles: two waves for each 32 rows (512 new rows, 32 query heads on 8 of 128: 20.4 us with one,
  // 19.4 with two; 500, 16 heads on 4 of 64: 14.9, 13.3; four prompts of 100, 32 on 8 of 128: 11.4, 13.2).
  p.halves = p.chunk && !cut && C->head_dim < 256 && p.tile_rows == 128 && groups <= cus &&
             span > 256;
  p.target = cut ? (int)((full + C->n_heads - 1) / C->n_heads) : 0;
  p.items = p.tiles + p.target;
  return p;
}

// Floats of a cut call's workspace: the pieces' rows, their bases and sums, the rows' records.
inline int64_t part_floats(const moe_kv_cache_t* C, int64_t items, int64_t tile_rows, int64_t rows) {
  return items * C->n_heads * tile_rows * (C->head_dim + 2) + 4 * rows;
}

// Bytes of workspace for calls of up to so many rows and sequences.  Cut calls have fewer than `full`
// tiles over all heads, so at most that many and their target pieces: no fewer rows or sequences need
// more.
inline int64_t attn_workspace(const moe_attn_t* A, const moe_kv_cache_t* C, int64_t rows, int64_t n_seqs,
                              int cus) {
  const int64_t heads = C->n_heads;
  const int64_t group = A->n_heads / heads;
  int64_t most = 0;
  for (int tile_rows : {16, 32, 64, 128, 256}) {
    const int64_t full = (tile_rows <= 64 ? 4 : tile_rows == 128 ? 2 : 1) * cus;
    const int64_t target = (full + heads - 1) / heads;
    int64_t tiles = tiles_of(rows, group, n_seqs, tile_rows);
    tiles = tiles < target ? tiles : target;
    const int64_t most_rows = target * tile_rows;
    const int64_t n = part_floats(C, tiles + target, tile_rows, rows < most_rows ? rows : most_rows);
    most = n > most ? n : most;
  }
  return most * 4;
}

}  // namespace moe
