// attn.h -- what the kernels of the attention over the 4-bit cache share: a call's arguments, the cut
// of its work, what a row sees, scores beyond the product, reductions.
#pragma once

#include "kv_cache.h"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kStep = 64;       // tokens of an iteration
constexpr int kLeastPart = 256; // tokens that are worth a workgroup: an iteration for each wave

struct AttnArgs {
  const void* q;
  void* out;
  const uint8_t* data;
  const int32_t* q_offsets;
  const int32_t* kv_lens;
  const int32_t* table;
  const int32_t* prefix;
  const float* slopes;
  float* part;  // partial results, NULL: tokens are not cut
  int64_t ld_q, hs_q, ld_out, hs_out, ld_table;
  int64_t ml_at;  // floats from `part` to the maxima and sums
  int rows, n_seqs, n_heads, kv_heads, group, page_log, n_pages, max_pages, window;
  int target;    // pieces that fill the chip (0: tokens are not cut)
  int64_t items; // of the grid
  int tile_rows; // rows of a tile
  float scale, softcap;
};

// A sequence's numbers, kept within what the arguments allow.
struct Seq {
  int row0, m, n, prefix;  // first row, rows, cached tokens, prefix
  __device__ void load(const AttnArgs& a, int s) {
    if (a.q_offsets) {
      int r0 = a.q_offsets[s], r1 = a.q_offsets[s + 1];
      r0 = r0 < 0 ? 0 : r0 > a.rows ? a.rows : r0;
      r1 = r1 < r0 ? r0 : r1 > a.rows ? a.rows : r1;
      row0 = r0;
      m = r1 - r0;
    } else {
      row0 = s;
      m = 1;
    }
    const int64_t most = (int64_t)a.max_pages << a.page_log;
    n = a.kv_lens[s];
    n = n < 0 ? 0 : n > most ? (int)most : n;
    prefix = a.prefix ? a.prefix[s] : 0;
  }
  // tokens that any row sees lie from here (a multiple of kStep) to n
  __device__ int first(const AttnArgs& a) const {
    const int64_t f = a.window > 0 ? (int64_t)n - m - a.window + 1 : 0;
    return f > 0 ? (int)f & ~(kStep - 1) : 0;
  }
  __device__ int tiles(const AttnArgs& a) const {
    return (int)(((int64_t)m * a.group + a.tile_rows - 1) / a.tile_rows);
  }
};

__device__ inline int64_t wave_sum_i64(int64_t v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Tokens of a piece: all of them, or as many as cut the batch's work into `target` pieces.
__device__ inline int piece_tokens(const AttnArgs& a) {
  int64_t work = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 64) {
    const int s = s0 + lane_id();
    if (s < a.n_seqs) {
      Seq q;
      q.load(a, s);
      work += (int64_t)q.tiles(a) * (q.n - q.first(a));
    }
  }
  work = wave_sum_i64(work);
  int64_t c = (work + a.target - 1) / a.target;
  c = (c + kStep - 1) / kStep * kStep;
  c = c < kLeastPart ? kLeastPart : c > 0x40000000 ? 0x40000000 : c;
  return uniform((int)c);
}

__device__ inline int pieces_of(const AttnArgs& a, const Seq& s, int cut) {
  const int span = s.n - s.first(a);
  return span <= cut ? 1 : (span + cut - 1) / cut;
}

// A sequence, its place in the batch, and where its items (pieces of tiles) begin.
struct Found {
  Seq seq;
  int at, pieces;
  int64_t first_item;
};

// Uncut calls: sequence s has its tiles from item q_offsets[s] * group / tile_rows + s on, which
// leaves room for a last tile that is not full; the item's sequence by 64 probes at a time.
__device__ inline bool find_tile(const AttnArgs& a, int64_t item, Found& f) {
  f.pieces = 1;
  if (!a.q_offsets) {  // a row each
    const int64_t each = ((int64_t)a.group + a.tile_rows - 1) / a.tile_rows;
    f.at = (int)(item / each);
    f.first_item = f.at * each;
    if (f.at >= a.n_seqs) return false;
    f.seq.load(a, f.at);
    return true;
  }
  int lo = 0, n = a.n_seqs;  // the last s of lo .. lo + n - 1 that begins at or before the item
  while (n > 1) {
    const int step = (n + 63) / 64, s = lo + step * lane_id();
    bool before = false;
    if (step * lane_id() < n) {
      int r0 = a.q_offsets[s];
      r0 = r0 < 0 ? 0 : r0 > a.rows ? a.rows : r0;
      before = (int64_t)r0 * a.group / a.tile_rows + s <= item;
    }
    const uint64_t b = __ballot(before);
    const int l = b ? 63 - __builtin_clzll(b) : 0;
    n = n - step * l < step ? n - step * l : step;
    lo += step * l;
  }
  f.at = lo;
  f.seq.load(a, lo);
  f.first_item = (int64_t)f.seq.row0 * a.group / a.tile_rows + lo;
  return item >= f.first_item && item - f.first_item < f.seq.tiles(a);
}

// Cut calls (few tiles, so few sequences): items are counted over the sequences.  The sequence of
// an item, or with `row` >= 0 of that row.
constexpr int kMostItems = 1 << 24;  // of one sequence (offsets that overlap could make it more)
__device__ inline bool find_piece(const AttnArgs& a, int cut, int64_t item, int row, Found& f) {
  int64_t before = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 64) {
    const int s = s0 + lane_id();
    Seq q = {0, 0, 0, 0};
    int pieces = 1, items = 0;
    if (s < a.n_seqs) {
      q.load(a, s);
      pieces = pieces_of(a, q, cut);
      const int64_t all = (int64_t)q.tiles(a) * pieces;
      items = all < kMostItems ? (int)all : kMostItems;
    }
    const int scan = wave_incl_scan(items);
    const int64_t end = before + scan;
    const bool mine = row >= 0 ? row >= q.row0 && row < q.row0 + q.m : item < end && item >= end - items;
    const uint64_t who = __ballot(mine);
    if (who) {
      const int l = __builtin_ctzll(who);
      f.at = s0 + l;
      f.first_item = before + __builtin_amdgcn_readlane(scan - items, l);
      f.pieces = __builtin_amdgcn_readlane(pieces, l);
      f.seq.row0 = __builtin_amdgcn_readlane(q.row0, l);
      f.seq.m = __builtin_amdgcn_readlane(q.m, l);
      f.seq.n = __builtin_amdgcn_readlane(q.n, l);
      f.seq.prefix = __builtin_amdgcn_readlane(q.prefix, l);
      return true;
    }
    before += __builtin_amdgcn_readlane(scan, 63);
  }
  return false;
}

// The tokens that a row sees: lo <= j < hi.
struct Sight {
  int lo, hi;
};
__device__ inline Sight sight_of(const AttnArgs& a, const Seq& s, int token) {
  const int i = s.n - s.m + token;  // the row's place
  Sight v;
  v.hi = i + 1 > s.prefix ? i + 1 : s.prefix;
  v.hi = v.hi < s.n ? v.hi : s.n;
  v.hi = v.hi > 0 ? v.hi : 0;
  const int64_t lo = a.window > 0 ? (int64_t)i - a.window + 1 : 0;
  v.lo = lo > 0 ? (int)lo : 0;
  return v;
}

__device__ inline float max16(float v) {  // over the lanes l % 16
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(t[0]), __uint_as_float(t[1]));
}
__device__ inline float sum16(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(t[0]) + __uint_as_float(t[1]);
}

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// softcap * tanh(s / softcap).  (1 - e^-2x) / (1 + e^-2x), its quotient refined once, loses a small
// x beside the 1; below 1/4 Taylor's series to x^9 is within 2^-25 of x.
__device__ inline float capped(float s, float cap, float inv) {
  const float x = s * inv, z = x * x;
  const float e = exp2_fast(-2.f * kLog2e * fabsf(x)), d = 1.f + e, rc = __builtin_amdgcn_rcpf(d);
  float big = (1.f - e) * rc;
  big = copysignf(fmaf(fmaf(-big, d, 1.f - e), rc, big), x);
  float p = 62.f / 2835.f;
  p = fmaf(p, z, -17.f / 315.f);
  p = fmaf(p, z, 2.f / 15.f);
  p = fmaf(p, z, -1.f / 3.f);
  const float small = fmaf(x * z, p, x);
  return cap * (fabsf(x) < 0.25f ? small : big);
}

// 4 scale bytes, any above kMaxScaleByte (253..255)?
__device__ inline uint32_t over_bytes(uint32_t x) {
  return ((x & 0x7F7F7F7Fu) + 0x03030303u) & x & 0x80808080u;
}
__device__ inline float scale_byte(uint32_t word, int b) {
  return __uint_as_float((b == 0 ? word << 23 : b == 3 ? word >> 1 : word >> (8 * b) << 23) & 0x7F800000u);
}

// x = sum of PARTS bf16 numbers (three hold every fp32 bit).
template <int PARTS>
__device__ inline void split(float x, __bf16 (&p)[PARTS]) {
  p[0] = (__bf16)x;
  if constexpr (PARTS == 3) {
    // (infinities and NaN: the first part has them, the others must not make NaN of infinity)
    const float r = fabsf(x) < __builtin_inff() ? x - (float)p[0] : 0.f;
    p[1] = (__bf16)r;
    p[2] = (__bf16)(r - (float)p[1]);
  }
}

// 256 rows or fewer of a sequence and one key head at a time, bf16 (attn_chunk.hip).
void attn_chunk_launch(const AttnArgs& a, int head_dim, int waves, hipStream_t stream);

}  // namespace moe
