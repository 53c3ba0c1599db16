// attn.h -- what the kernels of the attention over the 4-bit cache share: a call's arguments, the cut
// of its work, what a row sees, scores beyond the product, reductions.
#pragma once

#include "kv_cache.h"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kStep = 64;  // tokens to which pieces and the start of a pass are aligned

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
  int quantum;   // tokens of a piece: a multiple of this
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

__device__ inline int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_incl_scan(v), 63); }

// Cut calls (few tiles, so few sequences): a piece has `cut` tokens, as many for every sequence, and
// items are counted over the sequences.  The cut is the batch's work over `target` pieces where
// that makes no more than `target` of them (a sequence's last piece is a whole one there), or over
// fewer pieces by half a piece, or a whole one, for each tile.  Finds the sequence of an item, or
// with `row` >= 0 of that row.  (Counts of one sequence are kept below 2^24 or 2^25, so that offsets
// that overlap cannot make a sum of 64 overflow.)
__device__ inline bool find_piece(const AttnArgs& a, int64_t item, int row, Found& f, int& cut) {
  const int lane = lane_id();
  Seq q = {0, 0, 0, 0};
  int tiles = 0, span = 0;
  const auto take = [&](int s0) {
    q = {0, 0, 0, 0};
    tiles = span = 0;
    if (s0 + lane < a.n_seqs) {
      q.load(a, s0 + lane);
      tiles = q.tiles(a);
      tiles = tiles < (1 << 24) ? tiles : 1 << 24;
      span = q.n - q.first(a);
    }
  };
  const auto steps = [&] {
    const int64_t w = (int64_t)tiles * ((span + kStep - 1) / kStep);
    return w < (1 << 25) ? (int)w : (1 << 25) - 1;
  };
  const auto items_of = [&](int pieces) {
    const int64_t n = (int64_t)tiles * pieces;
    return n < (1 << 24) ? (int)n : 1 << 24;
  };
  take(0);
  int64_t work = wave_sum(steps()), all = wave_sum(tiles);
  const bool one = a.n_seqs <= 64;
  if (!one) {
    for (int s0 = 64; s0 < a.n_seqs; s0 += 64) {
      take(s0);
      work += wave_sum(steps());
      all += wave_sum(tiles);
    }
    take(0);
  }
  for (int k = one ? 0 : 2;; ++k) {
    int64_t over = a.target - all * k / 2;
    over = over > a.target / 2 ? over : a.target / 2 > 0 ? a.target / 2 : 1;
    int64_t c = (work * kStep + over - 1) / over;
    c = (c + a.quantum - 1) / a.quantum * a.quantum;
    cut = uniform((int)(c < a.quantum ? a.quantum : c > 0x40000000 ? 0x40000000 : c));
    if (k == 2 || wave_sum(items_of(span <= cut ? 1 : (span + cut - 1) / cut)) <= a.target) break;
  }
  int64_t before = 0;
  for (int s0 = 0;;) {
    const int pieces = span <= cut ? 1 : (span + cut - 1) / cut;
    const int items = items_of(pieces), scan = wave_incl_scan(items);
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
    s0 += 64;
    if (s0 >= a.n_seqs) return false;
    take(s0);
  }
}

// The item of a workgroup (false: there is none), the tokens of a piece.
__device__ inline bool find_item(const AttnArgs& a, int64_t item, Found& f, int& cut) {
  cut = 0x40000000;
  return a.target ? find_piece(a, item, -1, f, cut) : find_tile(a, item, f);
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

// 16 channels of a query row in two E4M3 planes, x = 2^(e - 127) (hi + 2^-5 lo), where e puts the
// largest magnitude of the block (bits `most`) at 128 .. 256.
__device__ inline int plane_exponent(uint32_t most) {
  const int e = (int)(most >> 23) - 7;
  return e < 16 ? 16 : e;
}
template <int AT>
__device__ inline void e4m3_planes(const float (&x)[16], int e, v8i32& hi, v8i32& lo) {
  const float down = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int h = 0, l = 0;
    float r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = x[4 * i + k] * down;
    h = __builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], h, false);
    h = __builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], h, true);
    r[0] = (r[0] - __builtin_amdgcn_cvt_f32_fp8(h, 0)) * 32.f;
    r[1] = (r[1] - __builtin_amdgcn_cvt_f32_fp8(h, 1)) * 32.f;
    r[2] = (r[2] - __builtin_amdgcn_cvt_f32_fp8(h, 2)) * 32.f;
    r[3] = (r[3] - __builtin_amdgcn_cvt_f32_fp8(h, 3)) * 32.f;
    l = __builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], l, false);
    l = __builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], l, true);
    hi[AT + i] = h;
    lo[AT + i] = l;
  }
}
__device__ inline uint32_t most_bits(const float (&x)[16]) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    most = b > most ? b : most;
  }
  return most;
}

// 256 rows or fewer of a sequence and one key head at a time, bf16 (attn_chunk.hip).
void attn_chunk_launch(const AttnArgs& a, int head_dim, int waves, hipStream_t stream);

}  // namespace moe
