// attn.h -- what the kernels of the attention over the 4-bit cache share: a call's arguments, the cut
// of its work, what a row sees, scores beyond the product, reductions.
#pragma once

#include "attn_plan.h"
#include "kv_cache.h"

namespace moe {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;

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
  int64_t ml_at, rec_at;  // floats from `part` to the pieces' bases and sums, to the rows' records
  int rows, n_seqs, n_heads, kv_heads, group, page_log, n_pages, max_pages, window;
  int target;    // pieces that fill the chip (0: tokens are not cut)
  int64_t items; // of the grid
  int quantum;   // tokens of a piece: a multiple of this power of two
  int tile_log;  // rows of a tile, as a power of two
  uint32_t group_inv;  // 2^32 / group + 1
  float scale, softcap;
};

// (token, head of the group) of rows near a tile's first, whose division is done once.
struct RowSplit {
  int tok0, rem0;
  __device__ __forceinline__ RowSplit(const AttnArgs& a, int row) {
    tok0 = uniform((int)((uint32_t)row / (uint32_t)a.group));
    rem0 = row - tok0 * a.group;
  }
  // of row + i, where (group + i) * group < 2^32: i < 256 and groups of up to 2^14
  __device__ __forceinline__ void at(const AttnArgs& a, int i, int& tok, int& head) const {
    const uint32_t x = rem0 + i, t = a.group == 1 ? x : __umulhi(x, a.group_inv);
    tok = tok0 + (int)t;
    head = (int)(x - t * a.group);
  }
};

// A sequence's numbers, kept within what the arguments allow.
struct Seq {
  int row0, m, n, prefix;  // first row, rows, cached tokens, prefix
  __device__ __forceinline__ void load(const AttnArgs& a, int s) {
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
  __device__ __forceinline__ int first(const AttnArgs& a) const {
    const int64_t f = a.window > 0 ? (int64_t)n - m - a.window + 1 : 0;
    return f > 0 ? (int)f & ~(kStep - 1) : 0;
  }
  __device__ __forceinline__ int tiles(const AttnArgs& a) const {  // (rows * group < 2^28)
    return (m * a.group + (1 << a.tile_log) - 1) >> a.tile_log;
  }
};

// A sequence, its place in the batch, and where its items (pieces of tiles) begin.
struct Found {
  Seq seq;
  int at, pieces, first_item;
};

// Uncut calls: sequence s has its tiles from item q_offsets[s] * group / (tile's rows) + s on, which
// leaves room for a last tile that is not full; the item's sequence by 64 probes at a time.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int item, Found& f) {
  f.pieces = 1;
  if (!a.q_offsets) {  // a row each
    const int each = (a.group + (1 << a.tile_log) - 1) >> a.tile_log;
    f.at = each == 1 ? item : item / each;
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
      before = ((r0 * a.group) >> a.tile_log) + s <= item;
    }
    const uint64_t b = __ballot(before);
    const int l = b ? 63 - __builtin_clzll(b) : 0;
    n = n - step * l < step ? n - step * l : step;
    lo += step * l;
  }
  f.at = lo;
  f.seq.load(a, lo);
  f.first_item = ((f.seq.row0 * a.group) >> a.tile_log) + lo;
  return item >= f.first_item && item - f.first_item < f.seq.tiles(a);
}

__device__ __forceinline__ int wave_sum(int v) {
  return __builtin_amdgcn_readlane(wave_incl_scan(v), 63);
}

__device__ __forceinline__ int64_t wave_sum(int64_t v) {  // of numbers below 2^48
  const int low = wave_sum((int)(v & 0xFFFFFF));
  return ((int64_t)wave_sum((int)(v >> 24)) << 24) + low;
}

// Cut calls (few tiles, so few sequences): a piece has `cut` tokens (choose_cut), as many for every
// sequence, and items are counted over the sequences.  (A sequence's rows are below 2^28, so its tiles
// below 2^24, and its pieces are kept below 2^24, so that offsets that overlap cannot make a sum of 64
// overflow.)
__device__ __forceinline__ bool find_piece(const AttnArgs& a, int item, Found& f, int& cut) {
  const int lane = lane_id();
  Seq q = {0, 0, 0, 0};
  int tiles = 0, span = 0;
  const auto take = [&](int s0) {
    q = {0, 0, 0, 0};
    tiles = span = 0;
    if (s0 + lane < a.n_seqs) {
      q.load(a, s0 + lane);
      tiles = q.tiles(a);
      span = q.n - q.first(a);
    }
  };
  const auto items_of = [&](int pieces) {
    const int64_t n = (int64_t)tiles * pieces;
    return n < (1 << 24) ? (int)n : 1 << 24;
  };
  take(0);
  int64_t work = wave_sum(steps_of(tiles, span)), all = wave_sum(tiles);
  const bool one = a.n_seqs <= 64;
  if (!one) {
    for (int s0 = 64; s0 < a.n_seqs; s0 += 64) {
      take(s0);
      work += wave_sum(steps_of(tiles, span));
      all += wave_sum(tiles);
    }
    take(0);
  }
  cut = uniform(choose_cut(work, all, a.target, a.quantum, one,
                           [&](int c) { return wave_sum(items_of(pieces_of(span, c))); }));
  int64_t before = 0;
  for (int s0 = 0;;) {
    const int pieces = pieces_of(span, cut);
    const int items = items_of(pieces), scan = wave_incl_scan(items);
    const int64_t end = before + scan;
    const bool mine = item < end && item >= end - items;
    const uint64_t who = __ballot(mine);
    if (who) {
      const int l = __builtin_ctzll(who);
      f.at = s0 + l;
      f.first_item = (int)before + __builtin_amdgcn_readlane(scan - items, l);
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

// Workgroups: key heads first, so that with 8 of them (or a multiple) each XCD's L2 has the tokens of
// its own; then items, in two dimensions.
constexpr unsigned kItemsY = 32768;
__device__ __forceinline__ int block_item() { return (int)(blockIdx.z * kItemsY + blockIdx.y); }
inline dim3 item_grid(int64_t items, int kv_heads) {
  const int64_t y = items < kItemsY ? items : kItemsY;
  return dim3((unsigned)kv_heads, (unsigned)y, (unsigned)((items + y - 1) / y));
}

// The item of a workgroup (false: there is none), the tokens of a piece.
__device__ __forceinline__ bool find_item(const AttnArgs& a, int item, Found& f, int& cut) {
  cut = 0x40000000;
  if (item >= a.items) return false;
  return a.target ? find_piece(a, item, f, cut) : find_tile(a, item, f);
}

// The tokens that a row sees: lo <= j < hi.
struct Sight {
  int lo, hi;
};
__device__ __forceinline__ Sight sight_of(const AttnArgs& a, const Seq& s, int token) {
  const int i = s.n - s.m + token;  // the row's place
  Sight v;
  v.hi = i + 1 > s.prefix ? i + 1 : s.prefix;
  v.hi = v.hi < s.n ? v.hi : s.n;
  v.hi = v.hi > 0 ? v.hi : 0;
  const int64_t lo = a.window > 0 ? (int64_t)i - a.window + 1 : 0;
  v.lo = lo > 0 ? (int)lo : 0;
  return v;
}

// What the joining launch has to know of a row; written by the workgroup of the sequence's first piece
// and key head.
struct RowRecord {
  int first_item, pieces, tiles, row0;  // pieces negative: the row sees nothing
};
__device__ __forceinline__ void put_record(const AttnArgs& a, const Found& f, int token,
                                           const Sight& see) {
  RowRecord r = {f.first_item, see.lo < see.hi ? f.pieces : -f.pieces, f.seq.tiles(a), f.seq.row0};
  if (f.pieces == 1) r.pieces = 1;
  ((RowRecord*)(a.part + a.rec_at))[f.seq.row0 + token] = r;
}

// find_item for a workgroup: by its first wave, for the others through LDS (the cut's arithmetic takes
// as long as half a step of a pass, and waves that share a SIMD would take turns at it).
struct FoundShared {
  int have, cut;
  Found f;
};
__device__ __forceinline__ bool find_item(const AttnArgs& a, int item, Found& f, int& cut, int wave,
                                          FoundShared& s) {
  if (!a.target && !a.q_offsets) return find_item(a, item, f, cut);
  if (wave == 0) {
    const bool have = find_item(a, item, f, cut);
    if (lane_id() == 0) s = {have, cut, f};
  }
  lds_barrier();
  f = s.f;
  cut = uniform(s.cut);
  f.at = uniform(f.at);
  f.pieces = uniform(f.pieces);
  f.first_item = uniform(f.first_item);
  f.seq.row0 = uniform(f.seq.row0);
  f.seq.m = uniform(f.seq.m);
  f.seq.n = uniform(f.seq.n);
  f.seq.prefix = uniform(f.seq.prefix);
  return uniform(s.have) != 0;
}

__device__ __forceinline__ float max16(float v) {  // over the lanes l % 16
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(t[0]), __uint_as_float(t[1]));
}
__device__ __forceinline__ float sum16(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(t[0]) + __uint_as_float(t[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// softcap * tanh(x), x = s / softcap; k = 2 log2(e) / softcap.  Caps up to kNearCap: bf16 calls
// cap - 2 cap / (1 + e^2x), f32 ones cap (1 - e^-2x) / (1 + e^-2x) with the reciprocal refined, off by
// at most 2^-23 and 2^-24 of the cap, which is what scores near it are rounded to.  Wider caps leave
// most scores far below them, where that would be much: below x = 1/4 the series of tanh x / x, whose
// first dropped term is 2^-26, and the quotient from there on.
constexpr float kNearCap = 64.f;
__device__ __forceinline__ float cap_factor(float cap) {
  return cap > 0.f ? fminf(2.f * kLog2e / cap, 3.4e38f) : 0.f;
}
__device__ __forceinline__ float capped_quotient(float s, float cap, float k) {
  const float e = exp2_fast(-k * fabsf(s)), d = 1.f + e;
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(fmaf(-d, r, 1.f), r, r);
  return copysignf(cap * ((1.f - e) * r), s);
}
template <bool F32>
__device__ __forceinline__ float capped(float s, float cap, float k) {
  if constexpr (F32) return capped_quotient(s, cap, k);
  else return fmaf(-2.f * cap, __builtin_amdgcn_rcpf(1.f + exp2_fast(s * k)), cap);
}
__device__ __forceinline__ float capped_wide(float s, float cap, float k) {
  const float x = s * (k * (0.5f / kLog2e)), z = x * x;
  float p = 2.1869489e-2f;  // 62/2835, -17/315, 2/15, -1/3
  p = fmaf(p, z, -5.3968254e-2f);
  p = fmaf(p, z, 1.3333333e-1f);
  p = fmaf(p, z, -3.3333333e-1f);
  return z < 0.0625f ? fmaf(s * z, p, s) : capped_quotient(s, cap, k);
}

// 4 scale bytes, any above kMaxScaleByte (253..255)?
__device__ __forceinline__ uint32_t over_bytes(uint32_t x) {
  return ((x & 0x7F7F7F7Fu) + 0x03030303u) & x & 0x80808080u;
}
__device__ __forceinline__ float scale_byte(uint32_t word, int b) {
  const uint32_t at = b == 0 ? word << 23 : b == 3 ? word >> 1 : word >> (8 * b) << 23;
  return __uint_as_float(at & 0x7F800000u);
}

// Eight numbers as sums of PARTS bf16 numbers.  Three hold every fp32 bit: the upper 8 bits of the
// significand, the next 8 and the last, each cut off (the rest of an infinity is NaN).  One is
// rounded to nearest.
template <int PARTS>
__device__ __forceinline__ void split8(const float (&x)[2][4], bf16x8 (&p)[PARTS]) {
  if constexpr (PARTS == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[0][i] = (__bf16)x[i / 4][i % 4];
  } else {
    u32x4 w[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[3], b[3];  // of numbers 2i and 2i + 1
      const auto cut = [](float v, uint32_t (&c)[3]) {
        c[0] = __float_as_uint(v);
        const float r = v - __uint_as_float(c[0] & 0xFFFF0000u);
        c[1] = __float_as_uint(r);
        c[2] = __float_as_uint(r - __uint_as_float(c[1] & 0xFFFF0000u));
      };
      cut(x[i / 2][2 * i % 4], a);
      cut(x[i / 2][2 * i % 4 + 1], b);
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k][i] = __builtin_amdgcn_perm(b[k], a[k], 0x07060302);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) p[k] = __builtin_bit_cast(bf16x8, w[k]);
  }
}

// 16 channels of a query row in two E4M3 planes, x = 2^(e - 127) (hi + 2^-5 lo), where e puts the
// largest magnitude of the block (bits `most`) at 128 .. 256.
__device__ __forceinline__ int plane_exponent(uint32_t most) {
  const int e = (int)(most >> 23) - 7;
  return e < 16 ? 16 : e;
}
template <int AT>
__device__ __forceinline__ void e4m3_planes(const float (&x)[16], int e, v8i32& hi, v8i32& lo) {
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
// Largest over blocks of 8, 16 or 32 neighbouring lanes.
template <int LANES>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  const auto step = [&](int o) { v = (uint32_t)o > v ? (uint32_t)o : v; };
  step(__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
  step(__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
  step(__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));  // row_half_mirror
  if constexpr (LANES >= 16)
    step(__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));  // row_mirror
  if constexpr (LANES == 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = s[0] > s[1] ? s[0] : s[1];
  }
  return v;
}
__device__ __forceinline__ uint32_t most_bits(const float (&x)[16]) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    most = b > most ? b : most;
  }
  return most;
}

// 256 rows or fewer of a sequence and one key head at a time, bf16 (attn_chunk.hip).
void attn_chunk_launch(const AttnArgs& a, int head_dim, int tile_rows, bool halves, hipStream_t stream);

}  // namespace moe
