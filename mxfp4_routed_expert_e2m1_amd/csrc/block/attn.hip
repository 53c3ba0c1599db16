// attn.hip -- attention of a ragged batch's rows over a 4-bit cache.
//
// One pass over the tokens with the running maximum and sum of a softmax: for 64 tokens at a time
//   S^T = K Q^T          (matrix core, tokens x rows)
//   m' = max(m, max S),  P = 2^(S - m'),  l = l 2^(m - m') + sum P
//   O^T = O^T 2^(m - m') + V^T P^T
// with S in units of log2.  A tile's rows are (token, query head of the key head's group) pairs,
// row r = token r / G, head r % G, so one pass over a key head's tokens serves its whole group.
//
// Operands without a detour through LDS.  E2M1 values times a power of two are exact in bf16, and
// the converter makes two of them in one instruction.  Lane l of a wave holds row l % 16 of an
// operand and 8 elements of the contraction, group l / 16; which 8 is free, as long as both
// operands agree:
//   scores: group g has the channels g D/4 .. + D/4, which lie side by side in the cache, 8 at a
//           time, so one load fetches a lane's part of a token;
//   out:    group g has the tokens 4g .. 4g+3 and 16 + 4g .. + 3 of 32, since that is what it
//           holds of S^T as the matrix core leaves it: P goes from one product into the next in
//           the registers where it was made.  V's order in the cache makes these 4 tokens of
//           D/16 channels one load.
// Rounding: q, K and V are exact.  P is rounded to bf16 (relative 2^-9, of either sign, averaged
// over the tokens); f32 calls split q and P into three bf16 parts each, which hold all 24 bits.
//
// Work.  A call's tiles (sequence, rows) times key heads fill the chip or not; where they do not, a
// sequence's tokens are cut into pieces of equal length, as many over all sequences as fill it,
// and a second launch joins them.  Lengths are on the GPU alone, so every wave works out the
// same cut from them.
#include "attn.h"

namespace moe {

// ------------------------------------------------------------------- the pass
// SHARED: the four waves of a workgroup have one tile of 16 NQ rows and take its tokens in turn,
// joined in LDS at the end; otherwise each wave has a tile of its own among the workgroup's 64 NQ.
template <typename T, int D, int NQ, bool SHARED>
__global__ __launch_bounds__(256) void attn_kernel(const AttnArgs a) {
  constexpr int NB = D / 32, NC = D / 16, PARTS = sizeof(T) == 4 ? 3 : 1;
  constexpr int SUB = kStep / 16;
  typedef uint32_t KRaw __attribute__((ext_vector_type(NB)));
  const int wave = uniform((int)(threadIdx.x >> 6)), lane = lane_id();
  const int r16 = lane & 15, g = lane >> 4;
  const int kvh = blockIdx.y;

  int cut = 0x40000000;
  Found f;
  if (a.target) {
    cut = piece_tokens(a);
    if (!find_piece(a, cut, blockIdx.x, -1, f)) return;
  } else {
    if (!find_tile(a, blockIdx.x, f)) return;
  }
  const Seq& sq = f.seq;
  const int local = (int)(blockIdx.x - f.first_item);
  const int tile = sq.tiles(a) - 1 - local / f.pieces, piece = local % f.pieces;
  const int trow0 = tile * a.tile_rows + (SHARED ? 0 : wave * 16 * NQ);
  const int rows_here = sq.m * a.group;  // (row, head) pairs of the sequence and key head

  // this lane's rows: trow0 + 16 nq + r16
  int tok[NQ], head[NQ];
  bool real[NQ];
  Sight see[NQ];
  float slope[NQ];
  bf16x8 q[NQ][PARTS][NB];
#pragma unroll
  for (int nq = 0; nq < NQ; ++nq) {
    const int r = trow0 + 16 * nq + r16;
    real[nq] = r < rows_here;
    const int rr = real[nq] ? r : 0;
    tok[nq] = rr / a.group;
    head[nq] = kvh * a.group + rr - tok[nq] * a.group;
    see[nq] = sight_of(a, sq, tok[nq]);
    if (!real[nq]) see[nq] = {0, 0};
    slope[nq] = a.slopes && real[nq] ? a.slopes[head[nq]] * kLog2e : 0.f;
    const T* qp = (const T*)a.q + (sq.row0 + tok[nq]) * a.ld_q + head[nq] * a.hs_q;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      float v[8] = {};
      if (real[nq]) to_f32<T>(load8(qp + 8 * (g * NB + i)), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        __bf16 p[PARTS];
        split<PARTS>(v[e], p);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) q[nq][k][i][e] = p[k];
      }
    }
  }

  // the tile's tokens: what its first row (window) and its last (causal) see
  const int last_row = trow0 + 16 * NQ - 1 < rows_here - 1 ? trow0 + 16 * NQ - 1 : rows_here - 1;
  const bool any = trow0 < rows_here;
  const Sight s0 = sight_of(a, sq, any ? trow0 / a.group : 0);
  const Sight s1 = sight_of(a, sq, any ? last_row / a.group : 0);
  // (rows all see what lies in [s1.lo, s0.hi))
  const int64_t p0 = sq.first(a) + (int64_t)piece * cut;
  int lo = p0 > s0.lo ? (int)p0 : s0.lo & ~(kStep - 1);
  int hi = p0 + cut < s1.hi ? (int)(p0 + cut) : s1.hi;
  if (!any) hi = lo;

  float m[NQ], l[NQ];
  f32x4 acc[NQ][NC];
#pragma unroll
  for (int nq = 0; nq < NQ; ++nq) {
    m[nq] = -__builtin_inff();
    l[nq] = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[nq][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const KvUnit<D> unit{1 << a.page_log};
  const int32_t* pages = a.table + f.at * a.ld_table;
  const float qk_scale = a.scale * (a.softcap > 0.f ? 1.f : kLog2e);
  const float inv_cap = a.softcap > 0.f ? 1.f / a.softcap : 0.f;

  for (int t0 = lo + (SHARED ? wave * kStep : 0); t0 < hi; t0 += SHARED ? 4 * kStep : kStep) {
    // ---- loads
    KRaw kr[SUB];
    uint32_t ks[SUB][NB > 4 ? 2 : 1];
    KRaw vr[SUB];
    uint32_t vs[SUB];
    bool bad[SUB];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const int t = t0 + 16 * u;
      bad[u] = false;
      kr[u] = KRaw{};
      vr[u] = KRaw{};
      vs[u] = 0;
      ks[u][0] = 0;
      if constexpr (NB > 4) ks[u][1] = 0;
      if (t < hi) {
        int pg = uniform(pages[t >> a.page_log]);
        bad[u] = pg < 0 || pg >= a.n_pages;
        pg = bad[u] ? 0 : pg;
        const uint8_t* at = a.data + ((int64_t)pg * a.kv_heads + kvh) * unit.bytes();
        const int in = t & ((1 << a.page_log) - 1);
        __builtin_memcpy(&kr[u], at + (in + r16) * (D / 2) + g * (4 * NB), 4 * NB);
        const uint8_t* sc = at + unit.k_scales() + (in + r16) * NB;
        if constexpr (NB == 2) ks[u][0] = sc[g >> 1];
        if constexpr (NB == 4) ks[u][0] = sc[g];
        if constexpr (NB == 8) {
          ks[u][0] = sc[2 * g];
          ks[u][1] = sc[2 * g + 1];
        }
        const int quad = (in >> 2) + g;
        __builtin_memcpy(&vr[u], at + unit.v_codes() + (quad * 16 + r16) * 4 * NB, 4 * NB);
        __builtin_memcpy(&vs[u], at + unit.v_scales() + (quad * NB + r16 * NB / 16) * 4, 4);
      }
    }

    // ---- scores
    float s[NQ][SUB][4];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      f32x4 c[NQ];
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) c[nq] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint32_t sb = ks[u][NB > 4 ? i / 4 : 0];
        bf16x8 k = fp4x8_to_bf16x8(kr[u][i], __uint_as_float(sb << 23));
        if (sb > kMaxScaleByte || bad[u]) {
#pragma unroll
          for (int e = 0; e < 8; ++e) k[e] = (__bf16)__builtin_nanf("");
        }
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
            c[nq] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[nq][p][i], c[nq], 0, 0, 0);
      }
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = c[nq][e] * qk_scale;
          if (a.softcap > 0.f) x = capped(x, a.softcap, inv_cap) * kLog2e;
          const int j = t0 + 16 * u + 4 * g + e;
          if (a.slopes) x -= slope[nq] * (float)abs(sq.n - sq.m + tok[nq] - j);
          s[nq][u][e] = j >= see[nq].lo && j < see[nq].hi ? x : -__builtin_inff();
        }
    }

    // ---- values that are NaN (or, behind the last token, anything): 0 in the product, and NaN
    // in the channels of the rows that see them
    uint32_t over = 0;
#pragma unroll
    for (int u = 0; u < SUB; ++u) over |= over_bytes(vs[u]);
    if (__ballot(over != 0)) {
#pragma unroll
      for (int h = 0; h < SUB / 2; ++h) {
        bf16x8 nan;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int u = 2 * h + e / 4;
          nan[e] = (__bf16)(((vs[u] >> (8 * (e & 3))) & 0xFF) > kMaxScaleByte ? 1.f : 0.f);
        }
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
          bf16x8 seen;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int u = 2 * h + e / 4, j = t0 + 16 * u + 4 * g + (e & 3);
            seen[e] = (__bf16)(j >= see[nq].lo && j < see[nq].hi ? 1.f : 0.f);
          }
          f32x4 c = {0.f, 0.f, 0.f, 0.f};
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nan, seen, c, 0, 0, 0);
          // (c: of the runs of channels 4g + e, which a block's scale covers whole)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c[e] > 0.f) {
#pragma unroll
              for (int j = 0; j < NC; ++j) acc[nq][j][e] = __builtin_nanf("");
            }
        }
      }
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (((vs[u] >> (8 * b)) & 0xFF) > kMaxScaleByte) vs[u] &= ~(0xFFu << (8 * b));
    }

    // ---- softmax
    bf16x8 p[NQ][PARTS][SUB / 2];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      float top = m[nq];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[nq][u][e]);
      top = max16(top);
      const float base = top == -__builtin_inff() ? 0.f : top;
      const float old = exp2_fast(m[nq] - base);
      if (__ballot(top > m[nq])) {
        l[nq] *= old;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nq][j][e] *= old;
      }
      m[nq] = top;
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = exp2_fast(s[nq][u][e] - base);
          l[nq] += w;
          __bf16 part[PARTS];
          split<PARTS>(w, part);
#pragma unroll
          for (int k = 0; k < PARTS; ++k) p[nq][k][u / 2][(u & 1) * 4 + e] = part[k];
        }
    }

    // ---- out
#pragma unroll
    for (int h = 0; h < SUB / 2; ++h) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        // channels 2b and 2b + 1 of the lane's run, 8 tokens
        bf16x8 v0, v1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int u = 2 * h + e / 4, byte = (e & 3) * NB + b;  // of the 4 NB loaded
          const float sc = scale_byte(vs[u], e & 3);
          const uint32_t w = vr[u][byte / 4];
          bf16x2 x;
          switch (byte & 3) {
            case 0: x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0); break;
            case 1: x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1); break;
            case 2: x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2); break;
            default: x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3); break;
          }
          v0[e] = x[0];
          v1[e] = x[1];
        }
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int k = 0; k < PARTS; ++k) {
            acc[nq][2 * b] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, p[nq][k][h], acc[nq][2 * b], 0, 0, 0);
            acc[nq][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, p[nq][k][h],
                                                                         acc[nq][2 * b + 1], 0, 0, 0);
          }
      }
    }
  }
#pragma unroll
  for (int nq = 0; nq < NQ; ++nq) l[nq] = sum16(l[nq]);

  // ---- the waves' parts into one
  if constexpr (SHARED) {
    constexpr int LD = D + 4;
    __shared__ float joined[4][16][LD];
    __shared__ float ml[4][16][2];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      if (nq) __syncthreads();
      if (g == 0) {
        ml[wave][r16][0] = m[nq];
        ml[wave][r16][1] = l[nq];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < NC; j += 4)
          *(f32x4*)&joined[wave][r16][NC * (4 * g + e) + j] =
              f32x4{acc[nq][j][e], acc[nq][j + 1][e], acc[nq][j + 2][e], acc[nq][j + 3][e]};
      __syncthreads();
      // thread: row t / 16, channels D/16 (t % 16) ..
      const int row = threadIdx.x >> 4, ch = (threadIdx.x & 15) * NC;
      float top = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[w][row][0]);
      const float base = top == -__builtin_inff() ? 0.f : top;
      float sum = 0.f, o[NC] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float lw = ml[w][row][1], k = exp2_fast(ml[w][row][0] - base);
        if (lw == 0.f) continue;
        sum += lw * k;
#pragma unroll
        for (int j = 0; j < NC; ++j) o[j] += joined[w][row][ch + j] * k;
      }
      const int r = trow0 + 16 * nq + row;
      if (r >= rows_here) continue;
      if (f.pieces > 1) {
        const int64_t slot = ((int64_t)blockIdx.x * a.kv_heads + kvh) * a.tile_rows + 16 * nq + row;
        float* po = a.part + slot * D + ch;
#pragma unroll
        for (int j = 0; j < NC; ++j) po[j] = o[j];
        if (ch == 0) {
          a.part[a.ml_at + 2 * slot] = top;
          a.part[a.ml_at + 2 * slot + 1] = sum;
        }
      } else {
        const int token = r / a.group, hd = kvh * a.group + r - token * a.group;
        const Sight sg = sight_of(a, sq, token);
        const float inv = sg.lo < sg.hi ? 1.f / sum : 0.f;
        T res[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j) res[j] = (T)(sg.lo < sg.hi ? o[j] * inv : 0.f);
        T* dst = (T*)a.out + (sq.row0 + token) * a.ld_out + hd * a.hs_out + ch;
        __builtin_memcpy(dst, res, sizeof(res));
      }
    }
  } else {
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      if (!real[nq]) continue;
      const bool sees = see[nq].lo < see[nq].hi;
      if (f.pieces > 1) {
        const int64_t slot = ((int64_t)blockIdx.x * a.kv_heads + kvh) * a.tile_rows +
                             wave * 16 * NQ + 16 * nq + r16;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < NC; ++j)
            a.part[slot * D + NC * (4 * g + e) + j] = acc[nq][j][e];
        if (g == 0) {
          a.part[a.ml_at + 2 * slot] = m[nq];
          a.part[a.ml_at + 2 * slot + 1] = l[nq];
        }
      } else {
        const float inv = sees ? 1.f / l[nq] : 0.f;
        T* dst = (T*)a.out + (sq.row0 + tok[nq]) * a.ld_out + head[nq] * a.hs_out;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          T res[NC];
#pragma unroll
          for (int j = 0; j < NC; ++j) res[j] = (T)(sees ? acc[nq][j][e] * inv : 0.f);
          __builtin_memcpy(dst + NC * (4 * g + e), res, sizeof(res));
        }
      }
    }
  }
}

// Pieces into rows: a wave for each (row, head).
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a) {
  constexpr int PER = D / 64;
  const int lane = lane_id();
  const int64_t at = (int64_t)blockIdx.x * 4 + uniform((int)(threadIdx.x >> 6));
  if (at >= (int64_t)a.rows * a.n_heads) return;
  const int row = (int)(at / a.n_heads), head = (int)(at - (int64_t)row * a.n_heads);
  const int cut = piece_tokens(a);
  Found f;
  if (!find_piece(a, cut, 0, row, f) || f.pieces == 1) return;
  const int kvh = head / a.group, token = row - f.seq.row0;
  const int r = token * a.group + head - kvh * a.group;
  const int tile = r / a.tile_rows;
  const int64_t item0 = f.first_item + (int64_t)(f.seq.tiles(a) - 1 - tile) * f.pieces;
  if (item0 + f.pieces > a.items) return;  // (sequences that overlap)
  const int64_t slot0 = (item0 * a.kv_heads + kvh) * a.tile_rows + (r - tile * a.tile_rows);
  const int64_t step = (int64_t)a.kv_heads * a.tile_rows;
  const float* ml = a.part + a.ml_at;
  float top = -__builtin_inff();
  for (int p = lane; p < f.pieces; p += 64) top = fmaxf(top, ml[2 * (slot0 + p * step)]);
  top = wave_max(top);
  const float base = top == -__builtin_inff() ? 0.f : top;
  float sum = 0.f, o[PER] = {};
  for (int p = 0; p < f.pieces; ++p) {
    const int64_t slot = slot0 + p * step;
    const float lp = ml[2 * slot + 1], k = exp2_fast(ml[2 * slot] - base);
    if (lp == 0.f) continue;
    sum += lp * k;
#pragma unroll
    for (int j = 0; j < PER; ++j) o[j] += a.part[slot * D + lane * PER + j] * k;
  }
  const Sight sg = sight_of(a, f.seq, token);
  const bool sees = sg.lo < sg.hi;
  const float inv = 1.f / sum;
  T* dst = (T*)a.out + row * a.ld_out + head * a.hs_out + lane * PER;
#pragma unroll
  for (int j = 0; j < PER; ++j) dst[j] = (T)(sees ? o[j] * inv : 0.f);
}

// ------------------------------------------------------------------ the host side
// How a call runs: the kernel and the rows of its tiles, the pieces to cut into.
struct AttnPlan {
  int chunk_waves; // 0: attn_kernel
  int nq;          // of attn_kernel
  bool shared;
  int tile_rows;
  int64_t tiles;   // at most, over all sequences
  int target;      // 0: tokens are not cut
  int64_t items;   // of the grid
};

static int64_t tiles_of(int64_t rows, int64_t group, int64_t n_seqs, int tile_rows) {
  return (rows * group + tile_rows - 1) / tile_rows + n_seqs;
}

static AttnPlan attn_plan(const moe_attn_t* A, const moe_kv_cache_t* C, bool f32, int64_t rows,
                          int64_t n_seqs, int cus) {
  AttnPlan p;
  const int64_t group = A->n_heads / C->n_heads;
  const int64_t each = (rows * group + n_seqs - 1) / n_seqs;  // rows of a sequence, on average
  p.shared = each <= 64;
  p.nq = f32 || each <= 16 ? 1 : 2;
  p.chunk_waves = f32 || p.shared ? 0 : 4;
  p.tile_rows = p.shared ? 16 * p.nq : f32 ? 64 : 128;
  int64_t full = 2 * cus;
  if (p.chunk_waves && C->head_dim < 256 &&
      tiles_of(rows, group, n_seqs, 256) * C->n_heads >= cus) {
    p.chunk_waves = 8;
    p.tile_rows = 256;
    full = cus;
  }
  p.tiles = tiles_of(rows, group, n_seqs, p.tile_rows);
  p.target = p.tiles * C->n_heads >= full ? 0 : (int)((full + C->n_heads - 1) / C->n_heads);
  p.items = p.tiles + p.target;
  return p;
}

static int64_t part_floats(const moe_kv_cache_t* C, int64_t items, int64_t tile_rows) {
  return items * C->n_heads * tile_rows * (C->head_dim + 2);
}

static bool attn_sizes_ok(const moe_attn_t* A, const moe_kv_cache_t* C) {
  return A->n_heads >= 1 && A->n_heads <= 65536 && A->n_heads % C->n_heads == 0;
}

template <typename T, int D>
static void attn_launch(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if (p.chunk_waves) {
    attn_chunk_launch(a, D, p.chunk_waves, stream);
  } else {
    const dim3 grid((unsigned)p.items, (unsigned)a.kv_heads);
    if constexpr (sizeof(T) == 4) {
      auto k = p.shared ? attn_kernel<T, D, 1, true> : attn_kernel<T, D, 1, false>;
      hipLaunchKernelGGL(k, grid, dim3(256), 0, stream, a);
    } else {
      auto k = p.nq == 1 ? attn_kernel<T, D, 1, true> : attn_kernel<T, D, 2, true>;
      hipLaunchKernelGGL(k, grid, dim3(256), 0, stream, a);
    }
  }
  if (p.target) {
    const int64_t waves = (int64_t)a.rows * a.n_heads;
    hipLaunchKernelGGL((attn_join_kernel<T, D>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0,
                       stream, a);
  }
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_attn_cache_workspace_bytes(const moe_attn_t* A, const moe_kv_cache_t* C,
                                                 int rows, int n_seqs) {
  if (!A || !C || !kv_sizes_ok(C) || !attn_sizes_ok(A, C) || rows <= 0 || n_seqs <= 0) return 0;
  int cus = device_cu_count();
  if (cus <= 0) cus = 256;
  // Cut calls have fewer than `full` tiles over all heads, so at most that many and their target
  // pieces: no fewer rows or sequences need more.
  const int64_t full = 2 * cus, heads = C->n_heads;
  const int64_t group = A->n_heads / heads;
  const int64_t target = (full + heads - 1) / heads;
  int64_t most = 0;
  for (int tile_rows : {16, 32, 64, 128, 256}) {
    int64_t tiles = ((int64_t)rows * group + tile_rows - 1) / tile_rows + n_seqs;
    const int64_t cap = (full + heads - 1) / heads;
    if (tiles > cap) tiles = cap;
    const int64_t n = part_floats(C, tiles + target, tile_rows);
    most = n > most ? n : most;
  }
  return (size_t)most * 4;
}

extern "C" int moe_attn_cache(const moe_attn_t* A, const moe_kv_cache_t* C, const void* q,
                              int type, int64_t ld_q, int64_t hs_q, int rows,
                              const int32_t* q_offsets, int n_seqs, const int32_t* kv_lens,
                              const int32_t* table, int64_t ld_table, int max_pages,
                              const int32_t* prefix, void* out, int64_t ld_out, int64_t hs_out,
                              void* ws, size_t ws_bytes, void* stream) {
  if (!A) return MOE_ERR_INVALID_ARG;
  const int rc = kv_cache_check(C);
  if (rc != MOE_OK) return rc;
  if (!attn_sizes_ok(A, C)) return MOE_ERR_SHAPE;
  if (A->window < 0 || !__builtin_isfinite(A->scale) || !__builtin_isfinite(A->softcap) ||
      A->softcap < 0.f || rows < 0 || n_seqs < 0 || max_pages < 0 || !type_ok(type))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0 || n_seqs == 0) return MOE_OK;
  if (!q || !out || q == out || !kv_lens || (!table && max_pages)) return MOE_ERR_INVALID_ARG;
  if (!q_offsets && rows != n_seqs) return MOE_ERR_INVALID_ARG;
  if ((int64_t)max_pages * C->page >= ((int64_t)1 << 30) ||
      (int64_t)rows * (A->n_heads / C->n_heads) >= ((int64_t)1 << 28) || n_seqs > (1 << 24))
    return MOE_ERR_SHAPE;
  if (!head_strides_ok(ld_q, hs_q, rows, A->n_heads, C->head_dim) ||
      !head_strides_ok(ld_out, hs_out, rows, A->n_heads, C->head_dim) ||
      (n_seqs > 1 && ld_table < max_pages))
    return MOE_ERR_STRIDE;
  const size_t size = type_size(type);
  if (!aligned(q, size) || !aligned(out, size) || !aligned(kv_lens, 4) || !aligned(table, 4) ||
      (q_offsets && !aligned(q_offsets, 4)) || (prefix && !aligned(prefix, 4)) ||
      (A->slopes && !aligned(A->slopes, 4)))
    return MOE_ERR_ALIGNMENT;
  int cus = device_cu_count();
  if (cus <= 0) cus = 256;
  AttnPlan p = attn_plan(A, C, type == MOE_TYPE_F32, rows, n_seqs, cus);
  if ((int64_t)max_pages * C->page <= kLeastPart) p.items -= p.target, p.target = 0;
  const int64_t need = p.target ? 4 * part_floats(C, p.items, p.tile_rows) : 0;
  if (need && !ws) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < (size_t)need) return MOE_ERR_WORKSPACE;
  if (need && !aligned(ws, 16)) return MOE_ERR_ALIGNMENT;
  if (!device_is_gfx950()) return MOE_ERR_UNSUPPORTED_ARCH;
  AttnArgs a;
  a.q = q;
  a.out = out;
  a.data = (const uint8_t*)C->data;
  a.q_offsets = q_offsets;
  a.kv_lens = kv_lens;
  a.table = table;
  a.prefix = prefix;
  a.slopes = A->slopes;
  a.part = (float*)ws;
  a.ld_q = ld_q;
  a.hs_q = hs_q;
  a.ld_out = ld_out;
  a.hs_out = hs_out;
  a.ld_table = n_seqs > 1 ? ld_table : 0;
  a.ml_at = p.items * C->n_heads * p.tile_rows * C->head_dim;
  a.rows = rows;
  a.n_seqs = n_seqs;
  a.n_heads = A->n_heads;
  a.kv_heads = C->n_heads;
  a.group = A->n_heads / C->n_heads;
  a.page_log = __builtin_ctz((unsigned)C->page);
  a.n_pages = C->n_pages;
  a.max_pages = max_pages;
  a.window = A->window;
  a.target = p.target;
  a.items = p.items;
  a.tile_rows = p.tile_rows;
  a.scale = A->scale;
  a.softcap = A->softcap;
  const hipStream_t st = (hipStream_t)stream;
  const bool f32 = type == MOE_TYPE_F32;
  switch (C->head_dim) {
    case 64: f32 ? attn_launch<float, 64>(a, p, st) : attn_launch<__bf16, 64>(a, p, st); break;
    case 128: f32 ? attn_launch<float, 128>(a, p, st) : attn_launch<__bf16, 128>(a, p, st); break;
    default: f32 ? attn_launch<float, 256>(a, p, st) : attn_launch<__bf16, 256>(a, p, st); break;
  }
  return launch_status();
}
